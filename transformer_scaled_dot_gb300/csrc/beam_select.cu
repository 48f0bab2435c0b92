// beam_select.cu -- one step of beam search: from the logits of every live
// hypothesis to the next beams and the ended hypotheses.
//
// With s_k the score of beam k of a sentence (its tokens' summed log
// probabilities) and x_k its row of logits,
//   total(k, v) = s_k + x_kv - log sum_u exp(x_ku).
// The best 2 K pairs (K without an end token: at most one pair of each beam
// ends it), by total and then by lowest k V + v, are the candidates. Those
// that are not the end token are the next beams, best first; those that are
// end there, scored total / ((5 + n) / 6)^alpha at n tokens, and compete with
// the hypotheses that ended before.
//
// Two launches. beam_tiles takes the rows in tiles of 1024 logits, a warp to a
// tile, and keeps of each its largest logit and the sum of exponentials
// relative to it: one pass over the logits, no list of best ones to carry. It
// is enough: a pair among the best M lies in one of the M tiles with the best
// maxima (each tile ahead of its own holds a pair that beats it). beam_pick, a
// block to a sentence, joins a row's tiles to its log-sum, picks those M tiles
// and then the M pairs in them. Sentences of few tiles go through beam_one, which
// is both in one launch.
// Totals that lie next to one another decide which token a beam takes: they
// are formed and compared as pairs of fp32, 48 bits. Exponentials and a tile's
// sum are in 32, relative to the tile's own maximum, as are the few tiles of a
// lane that joins them; lanes are joined in 48.
#include <cfloat>
#include <cstddef>

#include "kernels.h"
#include "sm103.cuh"

namespace tsd {

namespace {

constexpr int kTile = kBeamTile;          // logits of a warp's tile
constexpr int kTileWarps = 4;             // warps of a beam_tiles block
constexpr int kPickThreads = 512;
constexpr unsigned long long kDrainLimitNs = 100ull * 1000ull * 1000ull;  // 0.1 s
constexpr int kPickWarps = kPickThreads / 32;
static_assert(kPickWarps >= kBeamMaxBeams, "a warp joins a row's tiles");

template <bool F32>
__device__ __forceinline__ float load_logit(const void* p, int64_t at) {
  if constexpr (F32) return static_cast<const float*>(p)[at];
  return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[at]) << 16);
}

// A lane's 32 logits of a tile, as they lie in memory, two of bf16 to a word.
// ALIGNED: every row of the call starts on 16 bytes, and a lane's vector j holds
// the consecutive logits from (32 j + l) * (16 / size); otherwise a word j those
// from (32 j + l) * (4 / size). Which lane adds up a logit follows from its
// number alone, so that equal rows have equal sums wherever they start. Past the
// row's end -infinity.
template <bool F32, bool ALIGNED>
struct Tile {
  static constexpr int kSize = F32 ? 4 : 2;
  static constexpr int kPer = (ALIGNED ? 16 : 4) / kSize;  // consecutive logits of a lane
  static constexpr int kWords = 32 * kSize / 4;
  uint32_t w[kWords];

  static __device__ __forceinline__ int place(int t, int i, int lane) {
    return t * kTile + (i / kPer * 32 + lane) * kPer + i % kPer;
  }
  static __device__ __forceinline__ uint32_t one(const void* row, int v) {
    return F32 ? static_cast<const uint32_t*>(row)[v] : static_cast<const uint16_t*>(row)[v];
  }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (F32) return __uint_as_float(w[i]);
    return __uint_as_float(i & 1 ? w[i / 2 % kWords] & 0xffff0000u : w[i / 2 % kWords] << 16);
  }
  // what lies past the row's end
  __device__ __forceinline__ void cut(int t, int vocab, int lane) {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const bool past = place(t, i, lane) >= vocab;
      uint32_t& word = w[F32 ? i : i / 2 % kWords];
      if constexpr (F32) word = past ? 0xff800000u : word;
      else if (i & 1) word = past ? (word & 0xffffu) | 0xff800000u : word;
      else word = past ? (word & 0xffff0000u) | 0xff80u : word;
    }
  }
  // logit i, straight from memory
  __device__ __forceinline__ void load_one(const void* row, int t, int i, int vocab, int lane) {
    const int v = place(t, i, lane);
    const uint32_t x = v < vocab ? one(row, v) : F32 ? 0xff800000u : 0xff80u;
    if constexpr (F32) w[i] = x;
    else w[i / 2 % kWords] = i & 1 ? w[i / 2 % kWords] | x << 16 : x;
  }
  // straight from memory
  __device__ __forceinline__ void load(const void* row, int t, int vocab, int lane) {
    if constexpr (ALIGNED) {
#pragma unroll
      for (int j = 0; j < kWords / 4; ++j) {
        const int v = place(t, j * kPer, lane);
        if (v + kPer <= vocab) {
          const uint4 q = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(row) + static_cast<int64_t>(v) * kSize);
          w[4 * j] = q.x;
          w[4 * j + 1] = q.y;
          w[4 * j + 2] = q.z;
          w[4 * j + 3] = q.w;
        } else if (v >= vocab) {
          w[4 * j] = w[4 * j + 1] = w[4 * j + 2] = w[4 * j + 3] = F32 ? 0xff800000u : 0xff80ff80u;
        } else {
#pragma unroll
          for (int e = 0; e < kPer; ++e) load_one(row, t, j * kPer + e, vocab, lane);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) load_one(row, t, i, vocab, lane);
    }
  }
};

// A warp's ring of units of U tiles in shared memory, filled by bulk copies: one
// thread starts 4 KB, less at a row's end. They move 16-byte blocks of memory; a row
// that starts `skew` bytes into one has one block more to a unit.
template <bool F32, bool ALIGNED>
struct Ring {
  using T = Tile<F32, ALIGNED>;
  static constexpr int kStages = 2;
  static constexpr int U = F32 ? 1 : 2;
  static constexpr int kUnit = U * kTile;
  static constexpr int kUnitBytes = kUnit * T::kSize;
  static constexpr int kStageBytes = kUnitBytes + 16;
  alignas(16) uint8_t stage[kStages][kStageBytes];
  uint64_t full[kStages];

  static __device__ __forceinline__ int skew_of(const uint8_t* row) {
    return ALIGNED ? 0 : static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15u);
  }
  // Bytes of the copy of unit u, from `skew` bytes ahead of it; its first and
  // last blocks may hold logits of other rows. 0, no copy, where they would lie
  // outside of [begin, end), all rows' logits.
  static __device__ __forceinline__ int bytes(const uint8_t* row, int u, int vocab, const uint8_t* begin, const uint8_t* end) {
    const int skew = skew_of(row);
    const int there = (vocab - u * kUnit) * T::kSize + skew;
    const int n = min(kUnitBytes + (skew != 0 ? 16 : 0), (there + 15) & ~15);
    const uint8_t* from = row + static_cast<int64_t>(u) * kUnitBytes - skew;
    return from < begin || from + n > end ? 0 : n;
  }
  __device__ __forceinline__ void copy(int s, const uint8_t* row, int u, int n) {
    mbar_arrive_expect_tx(&full[s], static_cast<uint32_t>(n));
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(stage[s])),
                 "l"(row + static_cast<int64_t>(u) * kUnitBytes - skew_of(row)), "r"(n), "r"(smem_u32(&full[s]))
                 : "memory");
  }
  static __device__ __forceinline__ void read(T& x, const uint8_t* stage, const uint8_t* row, int lane) {
    if constexpr (ALIGNED) {
#pragma unroll
      for (int j = 0; j < T::kWords / 4; ++j) {
        const uint4 q = *reinterpret_cast<const uint4*>(stage + (j * 32 + lane) * 16);
        x.w[4 * j] = q.x;
        x.w[4 * j + 1] = q.y;
        x.w[4 * j + 2] = q.z;
        x.w[4 * j + 3] = q.w;
      }
    } else {
      const int skew = skew_of(row);
      const uint32_t* words = reinterpret_cast<const uint32_t*>(stage + (skew & ~3)) + lane;
      if (F32 || (skew & 3) == 0) {
#pragma unroll
        for (int j = 0; j < T::kWords; ++j) x.w[j] = words[j * 32];
      } else {  // each pair from two words
#pragma unroll
        for (int j = 0; j < T::kWords; ++j) x.w[j] = __funnelshift_r(words[j * 32], words[j * 32 + 1], 16);
      }
    }
  }
};

__device__ __forceinline__ float max_nan(float a, float b) {
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(a) : "f"(b));
  return a;
}
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(a) : "f"(b), "f"(c));
  return a;
}

// Over a warp: one instruction in place of five exchanges.
__device__ __forceinline__ float warp_max_nan(float x) {
  asm("redux.sync.max.NaN.f32 %0, %0, 0xffffffff;" : "+f"(x));
  return x;
}

// log2(e) as two numbers of 32 bits
constexpr float kLog2eHi = 1.4426950216293335f, kLog2eLo = 1.9259629911266175e-8f;

// The largest logit of a warp's tile and the sum of exponentials relative to it.
// 2^(x log2(e) - r), r = top log2(e) as fp32 has it, is one multiply-add; what r
// is off by is made good in the sum. What is left is the constant's own
// rounding, 2^-26 (x - top).
template <bool F32, bool ALIGNED>
__device__ __forceinline__ float2 tile_record(const Tile<F32, ALIGNED>& x) {
  float top = x.at(0);
#pragma unroll
  for (int i = 1; i < 31; i += 2) top = max3_nan(top, x.at(i), x.at(i + 1));
  top = warp_max_nan(max_nan(top, x.at(31)));
  float s = 0.f, off = 0.f;
  if (fabsf(top) < 1024.f) {  // r is off by 2^-14 at most
    const float r = top * kLog2eHi;
    const uint64_t neg = f2_pack(-r, -r), scale = f2_pack(kLog2eHi, kLog2eHi);
    uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float a, b;
      f2_unpack(ffma2(f2_pack(x.at(2 * i), x.at(2 * i + 1)), scale, neg), a, b);
      sum[i & 1] = fadd2(sum[i & 1], f2_pack(ex2(a), ex2(b)));
    }
    float a, b;
    f2_unpack(fadd2(sum[0], sum[1]), a, b);
    s = a + b;
    off = __fmaf_rn(top, kLog2eHi, -r);  // the largest one's exponent
  } else if (top > -INFINITY) {  // the differences first; a NaN or infinity among them
#pragma unroll
    for (int i = 0; i < 32; ++i) s += ex2((x.at(i) - top) * kLog2eHi);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return make_float2(top, __fmaf_rn(s, off * -0.693147181f, s));
}

// Persistent warps, each with a ring of two units of 4 KB, 24 warps to an SM.
// 134 MB of bf16 in 25 to 26 us, of fp32 in 22, launch included (5.2 and 6.1 TB/s;
// exponentials and all but the copies left out, 24 and 22). Loads by the lanes
// instead: 29 us, 40 where rows are not aligned, and for fp32 25; 2 KB to a copy
// and 4 stages 29; 8 KB 25, and slower where there are few tiles.
// Of a beam without a hypothesis nothing is loaded but the first unit of a
// warp, which does not wait for the score.
template <bool F32, bool ALIGNED>
__global__ void __launch_bounds__(32 * kTileWarps, 6)
    beam_tiles_kernel(const BeamProblem p, int tiles, int total) {
  using R = Ring<F32, ALIGNED>;
  constexpr int U = R::U;
  using T = Tile<F32, ALIGNED>;
  static_assert(sizeof(R) % 16 == 0 && R::kStageBytes % 16 == 0, "copies into shared memory start on 16 bytes");
  static_assert(R::kStages == 2, "the first copy ahead of the loop, the second by its first round");
  extern __shared__ __align__(16) uint8_t smem_raw[];
  R& ring = reinterpret_cast<R*>(smem_raw)[warp_id()];
  __shared__ uint32_t abort_word;
  volatile uint32_t* abort_flag = &abort_word;
  const int lane = static_cast<int>(lane_id());
  if (lane == 0) {
    for (int i = 0; i < R::kStages; ++i) mbar_init(&ring.full[i], 1);
    fence_mbar_init();
  }
  if (threadIdx.x == 0) abort_word = 0;
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  const int step = static_cast<int>(gridDim.x) * kTileWarps;
  int id = static_cast<int>(blockIdx.x) * kTileWarps + warp_id();
  if (id >= total) return;
  const int rows = p.B * p.beams;
  const uint8_t* logits = static_cast<const uint8_t*>(p.logits);
  const int64_t row_bytes = p.row_stride * (F32 ? 4 : 2);
  const uint8_t* logits_end = logits + (rows - 1) * row_bytes + p.vocab * T::kSize;
  const int units = (tiles + U - 1) / U;  // of a row
  const int step_rows = step / units, step_units = step - step_rows * units;
  struct At {
    int row, u;
  };
  auto next = [&](At at) {
    at.row += step_rows;
    at.u += step_units;
    if (at.u >= units) {
      at.u -= units;
      ++at.row;
    }
    return at;
  };
  auto score = [&](const At& at) { return at.row < rows ? __ldcg(p.scores + at.row) : -INFINITY; };
  At now = {id / units, id % units}, ahead = now;  // the unit at hand, and the next to copy
  uint32_t under_way = 0u;  // bit s: a copy into stage s
  auto copy = [&](int s, bool wanted) {
    if (wanted) {
      const uint8_t* row = logits + ahead.row * row_bytes;
      const int n = R::bytes(row, ahead.u, p.vocab, logits, logits_end);
      if (n > 0) {
        under_way |= 1u << s;
        if (lane == 0) ring.copy(s, row, ahead.u, n);
      }
    }
    ahead = next(ahead);
  };
  copy(0, true);
  At look = now;
  float scores[R::kStages];
#pragma unroll
  for (int i = 0; i < R::kStages; ++i) {
    scores[i] = score(look);
    look = next(look);
  }
  float pending = score(look);  // of the unit after them; looked at a round later
  look = next(look);
  uint32_t live = 0u;  // bit i: the unit i after the one at hand has a hypothesis
#pragma unroll
  for (int i = 0; i < R::kStages; ++i) live |= (scores[i] != -INFINITY ? 1u : 0u) << i;
  uint32_t parity = 0u;  // bit s: of stage s
  bool ok = true;
  for (int s = 0; id < total; id += step) {
    __syncwarp();  // the previous unit has been read
    copy(s == 0 ? R::kStages - 1 : s - 1, live >> (R::kStages - 1) & 1u);
    const bool wanted = live & 1u;
    live = live >> 1 | (pending != -INFINITY ? 1u : 0u) << (R::kStages - 1);
    pending = score(look);
    look = next(look);
    const uint8_t* row = logits + now.row * row_bytes;
    const bool copied = under_way >> s & 1u;
    if (copied) {
      ok = __all_sync(0xffffffffu, mbar_wait(&ring.full[s], parity >> s & 1u, abort_flag));
      if (!ok) break;
      parity ^= 1u << s;
      under_way &= ~(1u << s);
    }
    if (wanted) {
#pragma unroll
      for (int h = 0; h < U; ++h) {
        const int t = now.u * U + h;
        if (t >= tiles) break;
        Tile<F32, ALIGNED> x;
        if (copied) {
          R::read(x, ring.stage[s] + h * kTile * T::kSize, row, lane);
          if ((t + 1) * kTile > p.vocab) x.cut(t, p.vocab, lane);
        } else {
          x.load(row, t, p.vocab, lane);
        }
        const float2 record = tile_record(x);
        if (lane == 0) reinterpret_cast<float2*>(p.workspace)[static_cast<int64_t>(now.row) * tiles + t] = record;
      }
    }
    now = next(now);
    s = s + 1 == R::kStages ? 0 : s + 1;
  }
  if (!ok) {
    // this warp's copies still under way, a limited time
    volatile uint32_t never = 0;
    for (int s = 0; s < R::kStages; ++s)
      if (under_way >> s & 1u) mbar_wait(&ring.full[s], parity >> s & 1u, &never, kDrainLimitNs);
  }
}

// ---------------------------------------------------------------- pairs of fp32
// A number as the unevaluated sum of two of 32 bits, the second at most half a
// step of the first: 48 bits. Totals are kept so: 64-bit arithmetic has a
// sixtieth of the rate here and many times the latency (with it a sentence's
// choice took 13 us, 5 of them one logarithm and one power).

struct Pair {
  float h, l;
};
// a + b, exactly
__device__ __forceinline__ Pair two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
// h + l again with l at most half a step; |h| >= |l|, or h = 0
__device__ __forceinline__ Pair settled(float h, float l) {
  const float s = __fadd_rn(h, l);
  return {s, __fsub_rn(l, __fsub_rn(s, h))};
}
__device__ __forceinline__ Pair add(Pair a, Pair b) {
  const Pair s = two_sum(a.h, b.h);
  return settled(s.h, s.l + (a.l + b.l));
}

// ln 2 in two parts, the first of 14 bits, so that its products with exponents are exact
constexpr float kLn2Hi = 0x1.62e4p-1f, kLn2Lo = 1.4286068e-06f;

// ln(x) for a normal x.h, off by less than 2^-28: with x = 2^e m, m within
// sqrt(2) of 1, ln m = 2 atanh(z) = 2 (z + z^3 / 3 + z^5 / 5 + ..), z = (m - 1) / (m + 1),
// whose first term is carried as a pair.
__device__ __forceinline__ Pair log_pair(Pair x) {
  const int bits = __float_as_int(x.h);
  const int e = (bits - 0x3f3504f3) >> 23;  // sqrt(1/2) is 0x3f3504f3
  const float m = __int_as_float(bits - (e << 23));
  const float f = m - 1.f, d = 1.f + m, d_rest = m - (d - 1.f);
  const float inverse = __fdividef(1.f, d);  // what z is off by is in z_rest
  const float z = f * inverse;
  const float z_rest = (__fmaf_rn(-z, d, f) - z * d_rest) * inverse;
  const float z2 = z * z;
  float series = 1.f / 13.f;
  series = __fmaf_rn(series, z2, 1.f / 11.f);
  series = __fmaf_rn(series, z2, 1.f / 9.f);
  series = __fmaf_rn(series, z2, 1.f / 7.f);
  series = __fmaf_rn(series, z2, 1.f / 5.f);
  series = __fmaf_rn(series, z2, 1.f / 3.f);
  const float ef = static_cast<float>(e);
  const Pair s = two_sum(ef * kLn2Hi, 2.f * z);
  const float rest = 2.f * (z_rest + z * (z2 * series)) + __fdividef(x.l, x.h);
  return settled(s.h, s.l + (rest + ef * kLn2Lo));
}

// exp(x) = value * 2^exponent, to 2^-25 of it, |x| <= 300: the Taylor series over
// half of ln 2, its first two terms as a pair
__device__ __forceinline__ Pair exp_pair(Pair x, int* exponent) {
  const float k = rintf(x.h * kLog2eHi);
  *exponent = static_cast<int>(k);
  const Pair r = two_sum(__fmaf_rn(-k, kLn2Hi, x.h), x.l - k * kLn2Lo);
  float series = 1.f / 40320.f;
  series = __fmaf_rn(series, r.h, 1.f / 5040.f);
  series = __fmaf_rn(series, r.h, 1.f / 720.f);
  series = __fmaf_rn(series, r.h, 1.f / 120.f);
  series = __fmaf_rn(series, r.h, 1.f / 24.f);
  series = __fmaf_rn(series, r.h, 1.f / 6.f);
  series = __fmaf_rn(series, r.h, 0.5f);
  const Pair s = two_sum(1.f, r.h);
  return settled(s.h, s.l + (r.l + r.h * r.h * series));
}

// The length penalty ((5 + n) / 6)^alpha as value * 2^exponent.
__device__ __forceinline__ Pair length_penalty(int n, Pair alpha, int* exponent) {
  const int64_t top = static_cast<int64_t>(n) + 5;
  const float h = static_cast<float>(top);
  constexpr float kLn6Hi = 0x1.cab0cp+0f, kLn6Lo = -2.1738742e-08f;
  Pair base = add(log_pair({h, static_cast<float>(top - static_cast<int64_t>(h))}), {-kLn6Hi, -kLn6Lo});
  if (n == 1) base = {0.f, 0.f};  // exactly, whatever alpha is
  float x = alpha.h * base.h;
  float rest = __fmaf_rn(alpha.h, base.h, -x) + (alpha.h * base.l + alpha.l * base.h);
  // e^300 and e^-300 take every score to 0 or beyond fp32 already
  if (!(fabsf(x) < 300.f)) {
    x = copysignf(300.f, x);
    rest = 0.f;
  }
  return exp_pair(settled(x, rest), exponent);
}

// Pairs as whole numbers in the same order; 0: none.
__device__ __forceinline__ uint32_t order_bits(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);  // -0 is 0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float from_order_bits(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}
__device__ __forceinline__ Pair key_total(uint64_t key) {
  return {from_order_bits(static_cast<uint32_t>(key >> 32)), from_order_bits(static_cast<uint32_t>(key))};
}
// Whether a is ahead of b: by total, then by place.
__device__ __forceinline__ bool ahead(uint64_t a_key, int a_at, uint64_t b_key, int b_at) {
  return a_key > b_key || (a_key == b_key && a_at < b_at);
}

// A beam: total = base + (logit - top), so that no digits are lost where
// logits are large.
struct Beam {
  Pair base;  // s_k - log sum exp(x - top); h = -infinity: no live hypothesis
  float top;  // the row's largest logit
};
// The key of a logit's total; 0 where it is no candidate.
__device__ __forceinline__ uint64_t total_key(const Beam& beam, float x) {
  const Pair d = two_sum(x, -beam.top);
  const Pair s = two_sum(beam.base.h, d.h);
  if (!(s.h > -INFINITY)) return 0;
  const Pair t = settled(s.h, s.l + (beam.base.l + d.l));
  return static_cast<uint64_t>(order_bits(t.h)) << 32 | order_bits(t.l);
}

constexpr int kGroups = 64;     // of a sentence's tiles, or of the lanes of some
constexpr int kSubs = kPickThreads / kGroups;  // threads of a group
static_assert(kGroups == 2 * 32, "a group's lane");
// Where a thread's entries of a list lie, every 512th from here: those of a group at
// every 64th place or a few off, so that neighbours fall into different groups, and a
// warp's in different banks.
__device__ __forceinline__ int first_of_thread() {
  const int sub = static_cast<int>(threadIdx.x) % kSubs, group = static_cast<int>(threadIdx.x) / kSubs;
  return sub * kGroups + (group + sub * (32 / kSubs)) % kGroups;
}
constexpr int kListMost = 2048, kListStep = 3 * kPickThreads;
constexpr int kTileList = 64;   // chosen tiles that are looked through
constexpr int kPairList = 2 * kTileList * 2 * kBeamMaxBeams;
constexpr int kSpare = kPairList / 2;  // of it, for tiles with more than M
constexpr int kTileMost = 128;  // of one tile (a warp takes 6 us for 1024)
constexpr int kFewPairs = 96;

struct PickSmem {
  Beam beam[kBeamMaxBeams];
  uint64_t group_key[kGroups];
  int group_at[kGroups];
  uint64_t last_key;           // the M-th best group's largest total, and its place
  int last_at;
  int n_tiles, n_pairs;
  int claimed;                 // pairs of tiles that have more than M not behind the last
  int crowded;                 // they do not fit
  int tile[kListMost];         // chosen tiles
  uint64_t tile_key[kListMost];
  uint64_t pair_key[kPairList];
  int pair_at[kPairList];
  uint64_t best_key[2 * kBeamMaxBeams];
  int best_at[2 * kBeamMaxBeams];
  Pair penalty;
  int penalty_exponent, length;
  float end_score[2 * kBeamMaxBeams];
  int end_row[kBeamMaxBeams];
  // of every tile of the sentence first its record, then its largest total
  uint64_t key[1];
};

// Of n entries how many are ahead of entry i, by a warp.
__device__ __forceinline__ int rank_of(const uint64_t* key, const int* at, int n, int i, int lane) {
  int before = 0;
#pragma unroll 1
  for (int j = lane; j < n; j += 32) before += ahead(key[j], at[j], key[i], at[i]);
  return static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(before)));
}

// The M best of the listed tiles, at the list's front.
__device__ __noinline__ void keep_best_tiles(PickSmem& sm, int M) {
  const int warp = warp_id(), lane = static_cast<int>(lane_id()), tid = static_cast<int>(threadIdx.x);
  const int listed = sm.n_tiles;
#pragma unroll 1
  for (int i = warp; i < listed; i += kPickWarps) {
    const int rank = rank_of(sm.tile_key, sm.tile, listed, i, lane);
    if (lane == 0 && rank < M) {
      sm.best_key[rank] = sm.tile_key[i];
      sm.best_at[rank] = sm.tile[i];
    }
  }
  __syncthreads();
  if (tid < M) {
    sm.tile_key[tid] = sm.best_key[tid];
    sm.tile[tid] = sm.best_at[tid];
  }
  if (tid == 0) sm.n_tiles = M;
  __syncthreads();
}

// Groups of eight threads, each thread with its best (key 0: none), the places
// all different: the M-th best group's best into sm.last_key and sm.last_at;
// key 0 if so many groups have none.
__device__ __forceinline__ void last_of_groups(PickSmem& sm, uint64_t key, int at, int M) {
  const int tid = static_cast<int>(threadIdx.x);
#pragma unroll
  for (int o = 1; o < kSubs; o <<= 1) {
    const uint64_t other_key = __shfl_xor_sync(0xffffffffu, key, o);
    const int other_at = __shfl_xor_sync(0xffffffffu, at, o);
    if (ahead(other_key, other_at, key, at)) {
      key = other_key;
      at = other_at;
    }
  }
  if (tid % kSubs == 0) {
    sm.group_key[tid / kSubs] = key;
    sm.group_at[tid / kSubs] = at;
  }
  if (tid == 0) {
    sm.last_key = 0;
    sm.last_at = INT32_MAX;
  }
  __syncthreads();
  int before = 0;
#pragma unroll
  for (int j = 0; j < kGroups / kSubs; ++j) {
    const int g = j * kSubs + tid % kSubs;
    before += ahead(sm.group_key[g], sm.group_at[g], key, at);
  }
#pragma unroll
  for (int o = 1; o < kSubs; o <<= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
  if (before == M - 1 && key != 0 && tid % kSubs == 0) {
    sm.last_key = key;
    sm.last_at = at;
  }
  __syncthreads();
}

// Of the pairs those that are not behind the M-th best of 64 groups.
__device__ __noinline__ void keep_best_pairs(PickSmem& sm, int M) {
  constexpr int kMost = kPairList / kPickThreads;
  const int tid = static_cast<int>(threadIdx.x), first = first_of_thread();
  const int pairs = sm.n_pairs;
  uint64_t key[kMost], best_key = 0;
  int at[kMost], best_at = INT32_MAX;
#pragma unroll
  for (int j = 0; j < kMost; ++j) {
    key[j] = 0;
    if (j * kPickThreads >= pairs) continue;
    const int i = first + j * kPickThreads;
    key[j] = i < pairs ? sm.pair_key[i] : 0;
    at[j] = i < pairs ? sm.pair_at[i] : INT32_MAX;
    if (ahead(key[j], at[j], best_key, best_at)) {
      best_key = key[j];
      best_at = at[j];
    }
  }
  __syncthreads();
  if (tid == 0) sm.n_pairs = 0;
  last_of_groups(sm, best_key, best_at, M);
#pragma unroll
  for (int j = 0; j < kMost; ++j) {
    if (key[j] == 0 || ahead(sm.last_key, sm.last_at, key[j], at[j])) continue;
    const int to = atomicAdd(&sm.n_pairs, 1);
    sm.pair_key[to] = key[j];
    sm.pair_at[to] = at[j];
  }
  __syncthreads();
}

// Which of its logits of a tile with at least M a lane has among the best M, by total
// and then by place: the M-th largest logit, bit by bit of its place in the
// numbers' order; what has a larger total; then of what has the same one (logits that
// differ by less than its 48 bits are equal) from the front. 2 us for any M.
template <bool F32, bool ALIGNED>
__device__ __noinline__ uint32_t best_of_tile(Beam beam, const uint8_t* row, int t, int vocab, int M, int lane) {
  constexpr int kPer = Tile<F32, ALIGNED>::kPer;
  Tile<F32, ALIGNED> x;
  x.load(row, t, vocab, lane);
  auto count = [&](float least) {
    int n = 0;
#pragma unroll
    for (int j = 0; j < 32; ++j) n += x.at(j) >= least;
    return static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(n)));
  };
  uint32_t order = 0u;
  int at_least = 0;  // how many are `order` or above
#pragma unroll 1
  for (int bit = 31; bit >= 0 && at_least != M; --bit) {
    const int n = count(from_order_bits(order | 1u << bit));  // none for a NaN
    if (n < M) continue;
    order |= 1u << bit;
    at_least = n;
  }
  const float last = from_order_bits(order);
  // Equal totals have logits nearer than this: each total is off by less than 3 2^-48 of it.
  const float near = 0x1p-44f * (fabsf(beam.base.h) + fabsf(beam.top) + fabsf(last));
  uint32_t above = 0u, equal = 0u;
  bool close = false;
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    above |= (x.at(j) > last ? 1u : 0u) << j;
    equal |= (x.at(j) == last ? 1u : 0u) << j;
    close |= x.at(j) != last && fabsf(x.at(j) - last) <= near;
  }
  // Then by the totals (3 us). Above are at most M, and with the equal ones M or more,
  // whatever the totals' last bits are.
  if (__any_sync(0xffffffffu, close)) {
    const uint64_t last_key = total_key(beam, last);
    above = equal = 0u;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const uint64_t key = total_key(beam, x.at(j));
      const bool over = x.at(j) > last && key > last_key;
      above |= (over ? 1u : 0u) << j;
      equal |= (!over && key != 0 && (x.at(j) >= last || key >= last_key) ? 1u : 0u) << j;
    }
  }
  int left = M - static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(__popc(above))));
  // places go by vectors of kPer, then by lanes
#pragma unroll 1
  for (int j = 0; j < 32 && left > 0; j += kPer) {
    uint32_t mine = kPer == 32 ? equal : equal >> j & ((1u << kPer) - 1u);
    const int have = __popc(mine);
    int sum = have;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int other = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += other;
    }
    for (int drop = have - max(min(left - (sum - have), have), 0); drop > 0; --drop) mine &= ~(0x80000000u >> __clz(mine));
    above |= mine << j;
    left -= __shfl_sync(0xffffffffu, sum, 31);
  }
  return above;
}

// i / tiles, given 1 / tiles: i is below 2^14, and (i + 1/2) / tiles at least 2^-11 off
// a whole number.
__device__ __forceinline__ int beam_of(int i, float per_tile) {
  return static_cast<int>((static_cast<float>(i) + 0.5f) * per_tile);
}

// The logits of a sentence's beam k.
template <bool F32>
__device__ __forceinline__ const uint8_t* row_of(const BeamProblem& p, int b, int k) {
  return static_cast<const uint8_t*>(p.logits) + (static_cast<int64_t>(b) * p.beams + k) * p.row_stride * (F32 ? 4 : 2);
}

// The pairs of the listed tiles that are not behind the last one, a warp to a tile,
// the next one's logits on their way. AGAIN: at most M of a tile; else sm.crowded is
// set where a tile has many or they do not fit in the list.
template <bool F32, bool ALIGNED, bool AGAIN>
__device__ __forceinline__ void list_pairs(const BeamProblem& p, int tiles, float per_tile, int b, PickSmem& sm, int M,
                                           uint64_t least_key, int least_at) {
  const int warp = warp_id(), lane = static_cast<int>(lane_id());
  const int listed = sm.n_tiles;
  Tile<F32, ALIGNED> next;
  auto load = [&](int i) {
    const int tile = sm.tile[i], k = beam_of(tile, per_tile);
    next.load(row_of<F32>(p, b, k), tile - k * tiles, p.vocab, lane);
  };
  if (warp < listed) load(warp);
#pragma unroll 1
  for (int i = warp; i < listed; i += kPickWarps) {
    const int tile = sm.tile[i], k = beam_of(tile, per_tile), t = tile - k * tiles;
    const uint8_t* row = row_of<F32>(p, b, k);
    const Tile<F32, ALIGNED> x = next;
    if (i + kPickWarps < listed) load(i + kPickWarps);
    const Beam beam = sm.beam[k];
    // Logits below `least` are not among the best: the logit at which the
    // last one's total is reached, less what this sum of 32 bits may be off.
    const float last = key_total(least_key).h;
    const float slack = 0x1p-21f * (fabsf(last) + fabsf(beam.base.h) + fabsf(beam.top));
    float least = (last - beam.base.h) + beam.top - slack;
    if (least_key == 0 || !(least > -FLT_MAX)) least = -FLT_MAX;
    uint32_t in = 0u;  // of this lane's logits
#pragma unroll
    for (int j = 0; j < 32; ++j) in |= (x.at(j) >= least ? 1u : 0u) << j;
    const int count = static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(__popc(in))));
    if constexpr (AGAIN) {
      if (count > kPairList / kTileList) in = best_of_tile<F32, ALIGNED>(beam, row, t, p.vocab, M, lane);
    } else if (count > M) {
      int claimed = count > kTileMost ? kSpare + 1 : 0;
      if (lane == 0 && claimed == 0) claimed = atomicAdd(&sm.claimed, count) + count;
      if (__shfl_sync(0xffffffffu, claimed, 0) > kSpare) {
        if (lane == 0) sm.crowded = 1;
        break;
      }
    }
#pragma unroll 1
    for (; in != 0u; in &= in - 1u) {
      const int v = Tile<F32, ALIGNED>::place(t, __ffs(in) - 1, lane);
      const uint64_t key = total_key(beam, load_logit<F32>(row, v));
      if (key == 0 || ahead(least_key, least_at, key, k * p.vocab + v)) continue;
      const int at = atomicAdd(&sm.n_pairs, 1);
      sm.pair_key[at] = key;
      sm.pair_at[at] = k * p.vocab + v;
    }
  }
}

// Where a tile has many pairs (no more tiles than M, equal logits), the last one is
// looked for again, among the best of each lane of each tile, and the
// tiles once more.
template <bool F32, bool ALIGNED>
__device__ __noinline__ void look_again(const BeamProblem& p, int tiles, float per_tile, int b, PickSmem& sm, int M,
                                         uint64_t least_key) {
  const int tid = static_cast<int>(threadIdx.x), warp = warp_id(), lane = static_cast<int>(lane_id());
  const int listed = sm.n_tiles;
  int least_at = INT32_MAX;
#pragma unroll 1
  for (int i = warp; i < listed; i += kPickWarps) {
    const int tile = sm.tile[i], k = beam_of(tile, per_tile), t = tile - k * tiles;
    Tile<F32, ALIGNED> x;
    x.load(row_of<F32>(p, b, k), t, p.vocab, lane);
    float best = x.at(0);
#pragma unroll
    for (int j = 1; j < 32; ++j) best = fmaxf(best, x.at(j));
    int best_v = INT32_MAX;
#pragma unroll
    for (int j = 31; j >= 0; --j) {
      const int v = Tile<F32, ALIGNED>::place(t, j, lane);
      if (x.at(j) == best && v < best_v) best_v = v;
    }
    const uint64_t key = best > -INFINITY ? total_key(sm.beam[k], best) : 0;
    const int e = i * 32 + (lane + i) % 32;  // in a group's order in different banks
    sm.pair_key[e] = key;
    sm.pair_at[e] = key != 0 ? k * p.vocab + best_v : INT32_MAX;
  }
  if (tid == 0) sm.n_pairs = 0;
  __syncthreads();
  uint64_t key = 0;
  int at = INT32_MAX;
  // a group: one lane, every other tile (the best may all be in one tile)
#pragma unroll 1
  for (int i = tid / kSubs % 2 + 2 * (tid % kSubs); i < listed; i += 2 * kSubs) {
    const int e = i * 32 + (tid / (2 * kSubs) + i) % 32;
    if (ahead(sm.pair_key[e], sm.pair_at[e], key, at)) {
      key = sm.pair_key[e];
      at = sm.pair_at[e];
    }
  }
  last_of_groups(sm, key, at, M);
  if (sm.last_key != 0) {
    least_key = sm.last_key;
    least_at = sm.last_at;
  }
  list_pairs<F32, ALIGNED, true>(p, tiles, per_tile, b, sm, M, least_key, least_at);
  __syncthreads();
}

// A sum of numbers of 0 .. 2^20 in all over a warp, off by 2^-25 at most: their parts
// above and below 2^-6 as whole numbers, for which a warp has an instruction.
__device__ __forceinline__ Pair warp_sum(float x) {
  const float scaled = x * 64.f, whole = truncf(scaled);
  const unsigned high = __reduce_add_sync(0xffffffffu, static_cast<unsigned>(whole));
  const unsigned low = __reduce_add_sync(0xffffffffu, static_cast<unsigned>((scaled - whole) * 0x1p24f));
  const float h = static_cast<float>(high & 0xffffff00u);  // exact
  return settled(h * 0x1p-6f, static_cast<float>(high & 0xffu) * 0x1p-6f + static_cast<float>(low) * 0x1p-30f);
}

// The choice of sentence b by a block, given its tiles' records: in `records`,
// or (null) in sm.key already.
template <bool F32, bool ALIGNED>
__device__ __forceinline__ void pick(const BeamProblem& p, int tiles, int b, PickSmem& sm, const uint64_t* records) {
  const int K = p.beams;
  const int tid = static_cast<int>(threadIdx.x), warp = warp_id(), lane = static_cast<int>(lane_id());
  const int M = p.end >= 0 ? 2 * K : K;
  const int n = K * tiles;  // below 2^14

  if (records != nullptr) {
#pragma unroll 1
    for (int i0 = tid; i0 < n; i0 += 4 * kPickThreads) {
      unsigned long long r[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i0 + j * kPickThreads < n) r[j] = __ldcg(reinterpret_cast<const unsigned long long*>(records) + i0 + j * kPickThreads);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i0 + j * kPickThreads < n) sm.key[i0 + j * kPickThreads] = r[j];
    }
  }
  // what the last step needs
  float score = -INFINITY, ended = -INFINITY;
  int end_row = 0, end_length = 0;
  if (warp < K) score = __ldcg(p.scores + b * K + warp);
  if (p.end >= 0 && warp == 1 && lane < K) {
    ended = __ldcg(p.ended_scores + b * K + lane);
    end_row = __ldcg(p.ended_rows + b * K + lane);
    end_length = __ldcg(p.ended_lengths + b * K + lane);
  }
  if (tid == 0) {
    sm.n_tiles = sm.n_pairs = sm.claimed = sm.crowded = 0;
  }
  if (tid < 2 * kBeamMaxBeams) sm.best_at[tid] = INT32_MAX;
  int length = 0;
  if (warp == kPickWarps - 1 && p.end >= 0) length = max(__ldcg(p.lengths + b), 1);
  __syncthreads();

  // a row's log-sum, by a warp
  if (warp < K) {
    Beam beam = {{-INFINITY, 0.f}, 0.f};
    if (score != -INFINITY) {
      const float2* st = reinterpret_cast<const float2*>(sm.key) + warp * tiles;
      float top = -INFINITY;
      for (int t = lane; t < tiles; t += 32) top = max_nan(top, st[t].x);
      top = warp_max_nan(top);
      if (!(top < INFINITY) || !(score < INFINITY)) {
        if (lane == 0) atomicOr(&g_device_error, kErrValue);
      } else if (top > -INFINITY) {
        float sum = 0.f;
        for (int t = lane; t < tiles; t += 32) {
          const float2 r = st[t];
          const float d = r.x - top;
          sum = __fmaf_rn(r.y, ex2(__fmaf_rn(d, kLog2eHi, d * kLog2eLo)), sum);
        }
        const Pair log_sum = log_pair(warp_sum(sum));
        beam = {add({score, 0.f}, {-log_sum.h, -log_sum.l}), top};
      }
    }
    if (lane == 0) sm.beam[warp] = beam;
  }
  if (warp == kPickWarps - 1 && p.end >= 0) {  // the last warp mostly has no row
    int exponent;
    const Pair penalty = length_penalty(length, {p.alpha, p.alpha_rest}, &exponent);
    if (lane == 0) {
      sm.length = length;
      sm.penalty = penalty;
      sm.penalty_exponent = exponent;
    }
  }
  __syncthreads();

  // The tiles' largest totals, and the best of each group's.
  const float per_tile = __fdividef(1.f, static_cast<float>(tiles));
  uint64_t group_key = 0;
  int group_tile = INT32_MAX;
#pragma unroll 1
  for (int i = first_of_thread(); i < n; i += kPickThreads) {
    const Beam& beam = sm.beam[beam_of(i, per_tile)];
    uint64_t key = 0;
    if (beam.base.h > -INFINITY) {
      const float x = reinterpret_cast<const float2*>(sm.key)[i].x;
      if (x > -INFINITY) key = total_key(beam, x);
    }
    sm.key[i] = key;
    if (key > group_key) {
      group_key = key;
      group_tile = i;
    }
  }
  // The M-th of them: the tiles that are ahead of it, or are it, hold the M best
  // pairs, and no pair behind it is one.
  last_of_groups(sm, group_key, group_tile, M);
  const uint64_t last_key = sm.last_key;
  const int last_tile = sm.last_at;

  // those tiles. More than the list holds (the best ones in few groups): the
  // best M of it are kept and it is filled again.
#pragma unroll 1
  for (int i0 = 0; i0 < n; i0 += kListStep) {
#pragma unroll 1
    for (int i = i0 + tid; i < min(n, i0 + kListStep); i += kPickThreads) {
      const uint64_t key = sm.key[i];
      if (key != 0 && !ahead(last_key, last_tile, key, i)) {
        const int at = atomicAdd(&sm.n_tiles, 1);
        sm.tile[at] = i;
        sm.tile_key[at] = key;
      }
    }
    __syncthreads();
    const bool more = i0 + kListStep < n;
    if (sm.n_tiles > (more ? kListMost - kListStep : kTileList)) keep_best_tiles(sm, M);
    if (more) __syncthreads();  // all have seen the count before it grows
  }

  // their pairs
  const bool none = n <= M && p.vocab > kTileMost;  // the last one, if there is one, is the worst tile's best
  if (!none) list_pairs<F32, ALIGNED, false>(p, tiles, per_tile, b, sm, M, last_key, INT32_MAX);
  __syncthreads();
  if (none || sm.crowded) look_again<F32, ALIGNED>(p, tiles, per_tile, b, sm, M, last_key);

  // the best M in order (ranks cost the square of the pairs: of 512 40 us)
  if (sm.n_pairs > kFewPairs) keep_best_pairs(sm, M);
  const int pairs = sm.n_pairs;
#pragma unroll 1
  for (int i = warp; i < pairs; i += kPickWarps) {
    const int rank = rank_of(sm.pair_key, sm.pair_at, pairs, i, lane);
    if (lane == 0 && rank < M) {
      sm.best_key[rank] = sm.pair_key[i];
      sm.best_at[rank] = sm.pair_at[i];
    }
  }
  __syncthreads();
  if (warp > 1) return;

  // a lane to a candidate
  const int pair = lane < M ? sm.best_at[lane] : INT32_MAX;
  const bool real = pair != INT32_MAX;
  const Pair total = real ? key_total(sm.best_key[lane]) : Pair{0.f, 0.f};
  const int beam = real ? pair / p.vocab : 0, token = real ? pair - beam * p.vocab : 0;
  const bool ends = real && token == p.end;
  const uint32_t before = (1u << lane) - 1u;
  if (warp == 0) {  // the next beams
    const uint32_t going = __ballot_sync(0xffffffffu, real && !ends);
    const int rank = __popc(going & before);
    if (real && !ends && rank < K) {
      p.tokens[b * K + rank] = token;
      p.parents[b * K + rank] = b * K + beam;
      p.new_scores[b * K + rank] = total.h;
    }
    if (lane < K && lane >= __popc(going)) {  // no pair for this beam
      p.tokens[b * K + lane] = p.end >= 0 ? p.end : 0;
      p.parents[b * K + lane] = b * K + lane;
      p.new_scores[b * K + lane] = -INFINITY;
    }
    return;
  }
  if (p.end < 0) return;

  // the ended hypotheses: lanes below 16 hold the earlier ones, the others this step's
  const uint32_t ending = __ballot_sync(0xffffffffu, ends);
  if (ends) {
    // the quotient of two pairs, rounded once, and the exponent in four steps; of a
    // total near the lowest number (a masked end token's) a quarter is divided, as over a
    // value below 1 it is infinite where with the exponent it is not
    const Pair by = sm.penalty;
    const bool large = fabsf(total.h) > 0x1p100f;
    const float h = large ? 0.25f * total.h : total.h, l = large ? 0.25f * total.l : total.l;
    const float q = __fdividef(h, by.h);
    const float rest = __fmaf_rn(-q, by.h, h) + (l - q * by.l);
    float value = q + __fdividef(rest, by.h);
    int exponent = (large ? 2 : 0) - sm.penalty_exponent;  // within 435
#pragma unroll
    for (int j = 4; j > 0; --j) {
      const int part = exponent / j;
      value *= __int_as_float((127 + part) << 23);
      exponent -= part;
    }
    const int e = __popc(ending & before);  // below K: a beam ends once
    sm.end_score[e] = value;
    sm.end_row[e] = b * K + beam;
  }
  __syncwarp();
  float value = ended;
  if (lane >= kBeamMaxBeams && lane - kBeamMaxBeams < __popc(ending)) {
    value = sm.end_score[lane - kBeamMaxBeams];
    end_row = sm.end_row[lane - kBeamMaxBeams];
    end_length = sm.length;
  }
  if (!(value > -INFINITY)) value = -INFINITY;  // a NaN is no hypothesis
  int place = 0;
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    const float other = __shfl_sync(0xffffffffu, value, j);
    place += other > value || (other == value && j < lane);
  }
  const int held = __popc(__ballot_sync(0xffffffffu, value > -INFINITY));
  if (value > -INFINITY && place < K) {
    p.ended_scores[b * K + place] = value;
    p.ended_rows[b * K + place] = end_row;
    p.ended_lengths[b * K + place] = end_length;
  }
  if (lane < K && lane >= held) p.ended_scores[b * K + lane] = -INFINITY;
}

template <bool F32, bool ALIGNED>
__global__ void __launch_bounds__(kPickThreads) beam_pick_kernel(const BeamProblem p, int tiles) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  griddep_wait();
  griddep_launch_dependents();
  pick<F32, ALIGNED>(p, tiles, static_cast<int>(blockIdx.x), *reinterpret_cast<PickSmem*>(smem_raw),
                     static_cast<const uint64_t*>(p.workspace) + static_cast<int64_t>(blockIdx.x) * p.beams * tiles);
}

// Few tiles to a sentence in one launch: a block to a sentence, or a cluster of 2 to 8
// whose warps have a tile or two each. They take the tiles straight from memory and
// write their records into the first block's shared memory, which then chooses. In us,
// by blocks to a sentence, against two launches (and 2 us less on the host):
//   16 tiles   8 sentences 1: 7.5, two launches 9.0; 300: 15.9, 18.2
//   32         8 2: 6.3, 1: 6.9, two 7.0; 64 2: 7.6, 1: 7.0, two 7.8; 200 1: 14.0, two 14.1
//   64         8 4: 6.4, 2: 7.3, two 7.0; 64 4: 13.9, 2: 8.4, two 8.5; 150 1: 9.2, two 10.9
//   128        8 8: 6.5, 4: 7.3, two 6.9; 16 8: 9.5 (not all clusters fit), 4: 7.5, two 7.4
constexpr int kOneCtas = 8;
template <bool F32, bool ALIGNED>
__global__ void __launch_bounds__(kPickThreads) beam_one_kernel(const BeamProblem p, int tiles, int ctas) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  PickSmem& sm = *reinterpret_cast<PickSmem*>(smem_raw);
  if (ctas > 1) cluster_sync();  // every block has begun: the first one's shared memory may be written
  griddep_wait();
  griddep_launch_dependents();
  const int b = static_cast<int>(blockIdx.x) / ctas, rank = ctas > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int lane = static_cast<int>(lane_id());
  const int n = p.beams * tiles;
  for (int i = warp_id() * ctas + rank; i < n; i += ctas * kPickWarps) {
    const int k = i / tiles, row = b * p.beams + k;
    Tile<F32, ALIGNED> x;
    x.load(static_cast<const uint8_t*>(p.logits) + row * (p.row_stride * (F32 ? 4 : 2)), i - k * tiles, p.vocab, lane);
    if (__ldcg(p.scores + row) == -INFINITY) continue;
    const float2 record = tile_record(x);
    const uint64_t bits = static_cast<uint64_t>(__float_as_uint(record.y)) << 32 | __float_as_uint(record.x);
    if (lane == 0) {
      if (ctas > 1) st_cluster_u64(cluster_map(&sm.key[i], 0), bits);
      else sm.key[i] = bits;
    }
  }
  if (ctas > 1) cluster_sync();
  else __syncthreads();
  if (rank == 0) pick<F32, ALIGNED>(p, tiles, b, sm, nullptr);
}

// Blocks to a sentence of n tiles, or 0: two launches.
int one_launch_blocks(int B, int n, int sms) {
  if (n <= 16) return B <= 2 * sms ? 1 : 0;
  if (n <= 32 && B <= 48) return 2;
  if (n <= 64) return B <= 24 ? 4 : n > 32 && B <= 64 ? 2 : B <= sms ? 1 : 0;
  return n <= kOneCtas * kPickWarps && B <= 8 ? kOneCtas : 0;
}

int sm_count() {
  static int cached = 0;  // atomic accesses: launches may come from several host threads
  int n = __atomic_load_n(&cached, __ATOMIC_RELAXED);
  if (n == 0) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return 1;
    __atomic_store_n(&cached, n, __ATOMIC_RELAXED);
  }
  return n;
}

template <bool F32, bool ALIGNED>
cudaError_t launch_variant(const BeamProblem& p, cudaStream_t stream) {
  using R = Ring<F32, ALIGNED>;
  constexpr int kRingBytes = kTileWarps * static_cast<int>(sizeof(R));
  const int tiles = (p.vocab + kTile - 1) / kTile;
  // the largest call's tiles
  constexpr int kPickMost = static_cast<int>(sizeof(PickSmem)) + kBeamMaxBeams * (kBeamMaxVocab / kTile) * 8;
  static_assert(kPickMost <= 227 * 1024, "shared memory of a block");
  const size_t pick_bytes = sizeof(PickSmem) + static_cast<size_t>(p.beams) * tiles * sizeof(uint64_t);
  const int ctas = one_launch_blocks(p.B, p.beams * tiles, sm_count());
  if (ctas > 0) {
    static unsigned long long one_configured = 0;
    cudaError_t e = set_smem_once(beam_one_kernel<F32, ALIGNED>, kPickMost, &one_configured);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.B * ctas));
    cfg.blockDim = dim3(kPickThreads);
    cfg.dynamicSmemBytes = pick_bytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(ctas);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctas > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, beam_one_kernel<F32, ALIGNED>, p, tiles, ctas);
  }
  static unsigned long long tiles_configured = 0, pick_configured = 0;
  cudaError_t e = set_smem_once(beam_tiles_kernel<F32, ALIGNED>, kRingBytes, &tiles_configured);
  if (e == cudaSuccess) e = set_smem_once(beam_pick_kernel<F32, ALIGNED>, kPickMost, &pick_configured);
  if (e != cudaSuccess) return e;
  static int resident = 0;  // blocks on the device
  int fit = __atomic_load_n(&resident, __ATOMIC_RELAXED);
  if (fit == 0) {
    int per_sm = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, beam_tiles_kernel<F32, ALIGNED>, 32 * kTileWarps, kRingBytes);
    if (e != cudaSuccess) return e;
    fit = sm_count() * (per_sm > 0 ? per_sm : 1);
    __atomic_store_n(&resident, fit, __ATOMIC_RELAXED);
  }
  const int total = p.B * p.beams * ((tiles + R::U - 1) / R::U);
  const int blocks = (total + kTileWarps - 1) / kTileWarps;
  static_assert(kBeamMostTiles <= INT32_MAX - 2 * kTileWarps * 32768, "two rounds of any grid");
  e = launch_pdl(beam_tiles_kernel<F32, ALIGNED>, dim3(static_cast<unsigned>(blocks < fit ? blocks : fit)),
                 dim3(32 * kTileWarps), kRingBytes, stream, p, tiles, total);
  if (e != cudaSuccess) return e;
  return launch_pdl(beam_pick_kernel<F32, ALIGNED>, dim3(static_cast<unsigned>(p.B)), dim3(kPickThreads), pick_bytes,
                    stream, p, tiles);
}

}  // namespace

cudaError_t launch_beam_select(const BeamProblem& p, cudaStream_t stream) {
  const bool aligned = (reinterpret_cast<uintptr_t>(p.logits) & 15u) == 0 && p.row_stride % (p.f32 ? 4 : 8) == 0;
  if (p.f32) return aligned ? launch_variant<true, true>(p, stream) : launch_variant<true, false>(p, stream);
  return aligned ? launch_variant<false, true>(p, stream) : launch_variant<false, false>(p, stream);
}

TSD_DEFINE_ERROR_READER(take_device_error_beam)

}  // namespace tsd
