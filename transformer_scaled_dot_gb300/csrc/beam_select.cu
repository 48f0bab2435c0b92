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
// and then the M pairs in them.
// Totals that lie next to one another decide which token a beam takes: they
// are formed and compared in 64 bits. Exponentials and a tile's sum are in 32,
// relative to the tile's own maximum, as are the few tiles of a lane that joins
// them; lanes are joined in 64.
#include <cfloat>

#include "kernels.h"
#include "sm103.cuh"

namespace tsd {

namespace {

constexpr int kTile = kBeamTile;          // logits of a warp's tile
constexpr int kTileWarps = 8;             // warps of a beam_tiles block
constexpr int kPickThreads = 512;
constexpr int kPickWarps = kPickThreads / 32;
static_assert(kPickWarps >= kBeamMaxBeams, "a warp joins a row's tiles");

template <bool F32>
__device__ __forceinline__ float load_logit(const void* p, int64_t at) {
  if constexpr (F32) return static_cast<const float*>(p)[at];
  return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[at]) << 16);
}

// 32 logits of a lane. Aligned: 16-byte loads, lane l of load j holds the
// consecutive ones from (32 j + l) * (16 / size); otherwise one logit to a
// load, number 32 j + l. Past the row's end -infinity.
template <bool F32, bool ALIGNED>
__device__ __forceinline__ int tile_place(int t, int i, int lane) {
  constexpr int kPer = F32 ? 4 : 8;
  return t * kTile + (ALIGNED ? (i / kPer * 32 + lane) * kPer + i % kPer : i * 32 + lane);
}
template <bool F32, bool ALIGNED>
__device__ __forceinline__ void load_tile(const void* row, int t, int vocab, int lane, float (&x)[32]) {
  const int base = t * kTile;
  if constexpr (!ALIGNED) {
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const int v = base + j * 32 + lane;
      x[j] = v < vocab ? load_logit<F32>(row, v) : -INFINITY;
    }
  } else {
    constexpr int kPer = F32 ? 4 : 8;
#pragma unroll
    for (int j = 0; j < 32 / kPer; ++j) {
      const int v = base + (j * 32 + lane) * kPer;
      if (v + kPer <= vocab) {
        const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(row) + static_cast<int64_t>(v) * (16 / kPer));
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (F32) {
            x[j * kPer + i] = __uint_as_float(u[i]);
          } else {
            x[j * kPer + 2 * i] = __uint_as_float(u[i] << 16);
            x[j * kPer + 2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) x[j * kPer + i] = v + i < vocab ? load_logit<F32>(row, v + i) : -INFINITY;
      }
    }
  }
}

__device__ __forceinline__ float max_nan(float a, float b) {
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(a) : "f"(b));
  return a;
}
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(a) : "f"(b), "f"(c));
  return a;
}

// log2(e) as two numbers of 32 bits
constexpr float kLog2eHi = 1.4426950216293335f, kLog2eLo = 1.9259629911266175e-8f;

template <bool F32, bool ALIGNED>
__global__ void __launch_bounds__(32 * kTileWarps)
    beam_tiles_kernel(const BeamProblem p, int tiles, int total) {
  griddep_wait();
  griddep_launch_dependents();
  const int id = static_cast<int>(blockIdx.x) * kTileWarps + warp_id();
  if (id >= total) return;
  const int lane = static_cast<int>(lane_id());
  const int row = id / tiles, t = id % tiles;
  if (__ldcg(p.scores + row) == -INFINITY) return;  // no live hypothesis: beam_pick does not look here
  const uint8_t* x_row = static_cast<const uint8_t*>(p.logits) + row * p.row_stride * (F32 ? 4 : 2);
  float x[32];
  load_tile<F32, ALIGNED>(x_row, t, p.vocab, lane, x);
  float top = x[0];
#pragma unroll
  for (int i = 1; i < 31; i += 2) top = max3_nan(top, x[i], x[i + 1]);
  top = max_nan(top, x[31]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
  // the difference first, so that its rounding is its own (none for bf16 near the maximum)
  const float m = top == -INFINITY ? 0.f : top;
  const uint64_t neg = f2_pack(-m, -m), hi = f2_pack(kLog2eHi, kLog2eHi), lo = f2_pack(kLog2eLo, kLog2eLo);
  uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint64_t d = fadd2(f2_pack(x[2 * i], x[2 * i + 1]), neg);
    float a, b;
    f2_unpack(ffma2(d, hi, fmul2(d, lo)), a, b);
    sum[i & 1] = fadd2(sum[i & 1], f2_pack(ex2(a), ex2(b)));
  }
  float a, b;
  f2_unpack(fadd2(sum[0], sum[1]), a, b);
  float s = a + b;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) reinterpret_cast<float2*>(p.workspace)[id] = make_float2(top, s);
}

// Totals of 64 bits as whole numbers in the same order; 0: none.
__device__ __forceinline__ uint64_t order_key(double total) {
  const int64_t bits = __double_as_longlong(total + 0.0);  // -0 is 0
  return static_cast<uint64_t>(bits < 0 ? ~bits : bits | INT64_MIN);
}
__device__ __forceinline__ double key_total(uint64_t key) {
  const int64_t bits = static_cast<int64_t>(key);
  return __longlong_as_double(bits < 0 ? bits & INT64_MAX : ~bits);
}
// Whether a is ahead of b: by total, then by place.
__device__ __forceinline__ bool ahead(uint64_t a_key, int a_at, uint64_t b_key, int b_at) {
  return a_key > b_key || (a_key == b_key && a_at < b_at);
}

constexpr int kGroups = 128;    // of a sentence's tiles, each within a row
constexpr int kSubs = kPickThreads / kGroups;  // threads of a group
constexpr int kTileList = 64;   // chosen tiles that are looked through
constexpr int kPairList = kTileList * 2 * kBeamMaxBeams;

struct PickSmem {
  // total = base + (logit - top): no digits are lost where logits are large
  double base[kBeamMaxBeams];  // s_k - log sum exp(x - top); -infinity: no live hypothesis
  double top[kBeamMaxBeams];   // the row's largest logit
  float least[kBeamMaxBeams];  // logits of this beam below it are not among the best
  float group_top[kGroups];
  int group_tile[kGroups];
  uint64_t group_key[kGroups];
  uint64_t last_key;           // the M-th best group's largest total, and its tile
  int last_tile;
  int n_tiles, n_pairs;
  int tile[2 * kPickThreads];  // chosen tiles
  uint64_t tile_key[2 * kPickThreads];
  uint64_t pair_key[kPairList];
  int pair_at[kPairList];
  uint64_t best_key[2 * kBeamMaxBeams];
  int best_at[2 * kBeamMaxBeams];
  float end_score[2 * kBeamMaxBeams];
  int end_row[kBeamMaxBeams];
};

// Of n entries how many are ahead of entry i, by a warp.
__device__ __forceinline__ int rank_of(const uint64_t* key, const int* at, int n, int i, int lane) {
  int before = 0;
  for (int j = lane; j < n; j += 32) before += ahead(key[j], at[j], key[i], at[i]);
  return static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(before)));
}

template <bool F32, bool ALIGNED>
__global__ void __launch_bounds__(kPickThreads) beam_pick_kernel(const BeamProblem p, int tiles) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  PickSmem& sm = *reinterpret_cast<PickSmem*>(smem_raw);
  griddep_wait();
  griddep_launch_dependents();
  const int b = static_cast<int>(blockIdx.x), K = p.beams;
  const int tid = static_cast<int>(threadIdx.x), warp = warp_id(), lane = static_cast<int>(lane_id());
  const int M = p.end >= 0 ? 2 * K : K;
  const float2* tile_stats = reinterpret_cast<const float2*>(p.workspace) + static_cast<int64_t>(b) * K * tiles;

  // The largest logit of each group of tiles (of its lowest tile among equal
  // ones): beam group / per_beam, every per_beam-th tile of its row. The loads
  // do not wait for the log-sums.
  const int per_beam = kGroups / K;
  const int group = tid / kSubs, sub = tid % kSubs;
  const int group_beam = group / per_beam;
  float group_top = -INFINITY;
  int group_tile = INT32_MAX;
  if (group_beam < K && __ldcg(p.scores + b * K + group_beam) != -INFINITY) {
    const float2* st = tile_stats + static_cast<int64_t>(group_beam) * tiles;
#pragma unroll 4
    for (int t = group % per_beam + per_beam * sub; t < tiles; t += per_beam * kSubs) {
      const float x = __ldcg(&st[t].x);
      if (x > group_top) {
        group_top = x;
        group_tile = group_beam * tiles + t;
      }
    }
  }
#pragma unroll
  for (int o = 1; o < kSubs; o <<= 1) {
    const float x = __shfl_xor_sync(0xffffffffu, group_top, o);
    const int t = __shfl_xor_sync(0xffffffffu, group_tile, o);
    if (x > group_top || (x == group_top && t < group_tile)) {
      group_top = x;
      group_tile = t;
    }
  }
  if (sub == 0) {
    sm.group_top[group] = group_top;
    sm.group_tile[group] = group_tile;
  }
  if (tid == 0) {
    sm.n_tiles = sm.n_pairs = 0;
    sm.last_key = 0;
    sm.last_tile = INT32_MAX;
  }

  // a row's log-sum, by a warp: eight tiles to a lane at a time
  if (warp < K) {
    const float score = __ldcg(p.scores + b * K + warp);
    double base = -INFINITY;
    if (score != -INFINITY) {
      const float2* st = tile_stats + static_cast<int64_t>(warp) * tiles;
      float top = -INFINITY, sum = 0.f;
      for (int t0 = 0; t0 < tiles; t0 += 256) {
        float2 r[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int t = t0 + j * 32 + lane;
          r[j] = t < tiles ? __ldcg(&st[t]) : make_float2(-INFINITY, 0.f);
        }
        float now = top;
#pragma unroll
        for (int j = 0; j < 8; ++j) now = max_nan(now, r[j].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) now = max_nan(now, __shfl_xor_sync(0xffffffffu, now, o));
        if (!(now > -INFINITY && now < INFINITY)) {  // nothing yet, or no numbers
          top = now;
          continue;
        }
        auto weight = [&](float x) {
          const float d = x - now;
          return ex2(__fmaf_rn(d, kLog2eHi, d * kLog2eLo));
        };
        sum *= weight(top);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = __fmaf_rn(r[j].y, weight(r[j].x), sum);
        top = now;
      }
      if (!(top < INFINITY) || !(score < INFINITY)) {
        if (lane == 0) atomicOr(&g_device_error, kErrValue);
      } else if (top > -INFINITY) {
        double all = sum;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
        base = static_cast<double>(score) - log(all);
        if (lane == 0) sm.top[warp] = top;
      }
    }
    if (lane == 0) sm.base[warp] = base;
  }
  __syncthreads();

  // the groups' totals, and the M-th of them: the pairs that are ahead of it
  // or are it include the M best, and lie in tiles of which the same holds
  if (tid < kGroups) {
    const int tile = sm.group_tile[tid];
    uint64_t key = 0;
    if (tile != INT32_MAX) {
      const int k = tid / per_beam;
      if (sm.base[k] > -INFINITY) key = order_key(sm.base[k] + (sm.group_top[tid] - sm.top[k]));
    }
    sm.group_key[tid] = key;
  }
  __syncthreads();
  for (int i = warp; i < kGroups; i += kPickWarps) {
    if (sm.group_key[i] == 0) continue;
    if (rank_of(sm.group_key, sm.group_tile, kGroups, i, lane) == M - 1) {
      if (lane == 0) {
        sm.last_key = sm.group_key[i];
        sm.last_tile = sm.group_tile[i];
      }
      // lowered by what the sums may be off in 64 bits, and rounded down
      if (lane < K) {
        const double last = key_total(sm.group_key[i]), base = sm.base[lane], top = sm.top[lane];
        sm.least[lane] = __double2float_rd(fma(-0x1p-49, fabs(last) + fabs(base) + fabs(top), last - base + top));
      }
    }
  }
  __syncthreads();
  const uint64_t last_key = sm.last_key;
  const int last_tile = sm.last_tile;

  // those tiles. More than the list holds (the best ones in few groups): the
  // best M of it are kept and it is filled again.
  const int n = K * tiles;
  auto keep_best_tiles = [&]() {
    const int listed = sm.n_tiles;
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
  };
  for (int i0 = 0; i0 < n; i0 += kPickThreads) {
    const int i = i0 + tid, k = i / tiles;
    if (i < n && sm.base[k] > -INFINITY) {
      const float x = __ldcg(&tile_stats[i].x);
      if (x > -INFINITY && (last_key == 0 || x >= sm.least[k])) {
        const uint64_t key = order_key(sm.base[k] + (x - sm.top[k]));
        if (!ahead(last_key, last_tile, key, i)) {
          const int at = atomicAdd(&sm.n_tiles, 1);
          sm.tile[at] = i;
          sm.tile_key[at] = key;
        }
      }
    }
    if (i0 + kPickThreads < n || n > kTileList) {
      __syncthreads();
      const int listed = sm.n_tiles;
      __syncthreads();
      if (listed > (i0 + kPickThreads < n ? kPickThreads : kTileList)) keep_best_tiles();
    }
  }
  __syncthreads();

  // their pairs, a warp to a tile
  const int listed = sm.n_tiles;
  for (int i = warp; i < listed; i += kPickWarps) {
    const int tile = sm.tile[i], k = tile / tiles, t = tile % tiles;
    const uint8_t* row = static_cast<const uint8_t*>(p.logits) +
                         (static_cast<int64_t>(b) * K + k) * p.row_stride * (F32 ? 4 : 2);
    const float least = last_key == 0 ? -FLT_MAX : sm.least[k];
    float x[32];
    load_tile<F32, ALIGNED>(row, t, p.vocab, lane, x);
    uint32_t in = 0u;  // of this lane's logits
#pragma unroll
    for (int j = 0; j < 32; ++j) in |= (x[j] >= least ? 1u : 0u) << j;
    auto push = [&](int j) {
      const int v = tile_place<F32, ALIGNED>(t, j, lane);
      const int at = atomicAdd(&sm.n_pairs, 1);
      sm.pair_key[at] = order_key(sm.base[k] + (load_logit<F32>(row, v) - sm.top[k]));
      sm.pair_at[at] = k * p.vocab + v;
    };
    if (__reduce_add_sync(0xffffffffu, __popc(in)) <= static_cast<unsigned>(M)) {
      for (; in != 0u; in &= in - 1u) push(__ffs(in) - 1);
    } else {
      // more than M, as with many equal logits: the best M one by one
      for (int r = 0; r < M; ++r) {
        float best = -INFINITY;
        int best_j = 0, best_v = INT32_MAX;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const int v = tile_place<F32, ALIGNED>(t, j, lane);
          if ((in >> j & 1u) && (x[j] > best || (x[j] == best && v < best_v))) {
            best = x[j];
            best_j = j;
            best_v = v;
          }
        }
        float top = best;
        int top_v = best_v;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          const float other = __shfl_xor_sync(0xffffffffu, top, o);
          const int other_v = __shfl_xor_sync(0xffffffffu, top_v, o);
          if (other > top || (other == top && other_v < top_v)) {
            top = other;
            top_v = other_v;
          }
        }
        if (best_v == top_v) {
          push(best_j);
          in &= ~(1u << best_j);
        }
      }
    }
  }
  __syncthreads();

  // the best M in order
  const int pairs = sm.n_pairs;
  if (tid < 2 * kBeamMaxBeams) sm.best_at[tid] = INT32_MAX;
  __syncthreads();
  for (int i = warp; i < pairs; i += kPickWarps) {
    const int rank = rank_of(sm.pair_key, sm.pair_at, pairs, i, lane);
    if (lane == 0 && rank < M) {
      sm.best_key[rank] = sm.pair_key[i];
      sm.best_at[rank] = sm.pair_at[i];
    }
  }
  __syncthreads();
  if (warp != 0) return;

  // a lane to a candidate: the next beams
  const int pair = lane < M ? sm.best_at[lane] : INT32_MAX;
  const bool real = pair != INT32_MAX;
  const double pair_total = real ? key_total(sm.best_key[lane]) : 0.0;
  const int beam = real ? pair / p.vocab : 0, token = real ? pair % p.vocab : 0;
  const bool ends = real && token == p.end;
  const uint32_t before = (1u << lane) - 1u;
  const uint32_t going = __ballot_sync(0xffffffffu, real && !ends), ending = __ballot_sync(0xffffffffu, ends);
  const int rank = __popc(going & before);
  if (real && !ends && rank < K) {
    p.tokens[b * K + rank] = token;
    p.parents[b * K + rank] = b * K + beam;
    p.new_scores[b * K + rank] = static_cast<float>(pair_total);
  }
  if (lane < K && lane >= __popc(going)) {  // no pair for this beam
    p.tokens[b * K + lane] = p.end >= 0 ? p.end : 0;
    p.parents[b * K + lane] = b * K + lane;
    p.new_scores[b * K + lane] = -INFINITY;
  }
  if (p.end < 0) return;

  // the ended hypotheses: lanes below 16 hold the earlier ones, the others this step's
  const int length = max(__ldcg(p.lengths + b), 1);
  if (ends) {
    const double norm = pow((5.0 + length) / 6.0, static_cast<double>(p.alpha));
    const int e = __popc(ending & before);  // below K: a beam ends once
    sm.end_score[e] = static_cast<float>(pair_total / norm);
    sm.end_row[e] = b * K + beam;
  }
  __syncwarp();
  float value = -INFINITY;
  int end_row = 0, end_length = length;
  if (lane < kBeamMaxBeams) {
    if (lane < K) {
      value = __ldcg(p.ended_scores + b * K + lane);
      end_row = __ldcg(p.ended_rows + b * K + lane);
      end_length = __ldcg(p.ended_lengths + b * K + lane);
    }
  } else if (lane - kBeamMaxBeams < __popc(ending)) {
    value = sm.end_score[lane - kBeamMaxBeams];
    end_row = sm.end_row[lane - kBeamMaxBeams];
  }
  if (!(value > -INFINITY)) value = -INFINITY;  // a NaN is no hypothesis
  int place = 0;
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
cudaError_t launch_variant(const BeamProblem& p, cudaStream_t stream) {
  const int tiles = (p.vocab + kTile - 1) / kTile;
  const int total = p.B * p.beams * tiles;
  static unsigned long long configured = 0;
  cudaError_t e = set_smem_once(beam_pick_kernel<F32, ALIGNED>, sizeof(PickSmem), &configured);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>((total + kTileWarps - 1) / kTileWarps));
  e = launch_pdl(beam_tiles_kernel<F32, ALIGNED>, grid, dim3(32 * kTileWarps), 0, stream, p, tiles, total);
  if (e != cudaSuccess) return e;
  return launch_pdl(beam_pick_kernel<F32, ALIGNED>, dim3(static_cast<unsigned>(p.B)), dim3(kPickThreads), sizeof(PickSmem),
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
