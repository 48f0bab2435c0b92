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
// relative to the tile's own maximum; tiles are joined in 64.
#include <cuda_bf16.h>

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

struct Best {
  double total;
  int at;
};
// Whether a is ahead of b: by total, then by place. Neither is a NaN.
__device__ __forceinline__ bool ahead(const Best& a, const Best& b) {
  return a.total > b.total || (a.total == b.total && a.at < b.at);
}

struct PickSmem {
  // total = base + (logit - top): no digits are lost where logits are large
  double base[kBeamMaxBeams];  // s_k - log sum exp(x - top); -infinity: no live hypothesis
  double top[kBeamMaxBeams];   // the row's largest logit
  Best warp_best[kPickWarps];
  Best tiles[2 * kBeamMaxBeams];
  Best pairs[2 * kBeamMaxBeams];
  float end_score[2 * kBeamMaxBeams];
  int end_row[kBeamMaxBeams];
};

// The best of all threads' `mine`, in every thread.
__device__ __forceinline__ Best block_best(Best mine, PickSmem& sm) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Best other;
    other.total = __shfl_xor_sync(0xffffffffu, mine.total, o);
    other.at = __shfl_xor_sync(0xffffffffu, mine.at, o);
    if (ahead(other, mine)) mine = other;
  }
  __syncthreads();
  if (lane_id() == 0) sm.warp_best[warp_id()] = mine;
  __syncthreads();
  Best best = sm.warp_best[0];
  for (int w = 1; w < kPickWarps; ++w)
    if (ahead(sm.warp_best[w], best)) best = sm.warp_best[w];
  return best;
}

constexpr Best kNone = {-INFINITY, INT32_MAX};

template <bool F32>
__global__ void __launch_bounds__(kPickThreads) beam_pick_kernel(const BeamProblem p, int tiles) {
  __shared__ PickSmem sm;
  griddep_wait();
  griddep_launch_dependents();
  const int b = static_cast<int>(blockIdx.x), K = p.beams;
  const int tid = static_cast<int>(threadIdx.x), warp = warp_id(), lane = static_cast<int>(lane_id());
  const int M = p.end >= 0 ? 2 * K : K;
  const float2* tile_stats = reinterpret_cast<const float2*>(p.workspace) + static_cast<int64_t>(b) * K * tiles;

  if (warp < K) {
    const float score = __ldcg(p.scores + b * K + warp);
    double base = -INFINITY;
    if (score != -INFINITY) {
      const float2* st = tile_stats + static_cast<int64_t>(warp) * tiles;
      float top = -INFINITY;
      for (int t = lane; t < tiles; t += 32) top = max_nan(top, __ldcg(&st[t]).x);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
      if (!(top < INFINITY) || !(score < INFINITY)) {
        if (lane == 0) atomicOr(&g_device_error, kErrValue);
      } else if (top > -INFINITY) {
        double sum = 0.0;
        for (int t = lane; t < tiles; t += 32) {
          const float2 r = __ldcg(&st[t]);
          const float d = r.x - top;
          sum += static_cast<double>(r.y * ex2(__fmaf_rn(d, kLog2eHi, d * kLog2eLo)));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        base = static_cast<double>(score) - log(sum);
        if (lane == 0) sm.top[warp] = top;
      }
    }
    if (lane == 0) sm.base[warp] = base;
  }
  __syncthreads();

  // the M tiles with the best maxima
  const int n = K * tiles;  // at most 32 to a thread
  uint32_t gone = 0u;
  auto best_tile = [&]() {
    Best best = kNone;
    for (int j = 0, i = tid; i < n; ++j, i += kPickThreads) {
      const int k = i / tiles;
      if (sm.base[k] == -INFINITY || (gone >> j & 1u)) continue;
      const Best one = {sm.base[k] + (__ldcg(&tile_stats[i]).x - sm.top[k]), i};
      if (one.total > -INFINITY && ahead(one, best)) best = one;
    }
    return best;
  };
  Best mine = best_tile();
  for (int r = 0; r < M; ++r) {
    const Best best = block_best(mine, sm);
    if (tid == 0) sm.tiles[r] = best;
    if (best.at != INT32_MAX && best.at % kPickThreads == tid) {
      gone |= 1u << (best.at / kPickThreads);
      mine = best_tile();
    }
  }
  __syncthreads();

  // the M best pairs in them: 2 M pairs to a thread
  uint64_t taken = 0ull;
  auto best_pair = [&]() {
    Best best = kNone;
    for (int j = 0; j < M * (kTile / kPickThreads); ++j) {
      const int i = j * kPickThreads + tid;
      const int tile = sm.tiles[i / kTile].at;
      if (tile == INT32_MAX || (taken >> j & 1ull)) continue;
      const int k = tile / tiles, v = tile % tiles * kTile + i % kTile;
      if (v >= p.vocab) continue;
      const int64_t at = (static_cast<int64_t>(b) * K + k) * p.row_stride + v;
      const Best one = {sm.base[k] + (load_logit<F32>(p.logits, at) - sm.top[k]), k * p.vocab + v};
      if (one.total > -INFINITY && ahead(one, best)) best = one;
    }
    return best;
  };
  mine = best_pair();
  for (int r = 0; r < M; ++r) {
    const Best best = block_best(mine, sm);
    if (tid == 0) sm.pairs[r] = best;
    if (best.at != INT32_MAX && best.at == mine.at) {
      // its place among this thread's pairs
      for (int j = 0; j < M * (kTile / kPickThreads); ++j) {
        const int i = j * kPickThreads + tid;
        const int tile = sm.tiles[i / kTile].at;
        if (tile != INT32_MAX && tile / tiles * p.vocab + tile % tiles * kTile + i % kTile == best.at) taken |= 1ull << j;
      }
      mine = best_pair();
    }
  }
  __syncthreads();
  if (warp != 0) return;

  // a lane to a candidate: the next beams
  const Best mine_pair = lane < M ? sm.pairs[lane] : kNone;
  const bool real = mine_pair.at != INT32_MAX;
  const int beam = real ? mine_pair.at / p.vocab : 0, token = real ? mine_pair.at % p.vocab : 0;
  const bool ends = real && token == p.end;
  const uint32_t before = (1u << lane) - 1u;
  const uint32_t going = __ballot_sync(0xffffffffu, real && !ends), ending = __ballot_sync(0xffffffffu, ends);
  const int rank = __popc(going & before);
  if (real && !ends && rank < K) {
    p.tokens[b * K + rank] = token;
    p.parents[b * K + rank] = b * K + beam;
    p.new_scores[b * K + rank] = static_cast<float>(mine_pair.total);
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
    sm.end_score[e] = static_cast<float>(mine_pair.total / norm);
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

template <bool F32>
cudaError_t launch_type(const BeamProblem& p, cudaStream_t stream) {
  const int tiles = (p.vocab + kTile - 1) / kTile;
  const int total = p.B * p.beams * tiles;
  const int per = F32 ? 4 : 8;
  const bool aligned = (reinterpret_cast<uintptr_t>(p.logits) & 15u) == 0 && p.row_stride % per == 0;
  const dim3 grid(static_cast<unsigned>((total + kTileWarps - 1) / kTileWarps));
  cudaError_t e = launch_pdl(aligned ? beam_tiles_kernel<F32, true> : beam_tiles_kernel<F32, false>, grid,
                             dim3(32 * kTileWarps), 0, stream, p, tiles, total);
  if (e != cudaSuccess) return e;
  return launch_pdl(beam_pick_kernel<F32>, dim3(static_cast<unsigned>(p.B)), dim3(kPickThreads), 0, stream, p, tiles);
}

}  // namespace

cudaError_t launch_beam_select(const BeamProblem& p, cudaStream_t stream) {
  return p.f32 ? launch_type<true>(p, stream) : launch_type<false>(p, stream);
}

TSD_DEFINE_ERROR_READER(take_device_error_beam)

}  // namespace tsd
