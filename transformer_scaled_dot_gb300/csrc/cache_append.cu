// cache_append.cu -- writes the new tokens' keys and values into a paged
// key/value cache, rotating queries and keys by their positions on the way.
//
// Token t of sequence b (of m_b new ones) sits at position p = L_b - m_b + t.
// The rotation turns each pair (a, b) of a query's or key's columns by the
// angle that the table's row p gives the pair,
//   a' = a cos - b sin,   b' = b cos + a sin,
// in fp32 (each product and sum rounded by itself), rounded once to bf16.
// A 4-bit cache takes the fp32 values of each group of 16 columns to
//   s = e4m3(max|x| / (6 f)),  code = e2m1(x / (s f)),
// both to nearest even with the largest finite value as the limit (6 is the
// largest code, f the cache's factor); the quotient is a true division, so
// that a value halfway between two codes is found to be halfway. A group
// that holds an infinity or a NaN gets a NaN as its scale.
//
// It moves bytes and does little else: one read of the projections, one
// write of the queries and of the cache rows. A block takes one token; d / 16
// threads take a head's row, each two 16-byte chunks that are a half-rotation
// apart, so that both members of every pair are in one thread and its eight
// cosines and sines are loaded once for all the heads it takes.
#include <cuda_bf16.h>

#include "kernels.h"
#include "sm103.cuh"

namespace tsd {

namespace {

__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// a cos - b sin and b cos + a sin, no product fused into a sum
__device__ __forceinline__ void rotate(float& a, float& b, float c, float s) {
  const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = x;
}

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// The codes of one chunk of 8 columns, given the largest magnitude of its
// group of 16 (as bits, so that infinities and NaN are largest); the group's
// scale byte in `scale`.
__device__ __forceinline__ uint32_t quantise8(const float (&x)[8], uint32_t top, float factor,
                                              uint32_t* scale) {
  if (top >= 0x7f800000u) {
    *scale = 0x7fu;  // NaN
    return 0u;
  }
  const float want = __fdiv_rn(__uint_as_float(top), 6.f * factor);
  uint16_t s2;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(s2) : "f"(0.f), "f"(want));
  *scale = s2 & 0xffu;
  uint32_t f2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f2) : "h"(s2));
  float s;
  asm("{.reg .b16 lo, hi; mov.b32 {lo, hi}, %1; cvt.f32.f16 %0, lo;}" : "=f"(s) : "r"(f2));
  const float unit = __fmul_rn(s, factor);
  uint32_t codes = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float lo = unit > 0.f ? __fdiv_rn(x[2 * i], unit) : 0.f;
    const float hi = unit > 0.f ? __fdiv_rn(x[2 * i + 1], unit) : 0.f;
    uint32_t two;
    asm("{.reg .b8 c; cvt.rn.satfinite.e2m1x2.f32 c, %1, %2; cvt.u32.u8 %0, c;}"
        : "=r"(two) : "f"(hi), "f"(lo));
    codes |= two << (8 * i);
  }
  return codes;
}

// One block per token. kThreads / (D / 16) heads are taken at a time.
template <int D, bool Q4>
__global__ void cache_append_kernel(const AppendProblem p) {
  constexpr int kLanes = D / 16;  // threads of a row
  griddep_wait();  // inputs, lengths and tables may come from the previous kernel
  griddep_launch_dependents();
  const int b = static_cast<int>(blockIdx.x / static_cast<uint32_t>(p.n_new));
  const int t = static_cast<int>(blockIdx.x % static_cast<uint32_t>(p.n_new));
  const PagedCache& c = p.cache;
  const int m = c.new_lens ? min(max(c.new_lens[b], 0), p.n_new) : p.n_new;
  if (t >= m) return;
  const int64_t pos = static_cast<int64_t>(c.lens[b]) - m + t;
  if (pos < 0) return;
  int page = -1;
  if ((pos >> c.page_shift) < c.max_pages && (p.rope_kind == 0 || pos < p.rope_rows))
    page = c.table[static_cast<int64_t>(b) * c.max_pages + (pos >> c.page_shift)];
  if (page < 0 || page >= c.n_pages) {
    if (threadIdx.x == 0) atomicOr(&g_device_error, kErrIndex);
    return;
  }
  const int64_t page_size = 1ll << c.page_shift;
  const int64_t slot = pos & (page_size - 1);
  const int lane = static_cast<int>(threadIdx.x) % kLanes;

  // this thread's chunks (of 8 columns): the rotated columns' first and
  // second half side by side, likewise the columns past them
  const bool halves = p.rope_kind == kRopeHalves;
  const int half = (halves ? p.rope_dim : D) / 16;  // chunks of one half
  const int c0 = lane < half ? lane : half + lane;
  const int c1 = c0 + (lane < half ? half : kLanes - half);
  // cosines and sines: of the pairs (c0 * 8 + i, c1 * 8 + i), or of each
  // chunk's four neighbouring pairs
  float cs[8], sn[8];
  bool turn0 = false, turn1 = false;
  if (halves) {
    turn0 = turn1 = lane < half;
    if (turn0) {
      const float* r = p.rope + pos * p.rope_dim + 8 * c0;
#pragma unroll
      for (int i = 0; i < 8; ++i) cs[i] = r[i], sn[i] = r[i + p.rope_dim / 2];
    }
  } else if (p.rope_kind == kRopePairs) {
    turn0 = 8 * c0 < p.rope_dim;
    turn1 = 8 * c1 < p.rope_dim;
    const float* r = p.rope + pos * p.rope_dim;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (turn0) cs[i] = r[4 * c0 + i], sn[i] = r[4 * c0 + i + p.rope_dim / 2];
      if (turn1) cs[4 + i] = r[4 * c1 + i], sn[4 + i] = r[4 * c1 + i + p.rope_dim / 2];
    }
  }

  const int rows_q = p.q ? p.h : 0;
  const int rows = rows_q + 2 * c.h_kv;
  const int step = static_cast<int>(blockDim.x) / kLanes;
  // every thread takes the same number of rounds: a group's two threads
  // exchange their maxima
  for (int base = 0; base < rows; base += step) {
    const int row = base + static_cast<int>(threadIdx.x) / kLanes;
    const bool live = row < rows;
    const bool is_q = row < rows_q, is_v = row >= rows_q + c.h_kv;
    const int head = is_q ? row : (is_v ? row - rows_q - c.h_kv : row - rows_q);
    float x0[8], x1[8];
    if (live) {
      const uint16_t* src =
          is_q ? p.q + b * p.q_sb + head * p.q_sh + t * p.q_sr
               : (is_v ? p.v : p.k) + b * p.kv_sb + head * p.kv_sh + t * p.kv_sr;
      unpack8(*reinterpret_cast<const uint4*>(src + 8 * c0), x0);
      unpack8(*reinterpret_cast<const uint4*>(src + 8 * c1), x1);
      if (!is_v) {
        if (halves) {
          if (turn0) {
#pragma unroll
            for (int i = 0; i < 8; ++i) rotate(x0[i], x1[i], cs[i], sn[i]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (turn0) rotate(x0[2 * i], x0[2 * i + 1], cs[i], sn[i]);
            if (turn1) rotate(x1[2 * i], x1[2 * i + 1], cs[4 + i], sn[4 + i]);
          }
        }
      }
      if (is_q || (!is_v && p.k_out != nullptr)) {
        uint16_t* dst = is_q ? p.q_out + ((static_cast<int64_t>(b) * p.h + head) * p.n_new + t) * D
                             : p.k_out + ((static_cast<int64_t>(b) * c.h_kv + head) * p.n_new + t) * D;
        *reinterpret_cast<uint4*>(dst + 8 * c0) = pack8(x0);
        *reinterpret_cast<uint4*>(dst + 8 * c1) = pack8(x1);
      }
    }
    const int64_t at = (static_cast<int64_t>(page) * c.h_kv + head) * page_size + slot;
    if constexpr (!Q4) {
      if (live && !is_q) {
        uint16_t* dst = static_cast<uint16_t*>(is_v ? c.v : c.k) + at * D;
        *reinterpret_cast<uint4*>(dst + 8 * c0) = pack8(x0);
        *reinterpret_cast<uint4*>(dst + 8 * c1) = pack8(x1);
      }
    } else {
      // a group of 16 columns is chunk c0 (c1) of this thread and its neighbour
      uint32_t top0 = 0, top1 = 0;
      if (live && !is_q) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          top0 = max(top0, abs_bits(x0[i]));
          top1 = max(top1, abs_bits(x1[i]));
        }
      }
      top0 = max(top0, __shfl_xor_sync(0xffffffffu, top0, 1));
      top1 = max(top1, __shfl_xor_sync(0xffffffffu, top1, 1));
      if (live && !is_q) {
        const float f = is_v ? c.v_factor : c.k_factor;
        uint8_t* codes = static_cast<uint8_t*>(is_v ? c.v : c.k) + at * (D / 2);
        uint8_t* scales = (is_v ? c.v_scales : c.k_scales) + at * (D / 16);
        uint32_t s0, s1;
        *reinterpret_cast<uint32_t*>(codes + 4 * c0) = quantise8(x0, top0, f, &s0);
        *reinterpret_cast<uint32_t*>(codes + 4 * c1) = quantise8(x1, top1, f, &s1);
        if ((lane & 1) == 0) {
          scales[c0 / 2] = static_cast<uint8_t>(s0);
          scales[c1 / 2] = static_cast<uint8_t>(s1);
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_cache_append(const AppendProblem& p, cudaStream_t stream) {
  const int64_t tokens = static_cast<int64_t>(p.B) * p.n_new;
  if (tokens < 1 || tokens > INT32_MAX) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(tokens)), block(128);
  const bool q4 = p.cache.k_scales != nullptr;
  if (p.cache.d == 64)
    return launch_pdl(q4 ? cache_append_kernel<64, true> : cache_append_kernel<64, false>, grid,
                      block, 0, stream, p);
  if (p.cache.d == 128)
    return launch_pdl(q4 ? cache_append_kernel<128, true> : cache_append_kernel<128, false>, grid,
                      block, 0, stream, p);
  return cudaErrorInvalidValue;
}

TSD_DEFINE_ERROR_READER(take_device_error_append)

}  // namespace tsd
