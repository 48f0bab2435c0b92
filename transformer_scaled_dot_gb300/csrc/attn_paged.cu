// attn_paged.cu -- one decoding step against a paged key/value cache, bf16
// or 4-bit: softmax(scale q K^T) V of each query row over the rows it sees.
//
// A warp per query row walks the cache row by row, the running maximum and
// sum of the softmax in fp32; d / 32 columns per lane.
#include <cuda_bf16.h>

#include "kernels.h"
#include "sm103.cuh"

namespace tsd {

namespace {

__device__ __forceinline__ float bf16_f32(uint16_t w) {
  return __uint_as_float(static_cast<uint32_t>(w) << 16);
}

__device__ __forceinline__ float e2m1_f32(uint32_t code) {
  const uint32_t m = code & 7u;
  const float v = m < 4 ? 0.5f * m : (m == 4 ? 2.f : (m == 5 ? 3.f : (m == 6 ? 4.f : 6.f)));
  return (code & 8u) ? -v : v;
}

__device__ __forceinline__ float e4m3_f32(uint8_t s) {
  uint32_t f2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f2) : "h"(static_cast<uint16_t>(s)));
  float x;
  asm("{.reg .b16 lo, hi; mov.b32 {lo, hi}, %1; cvt.f32.f16 %0, lo;}" : "=f"(x) : "r"(f2));
  return x;
}

template <int D, bool Q4>
__global__ void __launch_bounds__(128) decode_paged_kernel(const PagedDecodeProblem p) {
  constexpr int kCols = D / 32;
  griddep_wait();
  griddep_launch_dependents();
  const PagedCache& c = p.cache;
  const int lane = static_cast<int>(threadIdx.x) & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (row >= static_cast<int64_t>(p.B) * p.h * p.n_q) return;
  const int t = static_cast<int>(row % p.n_q);
  const int head = static_cast<int>(row / p.n_q % p.h);
  const int b = static_cast<int>(row / p.n_q / p.h);
  const int g = head / (p.h / c.h_kv);
  const int capacity = c.max_pages << c.page_shift;
  const int L = c.lens ? min(max(c.lens[b], 0), capacity) : capacity;
  const int m = c.new_lens ? min(max(c.new_lens[b], 0), p.n_q) : p.n_q;
  const int seen = t >= m ? 0 : (p.causal ? L - m + t + 1 : L);  // rows 0 .. seen - 1
  float q[kCols], o[kCols];
#pragma unroll
  for (int i = 0; i < kCols; ++i) {
    q[i] = bf16_f32(p.q[row * D + lane * kCols + i]) * p.scale;
    o[i] = 0.f;
  }
  float top = -INFINITY, sum = 0.f;
  for (int j = 0; j < seen; ++j) {
    const int page = c.table[static_cast<int64_t>(b) * c.max_pages + (j >> c.page_shift)];
    if (page < 0 || page >= c.n_pages) {
      if (lane == 0) atomicOr(&g_device_error, kErrIndex);
      continue;
    }
    const int64_t at = (((static_cast<int64_t>(page) * c.h_kv + g) << c.page_shift) +
                        (j & ((1 << c.page_shift) - 1)));
    float k[kCols], v[kCols];
#pragma unroll
    for (int i = 0; i < kCols; ++i) {
      const int col = lane * kCols + i;
      if constexpr (Q4) {
        const uint8_t kc = static_cast<const uint8_t*>(c.k)[at * (D / 2) + col / 2];
        const uint8_t vc = static_cast<const uint8_t*>(c.v)[at * (D / 2) + col / 2];
        k[i] = e2m1_f32(kc >> (4 * (col & 1))) * e4m3_f32(c.k_scales[at * (D / 16) + col / 16]) *
               c.k_factor;
        v[i] = e2m1_f32(vc >> (4 * (col & 1))) * e4m3_f32(c.v_scales[at * (D / 16) + col / 16]) *
               c.v_factor;
      } else {
        k[i] = bf16_f32(static_cast<const uint16_t*>(c.k)[at * D + col]);
        v[i] = bf16_f32(static_cast<const uint16_t*>(c.v)[at * D + col]);
      }
    }
    float x = 0.f;
#pragma unroll
    for (int i = 0; i < kCols; ++i) x = fmaf(q[i], k[i], x);
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
    const float next = fmaxf(top, x);
    const float keep = top == -INFINITY ? 0.f : __expf(top - next);
    const float w = x == -INFINITY ? 0.f : __expf(x - next);
    sum = sum * keep + w;
#pragma unroll
    for (int i = 0; i < kCols; ++i) o[i] = fmaf(w, v[i], o[i] * keep);
    top = next;
  }
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
  for (int i = 0; i < kCols; ++i)
    reinterpret_cast<__nv_bfloat16*>(p.out)[row * D + lane * kCols + i] =
        __float2bfloat16_rn(o[i] * inv);
}

}  // namespace

size_t decode_paged_workspace_bytes(int, int, int, int, int, int, int) { return 256; }

cudaError_t launch_decode_paged(const PagedDecodeProblem& p, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(p.B) * p.h * p.n_q;
  if (rows < 1 || (rows + 3) / 4 > INT32_MAX) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>((rows + 3) / 4)), block(128);
  const bool q4 = p.cache.k_scales != nullptr;
  if (p.cache.d == 64)
    return launch_pdl(q4 ? decode_paged_kernel<64, true> : decode_paged_kernel<64, false>, grid,
                      block, 0, stream, p);
  if (p.cache.d == 128)
    return launch_pdl(q4 ? decode_paged_kernel<128, true> : decode_paged_kernel<128, false>, grid,
                      block, 0, stream, p);
  return cudaErrorInvalidValue;
}

TSD_DEFINE_ERROR_READER(take_device_error_paged)

}  // namespace tsd
