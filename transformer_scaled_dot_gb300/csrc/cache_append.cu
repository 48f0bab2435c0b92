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
// write of the queries and of the cache rows. A block takes a few consecutive
// tokens of a sequence, all their heads; d / 16 threads take a head's row,
// each two 16-byte chunks that are a half-rotation apart, so that both
// members of every pair are in one thread, and every thread kItems heads, for
// which a token's eight cosines and sines are loaded once. A thread keeps its
// heads from token to token, the next token's pieces on their way while it
// writes this one's. 8 prompts of 1900 to 4096 tokens, 48 rows of 64 each, in
// bf16: 325 MB in 52 us, 6.3 TB/s, 0.92 of a plain copy's rate. 3 prompts of
// 1203 to 2777, 48 rows of 128, in 4 bits: 140 MB in 32 us, 4.4 TB/s, at 0.67
// of the issue slots, with 24 warps to an SM (80 registers, 68 bytes of them
// spilled) and 2.3 rounds of blocks; 4 prompts of 8192 run at 0.80 of a copy's.
#include <cuda_bf16.h>

#include "kernels.h"
#include "sm103.cuh"

namespace tsd {

namespace {

constexpr int kMaxSpan = 4;      // tokens of a block; no more than the smallest page's 16
// Up to this many tokens a block takes one of them and a thread one head; above
// it a thread takes three heads, and a block a token more for each time this
// many, up to kMaxSpan (launch_cache_append).
constexpr int kFewTokens = 1520;

__device__ __forceinline__ float4 ld_f4(const float* p) {
  return *reinterpret_cast<const float4*>(p);
}

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

// The largest magnitude of eight values; NaN if one of them is.
__device__ __forceinline__ float largest8(const float (&x)[8]) {
  float m = fabsf(x[0]);
  asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(fabsf(x[1])), "f"(fabsf(x[2])));
  asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(fabsf(x[3])), "f"(fabsf(x[4])));
  asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(fabsf(x[5])), "f"(fabsf(x[6])));
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(fabsf(x[7])));
  return m;
}
__device__ __forceinline__ float largest2(float a, float b) {
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(a) : "f"(b));
  return a;
}

// Eight values times `r` as codes.
__device__ __forceinline__ uint32_t codes8(const float (&x)[8], float r) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = x[i] * r;
  uint32_t codes;
  asm("{.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};}"
      : "=r"(codes)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return codes;
}

// The codes of one chunk of 8 columns, given the largest magnitude of its
// group of 16; the group's scale byte in `scale`. Quotients are enclosed by
// products with a little less and a little more than the divisor's inverse
// (kLess, kMore: its error, 2^-23 at most, and two roundings of 2^-24 stay
// within 2^-21). Where both round to the same number it is the quotient's;
// where they do not, a quotient lies at or next to halfway between two
// numbers and the division itself decides. (Eight divisions for a chunk, each
// with a branch for its rare operands: 42 us for 8331 tokens, against 34.)
constexpr float kLess = 1.f - 0x1p-21f, kMore = 1.f + 0x1p-21f;
__device__ __forceinline__ uint32_t quantise8(const float (&x)[8], float top, float factor,
                                              float inverse6, uint32_t* scale) {
  if (!(top < INFINITY)) {
    *scale = 0x7fu;  // NaN
    return 0u;
  }
  uint16_t two;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
      : "=h"(two) : "f"(top * (inverse6 * kMore)), "f"(top * (inverse6 * kLess)));
  if ((two >> 8) != (two & 0xff)) {
    const float want = __fdiv_rn(top, 6.f * factor);
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %1;" : "=h"(two) : "f"(want));
  }
  *scale = two & 0xffu;
  if (*scale == 0u) return 0u;
  uint32_t f2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f2) : "h"(two));
  float s;
  asm("{.reg .b16 lo, hi; mov.b32 {lo, hi}, %1; cvt.f32.f16 %0, lo;}" : "=f"(s) : "r"(f2));
  const float unit = __fmul_rn(s, factor);
  float inverse;
  asm("rcp.approx.f32 %0, %1;" : "=f"(inverse) : "f"(unit));
  const uint32_t low = codes8(x, inverse * kLess), high = codes8(x, inverse * kMore);
  if (low == high) return low;
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = __fdiv_rn(x[i], unit);
  return codes8(y, 1.f);
}

template <int D, bool Q4, int kItems>
__global__ void __launch_bounds__(kItems == 1 ? 512 : 256, kItems == 1 ? 1 : 3)
    cache_append_kernel(const AppendProblem p, int span) {
  constexpr int kLanes = D / 16;  // threads of a row
  griddep_wait();  // inputs, lengths and tables may come from the previous kernel
  griddep_launch_dependents();
  const int groups = (p.n_new - 1) / span + 1;  // n_new + span may pass 32 bits
  const int b = static_cast<int>(blockIdx.x) / groups;
  const int t0 = static_cast<int>(blockIdx.x) % groups * span;
  const PagedCache& c = p.cache;
  const int len = __ldcg(c.lens + b);
  const int m = c.new_lens ? min(max(__ldcg(c.new_lens + b), 0), p.n_new) : p.n_new;
  // the tokens t0 .. t1 - 1 that are no padding and have a place
  const int64_t start = static_cast<int64_t>(len) - m;  // token t's position is start + t
  const int64_t places = static_cast<int64_t>(c.max_pages) << c.page_shift;
  const int64_t known = p.rope_kind != 0 ? min(places, static_cast<int64_t>(p.rope_rows)) : places;
  if (m <= t0) return;
  int t1 = m - t0 < span ? m : t0 + span;
  if (start + t1 > known) {
    if (threadIdx.x == 0) atomicOr(&g_device_error, kErrIndex);
    t1 = static_cast<int>(max(known - start, static_cast<int64_t>(t0)));
  }
  int t = start + t0 < 0 ? static_cast<int>(min(-start, static_cast<int64_t>(t1))) : t0;
  if (t >= t1) return;
  // span <= 16 <= page_size: two pages at most
  const int64_t first_page = (start + t) >> c.page_shift;
  const int32_t* table = c.table + static_cast<int64_t>(b) * c.max_pages + first_page;
  const int page0 = __ldcg(table);
  const int page1 = (start + t1 - 1) >> c.page_shift != first_page ? __ldcg(table + 1) : page0;

  // this thread's chunks (of 8 columns): the rotated columns' first and
  // second half side by side, likewise the columns past them
  const int lane = static_cast<int>(threadIdx.x) % kLanes;
  const bool halves = p.rope_kind == kRopeHalves;
  const int half = (halves ? p.rope_dim : D) / 16;  // chunks of one half
  const int c0 = lane < half ? lane : half + lane;
  const int c1 = c0 + (lane < half ? half : kLanes - half);
  // which of them are rotated
  const bool turn0 = halves ? lane < half : p.rope_kind == kRopePairs && 8 * c0 < p.rope_dim;
  const bool turn1 = halves ? lane < half : p.rope_kind == kRopePairs && 8 * c1 < p.rope_dim;
  // where its angles lie in a row of cosines (sines): of the pairs (c0 * 8 +
  // i, c1 * 8 + i), or of each chunk's four neighbouring pairs
  const float* rope0 = p.rope + (halves ? 8 * c0 : 4 * c0);
  const float* rope1 = p.rope + (halves ? 8 * c0 + 4 : 4 * c1);
  const int sines = p.rope_dim / 2;

  const int rows_q = p.q ? p.h : 0;
  const int rows = rows_q + 2 * c.h_kv;
  const int step = static_cast<int>(blockDim.x) / kLanes;
  const int tokens_begin = t;
  const float k_inverse6 = 1.f / (6.f * c.k_factor), v_inverse6 = 1.f / (6.f * c.v_factor);
  // every thread takes the same number of rounds: a group's two threads
  // exchange their maxima
  for (int round = 0; round < rows; round += kItems * step) {
    const uint16_t* src[kItems];
    uint4 w0[kItems], w1[kItems];
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int row = round + i * step + static_cast<int>(threadIdx.x) / kLanes;
      const bool is_q = row < rows_q, is_v = row >= rows_q + c.h_kv;
      src[i] = is_q ? p.q + b * p.q_sb + row * p.q_sh
                    : (is_v ? p.v : p.k) + b * p.kv_sb + (row - rows_q - (is_v ? c.h_kv : 0)) * p.kv_sh;
      if (row < rows) {
        const uint16_t* x = src[i] + tokens_begin * (is_q ? p.q_sr : p.kv_sr);
        w0[i] = *reinterpret_cast<const uint4*>(x + 8 * c0);
        w1[i] = *reinterpret_cast<const uint4*>(x + 8 * c1);
      }
    }
    for (t = tokens_begin; t < t1; ++t) {
      const int64_t pos = start + t;
      float4 cs[2], sn[2];
      if (turn0) cs[0] = ld_f4(rope0 + pos * p.rope_dim), sn[0] = ld_f4(rope0 + pos * p.rope_dim + sines);
      if (turn1) cs[1] = ld_f4(rope1 + pos * p.rope_dim), sn[1] = ld_f4(rope1 + pos * p.rope_dim + sines);
      const int page = (pos >> c.page_shift) == first_page ? page0 : page1;
      const bool has_page = page >= 0 && page < c.n_pages;
      if (!has_page && threadIdx.x == 0) atomicOr(&g_device_error, kErrIndex);
      const int64_t slot = pos & ((1ll << c.page_shift) - 1);
#pragma unroll
      for (int i = 0; i < kItems; ++i) {
        const int row = round + i * step + static_cast<int>(threadIdx.x) / kLanes;
        const bool live = row < rows && has_page;
        const bool is_q = row < rows_q, is_v = row >= rows_q + c.h_kv;
        const int head = row - (is_q ? 0 : is_v ? rows_q + c.h_kv : rows_q);
        float x0[8], x1[8];
        unpack8(w0[i], x0);
        unpack8(w1[i], x1);
        if (row < rows && t + 1 < t1) {
          const uint16_t* x = src[i] + (t + 1) * (is_q ? p.q_sr : p.kv_sr);
          w0[i] = *reinterpret_cast<const uint4*>(x + 8 * c0);
          w1[i] = *reinterpret_cast<const uint4*>(x + 8 * c1);
        }
        if (!is_v) {
          const float cc[8] = {cs[0].x, cs[0].y, cs[0].z, cs[0].w, cs[1].x, cs[1].y, cs[1].z, cs[1].w};
          const float ss[8] = {sn[0].x, sn[0].y, sn[0].z, sn[0].w, sn[1].x, sn[1].y, sn[1].z, sn[1].w};
          if (halves) {
            if (turn0) {
#pragma unroll
              for (int j = 0; j < 8; ++j) rotate(x0[j], x1[j], cc[j], ss[j]);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (turn0) rotate(x0[2 * j], x0[2 * j + 1], cc[j], ss[j]);
              if (turn1) rotate(x1[2 * j], x1[2 * j + 1], cc[4 + j], ss[4 + j]);
            }
          }
        }
        if (live && (is_q || (!is_v && p.k_out != nullptr))) {
          const int64_t at = is_q ? static_cast<int64_t>(b) * p.h + head
                                  : static_cast<int64_t>(b) * c.h_kv + head;
          uint16_t* dst = (is_q ? p.q_out : p.k_out) + (at * p.n_new + t) * D;
          *reinterpret_cast<uint4*>(dst + 8 * c0) = pack8(x0);
          *reinterpret_cast<uint4*>(dst + 8 * c1) = pack8(x1);
        }
        const int64_t at = ((static_cast<int64_t>(page) * c.h_kv + head) << c.page_shift) + slot;
        if constexpr (!Q4) {
          if (live && !is_q) {
            uint16_t* dst = static_cast<uint16_t*>(is_v ? c.v : c.k) + at * D;
            *reinterpret_cast<uint4*>(dst + 8 * c0) = pack8(x0);
            *reinterpret_cast<uint4*>(dst + 8 * c1) = pack8(x1);
          }
        } else {
          // a group of 16 columns is chunk c0 (c1) of this thread and its neighbour
          if (!__any_sync(0xffffffffu, live && !is_q)) continue;
          float top0 = largest8(x0), top1 = largest8(x1);
          top0 = largest2(top0, __shfl_xor_sync(0xffffffffu, top0, 1));
          top1 = largest2(top1, __shfl_xor_sync(0xffffffffu, top1, 1));
          if (live && !is_q) {
            const float f = is_v ? c.v_factor : c.k_factor;
            uint8_t* codes = static_cast<uint8_t*>(is_v ? c.v : c.k) + at * (D / 2);
            uint8_t* scales = (is_v ? c.v_scales : c.k_scales) + at * (D / 16);
            const float inverse6 = is_v ? v_inverse6 : k_inverse6;
            uint32_t s0, s1;
            *reinterpret_cast<uint32_t*>(codes + 4 * c0) = quantise8(x0, top0, f, inverse6, &s0);
            *reinterpret_cast<uint32_t*>(codes + 4 * c1) = quantise8(x1, top1, f, inverse6, &s1);
            if ((lane & 1) == 0) {
              scales[c0 / 2] = static_cast<uint8_t>(s0);
              scales[c1 / 2] = static_cast<uint8_t>(s1);
            }
          }
        }
      }
    }
  }
}

template <int D, bool Q4, int kItems>
cudaError_t launch_items(const AppendProblem& p, int span, cudaStream_t stream) {
  // threads for all of a token's rows at kItems each, in rounds where they are too many
  constexpr int kMost = kItems == 1 ? 512 : 256;
  const int rows = (p.q ? p.h : 0) + 2 * p.cache.h_kv;
  const int64_t wanted = (int64_t(rows) * (D / 16) + kItems - 1) / kItems;
  const unsigned threads = wanted >= kMost ? kMost : static_cast<unsigned>((wanted + 31) / 32 * 32);
  const int64_t groups = (p.n_new - 1) / span + 1;
  return launch_pdl(cache_append_kernel<D, Q4, kItems>, dim3(static_cast<unsigned>(p.B * groups)),
                    dim3(threads), 0, stream, p, span);
}

}  // namespace

cudaError_t launch_cache_append(const AppendProblem& p, cudaStream_t stream) {
  const int64_t tokens = static_cast<int64_t>(p.B) * p.n_new;
  if (tokens < 1 || tokens > INT32_MAX || (p.cache.d != 64 && p.cache.d != 128))
    return cudaErrorInvalidValue;
  const bool q4 = p.cache.k_scales != nullptr;
  // A head to a thread is the shortest way through, three heads' loads overlap.
  // One head against three, in us: 8 query and 2 x 8 key and value heads of 64,
  // bf16, 32 tokens 2.1 and 2.8, 400 2.6 and 3.0, 800 3.5 and 3.1, 1520 4.6 and
  // 3.5, 32768 85 and 36; 4 bits 2.8 and 4.7, 3.3 and 5.1, 4.6 and 5.2, 5.9 and
  // 5.5, 100 and 51. More rows to a token cross sooner: 32 and 2 x 8 heads of
  // 128, bf16, 96 tokens 2.8 and 3.0, 200 4.0 and 3.3, 800 10.0 and 5.0, 1520 21
  // and 9.3; 4 bits 3.3 and 4.2, 5.0 and 4.5, 12.8 and 6.7, 24 and 11. One number
  // for all fits the first of these in 4 bits, and is late for the others.
  // Of the larger choices, 32768 tokens of 48 rows of 64 in bf16: 52 us; two
  // heads 54, four 59; one, two or eight tokens to a block 66, 54 and 58. In 4
  // bits two heads take as long as three (8331 tokens of 48 rows of 128: 32.0).
  const bool wide = p.cache.d == 128;
  if (tokens <= kFewTokens) {
    if (wide) return q4 ? launch_items<128, true, 1>(p, 1, stream) : launch_items<128, false, 1>(p, 1, stream);
    return q4 ? launch_items<64, true, 1>(p, 1, stream) : launch_items<64, false, 1>(p, 1, stream);
  }
  const int64_t times = (tokens + kFewTokens - 1) / kFewTokens;
  const int span = times < kMaxSpan ? static_cast<int>(times) : kMaxSpan;
  if (wide) return q4 ? launch_items<128, true, 3>(p, span, stream) : launch_items<128, false, 3>(p, span, stream);
  return q4 ? launch_items<64, true, 3>(p, span, stream) : launch_items<64, false, 3>(p, span, stream);
}

TSD_DEFINE_ERROR_READER(take_device_error_append)

}  // namespace tsd
