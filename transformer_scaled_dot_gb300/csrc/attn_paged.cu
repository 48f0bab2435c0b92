// attn_paged.cu -- one decoding step against a paged key/value cache, bf16
// or 4-bit, with grouped query heads:
//   out_r = sum_j p_rj v_j / sum_j p_rj,  p_rj = 2^(x_rj - m_r),
//   x_rj = scale log2(e) q_r . k_j,  m_r the largest x_rj that row r sees.
// The R = (h / h_kv) n_q query rows of one sequence and key head share every
// cached row, so that each is read once for all of them.
//
// The step is bound by reading the cache, and is laid out around that (64
// sequences of 500 to 8192 rows in bf16, 32 query and 8 key heads of 128: 1.14
// GB in 172 us, 6.6 TB/s, 0.98 of a plain copy's rate; 4 bits are bound by
// turning codes into f16 too: 48 sequences of 1001 to 16384 rows, 64 and 8
// heads, 498 MB in 95 us, 5.3 TB/s, 0.58 of the issue slots):
//
//  * Work. A unit is 64 cached rows of one pair, a pair being a (sequence, key
//    head, tile of query rows); a few units more stand for what a pair costs
//    by itself. The units of the batch, in that order, are cut into as many
//    equal ranges as blocks fit on the device, from the lengths that the
//    device holds: sequences of uneven lengths keep all SMs reading to the end,
//    and pages that a sequence does not have cost nothing. A range's first and
//    last sequence may be shared with the neighbouring blocks; those leave
//    partial results (m, l = sum p, O = sum p v, in fp32) in the workspace
//    and the merge kernel joins them.
//  * Loads. A warp takes 16 rows at a time (they lie within one page) and
//    copies them asynchronously into a ring of its own in shared memory, a
//    few 16-row tiles ahead, so no warp waits for another within a range.
//  * Products. A handful of query rows is far too few for a tcgen05 tile of
//    128 rows, and the warp-wide m16n8k16 product reaches the cache's rate
//    with room to spare: S^T = K Q^T with the 16 cached rows as its M and 8
//    query rows as its N, then O^T += V^T P^T. S^T's accumulators become
//    P^T's operand through an 8 x 8 transpose within the warp (movmatrix).
//    bf16 fragments come from the ring by ldmatrix, V's transposed by it;
//    4-bit codes are turned into f16 in registers, and since a product's sum
//    does not care about the order of its terms, a thread's K columns are
//    the ones that its 16 bytes hold, Q being laid out to match, and the two
//    rows that share a register of V are interleaved before the conversion.
//  * Softmax. The exponents' reference m is 2^kShift below the running maximum
//    when it is set, and follows it only when a p would pass 2^(kShift +
//    kSlack): the common tile then needs no maximum over the warp, only a vote.
//
// Numbers: S, the softmax and O in fp32. With a bf16 cache P is split into
// two bf16 parts, p = hi + lo to within 1.1 2^-16 of p, at the cost of a second
// product that the tensor cores have time for. Neither is below 0, and lo is
// not 0 unless p is as good as that: an infinite value that a query sees, times
// either, is the same infinity (with hi rounded to nearest, lo is 0 or less
// half of the time, and the sum of the products would be no number). With a
// 4-bit cache code * scale has 6 significant bits and is formed in f16 without
// rounding; q is brought to f16 by a power of two per row, exactly down to 2^-25
// of the row's largest value, and within 2^-33 of that largest below; and P is
// rounded to f16: to 11 bits, well below the output's 8, where it is at least
// 2^-25 of the row's largest in its warp (m is 2^kShift below that), and to 2^-36
// of that below.
#include <type_traits>

#include <cuda_bf16.h>

#include "kernels.h"
#include "sm103.cuh"

namespace tsd {

namespace {

constexpr int kTile = 16;  // cached rows of a product, within one page
constexpr int kUnit = 64;  // cached rows of a unit of work: a tile for each of four warps
// Caches of at most this many rows are not split: a block takes each pair
// whole and no merge is launched. 7 sequences of 900 rows at 32 query and 8
// key heads of 128: 10.3 us against 11.4, 4-bit 10.4 against 14.5; of 300
// rows 6.1 against 9.9.
constexpr int64_t kUnsplitRows = 1280;
// Where there is an SM for every pair too, a block of eight warps is done with
// more than 256 rows sooner (3 sequences of 1100 rows, 8 key heads of 128: 9.4
// us in place of 11.3; of 100 rows 4.6 in place of 4.3, of 1900 rows 12.6, and
// split 11.6).
constexpr int64_t kAlone = 152, kFewRows = 256;
// What starting and ending a pair costs, in units. 1, 3, 6 and 12, in us: 48
// sequences of up to 16384 rows in 4 bits 101.6, 99.0, 94.9 and 96.0; 64 of up to
// 8192 in bf16 173.7, 172.4, 171.9 and 173.8; 7 of up to 5001 with 28 query rows
// 21.9, 20.9, 21.1 and 21.3; one of 131072 in 4 bits 36.5, 36.6, 37.1 and 37.3.
constexpr int kPairUnits = 6;
constexpr int kMaxBlocks = 608;          // 4 blocks on each of 152 SMs, more than fit
constexpr int kMergeThreads = 256;       // at most
constexpr float kLowest = -3.4028234e38f;  // m before the first row

// Query rows of a block's tile, 8, 16 or 32. A wide tile reads the cache once
// for all of its rows; a narrow one is done sooner, and its blocks share the
// cache's rows through L2 (but each copies them: 4 tokens of 28 heads over 4
// key heads, 41.6 MB of rows, bring 85 MB from L2 to the SMs in two tiles of
// 16). Tiles of 8, 16 and 32, in us, at (pairs x rows each); the first three unsplit:
//                        12x1000     64x1000     160x1000    40x2500     28x5000     128x4000
// 28 rows, d 128, bf16  11  14  19    15  16  20    40  33  28    25  23  26    33  27  27    158  73  57
//                4 bit  10  12  17    16  14  18    29  27  24    22  20  24    25  22  24     65  51  47
//           d 64, bf16   9  10  13    12  11  13    23  22  18    17  16  18    21  19  19     52  44  36
//                4 bit   8   9  11    11  10  12    20  19  14    17  16  18    19  17  17     46  37  30
// 12 rows, d 128, bf16  11  13  18    13  14  19    28  20  26    20  20  23    25  23  25     66  49  52
//                4 bit  10  12  16    11  12  16    16  15  22    17  17  20    19  18  23     38  30  42
//           d 64, bf16   9  10  13     9  10  13    13  13  17    14  14  16    16  16  18     35  31  32
//                4 bit   8   9  11     9   9  11    11  11  14    14  14  15    15  14  16     27  22  27
// 10 rows are like 12, and 24 like 28. What the rule takes is 10 % off the best
// of these three at most (64x1000 of 28 rows, d 128, bf16), and is better where
// eight warps are taken (12x1000: 6.7 to 9.5).
// All of it goes by the rows that the page table has room for: the host does not
// know the lengths. 24 sequences of 100 to 900 rows, 32 query and 8 key heads of
// 128, take 14.1 us (4 bits 10.8) under a table as wide as they need and 18.7
// (15.0) under one of 32768 rows.
struct Plan {
  int tile_rows;
  bool unsplit, eight_warps;
};
Plan plan(int rows, int64_t pairs, int64_t capacity) {
  auto tiles = [&](int tile) { return pairs * ((rows + tile - 1) / tile); };
  const bool unsplit = capacity <= kUnsplitRows;
  if (unsplit && tiles(8) <= kAlone) return {8, true, capacity > kFewRows};
  if (rows <= 8 || (unsplit && tiles(8) <= 200)) return {8, unsplit, false};
  if (rows <= 16 || (unsplit ? tiles(16) <= 304 : pairs * (capacity / kUnit) <= 4096))
    return {16, unsplit, false};
  return {32, unsplit, false};
}

struct PagedArgs {
  const uint16_t* q;
  uint16_t* out;
  const uint8_t* k;
  const uint8_t* v;
  const uint8_t* k_scales;
  const uint8_t* v_scales;
  const int32_t* table;
  const int32_t* lens;
  const int32_t* new_lens;
  // what the merge has to join: by_pair, entry p is pair p's (first block, last
  // block), first -1 if one block did it all; else entry i is the pair that
  // block i begins and others finish (or -1), and its last block
  int2* split;
  bool by_pair;
  float* part_o;   // [blocks][2][rows of a tile][d]
  float2* part_ml; // [blocks][2][rows of a tile]
  int B, h_kv, n_q, rows, row_tiles, n_pages, page_shift, max_pages;
  bool unsplit;  // every pair is one unit, whatever its rows
  bool causal;
  float scale_log2;  // scale log2(e), with the keys' factor
  float v_factor;
};

template <int D, int NT, bool Q4, int W>
struct Shape {
  static constexpr int kWarps = W, kThreads = 32 * W;
  static constexpr int kRows = 8 * NT;
  static constexpr int kRowBytes = Q4 ? D / 2 : 2 * D;
  static constexpr int kScaleBytes = Q4 ? D / 16 : 0;
  static constexpr int kHalves = Q4 ? 2 : 1;  // tiles of a warp's step
  static constexpr int kTileBytes = 2 * kTile * (kRowBytes + kScaleBytes);
  static constexpr int kStageBytes = kHalves * kTileBytes;
  static constexpr int kStages = 3;
  static constexpr int kRingBytes = kWarps * kStages * kStageBytes;
  static constexpr int kPitch = D + 4;  // floats of a row of O in shared memory
  // a 4-bit cache's inner loop has no registers to spare for Q
  static constexpr bool kQInSmem = Q4 || NT * D > 128;
  // p = 2^(x - m) is at most 2^(kShift + kSlack): f16 holds up to 2^15.99, and
  // a bf16 value times 1 is in fp32's range
  static constexpr float kShift = Q4 ? 11.f : -8.f, kSlack = Q4 ? 4.f : 8.f;
  static constexpr int kMergeBytes = kWarps * kRows * kPitch * 4;
  // a warp's part of O fits into one stage of its ring
  static constexpr bool kAhead = kRows * kPitch * 4 <= kStageBytes;
  static constexpr int kSmem = kAhead || kRingBytes > kMergeBytes ? kRingBytes : kMergeBytes;
  // blocks that share an SM: the registers that leaves each thread. A fourth
  // of a 4-bit cache's spills: 104 us in place of 95 (the batch above); two 105.
  static constexpr int kMinBlocks = NT > 1 || W > 4 ? 1 : (Q4 || D == 64 ? 3 : 2);
};

// ------------------------------------------------------------------ instructions

// FULL: 16 bytes; else `valid` decides whether they are read or zeros written.
template <bool FULL>
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src, bool valid) {
  if constexpr (FULL) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  } else {
    const int n = valid ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
                 : "memory");
  }
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a));
  return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 r;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a));
  return r;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t r;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t r;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint32_t r;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(r) : "r"(a));
  return r;
}

template <bool TRANS>
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t a) {
  if constexpr (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// c = a b, or c += a b
template <bool F16>
__device__ __forceinline__ void mma_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
template <bool F16>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// four bytes of two e2m1 codes each -> four pairs of f16
__device__ __forceinline__ void codes_f16x2(uint32_t w, uint32_t (&x)[4]) {
  asm("{.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;}"
      : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(w));
}
// one half of a pair twice (an operand's modifier, no instruction of its own)
template <bool HIGH>
__device__ __forceinline__ uint32_t twice(uint32_t x) {
  uint32_t r;
  if constexpr (HIGH) asm("{.reg .b16 l, h; mov.b32 {l, h}, %1; mov.b32 %0, {h, h};}" : "=r"(r) : "r"(x));
  else asm("{.reg .b16 l, h; mov.b32 {l, h}, %1; mov.b32 %0, {l, l};}" : "=r"(r) : "r"(x));
  return r;
}
// two e4m3 bytes -> a pair of f16 (exact)
__device__ __forceinline__ uint32_t scales_f16x2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
  return r;
}
__device__ __forceinline__ float bf16_f32(uint32_t bits) { return __uint_as_float(bits << 16); }

// Four values of O times the inverse of the weights' sum, then the values'
// factor, as bf16. (The factor over a sum of up to 2^45 may be below fp32's
// normal numbers.)
__device__ __forceinline__ uint2 output4(const float4& y, float inv, float factor) {
  return make_uint2(pack_bf16x2(y.x * inv * factor, y.y * inv * factor),
                    pack_bf16x2(y.z * inv * factor, y.w * inv * factor));
}

// ------------------------------------------------------------------ the ring

// Where the 4-bit tile's rows lie in shared memory, so that a warp's loads of
// K (rows by g, 16 or 8 bytes by t) and of V (rows by t, 8 or 4 bytes by g)
// touch every bank once. Row r of the products is cached row cached_row(r):
// the rows that one thread's V operand spans (2t, 2t+1, 2t+8, 2t+9) are t,
// t+4, t+8 and t+12.
__device__ __forceinline__ constexpr int cached_row(int r) {
  return (r & 8) | ((r & 1) << 2) | ((r & 7) >> 1);
}
template <int D>
__device__ __forceinline__ uint32_t k_code_offset(int row, int byte) {
  if constexpr (D == 128) return static_cast<uint32_t>((row ^ ((row >> 2) & 1)) * 64 + byte);
  return static_cast<uint32_t>((row ^ ((row >> 1) & 2)) * 32 + byte);
}
template <int D>
__device__ __forceinline__ uint32_t v_code_offset(int row, int byte) {
  if constexpr (D == 128) return static_cast<uint32_t>(row * 64 + (byte ^ ((row & 2) << 4)));
  return static_cast<uint32_t>(row * 32 + byte);
}

// A lane's part in copying tiles into stages. bf16: rows of 2 D bytes, keys
// then values, 16-byte piece c of row r at c ^ (r & 7), which ldmatrix reads
// from all banks; 4-bit: both sides' codes, rows moved as above, then their
// scales. Everything that does not depend on the tile is worked out once.
template <int D, bool Q4>
struct TileCopy {
  static constexpr int kRowBytes = Q4 ? D / 2 : 2 * D;
  static constexpr int kPieces = kRowBytes / 16;        // of a row
  static constexpr int kRounds = kTile * kPieces / 32;  // a lane's pieces of each side
  static constexpr int kStep = 32 / kPieces;            // rows from one round to the next
  // bf16: rounds whose rows have the same r & 7 share an offset
  static constexpr int kOffsets = Q4 ? 1 : (8 / kStep < kRounds ? 8 / kStep : kRounds);
  const uint8_t* k;  // this lane's first piece of row 0 of the pool
  const uint8_t* v;
  const uint8_t* scales;
  uint32_t k_off[kOffsets], v_off[kOffsets], scale_off;
  int row0;          // the row of its first piece
  int scale_row;     // the first row whose scales its 16 bytes of scales hold
  bool has_scales;

  __device__ __forceinline__ TileCopy(const PagedArgs& a, int lane) {
    k = a.k + lane * 16;
    v = a.v + lane * 16;
    row0 = lane / kPieces;
    const int piece = lane % kPieces;
#pragma unroll
    for (int i = 0; i < kOffsets; ++i) {
      if constexpr (Q4) {
        k_off[i] = k_code_offset<D>(row0, piece * 16);
        v_off[i] = kTile * kRowBytes + v_code_offset<D>(row0, piece * 16);
      } else {
        k_off[i] = row0 * kRowBytes + ((piece ^ ((row0 + i * kStep) & 7)) << 4);
        v_off[i] = k_off[i] + kTile * kRowBytes;
      }
    }
    // the scales of 16 rows: D bytes for keys, D for values
    const int part = lane % (D / 16);
    has_scales = Q4 && lane < D / 8;
    scales = (lane < D / 16 ? a.k_scales : a.v_scales) + part * 16;
    scale_off = kTile * D + lane * 16;
    scale_row = part * (256 / D);
  }

  // The `valid` first rows of the pools' tile `block` (rows 16 block on); the
  // rest become zeros. A row's scales past `valid` meet codes of zero.
  template <bool FULL>
  __device__ __forceinline__ void load(uint32_t stage, uint32_t block, int valid) const {
    const uint8_t* ks = k + static_cast<uint64_t>(block) * (kTile * kRowBytes);
    const uint8_t* vs = v + static_cast<uint64_t>(block) * (kTile * kRowBytes);
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
      const bool there = row0 + i * kStep < valid;
      cp_async_16<FULL>(stage + k_off[i % kOffsets] + i * 512, ks + i * 512, there);
      cp_async_16<FULL>(stage + v_off[i % kOffsets] + i * 512, vs + i * 512, there);
    }
    if constexpr (Q4) {
      if (has_scales)
        cp_async_16<FULL>(stage + scale_off, scales + static_cast<uint64_t>(block) * D,
                          scale_row < valid);
    }
  }
};

// ------------------------------------------------------------------ the work's order

// Sequence b's rows that count, and its units.
struct Sequence {
  int len, fresh;  // cached rows, new tokens
  int units;       // of rows
};
__device__ __forceinline__ Sequence sequence(const PagedArgs& a, int b) {
  Sequence s;
  const int capacity = a.max_pages << a.page_shift;
  s.len = a.lens ? min(max(__ldcg(a.lens + b), 0), capacity) : capacity;
  s.fresh = a.new_lens ? min(max(__ldcg(a.new_lens + b), 0), a.n_q) : a.n_q;
  s.units = s.fresh > 0 ? (s.len + kUnit - 1) / kUnit : 0;
  return s;
}
// The units of each of its pairs, the first `extra` of which stand for no
// rows; at least one, as its output has to be written.
__device__ __forceinline__ int pair_units(const Sequence& s, int extra) {
  return max(s.units + extra, 1);
}

// A block's consecutive units of one pair.
struct Segment {
  int64_t unit;  // the first one's number
  int b, pair;
  int units, chunk, take;  // of the pair: all, those before, those that are the block's
  int len, fresh;
};

// Floor of x / y, in 32 bits where they suffice.
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t y) {
  if (((x | y) >> 32) == 0) return static_cast<uint32_t>(x) / static_cast<uint32_t>(y);
  return x / y;
}

// ------------------------------------------------------------------ the kernel

template <int D, int NT, bool Q4, int W>
__global__ void __launch_bounds__(32 * W, Shape<D, NT, Q4, W>::kMinBlocks)
    decode_paged_kernel(const PagedArgs a) {
  using S = Shape<D, NT, Q4, W>;
  constexpr int kWarps = S::kWarps, kThreads = S::kThreads;
  constexpr int kSteps = D / 16;  // products of S, and blocks of 16 columns of O
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float2 s_ml[kWarps][S::kRows];
  __shared__ float2 s_join[S::kRows];
  __shared__ float s_mult[S::kRows];
  __shared__ int s_limit[S::kRows];
  __shared__ uint2 s_q[S::kQInSmem ? kSteps * NT : 1][32];
  // kept out of the registers that the inner loop needs
  __shared__ Segment s_seg;
  __shared__ int64_t s_rest, s_plan[2];  // units after the segment; all units, all blocks
  const int tid = static_cast<int>(threadIdx.x);
  const int warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  griddep_wait();  // the cache, queries, lengths and tables may come from the previous kernel
  griddep_launch_dependents();

  // this block's range of units: each warp by itself sums the sequences' units
  const int pairs = a.h_kv * a.row_tiles;  // (key head, row tile) of a sequence
  int64_t total = 0;
  int extra = 0;
  Sequence early = {};  // the first 32, not loaded again
  if (!a.unsplit) early = sequence(a, min(lane, a.B - 1));
  if (a.unsplit) {
    total = static_cast<int64_t>(a.B) * pairs;
  } else {
    int none = 0;  // sequences without rows
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      int u = b0 == 0 ? early.units : b0 + lane < a.B ? sequence(a, b0 + lane).units : 0;
      if (b0 + lane >= a.B) u = 0;
      none += __popc(__ballot_sync(0xffffffffu, b0 + lane < a.B && u == 0));
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) u += __shfl_xor_sync(0xffffffffu, u, s);
      total += u;
    }
    total *= pairs;
    // a pair's own cost counts as far as the blocks have that much to do: with
    // a unit or two for each it would only leave blocks without rows
    extra = static_cast<int>(min(quotient(total, gridDim.x), static_cast<int64_t>(kPairUnits)));
    total += static_cast<int64_t>(pairs) * (extra > 0 ? static_cast<int64_t>(a.B) * extra : none);
  }
  const int64_t blocks = min(static_cast<int64_t>(gridDim.x), total);
  const int64_t me = blockIdx.x;
  if (tid == 0 && !a.by_pair && !a.unsplit) a.split[me] = make_int2(-1, 0);
  if (me >= blocks) return;
  const int64_t each = quotient(total, blocks), over_all = total - each * blocks;
  Segment seg;
  seg.unit = me * each + quotient(me * over_all, blocks);
  int64_t rest = (me + 1) * each + quotient((me + 1) * over_all, blocks) - seg.unit;
  if (a.unsplit) {
    seg.b = static_cast<int>(quotient(seg.unit, pairs));
    seg.pair = static_cast<int>(seg.unit - static_cast<int64_t>(seg.b) * pairs);
    const Sequence seq = sequence(a, seg.b);
    seg.len = seq.len;
    seg.fresh = seq.fresh;
    seg.units = seg.take = 1;
    seg.chunk = 0;
    --rest;
  } else {
    const int64_t want = quotient(seg.unit, pairs);
    int64_t base = 0;  // units of one pair of all sequences before b
    for (int b0 = 0;; b0 += 32) {
      const Sequence seq = b0 == 0 ? early : sequence(a, min(b0 + lane, a.B - 1));
      const int u = b0 + lane < a.B ? pair_units(seq, extra) : 0;
      int upto = u;
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, s);
        if (lane >= s) upto += v;
      }
      const unsigned past = __ballot_sync(0xffffffffu, base + upto > want);
      if (past != 0u || b0 + 32 >= a.B) {  // the second: for certain to end
        const int first = past != 0u ? __ffs(past) - 1 : (a.B - 1) & 31;
        seg.b = b0 + first;
        base += __shfl_sync(0xffffffffu, upto - u, first);
        seg.len = __shfl_sync(0xffffffffu, seq.len, first);
        seg.fresh = __shfl_sync(0xffffffffu, seq.fresh, first);
        seg.units = __shfl_sync(0xffffffffu, u, first);
        break;
      }
      base += __shfl_sync(0xffffffffu, upto, 31);
    }
    const int64_t local = seg.unit - base * pairs;
    seg.pair = static_cast<int>(quotient(local, seg.units));
    seg.chunk = static_cast<int>(local - static_cast<int64_t>(seg.pair) * seg.units);
    seg.take = static_cast<int>(min(rest, static_cast<int64_t>(seg.units - seg.chunk)));
    rest -= seg.take;
  }
  if (tid == 0) {
    s_plan[0] = total;
    s_plan[1] = blocks;
  }

  const uint32_t ring = smem_u32(smem) + warp * (S::kStages * S::kStageBytes);
  const TileCopy<D, Q4> copy(a, lane);
  constexpr int kHalves = S::kHalves, kStride = kHalves * kWarps * kTile;
  constexpr uint32_t kNoBlock = 0xffffffffu;

  // the part of a segment that this warp's copies go by
  int first_key = 0, key1 = 0, head = 0;
  const int32_t* table = nullptr;
  int to_load = 0;             // rows from the next step to load to key1, less than 1: none
  int next_tile = 0, refill = 0;  // the next tile to load; where block runs out
  uint32_t block = 0, block_next = 0;  // of the steps' tiles, 32 at a time, one per lane
  uint32_t skipped = 0;        // bit kHalves s + h: tile h of stage s has no page
  int fill = 0, stage = 0;     // the stages that are filled and read next
  uint32_t fill_at = ring, at = ring;
  // tile j's place in the pools, in tiles (kNoBlock: its page is no page)
  auto block_of = [&](int j) {
    const int key = first_key + j / kHalves * kStride + j % kHalves * kTile;
    if (key >= key1) return 0u;
    const int page = __ldcg(table + (key >> a.page_shift));
    if (page < 0 || page >= a.n_pages) {
      atomicOr(&g_device_error, kErrIndex);
      return kNoBlock;
    }
    return ((static_cast<uint32_t>(page) * a.h_kv + head) << (a.page_shift - 4)) +
           ((key & ((1 << a.page_shift) - 1)) >> 4);
  };
  auto issue = [&]() {  // the next step's tiles into the next stage
    if (to_load > 0) {
      if (next_tile == refill) {
        block = block_next;
        refill += 32;
        block_next = block_of(refill + lane);
      }
      uint32_t from[kHalves];
      bool common = to_load >= kHalves * kTile;
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        from[h] = __shfl_sync(0xffffffffu, block, next_tile + h);  // of 32 lanes
        common = common && from[h] != kNoBlock;
      }
      if (common) {
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
          copy.template load<true>(fill_at + h * S::kTileBytes, from[h], kTile);
      } else {
#pragma unroll
        for (int h = 0; h < kHalves; ++h) {
          const bool missing = from[h] == kNoBlock;
          if (missing) skipped |= 1u << (fill * kHalves + h);
          copy.template load<false>(fill_at + h * S::kTileBytes, missing ? 0u : from[h],
                                    missing ? 0 : to_load - h * kTile);
        }
      }
      to_load -= kStride;
      next_tile += kHalves;
    }
    cp_async_commit();
    fill_at += S::kStageBytes;
    if (++fill == S::kStages) fill = 0, fill_at = ring;
  };
  // a segment's first copies, into all stages but the last; the ring is empty
  auto begin = [&](const Segment& sg) {
    fill = stage = 0;
    fill_at = at = ring;
    skipped = 0;
    head = sg.pair / a.row_tiles;
    table = a.table + static_cast<int64_t>(sg.b) * a.max_pages;
    // rows [key0, key1) of the cache; none if every token is padding
    const int key0 = max(sg.chunk - extra, 0) * kUnit;
    key1 = a.unsplit ? sg.len : min(sg.len, max(sg.chunk + sg.take - extra, 0) * kUnit);
    if (sg.fresh == 0) key1 = 0;
    // this warp's steps of kHalves tiles each, a stride apart
    first_key = key0 + warp * (kHalves * kTile);
    to_load = key1 - first_key;
    next_tile = 0;
    refill = 32;
    block = block_of(lane);
    block_next = block_of(32 + lane);
#pragma unroll
    for (int i = 0; i < S::kStages - 1; ++i) issue();
  };
  begin(seg);

  while (true) {
    const int row0 = seg.pair % a.row_tiles * S::kRows;
    const int rows = min(S::kRows, a.rows - row0);
    const int64_t q_row0 = (static_cast<int64_t>(seg.b) * a.h_kv + seg.pair / a.row_tiles) * a.rows + row0;

    // ---- queries as the products' operand: registers 0 and 1 of step s hold
    // the columns that the threads' K registers of that step hold. In shared
    // memory where they would take too many registers.
    constexpr int kMine = S::kQInSmem ? 1 : NT;  // column blocks of this warp
    uint32_t qf[kMine][kSteps][2];
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int r = (S::kQInSmem ? warp : i) * 8 + g;
      const bool live = r < rows;
      const uint16_t* qp = a.q + (q_row0 + r) * D;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        if constexpr (Q4) {
          const uint2 two = live ? __ldcg(reinterpret_cast<const uint2*>(qp + t * (D / 4) + 4 * s))
                                 : make_uint2(0, 0);
          qf[i][s][0] = two.x;
          qf[i][s][1] = two.y;
        } else {
          const uint32_t* src = reinterpret_cast<const uint32_t*>(qp + 16 * s + 2 * t);
          qf[i][s][0] = live ? __ldcg(src) : 0u;
          qf[i][s][1] = live ? __ldcg(src + 4) : 0u;
        }
      }
    }

#pragma unroll
    for (int n = 0; n < kMine; ++n) {
      uint32_t (&w)[kSteps][2] = qf[n];
      const int nt = S::kQInSmem ? warp : n;
      if (nt >= NT) continue;
      if constexpr (Q4) {
        // the row's largest magnitude decides a power of two that brings it to
        // 2^8 or more, below 2^9. f16's least step is 2^-24: a value of 8 bits is
        // exact from 2^-17 on (2^-25 of the largest or more), and smaller ones
        // are off by half that step, 2^-33 of the largest, at most
        uint32_t top = 0;
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            top = max(top, max(w[s][i] & 0x7fffu, (w[s][i] >> 16) & 0x7fffu));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // exponent field e of the largest: times 2^(135 - e) in two factors,
        // since 135 - e may pass a float's exponents by itself
        const int e = top == 0 ? 127 : min(max(static_cast<int>(top >> 7), 1), 254);
        const int up = 135 - e, up0 = up / 2, up1 = up - up0;
        const float f0 = __int_as_float((127 + up0) << 23), f1 = __int_as_float((127 + up1) << 23);
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            w[s][i] = pack_f16x2(bf16_f32(w[s][i] & 0xffffu) * f0 * f1, bf16_f32(w[s][i] >> 16) * f0 * f1);
        // the factor from S to x; not 0, which would make the masks' -inf no
        // number, and finite, as an infinite one would make so a product of 0
        const float d0 = __int_as_float((127 - up0) << 23), d1 = __int_as_float((127 - up1) << 23);
        if (t == 0) s_mult[nt * 8 + g] = fminf(fmaxf(a.scale_log2 * d0 * d1, 1.2e-38f), 3.4e38f);
      }
      if constexpr (S::kQInSmem) {
#pragma unroll
        for (int s = 0; s < kSteps; ++s) s_q[s * NT + nt][lane] = make_uint2(w[s][0], w[s][1]);
      }
    }
    if (tid < S::kRows) {  // row tid of the tile sees the cached rows before its limit
      const int token = (row0 + tid) % a.n_q;
      int limit = 0x7fffffff;  // rows that nobody reads need no mask
      if (tid < rows && token < seg.fresh) {
        limit = seg.len;
        if (a.causal) limit = min(limit, seg.len - seg.fresh + token + 1);
      }
      s_limit[tid] = limit;
    }
    if (tid == 0) {
      s_seg = seg;
      s_rest = rest;
    }
    // cached rows from here on are hidden from some row of the tile
    const int hidden = a.causal ? min(seg.len, seg.len - seg.fresh + 1) : seg.len;

    float o[NT][kSteps][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int s = 0; s < kSteps; ++s) o[nt][s][0] = o[nt][s][1] = o[nt][s][2] = o[nt][s][3] = 0.f;
      m[nt][0] = m[nt][1] = kLowest;
      l[nt][0] = l[nt][1] = 0.f;
    }

    __syncthreads();  // s_limit, s_mult, s_q, s_seg
    float mult[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) mult[nt][c] = Q4 ? s_mult[nt * 8 + 2 * t + c] : a.scale_log2;
    auto query = [&](int nt, int s) {
      if constexpr (S::kQInSmem) return s_q[s * NT + nt][lane];
      else return make_uint2(qf[nt][s][0], qf[nt][s][1]);
    };
    const int row_lo = Q4 ? cached_row(g) : g;  // of S^T's registers 0, 1; 8 further: 2, 3
    // one step; MASKED: some row of it may be hidden from some query
    auto step = [&](auto masked, int key) {
      constexpr bool kMasked = decltype(masked)::value;

      // ---- S^T = K Q^T; for one column block of one tile even and odd steps
      // apart, as one chain of dependent products would be waited for
      [[maybe_unused]] constexpr bool kTwoChains = NT * kHalves == 1;
      float x[kHalves][NT][4];
      if constexpr (!Q4) {
#pragma unroll
        for (int h = 0; h < kHalves; ++h) {
          [[maybe_unused]] float x2[NT][4];
          const uint32_t kat = at + h * S::kTileBytes + (lane & 15) * (2 * D);
          const uint32_t swz = (lane >> 4) ^ (lane & 7);
#pragma unroll
          for (int s = 0; s < kSteps; ++s) {
            uint32_t w[4];
            ldmatrix4<false>(w, kat + ((swz ^ (2 * s)) << 4));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const uint2 q = query(nt, s);
              float (&to)[4] = kTwoChains && (s & 1) ? x2[nt] : x[h][nt];
              if (s == 0 || (kTwoChains && s == 1)) mma_first<false>(to, w[0], w[1], w[2], w[3], q.x, q.y);
              else mma<false>(to, w[0], w[1], w[2], w[3], q.x, q.y);
            }
          }
          if constexpr (kTwoChains) {
#pragma unroll
            for (int c = 0; c < 4; ++c) x[h][0][c] += x2[0][c];
          }
        }
      } else {
        constexpr int kWords = D / 32;  // of this thread's codes of one row
        uint32_t w[kHalves][2][kWords], sc[kHalves][2];
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint32_t tile = at + h * S::kTileBytes;
            const int row = row_lo + 8 * half;
            if constexpr (D == 128) {
              const uint4 v = lds128(tile + k_code_offset<D>(row, t * 16));
              w[h][half][0] = v.x, w[h][half][1] = v.y, w[h][half][2] = v.z, w[h][half][3] = v.w;
              sc[h][half] = scales_f16x2(lds16(tile + kTile * D + row * 8 + t * 2));
            } else {
              const uint2 v = lds64(tile + k_code_offset<D>(row, t * 8));
              w[h][half][0] = v.x, w[h][half][1] = v.y;
              sc[h][half] = scales_f16x2(lds8(tile + kTile * D + row * 4 + t));
            }
          }
#pragma unroll
        for (int i4 = 0; i4 < kWords; ++i4)
#pragma unroll
          for (int h = 0; h < kHalves; ++h) {
            uint32_t lo[4], hi[4];
            codes_f16x2(w[h][0][i4], lo);
            codes_f16x2(w[h][1][i4], hi);
            // d = 128: words 0, 1 are of the thread's first group, 2, 3 of its second
            const uint32_t s0 = i4 < 2 ? twice<false>(sc[h][0]) : twice<true>(sc[h][0]);
            const uint32_t s1 = i4 < 2 ? twice<false>(sc[h][1]) : twice<true>(sc[h][1]);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              lo[c] = mul_f16x2(lo[c], s0);
              hi[c] = mul_f16x2(hi[c], s1);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const uint2 q0 = query(nt, 2 * i4), q1 = query(nt, 2 * i4 + 1);
              if (i4 == 0) mma_first<true>(x[h][nt], lo[0], hi[0], lo[1], hi[1], q0.x, q0.y);
              else mma<true>(x[h][nt], lo[0], hi[0], lo[1], hi[1], q0.x, q0.y);
              mma<true>(x[h][nt], lo[2], hi[2], lo[3], hi[3], q1.x, q1.y);
            }
          }
      }

      // ---- masks, in the sequence's last rows or where a page is missing;
      // there also: is any value of V not finite?
      bool odd = false;
      if constexpr (kMasked) {
        const uint32_t missing = (skipped >> (stage * kHalves)) & ((1u << kHalves) - 1);
        skipped &= ~(missing << (stage * kHalves));
#pragma unroll
        for (int h = 0; h < kHalves; ++h) {
          const int row = key + h * kTile + row_lo;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (row + (c < 2 ? 0 : 8) >= s_limit[nt * 8 + 2 * t + (c & 1)] || (missing >> h & 1))
                x[h][nt][c] = -INFINITY;
          const uint32_t vat = at + h * S::kTileBytes + kTile * S::kRowBytes;
          if constexpr (Q4) {  // a NaN among the scales: 16 rows of D / 16
            if (lane < D / 4) {
              const uint32_t w = lds32(vat + kTile * S::kRowBytes + D + lane * 4) & 0x7f7f7f7fu;
              odd |= ((w + 0x01010101u) & 0x80808080u) != 0;
            }
          } else {
#pragma unroll
            for (int j = 0; j < kTile * S::kRowBytes / 512; ++j) {
              const uint4 w = lds128(vat + j * 512 + lane * 16);
#pragma unroll
              for (uint32_t e : {w.x, w.y, w.z, w.w})
                odd |= (e & 0x7f80u) == 0x7f80u || (e & 0x7f800000u) == 0x7f800000u;
            }
          }
        }
        odd = __any_sync(0xffffffffu, odd);
      }

      // ---- x - m, and whether any passes what P may be
      float y[kHalves][NT][4];
#pragma unroll
      for (int h = 0; h < kHalves; ++h)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            y[h][nt][c] = fmaf(x[h][nt][c], mult[nt][c & 1], -m[nt][c & 1]);
          }
      float highest = kLowest;
#pragma unroll
      for (int h = 0; h < kHalves; ++h)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          highest = fmax3(highest, y[h][nt][0], y[h][nt][1]);
          highest = fmax3(highest, y[h][nt][2], y[h][nt][3]);
        }
      if (__any_sync(0xffffffffu, highest > S::kShift + S::kSlack)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float top = fmaxf(x[0][nt][c], x[0][nt][2 + c]);
            if constexpr (kHalves == 2) top = fmaxf(top, fmaxf(x[kHalves - 1][nt][c], x[kHalves - 1][nt][2 + c]));
            top *= mult[nt][c];
#pragma unroll
            for (int s = 4; s < 32; s <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
            const float next = fmaxf(m[nt][c], top - S::kShift);
            const float f = ex2(m[nt][c] - next);
            m[nt][c] = next;
            l[nt][c] *= f;
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
              o[nt][s][c] *= f;
              o[nt][s][2 + c] *= f;
            }
#pragma unroll
            for (int h = 0; h < kHalves; ++h) {
              y[h][nt][c] = fmaf(x[h][nt][c], mult[nt][c], -next);
              y[h][nt][2 + c] = fmaf(x[h][nt][2 + c], mult[nt][c], -next);
            }
          }
      }

      // ---- p, its sum, and P^T as the second product's operand
      uint32_t p_hi[kHalves][NT][2];
      [[maybe_unused]] uint32_t p_lo[kHalves][NT][2];  // bf16 only
#pragma unroll
      for (int h = 0; h < kHalves; ++h)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float p[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) p[c] = ex2(y[h][nt][c]);
          l[nt][0] += p[0] + p[2];
          l[nt][1] += p[1] + p[3];
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const float p0 = p[2 * half], p1 = p[2 * half + 1];
            if constexpr (Q4) {
              p_hi[h][nt][half] = transpose8x8(pack_f16x2(p0, p1));
            } else {
              // hi cut off, so that the rest is no less than 0; and 2^-20 of p
              // more, so that it is not 0
              const uint32_t hi = __byte_perm(__float_as_uint(p0), __float_as_uint(p1), 0x7632);
              constexpr float kAbove = 1.f + 0x1p-20f;
              p_hi[h][nt][half] = transpose8x8(hi);
              p_lo[h][nt][half] = transpose8x8(pack_bf16x2(fmaf(p0, kAbove, -bf16_f32(hi & 0xffffu)),
                                                           fmaf(p1, kAbove, -bf16_f32(hi >> 16))));
            }
          }
        }

      // ---- O^T += V^T P^T. Registers 0 and 1 of V's operand are two columns
      // of cached rows r0 and r1, registers 2 and 3 of the rows 8 further
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        [[maybe_unused]] const uint32_t vat = at + h * S::kTileBytes + kTile * S::kRowBytes;
        // 4-bit: [rows' half][cached rows r0, r1][word]. (Loading them before the
        // softmax hides their latency and costs registers: 97 us against 95.)
        [[maybe_unused]] uint32_t v_codes[2][2][D / 64], v_scale[2];
        if constexpr (Q4) {
          const uint32_t sat = vat + kTile * S::kRowBytes + D;
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int a0 = t + 8 * r, a1 = a0 + 4;
            if constexpr (D == 128) {
              const uint2 w0 = lds64(vat + v_code_offset<D>(a0, g * 8));
              const uint2 w1 = lds64(vat + v_code_offset<D>(a1, g * 8));
              v_codes[r][0][0] = w0.x, v_codes[r][0][1] = w0.y;
              v_codes[r][1][0] = w1.x, v_codes[r][1][1] = w1.y;
            } else {
              v_codes[r][0][0] = lds32(vat + v_code_offset<D>(a0, g * 4));
              v_codes[r][1][0] = lds32(vat + v_code_offset<D>(a1, g * 4));
            }
            const int group = D == 128 ? g : g >> 1;
            v_scale[r] = scales_f16x2(__byte_perm(lds8(sat + a0 * (D / 16) + group),
                                                  lds8(sat + a1 * (D / 16) + group), 0x0040));
          }
        }
        // the operand of kBlock blocks of 16 columns from block s0 on
        constexpr int kBlock = Q4 ? 4 : 1;
        auto v_operand = [&](int s0, uint32_t (&va)[kBlock][4]) {
          if constexpr (!Q4) {
            const uint32_t row = (lane & 7) + ((lane >> 4) << 3);
            ldmatrix4<true>(va[0], vat + row * (2 * D) +
                                       (((2 * s0) ^ ((lane >> 3) & 1) ^ (lane & 7)) << 4));
          } else {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const uint32_t u = v_codes[r][0][s0 / 4], v = v_codes[r][1][s0 / 4];
              uint32_t even[4], uneven[4];
              codes_f16x2((u & 0x0f0f0f0fu) | ((v << 4) & 0xf0f0f0f0u), even);
              codes_f16x2(((u >> 4) & 0x0f0f0f0fu) | (v & 0xf0f0f0f0u), uneven);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                va[e][2 * r] = mul_f16x2(even[e], v_scale[r]);
                va[e][2 * r + 1] = mul_f16x2(uneven[e], v_scale[r]);
              }
            }
          }
        };
        if (kMasked && odd) {
          // 0 times an infinity is no number: the products once for each new
          // token, with the rows that it does not see cleared, and only the
          // token's own columns of O taken from them
          const int r0 = key + h * kTile + (Q4 ? t : 2 * t), r1 = r0 + (Q4 ? 4 : 1);
          const int fresh = s_seg.fresh, len = s_seg.len;
          const int row0 = s_seg.pair % a.row_tiles * S::kRows;
          for (int token = 0; token < fresh; ++token) {
            const int seen = a.causal ? len - fresh + token + 1 : len;
            uint32_t keep[2];
#pragma unroll
            for (int r = 0; r < 2; ++r)
              keep[r] = (r0 + 8 * r < seen ? 0xffffu : 0u) | (r1 + 8 * r < seen ? 0xffff0000u : 0u);
#pragma unroll
            for (int s = 0; s < kSteps; s += kBlock) {
              uint32_t va[kBlock][4];
              v_operand(s, va);
#pragma unroll
              for (int e = 0; e < kBlock; ++e)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  const uint32_t a0 = va[e][0] & keep[0], a1 = va[e][1] & keep[0];
                  const uint32_t a2 = va[e][2] & keep[1], a3 = va[e][3] & keep[1];
                  float (&acc)[4] = o[nt][s + e];
                  float z[4] = {acc[0], acc[1], acc[2], acc[3]};
                  mma<Q4>(z, a0, a1, a2, a3, p_hi[h][nt][0], p_hi[h][nt][1]);
                  if constexpr (!Q4) mma<Q4>(z, a0, a1, a2, a3, p_lo[h][nt][0], p_lo[h][nt][1]);
                  if ((row0 + nt * 8 + 2 * t) % a.n_q == token) acc[0] = z[0], acc[2] = z[2];
                  if ((row0 + nt * 8 + 2 * t + 1) % a.n_q == token) acc[1] = z[1], acc[3] = z[3];
                }
            }
          }
        } else {
#pragma unroll
          for (int s = 0; s < kSteps; s += kBlock) {
            uint32_t va[kBlock][4];
            v_operand(s, va);
#pragma unroll
            for (int e = 0; e < kBlock; ++e)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma<Q4>(o[nt][s + e], va[e][0], va[e][1], va[e][2], va[e][3], p_hi[h][nt][0],
                        p_hi[h][nt][1]);
                if constexpr (!Q4)
                  mma<Q4>(o[nt][s + e], va[e][0], va[e][1], va[e][2], va[e][3], p_lo[h][nt][0],
                          p_lo[h][nt][1]);
              }
          }
        }
      }
    };
    const int tail = key1 + kHalves * kTile - hidden;  // closer to key1 than this: masks
    for (int rest_rows = key1 - first_key; rest_rows > 0; rest_rows -= kStride) {
      cp_async_wait<S::kStages - 2>();
      __syncwarp();  // the other lanes' copies; and all have read the stage that is filled next
      issue();
      if (rest_rows < tail || skipped != 0) step(std::true_type{}, key1 - rest_rows);
      else step(std::false_type{}, 0);
      at += S::kStageBytes;
      if (++stage == S::kStages) stage = 0, at = ring;
    }

    // ---- what comes next, its first copies on their way before this segment
    // is finished where O has room beside them: in the stage left free
    const Segment done = s_seg;
    rest = s_rest;
    const bool more = rest > 0;
    if (more) {
      seg.unit = done.unit + done.take;
      seg.b = done.b;
      seg.pair = done.pair + 1;
      seg.chunk = 0;
      seg.units = done.units;
      seg.len = done.len;
      seg.fresh = done.fresh;
      if (seg.pair == pairs) {
        seg.pair = 0;
        ++seg.b;
        const Sequence seq = sequence(a, seg.b);
        seg.len = seq.len;
        seg.fresh = seq.fresh;
        seg.units = a.unsplit ? 1 : pair_units(seq, extra);
      }
      seg.take = static_cast<int>(min(rest, static_cast<int64_t>(seg.units)));
      rest -= seg.take;
      if (S::kAhead) {
        __syncwarp();  // no lane reads a stage any more
        begin(seg);
      }
    }
    if (!S::kAhead || !more) cp_async_wait<0>();

    // ---- the warps' results of these units, joined in shared memory
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int s = 4; s < 32; s <<= 1) l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], s);
        if (g == 0) s_ml[warp][nt * 8 + 2 * t + c] = make_float2(m[nt][c], l[nt][c]);
      }
    __syncthreads();  // also: without kAhead no warp uses its ring any more
    // warp w's rows of O: [S::kRows][S::kPitch] floats
    auto o_smem = [&](int w) {
      return reinterpret_cast<float*>(
          smem + (S::kAhead ? (w * S::kStages + S::kStages - 1) * S::kStageBytes
                            : w * S::kRows * S::kPitch * 4));
    };
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = nt * 8 + 2 * t + c;
        float top = s_ml[0][r].x;
#pragma unroll
        for (int w = 1; w < kWarps; ++w) top = fmaxf(top, s_ml[w][r].x);
        const float f = ex2(m[nt][c] - top);  // a warp without a row has O = l = 0
        float* dst = o_smem(warp) + r * S::kPitch;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          // the two columns of block s that this thread has
          const int d0 = Q4 ? g * (D / 8) + 8 * (s >> 2) + 2 * (s & 3) : 16 * s + g;
          dst[d0] = o[nt][s][c] * f;
          dst[d0 + (Q4 ? 1 : 8)] = o[nt][s][2 + c] * f;
        }
      }
    if (tid < S::kRows) {
      float top = s_ml[0][tid].x, sum = 0.f;
#pragma unroll
      for (int w = 1; w < kWarps; ++w) top = fmaxf(top, s_ml[w][tid].x);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) sum += s_ml[w][tid].y * ex2(s_ml[w][tid].x - top);
      s_join[tid] = make_float2(top, sum);
    }
    __syncthreads();
    const bool whole = done.chunk == 0 && done.take == done.units;
    const int64_t slot = 2 * me + (done.chunk == 0 ? 1 : 0);
    const int done_row0 = done.pair % a.row_tiles * S::kRows;
    const int done_rows = min(S::kRows, a.rows - done_row0);
    const int64_t out_row0 =
        (static_cast<int64_t>(done.b) * a.h_kv + done.pair / a.row_tiles) * a.rows + done_row0;
    for (int i = tid; i < done_rows * (D / 4); i += kThreads) {
      const int r = i / (D / 4), d = i % (D / 4) * 4;
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 z = *reinterpret_cast<const float4*>(o_smem(w) + r * S::kPitch + d);
        y.x += z.x, y.y += z.y, y.z += z.z, y.w += z.w;
      }
      const float2 join = s_join[r];
      if (whole) {
        const bool real = (done_row0 + r) % a.n_q < done.fresh;
        // no row seen (sum 0), or padding: 0; a sum that is no number stays one
        const float inv = real && join.y != 0.f ? 1.f / join.y : 0.f;
        *reinterpret_cast<uint2*>(a.out + (out_row0 + r) * D + d) =
            inv == 0.f ? make_uint2(0u, 0u) : output4(y, inv, Q4 ? a.v_factor : 1.f);
      } else {
        *reinterpret_cast<float4*>(a.part_o + (slot * S::kRows + r) * D + d) = y;
        if (d == 0) a.part_ml[slot * S::kRows + r] = join;
      }
    }
    if (tid == 0 && done.chunk == 0 && !a.unsplit) {
      // the block of this pair's last unit
      const int64_t upto = done.unit + done.units;
      const int last = static_cast<int>(quotient(upto * s_plan[1] - 1, s_plan[0]));
      if (a.by_pair)
        a.split[done.b * pairs + done.pair] = make_int2(whole ? -1 : static_cast<int>(me), last);
      else if (!whole)
        a.split[me] = make_int2(done.b * pairs + done.pair, last);
    }
    __syncthreads();  // O's and the segment's shared memory is free
    if (!more) break;
    if (!S::kAhead) begin(seg);
  }
}

// Joins the partial results of one query row of a pair that several blocks
// worked on: groups of D / 4 threads share the contributions, 16
// bytes to a thread. It is a chain of three reads (who, m and l, O); a
// group's first O is read along with the second.
template <int D>
__global__ void __launch_bounds__(kMergeThreads) decode_paged_merge_kernel(const PagedArgs a,
                                                                          int tile_rows) {
  constexpr int kMostGroups = kMergeThreads / (D / 4);
  const int threads = static_cast<int>(blockDim.x), warps = threads / 32, groups = threads / (D / 4);
  __shared__ float weight[kMaxBlocks];
  __shared__ float4 part[kMostGroups][D / 4];
  __shared__ float red[kMergeThreads / 32], red_l[kMergeThreads / 32];
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const int group = tid / (D / 4), col = tid % (D / 4);
  griddep_wait();  // the partials are complete
  griddep_launch_dependents();
  const int2 split = a.split[blockIdx.x];
  if (split.x < 0) return;
  const int pairs = a.h_kv * a.row_tiles;
  const int whole_pair = a.by_pair ? static_cast<int>(blockIdx.x) : split.x;
  const int first = a.by_pair ? split.x : static_cast<int>(blockIdx.x), n = split.y - first + 1;
  const int b = whole_pair / pairs, pair = whole_pair % pairs;
  const int head = pair / a.row_tiles, row0 = pair % a.row_tiles * tile_rows;
  const int r = static_cast<int>(blockIdx.y);
  if (row0 + r >= a.rows) return;
  // contribution i: the first block's second slot, then the others' first
  auto slot = [&](int i) {
    return (static_cast<int64_t>(2 * (first + i)) + (i == 0 ? 1 : 0)) * tile_rows + r;
  };
  auto part_o = [&](int i) {
    return *reinterpret_cast<const float4*>(a.part_o + slot(i) * D + 4 * col);
  };
  float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
  if (group < n) y = part_o(group);
  float top = kLowest;
  for (int i = tid; i < n; i += threads) top = fmaxf(top, a.part_ml[slot(i)].x);
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
  if (lane == 0) red[warp] = top;
  __syncthreads();
  for (int w = 0; w < warps; ++w) top = fmaxf(top, red[w]);
  float sum = 0.f;
  for (int i = tid; i < n; i += threads) {
    const float2 ml = a.part_ml[slot(i)];
    const float w = ex2(ml.x - top);
    weight[i] = w;
    sum += w * ml.y;
  }
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
  if (lane == 0) red_l[warp] = sum;
  __syncthreads();
  sum = 0.f;
  for (int w = 0; w < warps; ++w) sum += red_l[w];
  if (group < n) {
    const float w = weight[group];
    y.x *= w, y.y *= w, y.z *= w, y.w *= w;
  }
#pragma unroll 8
  for (int i = group + groups; i < n; i += groups) {
    const float w = weight[i];
    const float4 o = part_o(i);
    y.x = fmaf(w, o.x, y.x), y.y = fmaf(w, o.y, y.y);
    y.z = fmaf(w, o.z, y.z), y.w = fmaf(w, o.w, y.w);
  }
  part[group][col] = y;
  __syncthreads();
  if (group == 0) {
    for (int g = 1; g < groups; ++g) {
      const float4 o = part[g][col];
      y.x += o.x, y.y += o.y, y.z += o.z, y.w += o.w;
    }
    const Sequence seq = sequence(a, b);
    const bool real = (row0 + r) % a.n_q < seq.fresh;
    const float inv = real && sum != 0.f ? 1.f / sum : 0.f;
    const int64_t row = (static_cast<int64_t>(b) * a.h_kv + head) * a.rows + row0 + r;
    *reinterpret_cast<uint2*>(a.out + row * D + 4 * col) =
        inv == 0.f ? make_uint2(0u, 0u) : output4(y, inv, a.v_factor);
  }
}

// ------------------------------------------------------------------ launch

struct Layout {
  int row_tiles, tile_rows;
  bool unsplit, eight_warps;
  int64_t units;          // at most
  int blocks;             // at most
  size_t ml_off, o_off, total;
};

Layout layout(int B, int h, int h_kv, int n_q, int d, int page_size, int max_pages) {
  Layout w;
  const int rows = h / h_kv * n_q;
  const Plan p = plan(rows, int64_t(B) * h_kv, int64_t(max_pages) * page_size);
  w.tile_rows = p.tile_rows;
  w.unsplit = p.unsplit;
  w.eight_warps = p.eight_warps;
  w.row_tiles = (rows + w.tile_rows - 1) / w.tile_rows;
  const int64_t per_pair = 1 + (int64_t(max_pages) * page_size + kUnit - 1) / kUnit;
  w.units = int64_t(B) * h_kv * w.row_tiles * per_pair;
  w.blocks = static_cast<int>(w.units < kMaxBlocks ? w.units : kMaxBlocks);
  auto align = [](size_t x) { return (x + 255u) & ~size_t(255u); };
  w.ml_off = align(size_t(w.blocks) * sizeof(int2));
  w.o_off = w.ml_off + align(size_t(w.blocks) * 2 * w.tile_rows * sizeof(float2));
  w.total = w.o_off + align(size_t(w.blocks) * 2 * w.tile_rows * d * sizeof(float));
  if (w.total < 256) w.total = 256;
  return w;
}

// Blocks of this instance that fit on the current device at once (cached per device).
template <typename Kernel>
cudaError_t resident_blocks(Kernel kernel, int threads, int smem, int* cache, int* out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int n = dev >= 0 && dev < 64 ? __atomic_load_n(&cache[dev], __ATOMIC_ACQUIRE) : 0;
  if (n == 0) {
    int sms = 0, per_sm = 0;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess)
      e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, smem);
    if (e != cudaSuccess) return e;
    if (sms < 1 || per_sm < 1) return cudaErrorInvalidConfiguration;
    n = sms * per_sm;
    if (dev >= 0 && dev < 64) __atomic_store_n(&cache[dev], n, __ATOMIC_RELEASE);
  }
  *out = n;
  return cudaSuccess;
}

template <int D, int NT, bool Q4, int W>
cudaError_t launch_instance(PagedArgs a, const Layout& w, cudaStream_t stream) {
  auto kernel = decode_paged_kernel<D, NT, Q4, W>;
  constexpr int smem = Shape<D, NT, Q4, W>::kSmem;
  static unsigned long long configured = 0;
  static int resident[64] = {};
  cudaError_t e = set_smem_once(kernel, smem, &configured);
  int fit = 0;
  if (e == cudaSuccess) e = resident_blocks(kernel, 32 * W, smem, resident, &fit);
  if (e != cudaSuccess) return e;
  const unsigned blocks = static_cast<unsigned>(fit < w.blocks ? fit : w.blocks);
  // few pairs: look at each for what has to be joined; many: at the blocks,
  // each of which begins at most one that others finish
  const int64_t pairs = int64_t(a.B) * a.h_kv * a.row_tiles;
  a.by_pair = pairs <= static_cast<int64_t>(blocks);
  e = launch_pdl(kernel, dim3(blocks), dim3(32 * W), smem, stream, a);
  if (e != cudaSuccess || a.unsplit) return e;
  const unsigned rows = static_cast<unsigned>(a.rows < w.tile_rows ? a.rows : w.tile_rows);
  // more threads to a row where a pair has many contributions on the average
  const unsigned threads = pairs * 4 <= static_cast<int64_t>(blocks) ? kMergeThreads : 128;
  return launch_pdl(decode_paged_merge_kernel<D>,
                    dim3(a.by_pair ? static_cast<unsigned>(pairs) : blocks, rows),
                    dim3(threads), 0, stream, a, w.tile_rows);
}

template <int D, bool Q4>
cudaError_t launch_rows(const PagedArgs& a, const Layout& w, cudaStream_t stream) {
  if (w.eight_warps) return launch_instance<D, 1, Q4, 8>(a, w, stream);
  if (w.tile_rows == 8) return launch_instance<D, 1, Q4, 4>(a, w, stream);
  if (w.tile_rows == 16) return launch_instance<D, 2, Q4, 4>(a, w, stream);
  return launch_instance<D, 4, Q4, 4>(a, w, stream);
}

}  // namespace

size_t decode_paged_workspace_bytes(int B, int h, int h_kv, int n_q, int d, int page_size,
                                    int max_pages) {
  return layout(B, h, h_kv, n_q, d, page_size, max_pages).total;
}

int64_t decode_paged_units(int B, int h, int h_kv, int n_q, int d, int page_size, int max_pages) {
  return layout(B, h, h_kv, n_q, d, page_size, max_pages).units;
}

cudaError_t launch_decode_paged(const PagedDecodeProblem& p, cudaStream_t stream) {
  const PagedCache& c = p.cache;
  const Layout w = layout(p.B, p.h, c.h_kv, p.n_q, c.d, 1 << c.page_shift, c.max_pages);
  if (p.B < 1 || p.h < 1 || p.n_q < 1 || w.units > kPagedMaxUnits) return cudaErrorInvalidValue;
  const bool q4 = c.k_scales != nullptr;
  PagedArgs a;
  a.q = p.q;
  a.out = p.out;
  a.k = static_cast<const uint8_t*>(c.k);
  a.v = static_cast<const uint8_t*>(c.v);
  a.k_scales = c.k_scales;
  a.v_scales = c.v_scales;
  a.table = c.table;
  a.lens = c.lens;
  a.new_lens = c.new_lens;
  uint8_t* ws = static_cast<uint8_t*>(p.workspace);
  a.split = reinterpret_cast<int2*>(ws);
  a.part_ml = reinterpret_cast<float2*>(ws + w.ml_off);
  a.part_o = reinterpret_cast<float*>(ws + w.o_off);
  a.B = p.B;
  a.h_kv = c.h_kv;
  a.n_q = p.n_q;
  a.rows = p.h / c.h_kv * p.n_q;
  a.row_tiles = w.row_tiles;
  a.n_pages = c.n_pages;
  a.page_shift = c.page_shift;
  a.max_pages = c.max_pages;
  a.unsplit = w.unsplit;
  a.causal = p.causal;
  a.scale_log2 = p.scale * 1.4426950408889634f * (q4 ? c.k_factor : 1.f);
  a.v_factor = q4 ? c.v_factor : 1.f;
  if (c.d == 64) return q4 ? launch_rows<64, true>(a, w, stream) : launch_rows<64, false>(a, w, stream);
  if (c.d == 128)
    return q4 ? launch_rows<128, true>(a, w, stream) : launch_rows<128, false>(a, w, stream);
  return cudaErrorInvalidValue;
}

TSD_DEFINE_ERROR_READER(take_device_error_paged)

}  // namespace tsd
