// cache_copy.cu -- copies rows of pages of a key/value cache by a list of
// (from page, to page, rows), for keys and values of all layers in one launch.
//
// It moves bytes: one read and one write of each. A pool is
// [layers][n_pages][h_kv][page_size][row bytes]; a whole page is one run of
// memory, the first rows of a page one run for each head. The runs of one
// (copy, layer, pool) end to end are cut into pieces of 4 KB, a warp to a piece,
// with eight 16-byte loads of every lane in flight before the first store. The
// list's length is read on the device (the call that made the list has just
// written it), so the grid is what fits and its warps walk over the pieces:
// all copies' first ones, then all second ones, so that the copies that are of
// whole pages and those of a few rows keep all warps busy. A piece past the end
// of a copy is passed over.
#include "kernels.h"
#include "sm103.cuh"

namespace tsd {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kInFlight = 8;
constexpr int kBlocksPerSm = 3;
constexpr int kShortList = 512;
constexpr int kPiece = 32 * kInFlight * 16;  // bytes

// Pieces of a page of rows or codes, and of their scales.
struct Pieces {
  int rows, scales;
};
// Pieces of so many 16-byte vectors.
__host__ __device__ __forceinline__ int pieces_of(int vectors) { return (vectors + kPiece / 16 - 1) / (kPiece / 16); }

__global__ void __launch_bounds__(kThreads, kBlocksPerSm) cache_copy_kernel(const CopyProblem p, Pieces pieces) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = static_cast<int>(lane_id());
  const int page_size = 1 << p.page_shift;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
  // The list's length; of a short list (mostly rows' last pages) the most rows of a
  // copy too, which most pages' later pieces lie past. One at least, and a whole page
  // where a number is negative: a unit of each copy checks its numbers.
  int n = p.max_copies, most_rows = page_size;
  if (p.max_copies <= kShortList) {
    int rows[kShortList / 32];
#pragma unroll
    for (int i = 0; i < kShortList / 32; ++i) rows[i] = i * 32 + lane < p.max_copies ? p.copies[3 * (i * 32 + lane) + 2] : 0;
    if (p.n_copies != nullptr) n = __ldcg(p.n_copies);
    unsigned most = 1u;
#pragma unroll
    for (int i = 0; i < kShortList / 32; ++i) most = max(most, i * 32 + lane < n ? static_cast<unsigned>(rows[i]) : 0u);
    most_rows = static_cast<int>(min(__reduce_max_sync(0xffffffffu, most), static_cast<unsigned>(page_size)));
  } else if (p.n_copies != nullptr) {
    n = __ldcg(p.n_copies);
  }
  if (n > p.max_copies && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&g_device_error, kErrIndex);
  n = min(max(n, 0), p.max_copies);
  if (most_rows < page_size) {
    pieces.rows = pieces_of((most_rows * p.row_bytes[0] + 15) / 16 * p.h_kv);
    if (pieces.scales > 0) pieces.scales = pieces_of((most_rows * p.row_bytes[2] + 15) / 16 * p.h_kv);
  }
  // units: all copies' and layers' first pieces, then their second ones, and so on;
  // of all pools while the scales have some
  const int quads = 4 * pieces.scales, in_layer = 2 * (pieces.rows + pieces.scales);
  const int64_t per_piece = static_cast<int64_t>(n) * p.n_layers;
  const int64_t units = per_piece * in_layer;
  const bool small = units < INT32_MAX;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + warp_id(); u < units; u += step) {
    const int q = static_cast<int>(small ? static_cast<int>(u) / static_cast<int>(per_piece) : u / per_piece);
    const int64_t rest = u - q * per_piece;
    const int c = static_cast<int>(small ? static_cast<int>(rest) / p.n_layers : rest / p.n_layers);
    const int layer = static_cast<int>(rest - static_cast<int64_t>(c) * p.n_layers);
    const int32_t* copy = p.copies + 3 * static_cast<int64_t>(c);
    const int from = copy[0], to = copy[1], rows = copy[2];
    if (from < 0 || from >= p.n_pages || to < 0 || to >= p.n_pages || rows < 0 || rows > page_size) {
      if (lane == 0) atomicOr(&g_device_error, kErrIndex);
      continue;
    }
    // pools 0 and 1 hold rows or codes, 2 and 3 scales
    const int pool = q < quads ? q & 3 : q & 1;
    const int piece = q < quads ? q >> 2 : pieces.scales + ((q - quads) >> 1);
    uint8_t* base = static_cast<uint8_t*>(p.pool[0]);
    int row = p.row_bytes[0];
#pragma unroll
    for (int i = 1; i < 4; ++i) {
      if (pool != i) continue;
      base = static_cast<uint8_t*>(p.pool[i]);
      row = p.row_bytes[i];
    }
    const int page_bytes = (p.h_kv * row) << p.page_shift;
    base += layer * p.layer_rows * row;
    const uint8_t* src = base + static_cast<int64_t>(from) * page_bytes;
    uint8_t* dst = base + static_cast<int64_t>(to) * page_bytes;
    // 16 bytes at a time; a run's last ones may be 4, 8 or 12: scales of a part
    // of a page, where a row has 4 bytes (64 columns) or 8
    const bool whole = rows == page_size;  // one run
    const int run_bytes = whole ? page_bytes : rows * row;
    const int per = (run_bytes + 15) / 16, rest_bytes = run_bytes & 15;
    const int vectors = whole ? per : p.h_kv * per;
    const int begin = piece * (kPiece / 16);
    if (begin >= vectors) continue;
    int at[kInFlight];  // where this lane's lie in the page; -1: none
    uint32_t cut = 0u;  // bit i: the i-th is a run's last and short
    const float inverse = 1.f / static_cast<float>(per);
#pragma unroll
    for (int i = 0; i < kInFlight; ++i) {
      const int e = begin + i * 32 + lane;
      at[i] = e * 16;
      if (!whole) {
        // the product is 1 / (2 per) off a whole number at least, and below 2^20 off by a quarter of that
        const int run = vectors < 1 << 20 ? static_cast<int>((static_cast<float>(e) + 0.5f) * inverse) : e / per;
        at[i] = run * (row << p.page_shift) + (e - run * per) * 16;
        if (rest_bytes != 0 && e - run * per == per - 1) cut |= 1u << i;
      }
      if (e >= vectors) at[i] = -1;
    }
    uint4 v[kInFlight];
    if (rest_bytes == 0) {
#pragma unroll
      for (int i = 0; i < kInFlight; ++i)
        if (at[i] >= 0) v[i] = __ldcs(reinterpret_cast<const uint4*>(src + at[i]));
#pragma unroll
      for (int i = 0; i < kInFlight; ++i)
        if (at[i] >= 0) *reinterpret_cast<uint4*>(dst + at[i]) = v[i];
    } else {
#pragma unroll
      for (int i = 0; i < kInFlight; ++i) {
        if (at[i] < 0) continue;
        const uint32_t* w = reinterpret_cast<const uint32_t*>(src + at[i]);
        if (cut >> i & 1u) {
          v[i].x = __ldcs(w);
          if (rest_bytes > 4) v[i].y = __ldcs(w + 1);
          if (rest_bytes > 8) v[i].z = __ldcs(w + 2);
        } else {
          v[i] = __ldcs(reinterpret_cast<const uint4*>(w));
        }
      }
#pragma unroll
      for (int i = 0; i < kInFlight; ++i) {
        if (at[i] < 0) continue;
        uint32_t* w = reinterpret_cast<uint32_t*>(dst + at[i]);
        if (cut >> i & 1u) {
          w[0] = v[i].x;
          if (rest_bytes > 4) w[1] = v[i].y;
          if (rest_bytes > 8) w[2] = v[i].z;
        } else {
          *reinterpret_cast<uint4*>(w) = v[i];
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_cache_copy(const CopyProblem& p, cudaStream_t stream) {
  static int cached = 0;  // atomic accesses: launches may come from several host threads
  int sms = __atomic_load_n(&cached, __ATOMIC_RELAXED);
  if (sms == 0) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    __atomic_store_n(&cached, sms, __ATOMIC_RELAXED);
  }
  // a page has 2^26 vectors at most, and its rows a multiple of 16 bytes between heads
  auto whole = [&](int row_bytes) {
    return pieces_of(static_cast<int>((static_cast<int64_t>(p.h_kv) * row_bytes << p.page_shift) / 16));
  };
  const Pieces pieces = {whole(p.row_bytes[0]), p.n_pools == 4 ? whole(p.row_bytes[2]) : 0};
  const int64_t units = static_cast<int64_t>(p.max_copies) * p.n_layers * 2 * (pieces.rows + pieces.scales);
  // A long list is shared out among more blocks than are resident, so that SMs
  // which are done sooner take more of them; a short one, which may be shorter
  // than it says and its pages than whole ones, goes to the resident ones (in us, 8
  // and 3 blocks to an SM: 2500 whole pages of 64 KB in 4 layers 177 and 192; up to
  // 384 parts of 64 KB pages in 2 layers 16.1 and 14.8 with the step).
  const int64_t blocks = (units + kWarps - 1) / kWarps, most = sms * (p.max_copies > kShortList ? 8 : kBlocksPerSm);
  const int64_t grid = blocks > most ? most : blocks;
  return launch_pdl(cache_copy_kernel, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, stream, p, pieces);
}

TSD_DEFINE_ERROR_READER(take_device_error_copy)

}  // namespace tsd
