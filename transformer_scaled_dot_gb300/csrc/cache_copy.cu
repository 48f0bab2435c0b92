// cache_copy.cu -- copies rows of pages of a key/value cache by a list of
// (from page, to page, rows), for keys and values of all layers in one launch.
//
// It moves bytes: one read and one write of each. A pool is
// [layers][n_pages][h_kv][page_size][row bytes]; a whole page is one run of
// memory, the first rows of a page one run for each head. The runs of one
// (copy, layer, pool) end to end are cut into pieces of 4 KB, a warp to a piece,
// with eight 16-byte loads of every lane in flight before the first store. The
// list's length is read on the device (the call that made the list has just
// written it), so the grid is what fits and its warps walk over the pieces;
// pieces are numbered as if every copy were of whole pages, and those past the
// end of a shorter one are passed over.
#include "kernels.h"
#include "sm103.cuh"

namespace tsd {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kInFlight = 8;
constexpr int kPiece = 32 * kInFlight * 16;  // bytes

struct Pieces {
  int before[4];  // of a copy's pieces in a layer, those of the pools before each
  int in_layer;
};

// Bytes [begin, begin + kPiece) of `runs` runs of run_bytes, `stride` apart, in
// vectors of `Vec` (a divisor of run_bytes).
template <typename Vec>
__device__ __forceinline__ void copy_runs(uint8_t* to, const uint8_t* from, int begin, int runs, int run_bytes, int stride,
                                          int lane) {
  constexpr int kBytes = static_cast<int>(sizeof(Vec));
  const int per = run_bytes / kBytes;
  const int n = min(runs * per, (begin + kPiece) / kBytes);
  for (int e0 = begin / kBytes + lane; e0 - lane < n; e0 += 32 * kInFlight) {
    Vec v[kInFlight];
    int64_t at[kInFlight];
#pragma unroll
    for (int i = 0; i < kInFlight; ++i) {
      const int e = e0 + i * 32;
      const int run = e / per;
      at[i] = static_cast<int64_t>(run) * stride + (e - run * per) * kBytes;
      if (e < n) v[i] = __ldcs(reinterpret_cast<const Vec*>(from + at[i]));
    }
#pragma unroll
    for (int i = 0; i < kInFlight; ++i)
      if (e0 + i * 32 < n) *reinterpret_cast<Vec*>(to + at[i]) = v[i];
  }
}

__global__ void __launch_bounds__(kThreads) cache_copy_kernel(const CopyProblem p, const Pieces pieces) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = static_cast<int>(lane_id());
  const int page_size = 1 << p.page_shift;
  const int64_t per_copy = static_cast<int64_t>(p.n_layers) * pieces.in_layer;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
  int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + warp_id();
  int64_t units = static_cast<int64_t>(p.max_copies) * per_copy;
  bool counted = p.n_copies == nullptr;
  for (; u < units; u += step) {
    const int64_t c = units < INT32_MAX ? static_cast<int>(u) / static_cast<int>(per_copy) : u / per_copy;
    const int64_t rest = u - c * per_copy;
    const int from = __ldcg(p.copies + 3 * c), to = __ldcg(p.copies + 3 * c + 1), rows = __ldcg(p.copies + 3 * c + 2);
    if (!counted) {  // the first copy is on its way
      const int n = __ldcg(p.n_copies);
      if (n > p.max_copies && u == 0 && lane == 0) atomicOr(&g_device_error, kErrIndex);
      units = static_cast<int64_t>(min(max(n, 0), p.max_copies)) * per_copy;
      counted = true;
      if (u >= units) break;
    }
    if (from < 0 || from >= p.n_pages || to < 0 || to >= p.n_pages || rows < 0 || rows > page_size) {
      if (lane == 0) atomicOr(&g_device_error, kErrIndex);
      continue;
    }
    const int layer = units < INT32_MAX ? static_cast<int>(rest) / pieces.in_layer : static_cast<int>(rest / pieces.in_layer);
    int piece = static_cast<int>(rest - static_cast<int64_t>(layer) * pieces.in_layer);
    int pool = 0;
#pragma unroll
    for (int i = 1; i < 4; ++i)
      if (i < p.n_pools && piece >= pieces.before[i]) pool = i;
    uint8_t* base = static_cast<uint8_t*>(p.pool[0]);
    int row = p.row_bytes[0], skipped = 0;
#pragma unroll
    for (int i = 1; i < 4; ++i) {
      if (pool != i) continue;
      base = static_cast<uint8_t*>(p.pool[i]);
      row = p.row_bytes[i];
      skipped = pieces.before[i];
    }
    piece -= skipped;
    const int page_bytes = (p.h_kv * row) << p.page_shift;
    base += layer * p.layer_rows * row;
    const uint8_t* src = base + static_cast<int64_t>(from) * page_bytes;
    uint8_t* dst = base + static_cast<int64_t>(to) * page_bytes;
    const int begin = piece * kPiece;
    const int run_bytes = rows * row;
    if (rows == page_size) {  // one run
      const int last = min(begin + kPiece, page_bytes) - begin;
      src += begin;
      dst += begin;
      uint4 v[kInFlight];
#pragma unroll
      for (int i = 0; i < kInFlight; ++i)
        if ((i * 32 + lane) * 16 < last) v[i] = __ldcs(reinterpret_cast<const uint4*>(src) + i * 32 + lane);
#pragma unroll
      for (int i = 0; i < kInFlight; ++i)
        if ((i * 32 + lane) * 16 < last) reinterpret_cast<uint4*>(dst)[i * 32 + lane] = v[i];
    } else if (begin < p.h_kv * run_bytes) {
      // scales of a row: 4 bytes for 64 columns, 8 for 128
      if (run_bytes % 16 == 0) copy_runs<uint4>(dst, src, begin, p.h_kv, run_bytes, row << p.page_shift, lane);
      else copy_runs<uint32_t>(dst, src, begin, p.h_kv, run_bytes, row << p.page_shift, lane);
    }
  }
}

}  // namespace

cudaError_t launch_cache_copy(const CopyProblem& p, cudaStream_t stream) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  Pieces pieces = {};
  for (int i = 0; i < p.n_pools; ++i) {
    pieces.before[i] = pieces.in_layer;
    pieces.in_layer += static_cast<int>(((static_cast<int64_t>(p.h_kv) * p.row_bytes[i] << p.page_shift) + kPiece - 1) / kPiece);
  }
  const int64_t units = static_cast<int64_t>(p.max_copies) * p.n_layers * pieces.in_layer;
  const int64_t blocks = (units + kWarps - 1) / kWarps, grid = static_cast<int64_t>(sms) * 8;
  return launch_pdl(cache_copy_kernel, dim3(static_cast<unsigned>(blocks < grid ? blocks : grid)), dim3(kThreads), 0, stream, p,
                    pieces);
}

TSD_DEFINE_ERROR_READER(take_device_error_copy)

}  // namespace tsd
