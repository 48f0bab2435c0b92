// cache_copy.cu -- copies rows of pages of a key/value cache by a list of
// (from page, to page, rows), for keys and values of all layers in one launch.
//
// It moves bytes: one read and one write of each. A pool is
// [layers][n_pages][h_kv][page_size][row bytes]; a whole page is one run of
// memory, the first rows of a page one run for each head. A block takes pieces
// of 16 KB of one (copy, layer, pool), four 16-byte loads of every thread in
// flight before the first store. The list's length is read on the device (the
// call that made the list has just written it), so the grid is what fits and
// its blocks walk over the pieces.
#include "kernels.h"
#include "sm103.cuh"

namespace tsd {

namespace {

constexpr int kThreads = 256;
constexpr int kInFlight = 4;
constexpr int kPiece = kThreads * kInFlight * 16;  // bytes

template <typename Vec>
__device__ __forceinline__ void copy_piece(uint8_t* to, const uint8_t* from, int piece, int runs, int run_bytes,
                                           int stride) {
  constexpr int kBytes = static_cast<int>(sizeof(Vec));
  const int per = run_bytes / kBytes;
  const int n = runs * per;
  const int begin = piece * (kPiece / 16);
  // a piece is as many vectors whatever their size: narrow ones make small pieces
  Vec v[kInFlight];
  int64_t at[kInFlight];
#pragma unroll
  for (int i = 0; i < kInFlight; ++i) {
    const int e = begin + i * kThreads + static_cast<int>(threadIdx.x);
    const int run = runs > 1 ? e / per : 0;
    at[i] = static_cast<int64_t>(run) * stride + static_cast<int64_t>(e - run * per) * kBytes;
    if (e < n) v[i] = __ldcs(reinterpret_cast<const Vec*>(from + at[i]));
  }
#pragma unroll
  for (int i = 0; i < kInFlight; ++i) {
    const int e = begin + i * kThreads + static_cast<int>(threadIdx.x);
    if (e < n) *reinterpret_cast<Vec*>(to + at[i]) = v[i];
  }
}

__global__ void __launch_bounds__(kThreads) cache_copy_kernel(const CopyProblem p, int pieces) {
  griddep_wait();
  griddep_launch_dependents();
  int n = p.n_copies ? __ldcg(p.n_copies) : p.max_copies;
  if (n > p.max_copies) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&g_device_error, kErrIndex);
    n = p.max_copies;
  }
  const int page_size = 1 << p.page_shift;
  const int64_t per_copy = static_cast<int64_t>(p.n_layers) * p.n_pools * pieces;
  const int64_t units = static_cast<int64_t>(n < 0 ? 0 : n) * per_copy;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t c = u / per_copy;
    const int64_t rest = u - c * per_copy;
    const int part = static_cast<int>(rest / pieces), piece = static_cast<int>(rest - static_cast<int64_t>(part) * pieces);
    const int layer = part / p.n_pools, pool = part - layer * p.n_pools;
    const int from = __ldcg(p.copies + 3 * c), to = __ldcg(p.copies + 3 * c + 1), rows = __ldcg(p.copies + 3 * c + 2);
    if (from < 0 || from >= p.n_pages || to < 0 || to >= p.n_pages || rows < 0 || rows > page_size) {
      if (threadIdx.x == 0) atomicOr(&g_device_error, kErrIndex);
      continue;
    }
    const int row = p.row_bytes[pool];
    uint8_t* base = static_cast<uint8_t*>(p.pool[pool]) + layer * p.layer_rows * row;
    const int64_t page_bytes = static_cast<int64_t>(p.h_kv) * page_size * row;
    // a whole page is one run
    const bool whole = rows == page_size;
    const int runs = whole ? 1 : p.h_kv;
    const int run_bytes = whole ? static_cast<int>(page_bytes) : rows * row;
    if (run_bytes % 16 == 0) {
      copy_piece<uint4>(base + to * page_bytes, base + from * page_bytes, piece, runs, run_bytes, page_size * row);
    } else {  // scales of a part of a page: 4 bytes for each row of 64 columns, 8 of 128
      copy_piece<uint32_t>(base + to * page_bytes, base + from * page_bytes, piece, runs, run_bytes, page_size * row);
    }
  }
}

}  // namespace

cudaError_t launch_cache_copy(const CopyProblem& p, cudaStream_t stream) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  int64_t most = 0;  // vectors of a page of any pool: 16 bytes, or 4 where a run may not be a multiple of 16
  for (int i = 0; i < p.n_pools; ++i) {
    const int64_t bytes = static_cast<int64_t>(p.h_kv) * p.row_bytes[i] << p.page_shift;
    const int64_t vecs = p.row_bytes[i] % 16 == 0 ? bytes / 16 : bytes / 4;
    most = vecs > most ? vecs : most;
  }
  const int pieces = static_cast<int>((most + kPiece / 16 - 1) / (kPiece / 16));
  const int64_t units = static_cast<int64_t>(p.max_copies) * p.n_layers * p.n_pools * pieces;
  const int64_t grid = static_cast<int64_t>(sms) * 8;
  return launch_pdl(cache_copy_kernel, dim3(static_cast<unsigned>(units < grid ? units : grid)), dim3(kThreads), 0, stream, p,
                    pieces);
}

TSD_DEFINE_ERROR_READER(take_device_error_copy)

}  // namespace tsd
