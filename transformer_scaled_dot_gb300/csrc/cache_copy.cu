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
constexpr int kBlocksPerSm = 3;
constexpr int kPiece = 32 * kInFlight * 16;  // bytes

struct Pieces {
  int before[4];  // of a copy's pieces in a layer, those of the pools before each
  int in_layer;
};

__global__ void __launch_bounds__(kThreads, kBlocksPerSm) cache_copy_kernel(const CopyProblem p, const Pieces pieces) {
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
    // 16 bytes at a time; a run's last ones may be 4, 8 or 12: scales of a part
    // of a page, where a row has 4 bytes (64 columns) or 8
    const bool whole = rows == page_size;  // one run
    const int run_bytes = whole ? page_bytes : rows * row;
    const int per = (run_bytes + 15) / 16, rest_bytes = run_bytes & 15;
    const int n = whole ? per : p.h_kv * per;
    const int begin = piece * (kPiece / 16);
    if (begin >= n) continue;
    int at[kInFlight];  // where this lane's lie in the page; -1: none
    uint32_t cut = 0u;  // bit i: the i-th is a run's last and short
    const float inverse = 1.f / static_cast<float>(per);
#pragma unroll
    for (int i = 0; i < kInFlight; ++i) {
      const int e = begin + i * 32 + lane;
      at[i] = e * 16;
      if (!whole) {
        // the product is 1 / (2 per) off a whole number at least, and below 2^20 off by a quarter of that
        const int run = n < 1 << 20 ? static_cast<int>((static_cast<float>(e) + 0.5f) * inverse) : e / per;
        at[i] = run * (row << p.page_shift) + (e - run * per) * 16;
        if (rest_bytes != 0 && e - run * per == per - 1) cut |= 1u << i;
      }
      if (e >= n) at[i] = -1;
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
  Pieces pieces = {};
  for (int i = 0; i < p.n_pools; ++i) {
    pieces.before[i] = pieces.in_layer;
    pieces.in_layer += static_cast<int>(((static_cast<int64_t>(p.h_kv) * p.row_bytes[i] << p.page_shift) + kPiece - 1) / kPiece);
  }
  const int64_t units = static_cast<int64_t>(p.max_copies) * p.n_layers * pieces.in_layer;
  // A long list is shared out among more blocks than are resident, so that SMs
  // which are done sooner take more of them; a short one goes to the resident
  // ones, as a block more costs more than a second round (in us, 8 and 3 blocks
  // to an SM: 2500 whole pages of 64 KB in 4 layers 176 and 184, 240 of 32 KB in 6
  // layers 17.7 and 18.4 with the plan; parts of 120 4-bit pages in 4 layers, 1152
  // blocks' pieces, 15.6 and 14.4 with the step).
  const int64_t blocks = (units + kWarps - 1) / kWarps, most = static_cast<int64_t>(sms) * 8, resident = sms * kBlocksPerSm;
  const int64_t grid = blocks > most ? most : blocks > resident ? resident : blocks;
  return launch_pdl(cache_copy_kernel, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, stream, p, pieces);
}

TSD_DEFINE_ERROR_READER(take_device_error_copy)

}  // namespace tsd
