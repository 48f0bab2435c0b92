// cache_pages.cu -- keeping the pages of a paged key/value cache: giving rows
// the pages of the rows they continue (fork), finding pages for new tokens
// (reserve), giving pages back (release), and moving the used pages to the
// front of the pool (compact).
//
// The state is the page table [B, max_pages], -1 where a row has no page, and
// how many table entries name each page (0: a free page). There is no list of
// free pages that one call would leave to the next: the lowest free pages are
// found in the counts, so that the pages a call takes follow from its
// arguments alone, and the pool stays dense by itself. The counts of 2^18
// pages are 1 MB, two microseconds' reading for one cluster.
//
// All of it is integer work on a few hundred kilobytes and bound by latency:
// dependent reads of the L2 and barriers between phases. What needs an order
// over all rows or pages (which page is the j-th free one, which row the j-th
// to need one) runs in one thread-block cluster, whose barrier costs less than
// a second launch.
#include "kernels.h"
#include "sm103.cuh"

namespace tsd {

namespace {

constexpr uint32_t kAll = 0xffffffffu;

// ---------------------------------------------------------------- fork

// Row r becomes row parents[r], all rows at once. A block takes kCols columns
// of every row through shared memory, which is what makes it safe in place:
// no other block reads or writes them. A count changes only where an entry
// does, so that the pages that a row shares with its parent already cost
// nothing.
constexpr int kForkThreads = 512;
constexpr int kForkEntries = kForkMaxRows;  // of a block: 128 KB of shared memory

__global__ void __launch_bounds__(kForkThreads)
    cache_fork_kernel(const PagesProblem p, int32_t* lens, const int32_t* parents, int cols_log2) {
  extern __shared__ int32_t old[];  // [B][cols]
  griddep_wait();
  griddep_launch_dependents();
  const int cols = 1 << cols_log2;
  const bool for_lens = lens != nullptr && blockIdx.x == gridDim.x - 1;
  const int n = for_lens ? p.B : p.B << cols_log2;
  const int col0 = static_cast<int>(blockIdx.x) << cols_log2;
  auto entry = [&](int i) -> int32_t* {
    if (for_lens) return lens + i;
    const int col = col0 + (i & (cols - 1));
    return col < p.max_pages ? p.table + static_cast<int64_t>(i >> cols_log2) * p.max_pages + col : nullptr;
  };
  for (int i = threadIdx.x; i < n; i += kForkThreads) {
    const int32_t* e = entry(i);
    old[i] = e ? *e : -1;
  }
  __syncthreads();
  const int shift = for_lens ? 0 : cols_log2;
  for (int i = threadIdx.x; i < n; i += kForkThreads) {
    const int r = i >> shift;
    const int parent = __ldg(parents + r);
    if (parent < -1 || parent >= p.B) {
      if (for_lens || blockIdx.x == 0) atomicOr(&g_device_error, kErrIndex);
      continue;
    }
    const int32_t was = old[i];
    const int32_t now = parent < 0 ? (for_lens ? 0 : -1) : old[(parent << shift) | (i & ((1 << shift) - 1))];
    if (now == was) continue;
    int32_t* e = entry(i);
    if (e == nullptr) continue;
    *e = now;
    if (for_lens) continue;
    if (now >= 0 && now < p.n_pages) atomicAdd(p.counts + now, 1);
    if (was >= 0 && was < p.n_pages) atomicSub(p.counts + was, 1);
    if (now >= p.n_pages || was >= p.n_pages) atomicOr(&g_device_error, kErrIndex);
  }
}

// ---------------------------------------------------------------- release

constexpr int kReleaseThreads = 256;

__global__ void __launch_bounds__(kReleaseThreads)
    cache_release_kernel(const PagesProblem p, const int32_t* keep_lens, int64_t items, int chunks) {
  griddep_wait();
  griddep_launch_dependents();
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int b = static_cast<int>(item / chunks);
    const int col = static_cast<int>(item % chunks) * kReleaseThreads + static_cast<int>(threadIdx.x);
    const int keep = keep_lens ? __ldg(keep_lens + b) : 0;
    // a negative number keeps the row as it is
    const int64_t first = keep < 0 ? p.max_pages : (static_cast<int64_t>(keep) + (1 << p.page_shift) - 1) >> p.page_shift;
    if (col < first || col >= p.max_pages) continue;
    int32_t* e = p.table + static_cast<int64_t>(b) * p.max_pages + col;
    const int page = *e;
    if (page == -1) continue;
    *e = -1;
    if (page >= 0 && page < p.n_pages) atomicSub(p.counts + page, 1);
    if (page >= p.n_pages) atomicOr(&g_device_error, kErrIndex);
  }
}

// ---------------------------------------------------------------- one cluster

constexpr int kClusterThreads = 1024;
constexpr int kMaxCtas = 8;  // of the cluster (the portable size)
constexpr int kWarps = kClusterThreads / 32;

struct ClusterSmem {
  uint64_t warp_sum[kWarps];
  uint64_t cta_sum[2][kMaxCtas];  // written by the cluster's CTAs; used in turn
};

// The sum of `v` over the threads before this one, CTAs in order of rank;
// *total over all. Threads of every CTA call it together. Which of the two
// rows of cta_sum it uses alternates, so that a CTA that is ahead does not
// overwrite what another still reads (between two uses of a row lies the
// barrier of the other).
__device__ __forceinline__ uint64_t cluster_scan(uint64_t v, ClusterSmem& sm, int row, uint32_t rank,
                                                 uint32_t ctas, uint64_t* total) {
  const int lane = static_cast<int>(lane_id()), warp = warp_id();
  uint64_t sum = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t other = __shfl_up_sync(kAll, sum, o);
    if (lane >= o) sum += other;
  }
  __syncthreads();  // warp_sum's previous use is over
  if (lane == 31) sm.warp_sum[warp] = sum;
  __syncthreads();
  uint64_t before = sum - v;
  uint64_t mine = sm.warp_sum[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t other = __shfl_up_sync(kAll, mine, o);
    if (lane >= o) mine += other;
  }
  const uint64_t cta_total = __shfl_sync(kAll, mine, 31);
  const uint64_t warps_before = __shfl_sync(kAll, mine, (warp + 31) & 31);
  if (warp > 0) before += warps_before;
  if (threadIdx.x < ctas) st_cluster_u64(cluster_map(&sm.cta_sum[row][rank], threadIdx.x), cta_total);
  cluster_sync();
  uint64_t all = 0;
  for (uint32_t c = 0; c < ctas; ++c) {
    const uint64_t t = sm.cta_sum[row][c];
    if (c < rank) before += t;
    all += t;
  }
  *total = all;
  return before;
}

// Pages of one warp: [begin, end), in steps of 128.
struct Slice {
  int begin, end;
};
__device__ __forceinline__ Slice warp_slice(int n_pages, uint32_t rank, uint32_t ctas) {
  const int warps = static_cast<int>(ctas) * kWarps;
  const int64_t len = ((static_cast<int64_t>(n_pages) + warps - 1) / warps + 127) / 128 * 128;
  const int64_t begin = len * (static_cast<int64_t>(rank) * kWarps + warp_id());
  return {static_cast<int>(begin < n_pages ? begin : n_pages),
          static_cast<int>(begin + len < n_pages ? begin + len : n_pages)};
}

// How many of a warp's pages are free, in every lane.
__device__ __forceinline__ int free_pages(const int32_t* counts, const Slice& s) {
  int n = 0;
  const int lane = static_cast<int>(lane_id());
#pragma unroll 8
  for (int i = s.begin + lane; i < s.end; i += 32) n += __ldcg(counts + i) == 0;
  return static_cast<int>(__reduce_add_sync(kAll, static_cast<unsigned>(n)));
}

// ---------------------------------------------------------------- reserve

// Row b's new tokens lie at the positions before .. len - 1; the pages of
// those positions are looked at, by 2^lanes_log2 lanes to a row.
struct RowRange {
  int first, last;  // pages
  int rows;         // rows of the first page that hold earlier tokens
};

__device__ __forceinline__ RowRange row_range(const ReserveProblem& p, int b) {
  const int64_t room = static_cast<int64_t>(p.pages.max_pages) << p.pages.page_shift;
  int64_t len = __ldg(p.lens + b);
  const int m = p.new_lens ? min(max(__ldg(p.new_lens + b), 0), p.n_new) : p.n_new;
  const int64_t start = len - m > 0 ? len - m : 0;
  if (len > room) {
    atomicOr(&g_device_error, kErrIndex);
    len = room;
  }
  if (m == 0 || len <= start) return {0, 0, 0};
  const int page = 1 << p.pages.page_shift;
  return {static_cast<int>(start >> p.pages.page_shift), static_cast<int>((len + page - 1) >> p.pages.page_shift),
          static_cast<int>(start & (page - 1))};
}

// A table entry that names a page which other entries name too is marked
// while the call works: -2 - page. The row's own lanes alone read its entries.
__device__ __forceinline__ bool marked(int entry) { return entry < -1; }
__device__ __forceinline__ int marked_page(int entry) { return -2 - entry; }

__global__ void __launch_bounds__(kClusterThreads) cache_reserve_kernel(const ReserveProblem p, int lanes_log2) {
  __shared__ ClusterSmem sm;
  griddep_wait();
  griddep_launch_dependents();
  const PagesProblem& pg = p.pages;
  const uint32_t rank = cluster_ctarank(), ctas = gridDim.x;
  const int lane = static_cast<int>(lane_id());
  const int lanes = 1 << lanes_log2;
  // this group of lanes takes the rows [b0, b1), the groups in order
  const int groups = static_cast<int>(ctas) * (kClusterThreads >> lanes_log2);
  const int group = (static_cast<int>(rank) * kClusterThreads + static_cast<int>(threadIdx.x)) >> lanes_log2;
  const int per = (p.pages.B + groups - 1) / groups;
  const int b0 = min(group * per, pg.B), b1 = min(b0 + per, pg.B);
  const int sub = lane & (lanes - 1);
  const uint32_t group_mask = (lanes == 32 ? kAll : ((1u << lanes) - 1u) << (lane & ~(lanes - 1)));
  const uint32_t before_mask = group_mask & ((1u << lane) - 1u);

  // f(row, its range, page number in the row, entry) for every page of the
  // group's rows; all lanes of a warp take the same number of rounds, so that
  // f may vote (k >= last: no page)
  auto for_pages = [&](auto f) {
    for (int i = 0; i < per; ++i) {
      const int b = b0 + i;
      const RowRange r = b < b1 ? row_range(p, b) : RowRange{0, 0, 0};
      for (int k = r.first + sub; __any_sync(kAll, k - sub < r.last); k += lanes)
        f(b, r, k, k < r.last ? pg.table + static_cast<int64_t>(b) * pg.max_pages + k : nullptr);
    }
  };

  // which entries name shared pages
  int any = 0;
  for_pages([&](int, const RowRange&, int, int32_t* e) {
    if (!e) return;
    int page = *e;
    if (page >= pg.n_pages) atomicOr(&g_device_error, kErrIndex);
    if (page < 0 || page >= pg.n_pages) {
      if (page != -1) *e = -1;
    } else if (__ldcg(pg.counts + page) > 1) {
      *e = -2 - page;
      any = 1;
    }
  });
  uint64_t sharing;
  cluster_scan(static_cast<uint64_t>(any), sm, 0, rank, ctas, &sharing);
  if (sharing) {
    // Every row leaves the shared pages that it writes. Where that takes a
    // page's count to 0, the first of them keeps it after all: its number is
    // left in the count.
    for_pages([&](int, const RowRange&, int, int32_t* e) {
      if (e && marked(*e)) atomicSub(pg.counts + marked_page(*e), 1);
    });
    cluster_sync();
    for_pages([&](int b, const RowRange&, int, int32_t* e) {
      if (e && marked(*e) && __ldcg(pg.counts + marked_page(*e)) <= 0) atomicMin(pg.counts + marked_page(*e), INT32_MIN + b);
    });
    cluster_sync();
  }
  auto keeps = [&](int b, int entry) { return __ldcg(pg.counts + marked_page(entry)) == INT32_MIN + b; };

  // what the rows need: pages, and copies of what pages held before
  uint64_t need = 0;  // pages, in the high half; copies
  for_pages([&](int b, const RowRange& r, int k, int32_t* e) {
    if (!e) return;
    const int entry = *e;
    if (entry == -1 || (marked(entry) && !keeps(b, entry)))
      need += (1ull << 32) + (marked(entry) && k == r.first && r.rows > 0 ? 1ull : 0ull);
  });
  uint64_t totals, n_free;
  uint64_t place = cluster_scan(need, sm, 1, rank, ctas, &totals);
  // a group's lanes share the place of its first
  place = __shfl_sync(kAll, place, lane & ~(lanes - 1));
  const Slice slice = warp_slice(pg.n_pages, rank, ctas);
  const int mine = free_pages(pg.counts, slice);
  uint64_t at = cluster_scan(lane == 0 ? static_cast<uint64_t>(mine) : 0ull, sm, 0, rank, ctas, &n_free);
  at = __shfl_sync(kAll, at, 0);
  const uint64_t wanted = totals >> 32;
  const bool enough = wanted <= n_free;
  if (rank == 0 && threadIdx.x == 0) {
    *p.n_copies = enough ? static_cast<int32_t>(totals & kAll) : 0;
    *p.n_missing = enough ? 0 : static_cast<int32_t>(wanted - n_free < INT32_MAX ? wanted - n_free : INT32_MAX);
  }
  if (!enough) {
    // as it was: the keepers' numbers out of the counts, then everybody back
    if (sharing) {
      for_pages([&](int b, const RowRange&, int, int32_t* e) {
        if (e && marked(*e) && keeps(b, *e)) pg.counts[marked_page(*e)] = 0;
      });
      cluster_sync();
      for_pages([&](int, const RowRange&, int, int32_t* e) {
        if (!e || !marked(*e)) return;
        atomicAdd(pg.counts + marked_page(*e), 1);
        *e = marked_page(*e);
      });
    }
    return;
  }

  // the lowest free pages, in order
  for (int i = slice.begin; i < slice.end && at < wanted; i += 32) {
    const bool free = i + lane < slice.end && __ldcg(pg.counts + i + lane) == 0;
    const uint32_t vote = __ballot_sync(kAll, free);
    const uint64_t to = at + __popc(vote & ((1u << lane) - 1u));
    if (free && to < wanted) p.free_ids[to] = i + lane;
    at += __popc(vote);
  }
  cluster_sync();

  for_pages([&](int b, const RowRange& r, int k, int32_t* e) {
    const int entry = e ? *e : 0;
    const bool shared = e && marked(entry);
    const bool kept = shared && keeps(b, entry);
    const bool wants = e && (entry == -1 || (shared && !kept));
    const bool copies = wants && shared && k == r.first && r.rows > 0;
    const uint32_t want_vote = __ballot_sync(kAll, wants), copy_vote = __ballot_sync(kAll, copies);
    if (kept) {
      *e = marked_page(entry);
      pg.counts[marked_page(entry)] = 1;
    }
    if (wants) {
      const int page = __ldcg(p.free_ids + (place >> 32) + __popc(want_vote & before_mask));
      *e = page;
      pg.counts[page] = 1;
      if (copies) {
        int32_t* c = p.copies + 3 * ((place & kAll) + __popc(copy_vote & before_mask));
        c[0] = marked_page(entry);
        c[1] = page;
        c[2] = r.rows;
      }
    }
    place += (static_cast<uint64_t>(__popc(want_vote & group_mask)) << 32) + __popc(copy_vote & group_mask);
  });
}

// ---------------------------------------------------------------- compact

// With U used pages, the k-th highest of those from U on moves into the k-th
// lowest free page below U. A page's rank follows from how many used pages
// lie before it: the holes' from below, the movers' from above.
__global__ void __launch_bounds__(kClusterThreads) cache_compact_kernel(const CompactProblem p) {
  __shared__ ClusterSmem sm;
  griddep_wait();
  griddep_launch_dependents();
  const PagesProblem& pg = p.pages;
  const uint32_t rank = cluster_ctarank(), ctas = gridDim.x;
  const int lane = static_cast<int>(lane_id());
  const Slice slice = warp_slice(pg.n_pages, rank, ctas);
  const int n = slice.end - slice.begin;
  const int mine = n - free_pages(pg.counts, slice);
  uint64_t total;
  uint64_t at = cluster_scan(lane == 0 ? static_cast<uint64_t>(mine) : 0ull, sm, 0, rank, ctas, &total);
  at = __shfl_sync(kAll, at, 0);
  const int used = static_cast<int>(total);
  const bool apart = p.counts_out != pg.counts;
  int movers = 0;
  for (int i = slice.begin; i < slice.end; i += 32) {
    const int page = i + lane;
    const bool in = page < slice.end;
    const int count = in ? __ldcg(pg.counts + page) : 0;
    const uint32_t vote = __ballot_sync(kAll, in && count != 0);
    const int before = static_cast<int>(at) + __popc(vote & ((1u << lane) - 1u));  // used pages before this
    at += __popc(vote);
    if (!in) continue;
    const bool high = page >= used;
    const bool moves = high && count != 0, hole = !high && count == 0;
    const int k = moves ? used - 1 - before : page - before;
    movers += moves;
    if ((moves || hole) && k < p.max_copies) {
      p.moves[2 * k + hole] = page;
      continue;  // its count and its place in the map are the move's
    }
    if (high) p.map[page] = page;
    if (apart) p.counts_out[page] = count;
  }
  uint64_t n_moves;
  cluster_scan(static_cast<uint64_t>(movers), sm, 1, rank, ctas, &n_moves);
  const int moved = static_cast<int>(n_moves) < p.max_copies ? static_cast<int>(n_moves) : p.max_copies;
  for (int k = static_cast<int>(rank) * kClusterThreads + static_cast<int>(threadIdx.x); k < moved;
       k += static_cast<int>(ctas) * kClusterThreads) {
    const int from = __ldcg(p.moves + 2 * k), to = __ldcg(p.moves + 2 * k + 1);
    p.copies[3 * k] = from;
    p.copies[3 * k + 1] = to;
    p.copies[3 * k + 2] = 1 << pg.page_shift;
    p.map[from] = to;
    p.counts_out[to] = __ldcg(pg.counts + from);
    p.counts_out[from] = 0;
  }
  if (rank == 0 && threadIdx.x == 0) {
    *p.n_copies = moved;
    *p.n_used = used;
  }
}

constexpr int kRemapThreads = 256;

__global__ void __launch_bounds__(kRemapThreads) cache_remap_kernel(const CompactProblem p, int64_t entries) {
  griddep_wait();
  griddep_launch_dependents();
  const int used = __ldcg(p.n_used);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kRemapThreads + threadIdx.x; i < entries;
       i += static_cast<int64_t>(gridDim.x) * kRemapThreads) {
    int page = p.pages.table[i];
    if (page >= p.pages.n_pages) {
      atomicOr(&g_device_error, kErrIndex);
    } else if (page >= used) {
      page = __ldcg(p.map + page);
    }
    p.table_out[i] = page;
  }
}

int sm_count() {
  static int cached = 0;
  int n = __atomic_load_n(&cached, __ATOMIC_RELAXED);
  if (n == 0) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
      n = 148;
    __atomic_store_n(&cached, n, __ATOMIC_RELAXED);
  }
  return n;
}

// One cluster for `work` pages or threads.
template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kernel)(KArgs...), int64_t work, cudaStream_t stream, Args&&... args) {
  unsigned ctas = 1;
  while (ctas < kMaxCtas && work > static_cast<int64_t>(ctas) * 4 * kClusterThreads) ctas *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kClusterThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

}  // namespace

cudaError_t launch_cache_fork(const PagesProblem& p, int32_t* lens, const int32_t* parents,
                              cudaStream_t stream) {
  // columns to a block: as many as fit, but no fewer blocks than SMs for it
  // (8 columns are a sector of memory)
  int cols_log2 = 5;
  while (cols_log2 > 0 && (static_cast<int64_t>(p.B) << cols_log2) > kForkEntries) --cols_log2;
  while (cols_log2 > 3 && (p.max_pages >> cols_log2) < sm_count()) --cols_log2;
  static unsigned long long configured = 0;
  cudaError_t e = set_smem_once(cache_fork_kernel, kForkEntries * 4, &configured);
  if (e != cudaSuccess) return e;
  const int64_t blocks = ((static_cast<int64_t>(p.max_pages) - 1) >> cols_log2) + 1 + (lens ? 1 : 0);
  return launch_pdl(cache_fork_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kForkThreads),
                    (static_cast<size_t>(p.B) << cols_log2) * 4, stream, p, lens, parents, cols_log2);
}

cudaError_t launch_cache_release(const PagesProblem& p, const int32_t* keep_lens, cudaStream_t stream) {
  const int chunks = (p.max_pages - 1) / kReleaseThreads + 1;
  const int64_t items = static_cast<int64_t>(p.B) * chunks;
  const int64_t most = static_cast<int64_t>(sm_count()) * 8;
  return launch_pdl(cache_release_kernel, dim3(static_cast<unsigned>(items < most ? items : most)),
                    dim3(kReleaseThreads), 0, stream, p, keep_lens, items, chunks);
}

cudaError_t launch_cache_reserve(const ReserveProblem& p, cudaStream_t stream) {
  // lanes to a row: for the most pages that its new tokens can touch
  const int64_t pages = ((static_cast<int64_t>(p.n_new) - 1) >> p.pages.page_shift) + 2;
  int lanes_log2 = 0;
  while (lanes_log2 < 5 && (1 << lanes_log2) < pages) ++lanes_log2;
  const int64_t threads = static_cast<int64_t>(p.pages.B) << lanes_log2;
  return launch_cluster(cache_reserve_kernel, threads * 4 > p.pages.n_pages ? threads * 4 : p.pages.n_pages, stream, p,
                        lanes_log2);
}

cudaError_t launch_cache_compact(const CompactProblem& p, cudaStream_t stream) {
  cudaError_t e = launch_cluster(cache_compact_kernel, p.pages.n_pages, stream, p);
  if (e != cudaSuccess) return e;
  const int64_t entries = static_cast<int64_t>(p.pages.B) * p.pages.max_pages;
  if (entries == 0) return cudaSuccess;
  const int64_t blocks = (entries + kRemapThreads - 1) / kRemapThreads, most = static_cast<int64_t>(sm_count()) * 8;
  return launch_pdl(cache_remap_kernel, dim3(static_cast<unsigned>(blocks < most ? blocks : most)), dim3(kRemapThreads), 0,
                    stream, p, entries);
}

TSD_DEFINE_ERROR_READER(take_device_error_pages)

}  // namespace tsd
