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
#include <type_traits>

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
  uint64_t warp_sum[2][kWarps];
  uint64_t cta_sum[4][kMaxCtas];  // written by the cluster's CTAs, each row once
};

// The sums of `v` and `w` over the threads before this one, CTAs in order of
// rank (returned, and in *w_before), and over all. Threads of every CTA call it
// together; row_v and row_w of cta_sum belong to this call.
__device__ __forceinline__ uint64_t cluster_scan(uint64_t v, ClusterSmem& sm, int row_v, uint32_t rank, uint32_t ctas,
                                                 uint64_t* v_total, uint64_t w, int row_w, uint64_t* w_total,
                                                 uint64_t* w_before) {
  const int lane = static_cast<int>(lane_id()), warp = warp_id();
  uint64_t sum_v = v, sum_w = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t other_v = __shfl_up_sync(kAll, sum_v, o), other_w = __shfl_up_sync(kAll, sum_w, o);
    if (lane >= o) {
      sum_v += other_v;
      sum_w += other_w;
    }
  }
  __syncthreads();  // warp_sum's previous use is over
  if (lane == 31) {
    sm.warp_sum[0][warp] = sum_v;
    sm.warp_sum[1][warp] = sum_w;
  }
  __syncthreads();
  uint64_t warp_v = sm.warp_sum[0][lane], warp_w = sm.warp_sum[1][lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t other_v = __shfl_up_sync(kAll, warp_v, o), other_w = __shfl_up_sync(kAll, warp_w, o);
    if (lane >= o) {
      warp_v += other_v;
      warp_w += other_w;
    }
  }
  uint64_t before_v = sum_v - v, before_w = sum_w - w;
  const uint64_t cta_v = __shfl_sync(kAll, warp_v, 31), cta_w = __shfl_sync(kAll, warp_w, 31);
  const uint64_t warps_v = __shfl_sync(kAll, warp_v, (warp + 31) & 31), warps_w = __shfl_sync(kAll, warp_w, (warp + 31) & 31);
  if (warp > 0) {
    before_v += warps_v;
    before_w += warps_w;
  }
  if (threadIdx.x < ctas) {
    st_cluster_u64(cluster_map(&sm.cta_sum[row_v][rank], threadIdx.x), cta_v);
    st_cluster_u64(cluster_map(&sm.cta_sum[row_w][rank], threadIdx.x), cta_w);
  }
  cluster_sync();
  uint64_t all_v = 0, all_w = 0;
  for (uint32_t c = 0; c < ctas; ++c) {
    const uint64_t t_v = sm.cta_sum[row_v][c], t_w = sm.cta_sum[row_w][c];
    if (c < rank) {
      before_v += t_v;
      before_w += t_w;
    }
    all_v += t_v;
    all_w += t_w;
  }
  *v_total = all_v;
  *w_total = all_w;
  *w_before = before_w;
  return before_v;
}

// Pages of one warp: [begin, end), in steps of 256: eight counts to a lane are
// loaded at a time.
constexpr int kBatch = 8;
struct Slice {
  int begin, end;
};
__device__ __forceinline__ Slice warp_slice(int n_pages, uint32_t rank, uint32_t ctas) {
  const int warps = static_cast<int>(ctas) * kWarps;
  const int64_t len = ((static_cast<int64_t>(n_pages) + warps - 1) / warps + 32 * kBatch - 1) / (32 * kBatch) * (32 * kBatch);
  const int64_t begin = len * (static_cast<int64_t>(rank) * kWarps + warp_id());
  return {static_cast<int>(begin < n_pages ? begin : n_pages),
          static_cast<int>(begin + len < n_pages ? begin + len : n_pages)};
}
// f(page, its count, whether it is one) for a warp's pages 32 at a time, while
// f returns true; all lanes call it together.
template <typename F>
__device__ __forceinline__ void for_slice(const int32_t* counts, const Slice& s, F f) {
  const int lane = static_cast<int>(lane_id());
  bool go = true;
#pragma unroll 1
  for (int i = s.begin; go && i < s.end; i += 32 * kBatch) {
    int c[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int page = i + 32 * j + lane;
      c[j] = page < s.end ? __ldcg(counts + page) : 0;
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int page = i + 32 * j + lane;
      go = go && f(page, c[j], page < s.end);
    }
  }
}
// How many of a warp's pages are free, in every lane.
__device__ __forceinline__ int free_pages(const int32_t* counts, const Slice& s) {
  int n = 0;
  for_slice(counts, s, [&](int, int count, bool in) {
    n += in && count == 0;
    return true;
  });
  return static_cast<int>(__reduce_add_sync(kAll, static_cast<unsigned>(n)));
}

// ---------------------------------------------------------------- reserve

// Row b's new tokens lie at the positions before .. len - 1: the pages
// [first, last) of the row.
struct RowRange {
  int first, last;
  int rows;  // rows of the first page that hold earlier tokens
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

// The pages of a row are cut into units of 2^lanes_log2, `units` of them to a row; a
// group of lanes takes consecutive units, so that the groups' order is the rows'
// and pages'. A call without shared pages, as most are, has two barriers: one
// that adds up what the rows need, with the free pages, and one after the free
// pages' numbers are written down. Pages that several rows name take three more.
// 256 rows of a token, 65536 pages: 5 us; 64 prompts of up to 8192 tokens, 33000
// pages of 262144: 10 us (with a row to a group, its pages one after the other,
// and the counts read 32 at a time: 11 and 38).
__global__ void __launch_bounds__(kClusterThreads) cache_reserve_kernel(const ReserveProblem p, int lanes_log2, int units) {
  __shared__ ClusterSmem sm;
  griddep_wait();
  griddep_launch_dependents();
  const PagesProblem& pg = p.pages;
  const uint32_t rank = cluster_ctarank(), ctas = gridDim.x;
  const int lane = static_cast<int>(lane_id());
  const int lanes = 1 << lanes_log2;
  const int groups = static_cast<int>(ctas) * (kClusterThreads >> lanes_log2);
  const int group = (static_cast<int>(rank) * kClusterThreads + static_cast<int>(threadIdx.x)) >> lanes_log2;
  const int64_t all_units = static_cast<int64_t>(pg.B) * units;
  const int64_t per = (all_units + groups - 1) / groups;
  const int sub = lane & (lanes - 1);
  const uint32_t group_mask = (lanes == 32 ? kAll : ((1u << lanes) - 1u) << (lane & ~(lanes - 1)));
  const uint32_t before_mask = group_mask & ((1u << lane) - 1u);

  // f(row, its range, page number in the row, address of the entry or null, the
  // entry) for every page of the group's units, U of them loaded at a time; all
  // lanes of a warp call f together, so that it may vote
  auto for_pages = [&](auto unroll, auto f) {
    constexpr int U = decltype(unroll)::value;
#pragma unroll 1
    for (int64_t i = 0; i < per; i += U) {
      int row[U], k[U], entry[U];
      RowRange r[U];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int64_t u = group * per + i + j;
        const bool is = i + j < per && u < all_units;
        row[j] = is ? units == 1 ? static_cast<int>(u) : static_cast<int>(u / units) : 0;
        r[j] = is ? row_range(p, row[j]) : RowRange{0, 0, 0};
        k[j] = is ? r[j].first + ((static_cast<int>(u - static_cast<int64_t>(row[j]) * units) << lanes_log2) | sub) : 0;
      }
#pragma unroll
      for (int j = 0; j < U; ++j)
        entry[j] = k[j] < r[j].last ? __ldcg(pg.table + static_cast<int64_t>(row[j]) * pg.max_pages + k[j]) : 0;
#pragma unroll
      for (int j = 0; j < U; ++j)
        f(row[j], r[j], k[j], k[j] < r[j].last ? pg.table + static_cast<int64_t>(row[j]) * pg.max_pages + k[j] : nullptr,
          entry[j]);
    }
  };
  using One = std::integral_constant<int, 1>;
  using Four = std::integral_constant<int, 4>;

  const Slice slice = warp_slice(pg.n_pages, rank, ctas);
  const int free_here = free_pages(pg.counts, slice);

  // what the rows need: pages, in the high half, and copies; and which entries
  // name shared pages
  uint64_t need = 0;
  bool any = false;
  for_pages(Four{}, [&](int, const RowRange&, int, int32_t* e, int page) {
    if (!e) return;
    if (page >= pg.n_pages) atomicOr(&g_device_error, kErrIndex);
    if (page < 0 || page >= pg.n_pages) {
      if (page != -1) *e = -1;
      need += 1ull << 32;
    } else if (__ldcg(pg.counts + page) > 1) {
      *e = -2 - page;
      any = true;
    }
  });
  uint64_t totals, more;  // more: free pages in the low half, threads with shared ones
  uint64_t at = cluster_scan((any ? 1ull << 32 : 0ull) + (lane == 0 ? static_cast<uint64_t>(free_here) : 0ull), sm, 1, rank,
                             ctas, &more, need, 0, &totals, &need);
  at = __shfl_sync(kAll, at & kAll, 0);
  const uint64_t n_free = more & kAll;
  const bool sharing = (more >> 32) != 0;
  uint64_t place = need;  // of this lane's group among the pages and copies
  auto keeps = [&](int b, int entry) { return __ldcg(pg.counts + marked_page(entry)) == INT32_MIN + b; };
  if (sharing) {
    // Every row leaves the shared pages that it writes. Where that takes a
    // page's count to 0, the first of them keeps it after all: its number is
    // left in the count.
    for_pages(One{}, [&](int, const RowRange&, int, int32_t* e, int entry) {
      if (e && marked(entry)) atomicSub(pg.counts + marked_page(entry), 1);
    });
    cluster_sync();
    for_pages(One{}, [&](int b, const RowRange&, int, int32_t* e, int entry) {
      if (e && marked(entry) && __ldcg(pg.counts + marked_page(entry)) <= 0)
        atomicMin(pg.counts + marked_page(entry), INT32_MIN + b);
    });
    cluster_sync();
    uint64_t now = 0, unused;
    for_pages(One{}, [&](int b, const RowRange& r, int k, int32_t* e, int entry) {
      if (e && (entry == -1 || (marked(entry) && !keeps(b, entry))))
        now += (1ull << 32) + (marked(entry) && k == r.first && r.rows > 0 ? 1ull : 0ull);
    });
    cluster_scan(0ull, sm, 3, rank, ctas, &unused, now, 2, &totals, &place);
  }
  // a group's lanes share the place of its first
  place = __shfl_sync(kAll, place, lane & ~(lanes - 1));
  const uint64_t wanted = totals >> 32;
  const bool enough = wanted <= n_free;
  if (rank == 0 && threadIdx.x == 0) {
    *p.n_copies = enough ? static_cast<int32_t>(totals & kAll) : 0;
    *p.n_missing = enough ? 0 : static_cast<int32_t>(wanted - n_free < INT32_MAX ? wanted - n_free : INT32_MAX);
  }
  if (!enough) {
    // as it was: the keepers' numbers out of the counts, then everybody back
    if (sharing) {
      for_pages(One{}, [&](int b, const RowRange&, int, int32_t* e, int entry) {
        if (e && marked(entry) && keeps(b, entry)) pg.counts[marked_page(entry)] = 0;
      });
      cluster_sync();
      for_pages(One{}, [&](int, const RowRange&, int, int32_t* e, int entry) {
        if (!e || !marked(entry)) return;
        atomicAdd(pg.counts + marked_page(entry), 1);
        *e = marked_page(entry);
      });
    }
    return;
  }

  // the lowest free pages, in order. (While pages are shared, a count that was
  // taken to 0 has its keeper's number.)
  if (free_here > 0 && at < wanted)
    for_slice(pg.counts, slice, [&](int page, int count, bool in) {
      const uint32_t vote = __ballot_sync(kAll, in && count == 0);
      const uint64_t to = at + __popc(vote & ((1u << lane) - 1u));
      if (in && count == 0 && to < wanted) p.free_ids[to] = page;
      at += __popc(vote);
      return at < wanted;
    });
  cluster_sync();

  for_pages(Four{}, [&](int b, const RowRange& r, int k, int32_t* e, int entry) {
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
  uint64_t total, unused, unused_before;
  uint64_t at = cluster_scan(lane == 0 ? static_cast<uint64_t>(mine) : 0ull, sm, 0, rank, ctas, &total, 0ull, 1, &unused,
                             &unused_before);
  at = __shfl_sync(kAll, at, 0);
  const int used = static_cast<int>(total);
  const bool apart = p.counts_out != pg.counts;
  int movers = 0;
  for_slice(pg.counts, slice, [&](int page, int count, bool in) {
    const uint32_t vote = __ballot_sync(kAll, in && count != 0);
    const int before = static_cast<int>(at) + __popc(vote & ((1u << lane) - 1u));  // used pages before this
    at += __popc(vote);
    if (!in) return true;
    const bool high = page >= used;
    const bool moves = high && count != 0, hole = !high && count == 0;
    const int k = moves ? used - 1 - before : page - before;
    movers += moves;
    if ((moves || hole) && k < p.max_copies) {
      p.moves[2 * k + hole] = page;
      return true;  // its count and its place in the map are the move's
    }
    if (high) p.map[page] = page;
    if (apart) p.counts_out[page] = count;
    return true;
  });
  uint64_t n_moves;
  cluster_scan(static_cast<uint64_t>(movers), sm, 2, rank, ctas, &n_moves, 0ull, 3, &unused, &unused_before);
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

// One cluster, of a block for each 8192 pages, 256 to a warp, and at most eight.
template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kernel)(KArgs...), int64_t work, cudaStream_t stream, Args&&... args) {
  unsigned ctas = 1;
  while (ctas < kMaxCtas && work > static_cast<int64_t>(ctas) * 8 * kClusterThreads) ctas *= 2;
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
  // lanes to a unit: for the most pages that a row's new tokens can touch
  int64_t pages = ((static_cast<int64_t>(p.n_new) - 1) >> p.pages.page_shift) + 2;
  if (pages > p.pages.max_pages) pages = p.pages.max_pages;
  int lanes_log2 = 0;
  while (lanes_log2 < 5 && (1 << lanes_log2) < pages) ++lanes_log2;
  const int units = static_cast<int>((pages + (1 << lanes_log2) - 1) >> lanes_log2);
  const int64_t threads = (static_cast<int64_t>(p.pages.B) * units) << lanes_log2;
  return launch_cluster(cache_reserve_kernel, threads * 4 > p.pages.n_pages ? threads * 4 : p.pages.n_pages, stream, p,
                        lanes_log2, units);
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
