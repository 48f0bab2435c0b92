// cache_pages.cu -- keeping the pages of a paged key/value cache: giving rows
// the pages of the rows they continue (fork), finding pages for new tokens
// (reserve), giving pages back (release), and moving the used pages to the
// front of the pool (compact).
//
// The state is the page table [B, max_pages], -1 where a row has no page, and
// how many table entries name each page (0: a free page). There is no list of
// free pages that one call would leave to the next: the lowest free pages are
// found in the counts, so that the pages a call takes follow from its
// arguments alone, and the pool stays dense by itself. Its price is to read
// them: 1 MB where there are 2^18 pages.
//
// All of it is integer work on a few hundred kilobytes and bound by latency:
// dependent reads of the L2 and barriers between phases. What needs an order
// over all rows or pages (which page is the j-th free one, which row the j-th
// to need one) runs in one thread-block cluster, whose barrier costs less than
// a second launch.
//
// Parents, lengths and what is kept may come from the launch before, which still
// runs when a block of these begins. They are read past the wait by ordinary loads:
// the read-only path is for what nobody writes while a kernel lives. (From the L2,
// by __ldcg, 64 prompts' reserve takes 13.2 us in place of 12.3: a row's length is
// read for each of its units.)
#include <type_traits>

#include "kernels.h"
#include "sm103.cuh"

namespace tsd {

namespace {

constexpr uint32_t kAll = 0xffffffffu;

// ---------------------------------------------------------------- fork

// Row r becomes row parents[r], all rows at once. A block takes some columns
// of every row through shared memory, which is what makes it safe in place:
// no other block reads or writes them. A count changes only where an entry
// does, so that the pages that a row shares with its parent already cost
// nothing.
constexpr int kForkThreads = 512;
constexpr int kForkEntries = kForkMaxRows;  // of a block at most
constexpr int kForkFew = 1024;              // where there are blocks enough
constexpr int kForkStaged = 16384;          // rows whose parents fit beside their entries
constexpr int kForkBytes = 4 * (kForkEntries + kForkStaged);
static_assert(kForkBytes <= 227 * 1024, "shared memory of a block");

__global__ void __launch_bounds__(kForkThreads)
    cache_fork_kernel(const PagesProblem p, int32_t* lens, const int32_t* parents, int cols_log2) {
  extern __shared__ int32_t old[];  // [B][cols], then the parents where both fit
  griddep_wait();
  griddep_launch_dependents();
  const bool for_lens = lens != nullptr && blockIdx.x == gridDim.x - 1;
  const int shift = for_lens ? 0 : cols_log2, mask = (1 << shift) - 1;
  const int n = p.B << shift;
  const int col0 = static_cast<int>(blockIdx.x) << shift;
  const bool staged = p.B <= kForkStaged;
  int32_t* parent_of = old + (p.B << cols_log2);
  auto entry = [&](int i) -> int32_t* {
    if (for_lens) return lens + i;
    const int col = col0 + (i & mask);
    return col < p.max_pages ? p.table + static_cast<int64_t>(i >> shift) * p.max_pages + col : nullptr;
  };
#pragma unroll 2
  for (int i = threadIdx.x; staged && i < p.B; i += kForkThreads) parent_of[i] = parents[i];
#pragma unroll 4
  for (int i = threadIdx.x; i < n; i += kForkThreads) {
    const int32_t* e = entry(i);
    old[i] = e ? *e : -1;
  }
  __syncthreads();
#pragma unroll 2
  for (int i = threadIdx.x; i < n; i += kForkThreads) {
    const int parent = staged ? parent_of[i >> shift] : parents[i >> shift];
    if (parent < -1 || parent >= p.B) {
      if (for_lens || blockIdx.x == 0) atomicOr(&g_device_error, kErrIndex);
      continue;
    }
    const int32_t was = old[i];
    const int32_t now = parent < 0 ? (for_lens ? 0 : -1) : old[(parent << shift) | (i & mask)];
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
    const int keep = keep_lens ? keep_lens[b] : 0;
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
constexpr int kMaxCtas = 16;     // of the cluster (above 8 where the device has room for it)
constexpr int kWarps = kClusterThreads / 32;

// A barrier of the cluster: of its one block where it has no more (a third of the
// time), which orders the block's accesses to global memory too.
__device__ __forceinline__ void sync_all(uint32_t ctas) {
  if (ctas == 1) __syncthreads();
  else cluster_sync();
}

// Two sums, over threads.
struct Sums {
  uint64_t v, w;
};
constexpr int kNear = 1024;
struct ClusterSmem {
  Sums warp[kWarps];      // of a warp, then of those before it
  Sums cta[2][kMaxCtas];  // written by the cluster's CTAs, each row once
  Sums before, all;
  int32_t free_ids[kNear];
};

// The sums of v and w over the threads before this one, the CTAs in order of
// rank; *all of them over all. A warp adds `more` to its w. Threads of every CTA
// call it together; `row` of sm.cta belongs to this call. LANES: which of the
// two differ within a warp (1: v, 2: both). One warp joins the warps' sums:
// 32 warps at once take an SM eight times as long for it.
template <int LANES>
__device__ __forceinline__ Sums cluster_scan(uint32_t v, uint32_t w, uint64_t more, ClusterSmem& sm, int row, uint32_t rank,
                                             uint32_t ctas, Sums* all) {
  const int lane = static_cast<int>(lane_id()), warp = warp_id();
  uint32_t sum_v = v, sum_w = w;
  if constexpr (LANES > 0) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t other_v = __shfl_up_sync(kAll, sum_v, o);
      if (lane >= o) sum_v += other_v;
      if constexpr (LANES > 1) {
        const uint32_t other_w = __shfl_up_sync(kAll, sum_w, o);
        if (lane >= o) sum_w += other_w;
      }
    }
  }
  if (lane == 31) sm.warp[warp] = {sum_v, sum_w + more};
  __syncthreads();
  if (warp == 0) {
    Sums mine = {0, 0};
    if (lane < static_cast<int>(blockDim.x >> 5)) mine = sm.warp[lane];
    Sums sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t other_v = __shfl_up_sync(kAll, sum.v, o), other_w = __shfl_up_sync(kAll, sum.w, o);
      if (lane >= o) {
        sum.v += other_v;
        sum.w += other_w;
      }
    }
    sm.warp[lane] = {sum.v - mine.v, sum.w - mine.w};
    if (ctas == 1 && lane == 31) {
      sm.before = {0, 0};
      sm.all = sum;
    }
    const uint64_t cta_v = __shfl_sync(kAll, sum.v, 31), cta_w = __shfl_sync(kAll, sum.w, 31);
    if (ctas > 1 && lane < static_cast<int>(ctas)) {
      const uint32_t to = cluster_map(&sm.cta[row][rank], static_cast<uint32_t>(lane));
      st_cluster_u64(to, cta_v);
      st_cluster_u64(to + 8, cta_w);
    }
  }
  if (ctas > 1) cluster_sync();
  if (ctas > 1 && warp == 0) {
    Sums mine = {0, 0};
    if (lane < static_cast<int>(ctas)) mine = sm.cta[row][lane];
    Sums sum = mine;
#pragma unroll
    for (int o = 1; o < kMaxCtas; o <<= 1) {
      const uint64_t other_v = __shfl_up_sync(kAll, sum.v, o), other_w = __shfl_up_sync(kAll, sum.w, o);
      if (lane >= o) {
        sum.v += other_v;
        sum.w += other_w;
      }
    }
    if (lane == static_cast<int>(rank)) sm.before = {sum.v - mine.v, sum.w - mine.w};
    if (lane == kMaxCtas - 1) sm.all = sum;
  }
  __syncthreads();
  *all = sm.all;
  const Sums warps = sm.warp[warp], ctas_before = sm.before;
  return {ctas_before.v + warps.v + (LANES > 0 ? sum_v - v : 0u), ctas_before.w + warps.w + (LANES > 1 ? sum_w - w : 0u)};
}

// Pages of one warp: [begin, end), in steps of 256: eight counts to a lane are
// loaded at a time.
constexpr int kBatch = 8;
struct Slice {
  int begin, end;
};
__device__ __forceinline__ Slice warp_slice(int n_pages, uint32_t rank, uint32_t ctas) {
  const int block_warps = static_cast<int>(blockDim.x) / 32, warps = static_cast<int>(ctas) * block_warps;
  const int64_t len = ((static_cast<int64_t>(n_pages) + warps - 1) / warps + 32 * kBatch - 1) / (32 * kBatch) * (32 * kBatch);
  const int64_t begin = len * (static_cast<int64_t>(rank) * block_warps + warp_id());
  return {static_cast<int>(begin < n_pages ? begin : n_pages),
          static_cast<int>(begin + len < n_pages ? begin + len : n_pages)};
}
// A batch of a warp's counts; a page past the slice counts as used.
struct Batch {
  int32_t c[kBatch];
};
__device__ __forceinline__ Batch load_batch(const int32_t* counts, const Slice& s, int begin, int lane) {
  Batch b;
#pragma unroll
  for (int j = 0; j < kBatch; ++j) {
    const int page = begin + 32 * j + lane;
    b.c[j] = page < s.end ? __ldcg(counts + page) : 1;
  }
  return b;
}
// f(page, its count) for a warp's pages 32 at a time, while go() holds ahead of
// a batch; all lanes call it together. `batch`: the slice's first.
template <typename F, typename G>
__device__ __forceinline__ void for_slice(const int32_t* counts, const Slice& s, Batch batch, int lane, F f, G go) {
#pragma unroll 1
  for (int i = s.begin; i < s.end && go(); i += 32 * kBatch) {
    const Batch now = batch;
    if (i + 32 * kBatch < s.end) batch = load_batch(counts, s, i + 32 * kBatch, lane);
#pragma unroll
    for (int j = 0; j < kBatch; ++j) f(i + 32 * j + lane, now.c[j]);
  }
}
// How many of a warp's pages are free, in every lane.
__device__ __forceinline__ int free_pages(const int32_t* counts, const Slice& s, const Batch& first, int lane) {
  int n = 0;
  for_slice(counts, s, first, lane, [&](int, int count) { n += count == 0; }, [] { return true; });
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
  const int room = p.pages.max_pages << p.pages.page_shift;  // 2^30 at most
  int len = p.lens[b];
  const int m = p.new_lens ? min(max(p.new_lens[b], 0), p.n_new) : p.n_new;
  const int start = len > m ? len - m : 0;
  if (len > room) {
    atomicOr(&g_device_error, kErrIndex);
    len = room;
  }
  if (m == 0 || len <= start) return {0, 0, 0};
  const int page = 1 << p.pages.page_shift;
  return {start >> p.pages.page_shift, (len + page - 1) >> p.pages.page_shift, start & (page - 1)};
}

// A table entry that names a page which other entries name too is marked
// while the call works: -2 - page. The row's own lanes alone read its entries.
__device__ __forceinline__ bool marked(int entry) { return entry < -1; }
__device__ __forceinline__ int marked_page(int entry) { return -2 - entry; }

// The pages of a row are cut into units of 2^lanes_log2, `units` of them to a row; a
// group of lanes takes consecutive units, so that the groups' order is the rows'
// and pages'. ONE: a group has one unit at most, and its entries stay in registers
// from phase to phase. A call without shared pages, as most are, has two
// barriers: one that adds up what the rows need, with the free pages, and one
// after the free pages' numbers are written down. Pages that several rows name
// take three more.
template <bool ONE>
__global__ void __launch_bounds__(kClusterThreads) cache_reserve_kernel(const ReserveProblem p, int lanes_log2, int units) {
  __shared__ ClusterSmem sm;
  const uint32_t rank = cluster_ctarank(), ctas = gridDim.x;
  if (ctas > 1) cluster_sync();  // every block has begun: its shared memory may be written
  griddep_wait();
  griddep_launch_dependents();
  const PagesProblem& pg = p.pages;
  const int lane = static_cast<int>(lane_id());
  const int lanes = 1 << lanes_log2;
  const int group = static_cast<int>(rank * blockDim.x + threadIdx.x) >> lanes_log2;
  const int64_t all_units = static_cast<int64_t>(pg.B) * units;
  const int groups = static_cast<int>(ctas * blockDim.x) >> lanes_log2;
  const int64_t per = ONE ? 1 : (all_units + groups - 1) / groups;
  const int sub = lane & (lanes - 1);
  const uint32_t group_mask = (lanes == 32 ? kAll : ((1u << lanes) - 1u) << (lane & ~(lanes - 1)));
  const uint32_t before_mask = group_mask & ((1u << lane) - 1u);

  // a lane's page of a unit
  struct Place {
    uint32_t id;    // in the order of the rows and of their pages, below 2^31
    int rows;       // of earlier tokens in the page, if it is the first to be written
    int entry;
    int32_t* at;    // the entry's address; null: no page
  };
  auto look_up = [&](int row, int unit, bool is) {
    Place q = {0, 0, 0, nullptr};
    if (!is) return q;
    const RowRange r = row_range(p, row);
    const int i = unit << lanes_log2 | sub, k = r.first + i;
    q.id = static_cast<uint32_t>(row) * static_cast<uint32_t>(p.width) + static_cast<uint32_t>(i);
    q.rows = i == 0 ? r.rows : 0;
    if (k < r.last) q.at = pg.table + static_cast<int64_t>(row) * pg.max_pages + k;
    return q;
  };
  const Slice slice = warp_slice(pg.n_pages, rank, ctas);
  const Batch first_batch = load_batch(pg.counts, slice, slice.begin, lane);
  const int row0 = ONE && units == 1 ? group : static_cast<int>(group * per / units);
  const int unit0 = static_cast<int>(group * per - static_cast<int64_t>(row0) * units);
  Place own = {0, 0, 0, nullptr};
  if constexpr (ONE) {
    own = look_up(row0, unit0, row0 < pg.B);
    if (own.at) own.entry = __ldcg(own.at);
  }
  // f(places, how many) for the group's units, U at a time; all lanes of a warp
  // call it together, so that it may vote
  auto for_pages = [&](auto unroll, auto f) {
    if constexpr (ONE) {
      f(&own, std::integral_constant<int, 1>{});
    } else {
      constexpr int U = decltype(unroll)::value;
      int row = row0, unit = unit0;
#pragma unroll 1
      for (int64_t i = 0; i < per; i += U) {
        Place q[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
          q[j] = {0, 0, 0, nullptr};
          if (i + j >= per) continue;
          q[j] = look_up(row, unit, row < pg.B);
          if (++unit == units) {
            unit = 0;
            ++row;
          }
        }
#pragma unroll
        for (int j = 0; j < U; ++j)
          if (q[j].at) q[j].entry = __ldcg(q[j].at);
        f(q, unroll);
      }
    }
  };
  using Single = std::integral_constant<int, 1>;
  using Two = std::integral_constant<int, 2>;

  const int free_here = free_pages(pg.counts, slice, first_batch, lane);

  // what the rows need, and which entries name shared pages
  uint32_t need = 0;
  bool any = false;
  for_pages(Two{}, [&](Place* q, auto n) {
    constexpr int U = decltype(n)::value;
    int count[U];
#pragma unroll
    for (int j = 0; j < U; ++j)
      count[j] = q[j].at && q[j].entry >= 0 && q[j].entry < pg.n_pages ? __ldcg(pg.counts + q[j].entry) : 0;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (!q[j].at) continue;
      const bool names = q[j].entry >= 0 && q[j].entry < pg.n_pages;
      if (q[j].entry >= pg.n_pages) atomicOr(&g_device_error, kErrIndex);
      if (!names) ++need;
      if ((names && count[j] > 1) || (!names && q[j].entry != -1)) {
        any |= names;
        q[j].entry = names ? -2 - q[j].entry : -1;
        *q[j].at = q[j].entry;
      }
    }
  });
  any = __any_sync(kAll, any);
  Sums all;  // pages needed; free pages, and above 32 bits the warps with shared ones
  const Sums first = cluster_scan<1>(need, 0u, static_cast<uint64_t>(free_here) + (any ? 1ull << 32 : 0ull), sm, 0, rank, ctas, &all);
  const uint32_t n_free = static_cast<uint32_t>(all.w);
  uint32_t free_at = static_cast<uint32_t>(first.w);  // free pages before this warp's
  const bool sharing = all.w >> 32 != 0;
  uint64_t page_at = first.v, copy_at = 0, wanted = all.v, n_copies = 0;
  auto keeper = [](const Place& q) { return static_cast<int>(0x80000000u + q.id); };  // below 0
  auto keeps = [&](const Place& q) { return __ldcg(pg.counts + marked_page(q.entry)) == keeper(q); };
  bool kept = false;  // ONE: the lane's page is shared, and its entry keeps it
  if (sharing) {
    // Every entry to be written leaves its shared page. Where that takes a page's
    // count to 0, the first of them keeps it after all: its number is left in the
    // count. (The entry's, not its row's: a row may name a page more than once.)
    for_pages(Single{}, [&](Place* q, auto) {
      if (q->at && marked(q->entry)) atomicSub(pg.counts + marked_page(q->entry), 1);
    });
    sync_all(ctas);
    for_pages(Single{}, [&](Place* q, auto) {
      if (q->at && marked(q->entry) && __ldcg(pg.counts + marked_page(q->entry)) <= 0)
        atomicMin(pg.counts + marked_page(q->entry), keeper(*q));
    });
    sync_all(ctas);
    need = 0;
    uint32_t copies = 0;
    for_pages(Single{}, [&](Place* q, auto) {
      if (!q->at) return;
      const bool shared = marked(q->entry);
      kept = shared && keeps(*q);
      if (q->entry != -1 && (!shared || kept)) return;
      ++need;
      copies += shared && q->rows > 0;
    });
    const Sums second = cluster_scan<2>(need, copies, 0ull, sm, 1, rank, ctas, &all);
    page_at = second.v;
    copy_at = second.w;
    wanted = all.v;
    n_copies = all.w;
  }
  // a group's lanes share the places of its first
  page_at = __shfl_sync(kAll, page_at, lane & ~(lanes - 1));
  copy_at = __shfl_sync(kAll, copy_at, lane & ~(lanes - 1));
  const bool enough = wanted <= n_free;
  if (rank == 0 && threadIdx.x == 0) {
    *p.n_copies = enough ? static_cast<int32_t>(n_copies) : 0;
    *p.n_missing = enough ? 0 : static_cast<int32_t>(wanted - n_free < INT32_MAX ? wanted - n_free : INT32_MAX);
  }
  if (!enough) {
    // as it was: the keepers' numbers out of the counts, then everybody back
    if (sharing) {
      for_pages(Single{}, [&](Place* q, auto) {
        if (q->at && marked(q->entry) && keeps(*q)) pg.counts[marked_page(q->entry)] = 0;
      });
      sync_all(ctas);
      for_pages(Single{}, [&](Place* q, auto) {
        if (!q->at || !marked(q->entry)) return;
        atomicAdd(pg.counts + marked_page(q->entry), 1);
        *q->at = marked_page(q->entry);
      });
    }
    return;
  }

  // the lowest free pages, in order: of one block's few in shared memory. (The
  // shared pages' counts were above 0 when this warp's first batch was read,
  // and are not 0 now: one that was taken there has its keeper's number.)
  const bool near = ctas == 1 && wanted <= kNear;
  int32_t* free_ids = near ? sm.free_ids : p.free_ids;
  const uint32_t most = static_cast<uint32_t>(wanted);  // n_free at most
  if (free_here > 0)
    for_slice(
        pg.counts, slice, first_batch, lane,
        [&](int page, int count) {
          const uint32_t vote = __ballot_sync(kAll, count == 0);
          const uint32_t to = free_at + __popc(vote & ((1u << lane) - 1u));
          if (count == 0 && to < most) free_ids[to] = page;
          free_at += __popc(vote);
        },
        [&] { return free_at < most; });
  if (near) __syncthreads();
  else sync_all(ctas);

  uint32_t page_to = static_cast<uint32_t>(page_at), copy_to = static_cast<uint32_t>(copy_at);
  for_pages(Two{}, [&](Place* q, auto n) {
    constexpr int U = decltype(n)::value;
    int page[U];
    int32_t* copy[U];
    bool stays[U], wants[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const bool shared = q[j].at && marked(q[j].entry);
      stays[j] = shared && (ONE ? kept : keeps(q[j]));
      wants[j] = most > 0 && q[j].at && (q[j].entry == -1 || (shared && !stays[j]));
      const bool copies = wants[j] && shared && q[j].rows > 0;
      const uint32_t want_vote = __ballot_sync(kAll, wants[j]), copy_vote = __ballot_sync(kAll, copies);
      // (only a table that its counts do not fit could want more than was counted)
      const uint32_t at = min(page_to + __popc(want_vote & before_mask), most - 1);
      page[j] = !wants[j] ? 0 : near ? sm.free_ids[at] : __ldcg(p.free_ids + at);
      copy[j] = copies ? p.copies + 3 * (copy_to + __popc(copy_vote & before_mask)) : nullptr;
      page_to += __popc(want_vote & group_mask);
      copy_to += __popc(copy_vote & group_mask);
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (!wants[j] && !stays[j]) continue;
      const int was = marked_page(q[j].entry), now = stays[j] ? was : page[j];
      *q[j].at = now;
      pg.counts[now] = 1;
      if (copy[j]) {
        copy[j][0] = was;
        copy[j][1] = now;
        copy[j][2] = q[j].rows;
      }
    }
  });
}

// ---------------------------------------------------------------- compact

// With U used pages, the k-th highest of those from U on moves into the k-th
// lowest free page below U. A page's rank follows from how many used pages
// lie before it: the holes' from below, the movers' from above. The table follows
// in a second launch, or, of up to kFewEntries entries to a thread, in the same: as
// soon on the GPU (456 entries 4.2 us against 4.6, 16000 in eight blocks 8.0 against
// 7.7), and 2 us less on the host; with eight 6.5 against 6.0.
constexpr int kFewEntries = 4;

// What the entries of the table from `first` on, every step-th, name afterwards.
__device__ __forceinline__ void remap(const CompactProblem& p, int used, int64_t first, int64_t step, int64_t entries) {
  constexpr int U = kFewEntries;
#pragma unroll 1
  for (int64_t i = first; i < entries; i += U * step) {
    int page[U];
#pragma unroll
    for (int j = 0; j < U; ++j) page[j] = i + j * step < entries ? p.pages.table[i + j * step] : -1;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (page[j] >= p.pages.n_pages) atomicOr(&g_device_error, kErrIndex);
      else if (page[j] >= used) page[j] = __ldcg(p.map + page[j]);
    }
#pragma unroll
    for (int j = 0; j < U; ++j)
      if (i + j * step < entries) p.table_out[i + j * step] = page[j];
  }
}

// entries: of the table, if it is to follow here, or 0
__global__ void __launch_bounds__(kClusterThreads) cache_compact_kernel(const CompactProblem p, int entries) {
  __shared__ ClusterSmem sm;
  const uint32_t rank = cluster_ctarank(), ctas = gridDim.x;
  if (ctas > 1) cluster_sync();  // every block has begun: its shared memory may be written
  griddep_wait();
  griddep_launch_dependents();
  const PagesProblem& pg = p.pages;
  const int lane = static_cast<int>(lane_id());
  const Slice slice = warp_slice(pg.n_pages, rank, ctas);
  const int n = slice.end - slice.begin;
  const Batch first_batch = load_batch(pg.counts, slice, slice.begin, lane);
  const int mine = n - free_pages(pg.counts, slice, first_batch, lane);
  Sums all;
  int at = static_cast<int>(cluster_scan<0>(0u, 0u, static_cast<uint64_t>(mine), sm, 0, rank, ctas, &all).w);  // before this warp's
  const int used = static_cast<int>(all.w);
  const bool apart = p.counts_out != pg.counts;
  int movers = 0;
  for_slice(pg.counts, slice, first_batch, lane, [&](int page, int count) {
    const bool in = page < slice.end;
    const uint32_t vote = __ballot_sync(kAll, in && count != 0);
    const int before = at + __popc(vote & ((1u << lane) - 1u));  // used pages before this
    at += __popc(vote);
    if (!in) return;
    const bool high = page >= used;
    const bool moves = high && count != 0, hole = !high && count == 0;
    const int k = moves ? used - 1 - before : page - before;
    movers += moves;
    if ((moves || hole) && k < p.max_copies) {
      p.moves[2 * k + hole] = page;
      return;  // its count and its place in the map are the move's
    }
    if (high) p.map[page] = page;
    if (apart) p.counts_out[page] = count;
  }, [] { return true; });
  movers = static_cast<int>(__reduce_add_sync(kAll, static_cast<unsigned>(movers)));
  cluster_scan<0>(0u, 0u, static_cast<uint64_t>(movers), sm, 1, rank, ctas, &all);
  const int moved = static_cast<int>(all.w) < p.max_copies ? static_cast<int>(all.w) : p.max_copies;
  for (int k = static_cast<int>(rank * blockDim.x + threadIdx.x); k < moved; k += static_cast<int>(ctas * blockDim.x)) {
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
  if (entries == 0) return;
  sync_all(ctas);  // the map is complete
  remap(p, used, rank * blockDim.x + threadIdx.x, ctas * blockDim.x, entries);
}

constexpr int kRemapThreads = 256;

__global__ void __launch_bounds__(kRemapThreads) cache_remap_kernel(const CompactProblem p, int64_t entries) {
  griddep_wait();
  griddep_launch_dependents();
  remap(p, __ldcg(p.n_used), static_cast<int64_t>(blockIdx.x) * kRemapThreads + threadIdx.x,
        static_cast<int64_t>(gridDim.x) * kRemapThreads, entries);
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

// The cluster for so many pages and threads. Blocks: one up to 16384 pages, else
// 256 pages to a warp; and enough for `threads`; or as many as there can be. (In us: a
// step with shared pages and 13000 pages in one block 15.6, in two 18.0; a step with
// 65536 in eight 6.5, in four 7.1, in one 7.9; 64 prompts with 262144 in 16 12.5, in
// eight 17.6.) One block has no more threads than that takes, as it waits for its
// barriers: a step of 128 rows with 973 pages takes 10 with its fork and copies,
// with 1024 threads 11.2.
struct Shape {
  unsigned ctas, threads;
};
Shape cluster_shape(int64_t n_pages, int64_t threads, unsigned most) {
  unsigned ctas = 1;
  while (ctas < most && ((n_pages > 16384 && n_pages > static_cast<int64_t>(ctas) * 256 * kWarps) ||
                         threads > static_cast<int64_t>(ctas) * kClusterThreads))
    ctas *= 2;
  if (ctas > 1) return {ctas, kClusterThreads};
  const int64_t wanted = (threads > n_pages / 8 ? threads : n_pages / 8) + 31;
  return {1, wanted >= kClusterThreads ? kClusterThreads : wanted < 128 ? 128u : static_cast<unsigned>(wanted) & ~31u};
}

cudaLaunchConfig_t cluster_config(const Shape& shape, cudaStream_t stream, cudaLaunchAttribute (&attr)[2]) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(shape.ctas);
  cfg.blockDim = dim3(shape.threads);
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = shape.ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cfg;
}

// The largest cluster of a kernel that the current device takes: 16 blocks, or the
// portable 8. Asked once for each kernel and device (`known` is the kernel's own).
constexpr int kDevices = 64;
template <typename Kernel>
cudaError_t most_blocks(Kernel kernel, unsigned (&known)[kDevices], unsigned* most) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  unsigned* mine = dev >= 0 && dev < kDevices ? &known[dev] : nullptr;
  *most = mine ? __atomic_load_n(mine, __ATOMIC_ACQUIRE) : 0;
  if (*most != 0) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = cluster_config({kMaxCtas, kClusterThreads}, nullptr, attr);
  cfg.numAttrs = 1;
  int fit = 0;
  if (cudaOccupancyMaxActiveClusters(&fit, kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();
    fit = 0;
  }
  *most = fit > 0 ? kMaxCtas : 8;
  if (mine) __atomic_store_n(mine, *most, __ATOMIC_RELEASE);
  return cudaSuccess;
}

template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kernel)(KArgs...), const Shape& shape, cudaStream_t stream, Args&&... args) {
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = cluster_config(shape, stream, attr);
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

}  // namespace

cudaError_t launch_cache_fork(const PagesProblem& p, int32_t* lens, const int32_t* parents,
                              cudaStream_t stream) {
  // columns to a block: two entries to a thread, or up to 32 columns (a line of
  // memory) where that leaves four blocks to an SM
  int cols_log2 = 0;
  while (cols_log2 < 5 && (static_cast<int64_t>(p.B) << (cols_log2 + 1)) <= kForkEntries &&
         ((p.B << (cols_log2 + 1)) <= kForkFew || (p.max_pages >> (cols_log2 + 1)) >= 4 * sm_count()))
    ++cols_log2;
  static unsigned long long configured = 0;
  cudaError_t e = set_smem_once(cache_fork_kernel, kForkBytes, &configured);
  if (e != cudaSuccess) return e;
  const int64_t blocks = ((static_cast<int64_t>(p.max_pages) - 1) >> cols_log2) + 1 + (lens ? 1 : 0);
  return launch_pdl(cache_fork_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kForkThreads),
                    ((static_cast<size_t>(p.B) << cols_log2) + (p.B <= kForkStaged ? p.B : 0)) * 4, stream, p, lens, parents, cols_log2);
}

cudaError_t launch_cache_release(const PagesProblem& p, const int32_t* keep_lens, cudaStream_t stream) {
  const int chunks = (p.max_pages - 1) / kReleaseThreads + 1;
  const int64_t items = static_cast<int64_t>(p.B) * chunks;
  const int64_t most = static_cast<int64_t>(sm_count()) * 8;
  return launch_pdl(cache_release_kernel, dim3(static_cast<unsigned>(items < most ? items : most)),
                    dim3(kReleaseThreads), 0, stream, p, keep_lens, items, chunks);
}

cudaError_t launch_cache_reserve(const ReserveProblem& p, cudaStream_t stream) {
  // lanes to a unit: for the most pages that a row's new tokens can lie in
  int lanes_log2 = 0;
  while (lanes_log2 < 5 && (1 << lanes_log2) < p.width) ++lanes_log2;
  const int units = (p.width + (1 << lanes_log2) - 1) >> lanes_log2;
  const int64_t threads = (static_cast<int64_t>(p.pages.B) * units) << lanes_log2;
  static unsigned known_one[kDevices], known_many[kDevices];
  unsigned most_one = 0, most_many = 0;
  cudaError_t e = most_blocks(cache_reserve_kernel<true>, known_one, &most_one);
  if (e == cudaSuccess) e = most_blocks(cache_reserve_kernel<false>, known_many, &most_many);
  if (e != cudaSuccess) return e;
  const Shape shape = cluster_shape(p.pages.n_pages, threads, most_one < most_many ? most_one : most_many);
  return threads <= static_cast<int64_t>(shape.ctas) * shape.threads
             ? launch_cluster(cache_reserve_kernel<true>, shape, stream, p, lanes_log2, units)
             : launch_cluster(cache_reserve_kernel<false>, shape, stream, p, lanes_log2, units);
}

cudaError_t launch_cache_compact(const CompactProblem& p, cudaStream_t stream) {
  static unsigned known[kDevices];
  unsigned most_ctas = 0;
  cudaError_t e = most_blocks(cache_compact_kernel, known, &most_ctas);
  if (e != cudaSuccess) return e;
  const Shape shape = cluster_shape(p.pages.n_pages, kClusterThreads, most_ctas);  // threads: for the moves and entries
  const int64_t entries = static_cast<int64_t>(p.pages.B) * p.pages.max_pages;
  const bool few = entries <= static_cast<int64_t>(kFewEntries) * shape.ctas * shape.threads;
  e = launch_cluster(cache_compact_kernel, shape, stream, p, few ? static_cast<int>(entries) : 0);
  if (e != cudaSuccess || few) return e;
  const int64_t blocks = (entries + kRemapThreads - 1) / kRemapThreads, most = static_cast<int64_t>(sm_count()) * 8;
  return launch_pdl(cache_remap_kernel, dim3(static_cast<unsigned>(blocks < most ? blocks : most)), dim3(kRemapThreads), 0,
                    stream, p, entries);
}

TSD_DEFINE_ERROR_READER(take_device_error_pages)

}  // namespace tsd
