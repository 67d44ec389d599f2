// The page table of a paged cache: whose pages are whose.
//
//   table [B, M] pages of each sequence in order, -1: none;  uses [pages], in how many places of the table a page
//   stands, 0: free.
//
//   fork     row b becomes what row parent[b] was, or empty; the uses follow.  Any reordering, in place: a CTA holds
//            a few columns of the whole table in shared memory.  Counts are integers, so the atomics' order does not show.
//   reserve  every page that the next tokens of a sequence touch and that is missing or has other users is replaced by a
//            free one: the lowest free pages in the order of the sequences and their pages.  Of a shared page that
//            holds tokens already the content is copied.  One cluster counts and ranks wants and free pages (the prefix
//            sums cross its CTAs through distributed shared memory) and hands the pages out; a second launch copies.
//   compact  the pages in use, in order, into another pool; ranks by the same cluster, then copies over the whole GPU.
//
// Bound: reserve by latency (a few dependent loads and three cluster barriers), the copies by HBM.
#include "paged.cuh"

namespace raattn {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kCopyThreads = 256, kCopyAhead = 4;
constexpr int kChunk = kCopyThreads * kCopyAhead * 16;   // bytes of a page that a CTA copies at a time

__device__ __forceinline__ bool is_page(int id, int pages) { return static_cast<unsigned>(id) < static_cast<unsigned>(pages); }

// ---------------------------------------------------------------------------------------------
// fork
// ---------------------------------------------------------------------------------------------
template <int W>   // columns of a CTA
__global__ void __launch_bounds__(kThreads) page_fork_kernel(const PageFork a) {
  extern __shared__ int old[];   // [B][W], the parents, and in the first CTA the lengths
  const int c0 = blockIdx.x * W, n = a.B * W;
  int *parent = old + n, *lengths = parent + a.B;
  await_previous();
  release_dependents();
  for (int b = threadIdx.x; b < a.B; b += kThreads) {
    parent[b] = a.parent[b];
    if (blockIdx.x == 0) lengths[b] = a.length[b];
  }
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int c = c0 + i % W;
    old[i] = c < a.M ? a.table[static_cast<int64_t>(i / W) * a.M + c] : -1;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int b = i / W, c = c0 + i % W, from = parent[b];
    if (c >= a.M || from == b) continue;
    const int was = old[i], is = is_page(from, a.B) ? old[from * W + i % W] : -1;
    if (was == is) continue;
    a.table[static_cast<int64_t>(b) * a.M + c] = is;
    if (is_page(was, a.pages)) atomicSub(a.uses + was, 1);
    if (is_page(is, a.pages)) atomicAdd(a.uses + is, 1);
  }
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < a.B; b += kThreads) {
      const int from = parent[b];
      if (from != b) a.length[b] = is_page(from, a.B) ? lengths[from] : 0;
    }
}

// ---------------------------------------------------------------------------------------------
// ranks over a cluster
// ---------------------------------------------------------------------------------------------
// Exclusive prefix sums of two counts per warp over the warps of a cluster of C CTAs, and their totals.  All threads;
// counts are the same in all lanes of a warp.  C = 1: an ordinary CTA.
struct ClusterSums {
  int2 warp[kWarps];
  int2 total;
};
template <int C>
__device__ __forceinline__ void all_sync() {
  if (C > 1) cluster_sync();
  else __syncthreads();
}
template <int C>
__device__ __forceinline__ int2 cluster_exclusive(ClusterSums& s, int2 mine, int2* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  if (lane == 0) s.warp[w] = mine;
  __syncthreads();
  int2 inc = s.warp[lane];
  const int2 own = inc;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, inc.x, o), y = __shfl_up_sync(0xffffffffu, inc.y, o);
    if (lane >= o) {
      inc.x += x;
      inc.y += y;
    }
  }
  int2 before = make_int2(__shfl_sync(0xffffffffu, inc.x - own.x, w), __shfl_sync(0xffffffffu, inc.y - own.y, w));
  *total = make_int2(__shfl_sync(0xffffffffu, inc.x, 31), __shfl_sync(0xffffffffu, inc.y, 31));
  if constexpr (C > 1) {
    if (threadIdx.x == 0) s.total = *total;
    cluster_sync();
    const uint32_t at = smem_u32(&s.total), rank = cluster_ctarank();
    int2 x[C];
#pragma unroll
    for (uint32_t r = 0; r < C; ++r)
      asm volatile("ld.shared::cluster.v2.s32 {%0, %1}, [%2];" : "=r"(x[r].x), "=r"(x[r].y) : "r"(mapa_shared(at, r)) : "memory");
    *total = make_int2(0, 0);
#pragma unroll
    for (uint32_t r = 0; r < C; ++r) {
      if (r < rank) {
        before.x += x[r].x;
        before.y += x[r].y;
      }
      total->x += x[r].x;
      total->y += x[r].y;
    }
  }
  return before;
}

// A warp's contiguous share [first, last) of n items, in whole steps of 32 R items.
template <int C, int R>
__device__ __forceinline__ int2 share_of(int n) {
  const int w = (C > 1 ? static_cast<int>(cluster_ctarank()) * kWarps : 0) + (threadIdx.x >> 5);
  const int64_t steps = (static_cast<int64_t>(n) + 32 * R - 1) / (32 * R), per = (steps + C * kWarps - 1) / (C * kWarps) * (32 * R);
  const int64_t first = w * per;
  return make_int2(static_cast<int>(first < n ? first : n), static_cast<int>(first + per < n ? first + per : n));
}
constexpr int kPer = 8;   // loads of a lane in flight

// A warp's share of the pages; LIVE: those in use count, else the free ones.  The first step's uses stay in registers.
template <int C, bool LIVE>
struct Pages {
  const int32_t* uses;
  int2 range;
  int held[kPer];
  __device__ __forceinline__ Pages(const int32_t* uses_, int n) : uses(uses_), range(share_of<C, kPer>(n)) { load(range.x, held); }
  __device__ __forceinline__ void load(int p0, int (&u)[kPer]) const {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int p = p0 + 32 * i + static_cast<int>(threadIdx.x & 31);
      u[i] = p < range.y ? uses[p] : LIVE ? 0 : 1;
    }
  }
  static __device__ __forceinline__ bool counts(int u) { return LIVE ? u > 0 : u == 0; }
  __device__ __forceinline__ int count() const {
    int n = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) n += counts(held[i]);
    for (int p0 = range.x + 32 * kPer; p0 < range.y; p0 += 32 * kPer) {
      int u[kPer];
      load(p0, u);
#pragma unroll
      for (int i = 0; i < kPer; ++i) n += counts(u[i]);
    }
    return __reduce_add_sync(0xffffffffu, n);
  }
  template <typename F>
  __device__ __forceinline__ void step(int p0, const int (&u)[kPer], int& rank, F f) const {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int p = p0 + 32 * i + lane;
      const unsigned all = __ballot_sync(0xffffffffu, counts(u[i]));
      if (p < range.y) f(p, u[i], counts(u[i]), rank + __popc(all & ((1u << lane) - 1u)));
      rank += __popc(all);
    }
  }
  // f(page, uses, whether it counts, its rank); `rank`: of the warp's first that counts.
  template <typename F>
  __device__ __forceinline__ void each(int rank, F f) const {
    if (range.x < range.y) step(range.x, held, rank, f);
    for (int p0 = range.x + 32 * kPer; p0 < range.y; p0 += 32 * kPer) {
      int u[kPer];
      load(p0, u);
      step(p0, u, rank, f);
    }
  }
};

// ---------------------------------------------------------------------------------------------
// reserve
// ---------------------------------------------------------------------------------------------
// Place k of sequence b among the pages that its new tokens touch.
struct Want {
  int b, k, at, length, tokens;
  int old;        // the page there, or -1
  bool touched, wanted;
};
__device__ __forceinline__ Want want_of(const PageReserve& a, int item) {
  Want w;
  w.b = item / a.per_row;
  w.k = item - w.b * a.per_row;
  const int64_t most = static_cast<int64_t>(a.M) << a.pool.shift;
  w.length = static_cast<int>(min(static_cast<int64_t>(max(a.length[w.b], 0)), most));
  w.tokens = a.count ? min(max(a.count[w.b], 0), a.tokens) : a.tokens;
  w.at = (w.length >> a.pool.shift) + w.k;
  w.touched = w.tokens > 0 && w.at < a.M && (static_cast<int64_t>(w.at) << a.pool.shift) < static_cast<int64_t>(w.length) + w.tokens;
  w.old = w.touched ? paged::page_at(a.pool, a.table + static_cast<int64_t>(w.b) * a.M, w.at) : -1;
  return w;
}

template <int C>
__global__ void __cluster_dims__(C, 1, 1) __launch_bounds__(kThreads) page_reserve_kernel(const PageReserve a) {
  __shared__ ClusterSums sums;
  const int lane = threadIdx.x & 31, items = a.B * a.per_row;
  const int2 mine = share_of<C, 1>(items);
  await_previous();
  release_dependents();
  const Pages<C, false> pages(a.uses, a.pool.pages);
  // wants, left in the workspace as ranks within the warp's share: the uses that they go by change below
  int wants = 0;
  for (int i0 = mine.x; i0 < mine.y; i0 += 32) {
    const int item = i0 + lane;
    bool wanted = false;
    if (item < mine.y) {
      const Want w = want_of(a, item);
      wanted = w.touched && (w.old < 0 || a.uses[w.old] > 1);
      if (w.k == 0) {
        const int64_t room = (static_cast<int64_t>(a.M) << a.pool.shift) - w.length;
        a.granted[w.b] = static_cast<int>(min(static_cast<int64_t>(w.tokens), room));
        a.copy[2 * w.b] = -1;
      }
    }
    const unsigned all = __ballot_sync(0xffffffffu, wanted);
    if (item < mine.y) a.place[item] = wanted ? wants + __popc(all & ((1u << lane) - 1u)) : -1;
    wants += __popc(all);
  }
  int2 total;
  const int2 before = cluster_exclusive<C>(sums, make_int2(wants, pages.count()), &total);
  if (total.x > 0)   // the same in all CTAs
    pages.each(before.y, [&](int p, int, bool free, int rank) {
      if (free && rank < total.x) a.freed[rank] = p;
    });
  all_sync<C>();   // and no CTA ends while another reads its counts
  if (total.x == 0) return;
  for (int i0 = mine.x; i0 < mine.y; i0 += 32) {
    const int item = i0 + lane;
    if (item >= mine.y || a.place[item] < 0) continue;
    const int rank = before.x + a.place[item];
    const Want w = want_of(a, item);   // its own place in the table, which no other thread changes
    if (rank < total.y) {
      const int id = __ldcg(a.freed + rank);
      a.table[static_cast<int64_t>(w.b) * a.M + w.at] = id;
      a.uses[id] = 1;
      if (w.old >= 0) {
        atomicSub(a.uses + w.old, 1);
        if (w.k == 0 && (w.length & (a.pool.page - 1))) {   // tokens that stay
          a.copy[2 * w.b + 1] = id;
          a.copy[2 * w.b] = w.old;
        }
      }
    } else {
      atomicMin(a.granted + w.b, max(static_cast<int>((static_cast<int64_t>(w.at) << a.pool.shift) - w.length), 0));
    }
  }
}

// ---------------------------------------------------------------------------------------------
// copies
// ---------------------------------------------------------------------------------------------
__device__ __forceinline__ void copy_chunk(uint8_t* to, const uint8_t* from, int64_t at, int64_t bytes) {
  uint4 x[kCopyAhead];
#pragma unroll
  for (int i = 0; i < kCopyAhead; ++i) {
    const int64_t o = at + (i * kCopyThreads + threadIdx.x) * 16;
    if (o < bytes) x[i] = __ldcs(reinterpret_cast<const uint4*>(from + o));
  }
#pragma unroll
  for (int i = 0; i < kCopyAhead; ++i) {
    const int64_t o = at + (i * kCopyThreads + threadIdx.x) * 16;
    if (o < bytes) __stcs(reinterpret_cast<uint4*>(to + o), x[i]);
  }
}

__global__ void __launch_bounds__(kCopyThreads) page_copy_kernel(const PageReserve a, int chunks) {
  await_previous();
  const int64_t items = static_cast<int64_t>(a.B) * chunks;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int b = static_cast<int>(item / chunks);
    const int from = __ldcg(a.copy + 2 * b);
    if (from < 0) continue;
    const int to = __ldcg(a.copy + 2 * b + 1);
    copy_chunk(a.pool.base + static_cast<int64_t>(to) * a.pool.page_stride, a.pool.base + static_cast<int64_t>(from) * a.pool.page_stride,
               (item - static_cast<int64_t>(b) * chunks) * kChunk, a.page_bytes);
  }
}

// ---------------------------------------------------------------------------------------------
// compact
// ---------------------------------------------------------------------------------------------
template <int C>
__global__ void __cluster_dims__(C, 1, 1) __launch_bounds__(kThreads) page_rank_kernel(const PageCompact a) {
  __shared__ ClusterSums sums;
  await_previous();
  release_dependents();
  const Pages<C, true> pages(a.uses, a.pages);
  int2 total;
  const int2 before = cluster_exclusive<C>(sums, make_int2(pages.count(), 0), &total);
  pages.each(before.x, [&](int p, int uses, bool live, int rank) {
    a.rank[p] = live && rank < a.pages_out ? rank : -1;
    if (live && rank < a.pages_out) {
      a.order[rank] = p;
      a.uses_out[rank] = uses;
    }
  });
  const int here = (C > 1 ? static_cast<int>(cluster_ctarank()) * kThreads : 0) + threadIdx.x;
  for (int64_t p = static_cast<int64_t>(total.x) + here; p < a.pages_out; p += C * kThreads) a.uses_out[p] = 0;
  if (here == 0) a.live[0] = total.x;
  all_sync<C>();   // no CTA ends while another reads its counts
}

__global__ void __launch_bounds__(kCopyThreads) page_move_kernel(const PageCompact a, int chunks) {
  await_previous();
  const int64_t places = static_cast<int64_t>(a.B) * a.M;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kCopyThreads + threadIdx.x; i < places;
       i += static_cast<int64_t>(gridDim.x) * kCopyThreads) {
    const int id = a.table[i];
    a.table_out[i] = is_page(id, a.pages) ? __ldcg(a.rank + id) : -1;
  }
  const int64_t items = static_cast<int64_t>(min(__ldcg(a.live), a.pages_out)) * chunks;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int page = static_cast<int>(item / chunks);
    copy_chunk(a.to + page * a.to_stride, a.from + __ldcg(a.order + page) * a.from_stride,
               (item - static_cast<int64_t>(page) * chunks) * kChunk, a.page_bytes);
  }
}

int chunks_of(int64_t page_bytes) { return static_cast<int>((page_bytes + kChunk - 1) / kChunk); }
unsigned copy_grid(int64_t items) { return static_cast<unsigned>(items < 1 ? 1 : items < 8 * kSms ? items : 8 * kSms); }

}  // namespace

cudaError_t launch_page_fork(const PageFork& a, cudaStream_t st) {
  constexpr int kWide = 8, kNarrow = 4;
  constexpr int kMost = 220 * 1024;   // bytes of shared memory: W columns, the parents and the lengths
  static_assert((kNarrow + 2) * kMostForkRows * 4 <= kMost, "every table fits");
  const bool wide = (kWide + 2) * a.B * 4 <= kMost;
  cudaError_t e = wide ? set_up_kernel<page_fork_kernel<kWide>>(kMost, false) : set_up_kernel<page_fork_kernel<kNarrow>>(kMost, false);
  if (e != cudaSuccess) return e;
  const int W = wide ? kWide : kNarrow, grid = (a.M + W - 1) / W, smem = (W + 2) * a.B * 4;
  return wide ? launch_dependent(page_fork_kernel<kWide>, grid, kThreads, smem, st, a)
              : launch_dependent(page_fork_kernel<kNarrow>, grid, kThreads, smem, st, a);
}

// One CTA where it has a step or two of pages and a few of places, else a cluster (fork and reserve of B256, 8192 pages: 10.9 us
// against 12.4; of B16, 256 pages 7.4 against 8.8).
bool one_cta(int pages, int items) { return pages <= 2 * 32 * kPer * kWarps && items <= 4 * kThreads; }
constexpr int kCluster = 8;

cudaError_t launch_page_reserve(const PageReserve& a, cudaStream_t st) {
  const cudaError_t e = one_cta(a.pool.pages, a.B * a.per_row)
                            ? launch_dependent(page_reserve_kernel<1>, 1, kThreads, 0, st, a)
                            : launch_dependent(page_reserve_kernel<kCluster>, kCluster, kThreads, 0, st, a);
  if (e != cudaSuccess) return e;
  const int chunks = chunks_of(a.page_bytes);
  return launch_dependent(page_copy_kernel, copy_grid(static_cast<int64_t>(a.B) * chunks), kCopyThreads, 0, st, a, chunks);
}

cudaError_t launch_page_compact(const PageCompact& a, cudaStream_t st) {
  const cudaError_t e = one_cta(a.pages, 0) ? launch_dependent(page_rank_kernel<1>, 1, kThreads, 0, st, a)
                                            : launch_dependent(page_rank_kernel<kCluster>, kCluster, kThreads, 0, st, a);
  if (e != cudaSuccess) return e;
  const int chunks = chunks_of(a.page_bytes);
  const int64_t most = a.pages < a.pages_out ? a.pages : a.pages_out, table = (static_cast<int64_t>(a.B) * a.M + kCopyThreads - 1) / kCopyThreads;
  const int64_t items = most * chunks;
  return launch_dependent(page_move_kernel, copy_grid(items > table ? items : table), kCopyThreads, 0, st, a, chunks);
}

}  // namespace raattn
