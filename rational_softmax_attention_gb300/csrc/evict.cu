// Eviction from a key/value cache by accumulated attention weight.
//
// Per (sequence, key head), with n = length[b], last = min(recent, n) and m = min(n, keep): the
// last `last` entries stay, and of the others the m - last with the largest weight (of equal
// weights the lowest slots).  The kept entries' keys, values and weights are written, in their
// order, to the first m slots of another cache.
//
//   select   a cluster of CTAs per (sequence, head), each with a slice of the entries: the threshold
//            by a radix selection over the weights' order-preserving bits (eight at a time; the
//            CTAs' counts are added through distributed shared memory, whose reads cost more than
//            a fourth pass: with 2048 bins they took 3 us a pass), then the kept
//            slots in order by prefix sums.  Each pass has counters of its own, so that one barrier of
//            the cluster per pass is enough.  Counts are integers, so nothing depends on the order
//            of the atomics.  A CTA's first 8192 weights stay in registers between the passes.
//   gather   the kept entries, 16 bytes per lane.
// Bound: select by latency (four passes, each of atomics that meet in few bins where weights have few exponents, and a
// barrier; the two were not timed apart: 14 us for 32 rows of 32768), gather by HBM
// (B32 H8 4352 -> 4096, D128 bf16: 849 MB in 133 us, 6.4 TB/s).  Both together, in a graph: B4 H8
// 32768 -> 2048 21.5 us.
#include "kernels.cuh"

namespace raattn {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kBins = 256, kPasses = 4;

// Order-preserving bits of a weight: larger weights give larger bits; -0 and 0 are equal; NaN above all.
__device__ __forceinline__ uint32_t order_bits(float w) {
  const uint32_t u = __float_as_uint(w == 0.0f ? 0.0f : w);
  if (w != w) return 0xffffffffu;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

constexpr uint32_t kZeroBits = 0x80000000u;   // order_bits(0)

// Exclusive prefix sum of v over the CTA; *total the sum.  All threads.
__device__ __forceinline__ int block_exclusive(int v, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    int s = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += x;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  *total = warp_sums[31];
  return inc - v + (warp ? warp_sums[warp - 1] : 0);
}

constexpr int kPer = 4;                        // consecutive entries of a thread in a chunk
constexpr int kChunk = kSelThreads * kPer;
constexpr int kHeld = 2;                       // chunks held in registers

template <int S>   // CTAs of a cluster
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a) {
  __shared__ int hist[kPasses][kBins];   // a pass's own: one barrier of the cluster per pass
  __shared__ int warp_sums[32];
  __shared__ int found[kPasses], left;
  __shared__ int2 counts;   // entries of this CTA's slice above the threshold, and equal to it
  const int rank = S > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int bk = blockIdx.x / S, b = bk / a.Hkv, kv = bk - b * a.Hkv;
  release_dependents();
  const int n = min(max(a.length[b], 0), a.C), m = min(n, a.keep), last = min(a.recent, n);
  const int cand = n - last, need = m - last;
  const float* w = a.weight + static_cast<int64_t>(bk) * a.C;
  int* index = a.index + static_cast<int64_t>(bk) * a.keep;
  if (rank == 0 && kv == 0 && threadIdx.x == 0) a.length_out[b] = m;
  for (int i = m + rank * kSelThreads + threadIdx.x; i < a.keep; i += S * kSelThreads) index[i] = -1;
  for (int i = rank * kSelThreads + threadIdx.x; i < last; i += S * kSelThreads) index[need + i] = cand + i;
  if (need == cand || need == 0) {   // all others stay, or none
    for (int i = rank * kSelThreads + threadIdx.x; i < need; i += S * kSelThreads) index[i] = i;
    return;   // uniform over the cluster
  }
  // this CTA's slice, in whole chunks
  const int chunks = (cand + kChunk - 1) / kChunk, per = (chunks + S - 1) / S;
  const int q0 = min(rank * per, chunks), q1 = min(q0 + per, chunks);
  auto load = [&](int q, uint32_t (&u)[kPer]) {   // 0, below every weight's bits, past the last
    const int i = q * kChunk + threadIdx.x * kPer;
#pragma unroll
    for (int j = 0; j < kPer; ++j) u[j] = i + j < cand ? order_bits(w[i + j]) : 0u;
  };
  uint32_t held[kHeld][kPer];
#pragma unroll
  for (int h = 0; h < kHeld; ++h)
    if (q0 + h < q1) load(q0 + h, held[h]);
  // f(entry bits of a chunk) for every chunk of the slice
  auto each = [&](auto f) {
#pragma unroll
    for (int h = 0; h < kHeld; ++h)
      if (q0 + h < q1) f(q0 + h, held[h]);
    for (int q = q0 + kHeld; q < q1; ++q) {
      uint32_t u[kPer];
      load(q, u);
      f(q, u);
    }
  };
  // The threshold: the need-th largest.  `rest` counts what is still wanted among the entries that
  // share the bits found so far.
  static_assert(kPasses * kBins == kSelThreads, "a thread per bin");
  hist[0][threadIdx.x] = 0;
  if (threadIdx.x == 0) counts = make_int2(0, 0);
  __syncthreads();
  uint32_t prefix = 0;
  int rest = need;
#pragma unroll 1
  for (int pass = 0; pass < kPasses; ++pass) {
    const int shift = 24 - 8 * pass, done = 8 * pass;   // done: bits found
    each([&](int, const uint32_t (&u)[kPer]) {
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const bool in = u[j] && (done == 0 || u[j] >> (32 - done) == prefix);
        // weights of exactly 0 (entries outside every query's support) are many: one addition for a warp's
        const unsigned zeros = __ballot_sync(0xffffffffu, in && u[j] == kZeroBits);
        if (zeros && (threadIdx.x & 31) == 0) atomicAdd(&hist[pass][kZeroBits >> shift & 255u], __popc(zeros));
        if (in && u[j] != kZeroBits) atomicAdd(&hist[pass][u[j] >> shift & 255u], 1);
      }
    });
    if (S > 1) cluster_sync();
    else __syncthreads();
    // bins from the top, one thread each
    const int bin = kBins - 1 - static_cast<int>(threadIdx.x);
    int c = 0, sum = 0;
    if (threadIdx.x < kBins) {
      if (S > 1) {
        const uint32_t at = smem_u32(&hist[pass][bin]);
        int x[S];
#pragma unroll
        for (int r = 0; r < S; ++r)
          asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(x[r]) : "r"(mapa_shared(at, r)) : "memory");
#pragma unroll
        for (int r = 0; r < S; ++r) c += x[r];
      } else {
        c = hist[pass][bin];
      }
      sum = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, sum, o);
        if ((threadIdx.x & 31) >= o) sum += x;
      }
      if ((threadIdx.x & 31) == 31) warp_sums[threadIdx.x >> 5] = sum;
    }
    __syncthreads();
    if (threadIdx.x < kBins) {
      int before = sum - c;
      for (int w = 0; w < static_cast<int>(threadIdx.x >> 5); ++w) before += warp_sums[w];
      if (before < rest && rest <= before + c) {
        found[pass] = bin;
        left = rest - before;
      }
    }
    __syncthreads();
    prefix = prefix << 8 | static_cast<uint32_t>(found[pass]);
    rest = left;   // written again only behind the next pass's barriers
  }
  // The kept slots in order: entries above the threshold and the first `rest` equal to it.  Both
  // counts of a chunk (at most 4096) go through one prefix sum.  A slice's counts are in its bins: above
  // the threshold lie those above the found bin of each pass.
  int above = 0, equal = 0;   // of the entries before this chunk
  if (S > 1) {
    const int pass = threadIdx.x / kBins, bin = threadIdx.x % kBins;
    const int mine = __reduce_add_sync(0xffffffffu, bin > found[pass] ? hist[pass][bin] : 0);
    if ((threadIdx.x & 31) == 0 && mine) atomicAdd(&counts.x, mine);
    if (threadIdx.x == 0) counts.y = hist[kPasses - 1][found[kPasses - 1]];
    cluster_sync();
    int x[S], y[S];
#pragma unroll
    for (int r = 0; r < S; ++r)
      asm volatile("ld.shared::cluster.v2.s32 {%0, %1}, [%2];"
                   : "=r"(x[r]), "=r"(y[r])
                   : "r"(mapa_shared(smem_u32(&counts), r))
                   : "memory");
#pragma unroll
    for (int r = 0; r < S; ++r) {
      above += r < rank ? x[r] : 0;
      equal += r < rank ? y[r] : 0;
    }
  }
  each([&](int q, const uint32_t (&u)[kPer]) {
    int gt = 0, eq = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      gt += u[j] > prefix ? 1 : 0;
      eq += u[j] == prefix ? 1 : 0;
    }
    int total;
    const int x = block_exclusive(gt << 16 | eq, warp_sums, &total);
    int a0 = above + (x >> 16), e0 = equal + (x & 0xffff);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const bool hi = u[j] > prefix, tie = u[j] == prefix;
      if (hi || (tie && e0 < rest)) index[a0 + min(e0, rest)] = q * kChunk + threadIdx.x * kPer + j;
      a0 += hi ? 1 : 0;
      e0 += tie ? 1 : 0;
    }
    above += total >> 16;
    equal += total & 0xffff;
  });
  if (S > 1) cluster_sync();   // nobody leaves while its counts may be read
}

constexpr int kGatherThreads = 256;

// Threads over the kept entries' vectors; an entry's K and V vectors are read together.
__global__ void __launch_bounds__(kGatherThreads) evict_gather_kernel(const EvictArgs a) {
  const int vecs = a.row_bytes / 16;
  const int64_t per_head = static_cast<int64_t>(a.keep) * vecs;
  const int64_t total = static_cast<int64_t>(a.B) * a.Hkv * per_head;
  await_previous();
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kGatherThreads + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * kGatherThreads) {
    const int64_t bk = i / per_head, r = i - bk * per_head;
    const int e = static_cast<int>(r / vecs), c = static_cast<int>(r - static_cast<int64_t>(e) * vecs);
    const int from = a.index[bk * a.keep + e];
    if (from < 0) continue;
    const int64_t src = (bk * a.C + from) * vecs + c, dst = (bk * a.C_out + e) * vecs + c;
    const uint4 x = static_cast<const uint4*>(a.k)[src], y = static_cast<const uint4*>(a.v)[src];
    static_cast<uint4*>(a.k_out)[dst] = x;
    static_cast<uint4*>(a.v_out)[dst] = y;
    if (c == 0) a.weight_out[bk * a.C_out + e] = a.weight[bk * a.C + from];
  }
}

template <int S>
cudaError_t select(const EvictArgs& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.B) * a.Hkv * S);
  cfg.blockDim = dim3(kSelThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = S;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = S > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, evict_select_kernel<S>, a);
}

}  // namespace

// CTAs of a row's cluster: as many as give every SM one at most, while each still gets a chunk of
// 4096 entries.  (Two per SM do not all find room in clusters of eight: 32 rows of 32768 took 44 us
// so, gather included, when clusters of four took 23; with one CTA per row 42.)
cudaError_t launch_evict(const EvictArgs& a, cudaStream_t st) {
  const int64_t rows = static_cast<int64_t>(a.B) * a.Hkv, chunks = (a.C + kChunk - 1) / kChunk;
  int s = 1;
  while (s < 8 && rows * 2 * s <= kSms && 2 * s <= chunks) s *= 2;
  const cudaError_t e = s == 8 ? select<8>(a, st) : s == 4 ? select<4>(a, st) : s == 2 ? select<2>(a, st) : select<1>(a, st);
  if (e != cudaSuccess) return e;
  const int64_t total = rows * a.keep * (a.row_bytes / 16);
  const int64_t blocks = (total + kGatherThreads - 1) / kGatherThreads;
  return launch_dependent(evict_gather_kernel, static_cast<unsigned>(blocks < 16 * kSms ? blocks : 16 * kSms),
                          kGatherThreads, 0, st, a);
}

}  // namespace raattn
