// Eviction from a key/value cache by accumulated attention weight.
//
// Per (sequence, key head), with n = length[b], last = min(recent, n) and m = min(n, keep): the
// last `last` entries stay, and of the others the m - last with the largest weight (of equal
// weights the lowest slots).  The kept entries' keys, values and weights are written, in their
// order, to the first m slots of another cache.
//
//   select   one CTA per (sequence, head): the threshold by a radix selection over the weights'
//            order-preserving bits, then the kept slots in order by prefix sums;
//   gather   the kept entries, 16 bytes per lane: HBM-bound.
#include "kernels.cuh"

namespace raattn {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kBins = 2048;

// Order-preserving bits of a weight: larger weights give larger bits; -0 and 0 are equal; NaN above all.
__device__ __forceinline__ uint32_t order_bits(float w) {
  const uint32_t u = __float_as_uint(w == 0.0f ? 0.0f : w);
  if (w != w) return 0xffffffffu;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

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

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a) {
  __shared__ int hist[kBins];
  __shared__ int warp_sums[32];
  __shared__ uint32_t found;
  __shared__ int left;
  const int bk = blockIdx.x, b = bk / a.Hkv, kv = bk - b * a.Hkv;
  const int n = min(max(a.length[b], 0), a.C), m = min(n, a.keep), last = min(a.recent, n);
  const int cand = n - last, need = m - last;
  const float* w = a.weight + static_cast<int64_t>(bk) * a.C;
  int* index = a.index + static_cast<int64_t>(bk) * a.keep;
  if (kv == 0 && threadIdx.x == 0) a.length_out[b] = m;
  for (int i = m + threadIdx.x; i < a.keep; i += kSelThreads) index[i] = -1;
  if (need == cand) {   // everything stays
    for (int i = threadIdx.x; i < m; i += kSelThreads) index[i] = i;
    return;
  }
  // The threshold: the need-th largest, 11 + 11 + 10 bits at a time.  `rank` counts what is still
  // wanted among the entries that share the bits found so far.
  uint32_t prefix = 0;
  int rank = need;
  int done = 0;   // bits found
  if (need > 0) {
    for (int pass = 0; pass < 3; ++pass) {
      const int bits = pass < 2 ? 11 : 10, shift = 32 - done - bits;
      for (int i = threadIdx.x; i < kBins; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      for (int i = threadIdx.x; i < cand; i += kSelThreads) {
        const uint32_t u = order_bits(w[i]);
        if (done == 0 || u >> (32 - done) == prefix) atomicAdd(&hist[(u >> shift) & ((1u << bits) - 1u)], 1);
      }
      __syncthreads();
      // bins from the top: thread t owns the t-th pair of bins counted from the highest
      const int hi = kBins - 1 - 2 * static_cast<int>(threadIdx.x), c1 = hist[hi], c0 = hist[hi - 1];
      int total;
      const int before = block_exclusive(c1 + c0, warp_sums, &total);
      if (before < rank && rank <= before + c1 + c0) {
        const bool upper = rank <= before + c1;
        found = static_cast<uint32_t>(upper ? hi : hi - 1);
        left = rank - before - (upper ? 0 : c1);
      }
      __syncthreads();
      prefix = prefix << bits | found;
      rank = left;
      done += bits;
      __syncthreads();
    }
  }
  // The kept slots in order: entries above the threshold and the first `rank` equal to it.
  int kept = 0, equal = 0;
  for (int i0 = 0; i0 < cand; i0 += kSelThreads) {
    const int i = i0 + threadIdx.x;
    const uint32_t u = i < cand && need > 0 ? order_bits(w[i]) : 0u;
    const bool in = i < cand && need > 0;
    const int eq = in && u == prefix, gt = in && u > prefix;
    int teq, tall;
    const int eq_before = equal + block_exclusive(eq, warp_sums, &teq);
    const int take = gt || (eq && eq_before < rank);
    const int at = kept + block_exclusive(take, warp_sums, &tall);
    if (take) index[at] = i;
    kept += tall;
    equal += teq;
  }
  for (int i = threadIdx.x; i < last; i += kSelThreads) index[need + i] = cand + i;
}

constexpr int kGatherThreads = 256;

// Lane groups of one entry's vectors; an entry's K and V vectors are read together.
__global__ void __launch_bounds__(kGatherThreads) evict_gather_kernel(const EvictArgs a) {
  const int vecs = a.row_bytes / 16;
  const int64_t per_head = static_cast<int64_t>(a.keep) * vecs;
  const int64_t total = static_cast<int64_t>(a.B) * a.Hkv * per_head;
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

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t st) {
  evict_select_kernel<<<a.B * a.Hkv, kSelThreads, 0, st>>>(a);
  const int64_t total = static_cast<int64_t>(a.B) * a.Hkv * a.keep * (a.row_bytes / 16);
  const int64_t blocks = (total + kGatherThreads - 1) / kGatherThreads;
  evict_gather_kernel<<<static_cast<int>(blocks < 16 * kSms ? blocks : 16 * kSms), kGatherThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace raattn
