// What the decode kernels share: how their work is split, phi, copies into shared memory, and how a row's partial
// results are folded (decode.cu: a contiguous cache; decode_paged.cu: pages held in 4 bits).
#pragma once

#include "decode_split.cuh"

namespace raattn {
namespace decode {

constexpr int kThreads = kDecodeThreads, kWarps = kThreads / 32;
constexpr int kRows = kDecodeRows;
using Split = DecodeSplit;
constexpr float kInf = __builtin_huge_valf();

__device__ __forceinline__ float phi_fast(float d) {   // bf16 inputs: 1 ulp reciprocal, exactly 1 at d = 0
  const float q = fmaxf(16.0f - d, 0.0f) * rcp_approx(16.0f + d);
  const float q2 = q * q, q4 = q2 * q2;
  return q4 * q4;
}
__device__ __forceinline__ float phi_exact(float d) {   // fp32 inputs: IEEE division
  const bool in = !(d >= 16.0f);   // NaN stays NaN
  d = in ? d : 0.0f;   // always a plain quotient: a division's special cases are slow
  const float q = in ? (16.0f - d) / (16.0f + d) : 0.0f;
  const float q2 = q * q, q4 = q2 * q2;
  return q4 * q4;
}
template <typename T>
__device__ __forceinline__ float phi_t(float d) {
  return sizeof(T) == 2 ? phi_fast(d) : phi_exact(d);
}

// ---------------------------------------------------------------------------------------------
// the split
// ---------------------------------------------------------------------------------------------
// The sequences' entries and own blocks: cum[b] = blocks per stream of the sequences before b, for
// b <= B, and behind it their lengths; returns the most blocks of one.  All threads.
template <int KEYS>
__device__ __forceinline__ int count_blocks(int* cum, const DecodeArgs& a) {
  __shared__ int sums[kWarps], longest[kWarps];
  int* len = cum + a.B + 1;
  const int per = (a.B + kThreads - 1) / kThreads, b0 = threadIdx.x * per;
  int mine = 0, most = 0;
  for (int i = b0; i < b0 + per && i < a.B; ++i) {
    const int n = decode_own_length(a, i), blocks = (n + KEYS - 1) / KEYS;
    len[i] = n;
    mine += blocks;
    most = max(most, blocks);
  }
  most = __reduce_max_sync(0xffffffffu, most);
  if ((threadIdx.x & 31) == 0) longest[threadIdx.x >> 5] = most;
  int inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if ((threadIdx.x & 31) >= o) inc += v;
  }
  if ((threadIdx.x & 31) == 31) sums[threadIdx.x >> 5] = inc;
  __syncthreads();
  for (int w = 0; w < static_cast<int>(threadIdx.x >> 5); ++w) inc += sums[w];
  int run = inc - mine;
  for (int i = b0; i < b0 + per && i < a.B; ++i) {
    cum[i] = run;
    run += (len[i] + KEYS - 1) / KEYS;
  }
  if (b0 < a.B && b0 + per >= a.B) cum[a.B] = run;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) most = max(most, longest[w]);
  return most;
}
template <int KEYS>
__device__ __forceinline__ Split make_split(int* cum, const DecodeArgs& a, int* most_blocks) {
  *most_blocks = count_blocks<KEYS>(cum, a);
  return decode_split(a, cum[a.B], *most_blocks);
}

// A stream's part in a run.
struct Part {
  int first, count;    // blocks of the stream
  int keys;            // keys of the stream
  int slot;            // its place among a row's partial results
  int kv, b;           // key head; sequence, or -1: shared keys
  int row0, rows;      // rows: within the head's G (own) or the batch's B G (shared)
};

// The part that begins at block u of run `run`, which ends at `end`.
__device__ __forceinline__ Part get_part(int u, int run, int end, const int* cum, const Split& s, const DecodeArgs& a) {
  Part p;
  int stream0, blocks, stream;   // the stream's first block among all; its blocks
  if (u < s.own0) {
    blocks = a.pblocks;
    stream = u / blocks;
    stream0 = stream * blocks;
    p.kv = stream / a.shared_rowblocks;
    p.b = -1;
    p.keys = a.P;
    p.row0 = (stream - p.kv * a.shared_rowblocks) * kRows;
    p.rows = min(a.B * a.G - p.row0, kRows);
    p.slot = 0;
  } else {
    const int streams = a.Hkv * a.own_rowblocks, x = u - s.own0, c = x / streams;
    int lo = 0, hi = a.B - 1;   // the last b with cum[b] <= c: c lies in its blocks
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (cum[mid] <= c) lo = mid; else hi = mid - 1;
    }
    blocks = cum[lo + 1] - cum[lo];
    const int seq0 = cum[lo] * streams;
    stream = (x - seq0) / blocks;
    stream0 = s.own0 + seq0 + stream * blocks;
    p.kv = a.own_rowblocks == 1 ? stream : stream / a.own_rowblocks;
    p.b = lo;
    p.keys = cum[a.B + 1 + lo];
    p.row0 = (stream - p.kv * a.own_rowblocks) * kRows;
    p.rows = min(a.G - p.row0, kRows);
    p.slot = a.pslots;
  }
  p.first = u - stream0;
  p.count = min(blocks - p.first, end - u);
  p.slot += run - stream0 / s.per;
  return p;
}

// With a run per CTA: run `run` of the streams in order, each cut for itself; false where there is none.  All
// lanes; few streams, so few sequences: two per lane.
__device__ __forceinline__ bool get_run(int run, const int* cum, const Split& s, const DecodeArgs& a, Part& p) {
  int blocks, i;   // the stream's blocks; the run's place in it
  const int shared_runs = (a.pblocks + s.per - 1) / s.per, shared_streams = a.Hkv * a.shared_rowblocks;
  if (run < shared_runs * shared_streams) {
    const int stream = run / shared_runs;
    i = run - stream * shared_runs;
    blocks = a.pblocks;
    p.kv = stream / a.shared_rowblocks;
    p.b = -1;
    p.keys = a.P;
    p.row0 = (stream - p.kv * a.shared_rowblocks) * kRows;
    p.rows = min(a.B * a.G - p.row0, kRows);
    p.slot = i;
  } else {
    const int lane = threadIdx.x & 31, streams = a.Hkv * a.own_rowblocks;
    int at = run - shared_runs * shared_streams;
    int b = -1, n = 0, seq0 = 0;   // the sequence, its runs per stream and all before it
    for (int b0 = 0; b0 < a.B && b < 0; b0 += 32) {
      const int mine = b0 + lane < a.B ? (cum[b0 + lane + 1] - cum[b0 + lane] + s.per - 1) / s.per : 0;
      int upto = mine * streams;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
      }
      const unsigned past = __ballot_sync(0xffffffffu, seq0 + upto > at);
      const int l = past ? __ffs(past) - 1 : 31;
      n = __shfl_sync(0xffffffffu, mine, l);
      if (past) {
        b = b0 + l;
        seq0 += __shfl_sync(0xffffffffu, upto, l) - n * streams;
      } else {
        seq0 += __shfl_sync(0xffffffffu, upto, 31);
      }
    }
    if (b < 0) return false;
    at -= seq0;
    const int stream = at / n;
    i = at - stream * n;
    blocks = cum[b + 1] - cum[b];
    p.kv = stream / a.own_rowblocks;
    p.b = b;
    p.keys = cum[a.B + 1 + b];
    p.row0 = (stream - p.kv * a.own_rowblocks) * kRows;
    p.rows = min(a.G - p.row0, kRows);
    p.slot = a.pslots + i;
  }
  p.first = i * s.per;
  p.count = min(blocks - p.first, s.per);
  return true;
}

// A short prefix counts for more blocks than it has, see plan_decode: those that it has of them.
__device__ __forceinline__ void clip(Part& p, const DecodeArgs& a) {
  if (p.b < 0) p.count = max(min(p.count, (a.P + a.block - 1) / a.block - p.first), 0);
}

// f(part) for the parts of this team's run.
template <int TW, typename F>
__device__ __forceinline__ void each_part(int team, const int* cum, const Split& s, const DecodeArgs& a, F f) {
  if constexpr (TW == 1) {   // runs go to the CTAs in turn, so that few runs spread over the SMs
    const int run = team * gridDim.x + blockIdx.x, end = min((run + 1) * s.per, s.total);
    for (int u = run * s.per; u < end;) {
      Part p = get_part(u, run, end, cum, s, a);
      u += p.count;
      clip(p, a);
      f(p);
    }
  } else {
    Part p;
    if (get_run(blockIdx.x, cum, s, a, p)) {
      clip(p, a);
      f(p);
    }
  }
}

// Teams of TW warps.  Blocks of a part that this warp takes: every TW-th.
template <int TW>
__device__ __forceinline__ int warp_of_team() { return static_cast<int>(threadIdx.x >> 5) % TW; }
template <int TW>
__device__ __forceinline__ int blocks_of_warp(const Part& p) { return (p.count - warp_of_team<TW>() + TW - 1) / TW; }
template <int TW>
__device__ __forceinline__ void team_sync() {
  static_assert(TW == 1 || TW == kWarps, "a warp or the CTA");
  if (TW == 1) __syncwarp();
  else __syncthreads();
}

// Row r of a part (its last one for those past it) as an index into [B, H_q].
__device__ __forceinline__ int row_of(const Part& p, int r, const DecodeArgs& a) {
  const int x = p.row0 + min(r, p.rows - 1);
  if (p.b >= 0) return p.b * a.Hq + p.kv * a.G + x;
  const int b = x / a.G;
  return b * a.Hq + p.kv * a.G + x - b * a.G;
}
__device__ __forceinline__ float* score_row(const Part& p, int row, const DecodeArgs& a) {
  return p.b >= 0 ? a.s_own + static_cast<int64_t>(row) * a.own_width
                  : a.s_pre + static_cast<int64_t>(row) * a.pre_width;
}
// ---------------------------------------------------------------------------------------------
// asynchronous copies
// ---------------------------------------------------------------------------------------------
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool in) {   // zeros when not in
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
// The same without the choice, for keys and values: no later kernel reads them, so they are the first to leave
// L2, where the scores had better stay (B64 H32/8 D128 C2048, whole call: 111.5 us -> 99.0).  So too where several
// row blocks read them, close to one another in time: with the ordinary policy B8 H32/1 D128 C32768 takes 50.8 us
// instead of 44.8, B1 H24/1 D128 C524288 94.5 instead of 88.4, fp32 B32 H8 D64 P16384 130.5 instead of 128.5.
__device__ __forceinline__ void copy16_once(uint32_t dst, const void* src, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "l"(policy) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 u;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "r"(addr));
  return u;
}

// A row's values v[] over its slots, folded by f over N neighbouring lanes, of which this is lane t;
// x0 is neutral.  Eight loads at a time are in flight.
template <int N, typename F>
__device__ __forceinline__ float fold_slots(const float* v, int shared, int own, int pslots, int t, float x0, F f) {
  float x = x0;
  for (int i0 = t; i0 < shared + own; i0 += 8 * N) {
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = i0 + j * N;
      y[j] = i < shared + own ? __ldcg(v + (i < shared ? i : pslots + i - shared)) : x0;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) x = f(x, y[j]);
  }
#pragma unroll
  for (int o = 1; o < N; o <<= 1) x = f(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
// The maxima of a part's rows, each by 2 TW of the team's threads.
template <int TW>
__device__ __forceinline__ void part_maxima(float* rowm, const Part& p, const int* cum, const Split& s,
                                            const DecodeArgs& a) {
  const int tt = threadIdx.x % (32 * TW), r = tt / (2 * TW), row = row_of(p, r, a), b = row / a.Hq;
  int shared, own;
  decode_row_slots(b, p.kv, row - b * a.Hq - p.kv * a.G, cum[b], cum[b + 1], s, a, shared, own);
  const float m = fold_slots<2 * TW>(a.row_max + static_cast<int64_t>(row) * a.slots, shared, own, a.pslots,
                                     tt % (2 * TW), -kInf, [](float x, float y) { return fmaxf(x, y); });
  if (tt % (2 * TW) == 0) rowm[r] = m;
}

}  // namespace decode
}  // namespace raattn
