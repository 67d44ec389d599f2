// Attention of one query token per sequence against a ragged key/value cache and a prefix that
// the whole batch shares.
//
//   s_j = scale q . k_j over the shared keys and the sequence's own first length[b];
//   m = max s,  phi_j = ((16 - d) / (16 + d))^8 for d = m - s_j < 16, else exactly 0;
//   O = sum phi_j v_j / sum phi_j;  optionally weight[b, kv head, j] += sum over its query
//   heads of phi_j / sum phi, over the sequence's own keys.
//
// phi(d + c) is no multiple of phi(d), so a running maximum cannot rescale what was summed
// before it, as an exponential's can: the maximum comes first.  Three launches, each with its
// work split over the keys:
//   scores   the keys are read once per 16 query rows; unscaled scores go to the workspace in fp32 (4 bytes per
//            query head against the key's 2 D), with each part's maximum;
//   values   phi from the scores and the final maximum; the values are read, likewise;
//            partial sums (fp32) per part.  Sums need no rescaling: all parts share one maximum;
//   join     adds an output row's partial sums in a fixed order, and the weights.
// The shared keys of many rows go to the tensor cores instead (decode_prefix_tc.cu).
//
// The unit of work is a block of keys (kKeys) of one stream: a key head's own keys of one
// sequence, or its shared keys, for a block of up to 16 query rows that read them.  All blocks of
// all streams, in order, are cut into equal runs over a grid that fills every SM once, so a ragged
// batch loads all SMs alike however its lengths lie; a stream's part in a run is one partial
// result.  (Few streams are cut one by one, so that no CTA starts on a second one: fp32 B5 H12/4 C1003 P777
// 27.3 us -> 19.4, bf16 B1 H16 C512 11.5 -> 10.1.)  Every CTA counts the blocks from the lengths by
// itself: no host copy of them is needed, and a cache much larger than what it holds costs nothing.
//
// A run belongs to a team of warps: one warp where streams are many, which then needs no barrier
// beyond its lanes; the CTA's four where they are few, so that a long stream has a quarter of the
// partial results (the team's warps take a part's blocks in turn and add theirs at its end).
// bf16, whole call in a graph, with 1 / with 4: B2 H24/1 D64 C65537 76 / 24 us, B4 H8 D128 C8192 38.6 /
// 34.3; with 128 streams B16 H8 C512 16.2 / 15.2, C2048 36.5 / 36.3; B12 H8 C4096 48.7 / 50.0, B32 H8 C1024 36.1 / 37.0.
// Each warp streams its blocks through a small ring of its own in shared memory with asynchronous
// copies (which also zero the keys past a stream's end, so that nothing in a cache's unused slots
// can reach a sum).  bf16: m16n8k16 products, query
// rows as M; the chunks of a row are permuted in shared memory so that the 16-byte fragment reads
// below meet no bank conflict.  fp32: FFMA.
//
// Bound: HBM, K and V once (the row blocks of more than 16 query rows share them through L2), where there is
// much of them: B1 H32/8 D128 C131072 reads 537 MB in 92 us, 5.8
// TB/s; B64 H32/8, 2000 keys each, 524 MB in 92 us.  Latency below that: B1 H16 C512 takes 9.0 us in a
// graph, three launches of a few dependent loads each.  fp32 rows against a long prefix: the query loads, one of
// 16 bytes for four FMAs, and the keys anew for every 16 rows (B32 H8 D64 C64 P16384: 128 us, 8 TFLOP/s).
#include <climits>

#include "decode_split.cuh"

namespace raattn {
namespace {

constexpr int kThreads = kDecodeThreads, kWarps = kThreads / 32, kCtasPerSm = kDecodeCtasPerSm;
constexpr int kRows = kDecodeRows;
using Split = DecodeSplit;
constexpr float kInf = __builtin_huge_valf();

template <typename T, int D>
struct Cfg {
  static constexpr bool BF = sizeof(T) == 2;
  static constexpr int kKeys = decode_block_keys(BF, D);
  static constexpr int kChunks = D * static_cast<int>(sizeof(T)) / 16;   // of a key's or value's row
  static constexpr int kBlockBytes = kKeys * kChunks * 16;
  static constexpr int kStages = kBlockBytes >= 4096 ? 3 : 4;
  // floats of a row of scores in shared memory; bf16: no padding, the 16-byte pieces permuted (piece_of)
  static constexpr int kScoreStride = BF ? kKeys : kKeys + 4;
  static constexpr int kStageK = kBlockBytes;
  static constexpr int kStageV = kBlockBytes + kRows * kScoreStride * 4;
};

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
// b <= B, and behind it their lengths.  All threads.
template <int KEYS>
__device__ __forceinline__ Split make_split(int* cum, const DecodeArgs& a, int* most_blocks) {
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
  *most_blocks = most;
  return decode_split(a, cum[a.B], most);
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
template <typename T, int D>
__device__ __forceinline__ const char* stream_of(const Part& p, const void* own, const void* pre, const DecodeArgs& a) {
  const T* x = p.b >= 0 ? static_cast<const T*>(own) + (static_cast<int64_t>(p.b) * a.Hkv + p.kv) * a.C * D
                        : static_cast<const T*>(pre) + static_cast<int64_t>(p.kv) * a.P * D;
  return reinterpret_cast<const char*>(x);
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

// Where chunk c of row r of a block stands.  K16, V16: the bf16 fragment reads of eight lanes
// (two keys by four chunks; four keys by two chunks); F32: eight keys by one chunk.
enum Layout { K16, V16, F32 };
template <Layout LAY, int CHUNKS>
__device__ __forceinline__ int place(int r, int c) {
  if (LAY == K16) return r * CHUNKS + (c ^ ((r & 1) << 2));
  if (LAY == V16) return r * CHUNKS + (c ^ (((r >> 1) & 3) << 1));
  return r * CHUNKS + (CHUNKS >= 8 ? c ^ (r & 7) : c ^ ((r >> 1) & 3));
}

// A lane's share of the copies of a block: chunk c of rows r, r + kRowsPerCopy, ..; rows and places
// are constants from one copy to the next.
template <int KEYS, int CHUNKS, Layout LAY>
struct Fetch {
  static constexpr int kRowsPerCopy = 32 / CHUNKS, kCopies = KEYS / kRowsPerCopy;
  const char* src;   // the lane's chunk of the stream's row `lane / CHUNKS`
  int r, c;
  uint64_t policy;
  __device__ __forceinline__ Fetch(const char* stream, int lane) : r(lane / CHUNKS), c(lane % CHUNKS) {
    src = stream + lane * 16;
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  }
  // the block of keys first .. of a stream of `keys`
  __device__ __forceinline__ void operator()(uint32_t stage, int first, int keys) const {
    const char* s = src + static_cast<int64_t>(first) * (CHUNKS * 16);
    if (first + KEYS <= keys) {
#pragma unroll
      for (int i = 0; i < kCopies; ++i)
        copy16_once(stage + place<LAY, CHUNKS>(r + i * kRowsPerCopy, c) * 16, s + i * 512, policy);
    } else {
      const int left = keys - first - r;
#pragma unroll
      for (int i = 0; i < kCopies; ++i) {
        const bool in = i * kRowsPerCopy < left;
        copy16(stage + place<LAY, CHUNKS>(r + i * kRowsPerCopy, c) * 16, in ? s + i * 512 : src - r * (CHUNKS * 16), in);
      }
    }
  }
};

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 u;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "r"(addr));
  return u;
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// ---------------------------------------------------------------------------------------------
// scores
// ---------------------------------------------------------------------------------------------
// bf16.  Lane (g, t) = (lane / 4, lane % 4) reads, of key g of a block of eight, the chunks t,
// t + 4, .. of its row: words 0, 1 of chunk 4 c + t are the B operand of product 2 c, words 2, 3 of
// product 2 c + 1, and the query's chunks give the A operand in the same order (any order of the
// D products of a score is the score).
template <int D, int TW>
__device__ __forceinline__ void part_scores(const Part& p, const DecodeArgs& a, uint32_t ring, float* best_s,
                                            __nv_bfloat16*) {
  using C = Cfg<__nv_bfloat16, D>;
  constexpr int NV = D / 32;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int mine = blocks_of_warp<TW>(p), first = (p.first + warp_of_team<TW>()) * C::kKeys;
  constexpr int kStep = TW * C::kKeys;
  const char* keys = stream_of<__nv_bfloat16, D>(p, a.k, a.pk, a);
  const Fetch<C::kKeys, C::kChunks, K16> fetch(keys, lane);
#pragma unroll
  for (int i = 0; i < C::kStages - 1; ++i) {
    if (i < mine) fetch(ring + i * C::kStageK, first + i * kStep, p.keys);
    copy_commit();
  }
  uint4 q0[NV], q1[NV];
  const int r0 = row_of(p, g, a), r1 = row_of(p, g + 8, a);
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q);
#pragma unroll
  for (int c = 0; c < NV; ++c) {
    q0[c] = *reinterpret_cast<const uint4*>(q + static_cast<int64_t>(r0) * D + c * 32 + t * 8);
    q1[c] = *reinterpret_cast<const uint4*>(q + static_cast<int64_t>(r1) * D + c * 32 + t * 8);
  }
  float* s0 = score_row(p, r0, a);
  float* s1 = score_row(p, r1, a);
  const bool w0 = g < p.rows, w1 = g + 8 < p.rows;
  float m0 = -kInf, m1 = -kInf;
  for (int i = 0; i < mine; ++i) {
    copy_wait<C::kStages - 2>();
    __syncwarp();   // block i has landed for all lanes, and all have read block i - 1
    const int ahead = i + C::kStages - 1;
    if (ahead < mine) fetch(ring + ahead % C::kStages * C::kStageK, first + ahead * kStep, p.keys);
    copy_commit();
    const uint32_t stage = ring + i % C::kStages * C::kStageK;
#pragma unroll
    for (int nb = 0; nb < C::kKeys / 8; ++nb) {
      float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int c = 0; c < NV; ++c) {
        const uint4 x = lds128(stage + place<K16, C::kChunks>(nb * 8 + g, c * 4 + t) * 16);
        mma_bf16(s, q0[c].x, q1[c].x, q0[c].y, q1[c].y, x.x, x.y);
        mma_bf16(s, q0[c].z, q1[c].z, q0[c].w, q1[c].w, x.z, x.w);
      }
      const int key = first + i * kStep + nb * 8 + 2 * t;
#pragma unroll
      for (int e = 0; e < 4; ++e) s[e] = key + (e & 1) < p.keys ? s[e] : -kInf;
      m0 = fmaxf(m0, fmaxf(s[0], s[1]));
      m1 = fmaxf(m1, fmaxf(s[2], s[3]));
      if (w0) *reinterpret_cast<float2*>(s0 + key) = make_float2(s[0], s[1]);
      if (w1) *reinterpret_cast<float2*>(s1 + key) = make_float2(s[2], s[3]);
    }
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, o));
    m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, o));
  }
  if (t == 0) {
    best_s[(threadIdx.x >> 5) * kRows + g] = m0;
    best_s[(threadIdx.x >> 5) * kRows + g + 8] = m1;
  }
}

// fp32: 32 / kKeys lanes per key.
template <int D, int TW>
__device__ __forceinline__ void part_scores(const Part& p, const DecodeArgs& a, uint32_t ring, float* best_s, float*) {
  using C = Cfg<float, D>;
  constexpr int PARTS = 32 / C::kKeys;
  const int lane = threadIdx.x & 31, kk = lane / PARTS, part = lane % PARTS;
  const int mine = blocks_of_warp<TW>(p), first = (p.first + warp_of_team<TW>()) * C::kKeys;
  constexpr int kStep = TW * C::kKeys;
  const char* keys = stream_of<float, D>(p, a.k, a.pk, a);
  const Fetch<C::kKeys, C::kChunks, F32> fetch(keys, lane);
#pragma unroll 1
  for (int i = 0; i < C::kStages - 1; ++i) {
    if (i < mine) fetch(ring + i * C::kStageK, first + i * kStep, p.keys);
    copy_commit();
  }
  // Rows four at a time (independent chains) in a loop that is not unrolled: a part is short, and
  // fetching the code of all sixteen would cost more than running it.  best_s holds this warp's
  // maxima.
  float* best = best_s + (threadIdx.x >> 5) * kRows;
  if (lane < kRows) best[lane] = -kInf;
  const int row_lane = row_of(p, lane, a);   // of lane's row
  const float* q0 = static_cast<const float*>(a.q) + part * 4;
  for (int x = lane; x < p.rows * C::kChunks; x += 32)   // the queries, which every block reads, into L1
    asm volatile("prefetch.global.L1 [%0];" ::"l"(static_cast<const float*>(a.q) +
                                                  static_cast<int64_t>(row_of(p, x / C::kChunks, a)) * D +
                                                  x % C::kChunks * 4));
  __syncwarp();
  for (int i = 0; i < mine; ++i) {
    copy_wait<C::kStages - 2>();
    __syncwarp();
    const int ahead = i + C::kStages - 1;
    if (ahead < mine) fetch(ring + ahead % C::kStages * C::kStageK, first + ahead * kStep, p.keys);
    copy_commit();
    const uint32_t stage = ring + i % C::kStages * C::kStageK;
    float4 kx[C::kChunks / PARTS];
#pragma unroll
    for (int c = 0; c < C::kChunks / PARTS; ++c) {
      const uint4 u = lds128(stage + place<F32, C::kChunks>(kk, c * PARTS + part) * 16);
      kx[c] = make_float4(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w));
    }
    const int key = first + i * kStep + kk;
#pragma unroll 1
    for (int r0 = 0; r0 < p.rows; r0 += 4) {
      float s[4];
      int row[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        row[j] = __shfl_sync(0xffffffffu, row_lane, r0 + j);
        const float4* q = reinterpret_cast<const float4*>(q0 + static_cast<int64_t>(row[j]) * D);
        float u = 0.0f, v = 0.0f;
#pragma unroll
        for (int c = 0; c < C::kChunks / PARTS; ++c) {
          const float4 y = __ldg(q + c * PARTS);
          u = fmaf(y.x, kx[c].x, fmaf(y.y, kx[c].y, u));
          v = fmaf(y.z, kx[c].z, fmaf(y.w, kx[c].w, v));
        }
        s[j] = u + v;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
#pragma unroll
        for (int o = 1; o < PARTS; o <<= 1) s[j] += __shfl_xor_sync(0xffffffffu, s[j], o);
        s[j] = key < p.keys ? s[j] : -kInf;
        if (part == 0 && r0 + j < p.rows) score_row(p, row[j], a)[key] = s[j];
#pragma unroll
        for (int o = 16; o >= PARTS; o >>= 1) s[j] = fmaxf(s[j], __shfl_xor_sync(0xffffffffu, s[j], o));
      }
      if (lane < 4) best[r0 + lane] = fmaxf(best[r0 + lane], lane == 0 ? s[0] : lane == 1 ? s[1] : lane == 2 ? s[2] : s[3]);
    }
  }
}

template <typename T, int D, int TW>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) decode_scores_kernel(const DecodeArgs a) {
  extern __shared__ uint4 dyn[];
  constexpr int kRing = Cfg<T, D>::kStages * Cfg<T, D>::kStageK;
  int* cum = reinterpret_cast<int*>(reinterpret_cast<char*>(dyn) + kWarps * kRing);
  __shared__ float best[kWarps * kRows];
  const int warp = threadIdx.x >> 5, team = warp / TW, tt = threadIdx.x % (32 * TW);
  release_dependents();   // the next kernel's first values are on their way while this one ends
  int longest;
  const Split s = make_split<Cfg<T, D>::kKeys>(cum, a, &longest);
  if (blockIdx.x == 0) {   // for the kernels that look up a row's slots
    for (int b = threadIdx.x; b <= a.B; b += kThreads) a.cum[b] = cum[b];
    if (threadIdx.x == 0) a.cum[a.B + 1] = longest;
  }
  each_part<TW>(team, cum, s, a, [&](const Part& p) {
    part_scores<D, TW>(p, a, smem_u32(dyn) + warp * kRing, best, static_cast<T*>(nullptr));
    team_sync<TW>();
    if (tt < p.rows) {
      float m = best[team * TW * kRows + tt];
#pragma unroll
      for (int w = 1; w < TW; ++w) m = fmaxf(m, best[(team * TW + w) * kRows + tt]);
      a.row_max[static_cast<int64_t>(row_of(p, tt, a)) * a.slots + p.slot] = m;
    }
    team_sync<TW>();   // the maxima are read, and the rings are free
  });
  // The tensor cores' part, if any: whoever awaits this kernel awaits that too.  One CTA sees to it; the
  // others make room for the next ones.
  if (blockIdx.x == gridDim.x - 1) await_previous();
}

// ---------------------------------------------------------------------------------------------
// values
// ---------------------------------------------------------------------------------------------
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

// Where piece c (four keys) of row r's scores stands: in bf16 so that the reads of sixteen lanes (four
// rows, eight keys) meet no bank conflict.
template <bool BF>
__device__ __forceinline__ int piece_of(int r, int c) { return BF ? c ^ (r & 2) : c; }

// Blocks of values and their scores into a stage.
template <typename T, int D, int TW, Layout LAY>
struct FetchValues {
  using C = Cfg<T, D>;
  static constexpr int kPieces = C::kKeys / 4;                              // 16-byte pieces of a row of scores
  static constexpr int kLoads = (kRows * kPieces + 31) / 32, kRowsPerLoad = 32 / kPieces;
  Fetch<C::kKeys, C::kChunks, LAY> values;
  const float* src[kLoads];
  int r, keys, first;
  uint32_t at;
  __device__ __forceinline__ FetchValues(const char* vals, const Part& p, const DecodeArgs& a, int lane)
      : values(vals, lane), r(lane / kPieces), keys(p.keys), first((p.first + warp_of_team<TW>()) * C::kKeys) {
    const int c = lane % kPieces;
    at = C::kBlockBytes + (r * C::kScoreStride + piece_of<C::BF>(r, c) * 4) * 4;   // rows kRowsPerLoad apart: alike
#pragma unroll
    for (int j = 0; j < kLoads; ++j) src[j] = score_row(p, row_of(p, r + j * kRowsPerLoad, a), a) + c * 4;
  }
  __device__ __forceinline__ void block(uint32_t stage, int i) const { values(stage, first + i * (TW * C::kKeys), keys); }
  __device__ __forceinline__ void scores(uint32_t stage, int i, int rows) const {
    const int k = first + i * (TW * C::kKeys);
#pragma unroll
    for (int j = 0; j < kLoads; ++j)
      if (r + j * kRowsPerLoad < rows) copy16(stage + at + j * kRowsPerLoad * C::kScoreStride * 4, src[j] + k, true);
  }
  __device__ __forceinline__ void operator()(uint32_t stage, int i, int rows) const {
    block(stage, i);
    scores(stage, i, rows);
  }
  // The first blocks of a part; their values do not wait for the scores (B32 H32/8 C1024 34.3 us -> 33.4, B2 H24/1
  // C65537 19.2 -> 17.6, with the early start of the kernel).
  __device__ __forceinline__ void start(uint32_t ring, int blocks, int rows, bool wait) const {
#pragma unroll
    for (int i = 0; i < C::kStages - 1; ++i)
      if (i < blocks) block(ring + i * C::kStageV, i);
    if (wait) await_previous();
#pragma unroll
    for (int i = 0; i < C::kStages - 1; ++i) {
      if (i < blocks) scores(ring + i * C::kStageV, i, rows);
      copy_commit();   // the first group has all values
    }
  }
};

// bf16.  Lane (g, t) reads, of keys 2 t, 2 t + 1, 2 t + 8 and 2 t + 9 of sixteen, the dimensions
// 8 g .. 8 g + 7 of every 64: words of two keys, interleaved, are the B operand of the product
// whose column g stands for dimension 8 g + j.  phi of the scores at the same keys is the A operand.
// TWO: the part has more than eight query rows, so the weights' second halves take a product of their
// own; otherwise they stand in the upper eight rows of the same one.
template <int D, int TW, bool TWO>
__device__ __forceinline__ void bf16_values(const Part& p, const DecodeArgs& a, const Split& s, const int* cum,
                                            uint32_t ring, char* ring_ptr, float* rowm, float* sums, __nv_bfloat16*) {
  using C = Cfg<__nv_bfloat16, D>;
  constexpr int NC = D / 64;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int mine = blocks_of_warp<TW>(p);
  const char* vals = stream_of<__nv_bfloat16, D>(p, a.v, a.pv, a);
  const FetchValues<__nv_bfloat16, D, TW, V16> fetch(vals, p, a, lane);
  fetch.start(ring, mine, p.rows, !a.tc);
  part_maxima<TW>(rowm, p, cum, s, a);
  team_sync<TW>();
  const bool w0 = g < p.rows, w1 = TWO && g + 8 < p.rows;
  const float m0 = rowm[g], m1 = rowm[g + 8];
  float acc[NC][8][4];
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[c][j][0] = acc[c][j][1] = acc[c][j][2] = acc[c][j][3] = 0.0f;
  float t0 = 0.0f, t1 = 0.0f;
  for (int i = 0; i < mine; ++i) {
    copy_wait<C::kStages - 2>();
    __syncwarp();
    const int ahead = i + C::kStages - 1;
    if (ahead < mine) fetch(ring + ahead % C::kStages * C::kStageV, ahead, p.rows);
    copy_commit();
    const uint32_t stage = ring + i % C::kStages * C::kStageV;
    const float* sc = reinterpret_cast<const float*>(ring_ptr + i % C::kStages * C::kStageV + C::kBlockBytes);
    uint32_t w[4] = {0u, 0u, 0u, 0u}, rest[4] = {0u, 0u, 0u, 0u};
    bool live = false;   // some weight that is not 0 (a NaN is not)
    const int at = 2 * t, flip = (g & 2) << 2;   // piece_of: pieces 2 e + t / 2, flipped by two in rows 2, 3, 6, 7
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      // V is bf16, so phi goes into the product as two bf16: one alone would cost as much as the
      // rounding of the output.  Scores past the last key are -inf.
      if (w0) {
        const float2 x = *reinterpret_cast<const float2*>(sc + g * C::kScoreStride + at + ((e * 8) ^ flip));
        const float f0 = phi_fast((m0 - x.x) * a.scale), f1 = phi_fast((m0 - x.y) * a.scale);
        t0 += f0 + f1;
        live |= f0 + f1 != 0.0f;
        split_bf16x2(f0, f1, w[2 * e], rest[2 * e]);
      }
      if (w1) {
        const float2 x = *reinterpret_cast<const float2*>(sc + (g + 8) * C::kScoreStride + at + ((e * 8) ^ flip));
        const float f0 = phi_fast((m1 - x.x) * a.scale), f1 = phi_fast((m1 - x.y) * a.scale);
        t1 += f0 + f1;
        live |= f0 + f1 != 0.0f;
        split_bf16x2(f0, f1, w[2 * e + 1], rest[2 * e + 1]);
      }
    }
    if (!__any_sync(0xffffffffu, live)) continue;   // every weight is exactly 0
    if constexpr (!TWO) {
      w[1] = rest[0];
      w[3] = rest[2];
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      uint4 v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        v[e] = lds128(stage + place<V16, C::kChunks>((e >> 1) * 8 + 2 * t + (e & 1), c * 8 + g) * 16);
      const uint32_t x0[4] = {v[0].x, v[0].y, v[0].z, v[0].w}, x1[4] = {v[1].x, v[1].y, v[1].z, v[1].w};
      const uint32_t x2[4] = {v[2].x, v[2].y, v[2].z, v[2].w}, x3[4] = {v[3].x, v[3].y, v[3].z, v[3].w};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t sel = j & 1 ? 0x7632u : 0x5410u;
        const uint32_t b0 = __byte_perm(x0[j >> 1], x1[j >> 1], sel), b1 = __byte_perm(x2[j >> 1], x3[j >> 1], sel);
        mma_bf16(acc[c][j], w[0], w[1], w[2], w[3], b0, b1);
        if constexpr (TWO) mma_bf16(acc[c][j], rest[0], rest[1], rest[2], rest[3], b0, b1);
      }
    }
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    t0 += __shfl_xor_sync(0xffffffffu, t0, o);
    t1 += __shfl_xor_sync(0xffffffffu, t1, o);
  }
  if (t == 0) {
    sums[(threadIdx.x >> 5) * kRows + g] = t0;
    sums[(threadIdx.x >> 5) * kRows + g + 8] = t1;
  }
  // Into this warp's ring (its blocks have been read).  Accumulator columns 2 t, 2 t + 1 stand for
  // dimensions 16 t + j and 16 t + 8 + j.
  __syncwarp();
  float* out = reinterpret_cast<float*>(ring_ptr);
  if constexpr (!TWO) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        acc[c][j][0] += acc[c][j][2];
        acc[c][j][1] += acc[c][j][3];
      }
  }
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int j = 0; j < 8; j += 4)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < 2 ? w0 : w1)
          *reinterpret_cast<float4*>(out + (g + (e >> 1) * 8) * D + c * 64 + t * 16 + (e & 1) * 8 + j) =
              make_float4(acc[c][j][e], acc[c][j + 1][e], acc[c][j + 2][e], acc[c][j + 3][e]);
}

template <int D, int TW>
__device__ __forceinline__ void part_values(const Part& p, const DecodeArgs& a, const Split& s, const int* cum,
                                            uint32_t ring, char* ring_ptr, float* rowm, float* sums, __nv_bfloat16* t) {
  if (p.rows > 8)
    bf16_values<D, TW, true>(p, a, s, cum, ring, ring_ptr, rowm, sums, t);
  else
    bf16_values<D, TW, false>(p, a, s, cum, ring, ring_ptr, rowm, sums, t);
}

// fp32: D / 4 lanes across the dimensions, the other lanes over the keys; phi replaces the scores in
// shared memory.
template <int D, int TW>
__device__ __forceinline__ void part_values(const Part& p, const DecodeArgs& a, const Split& s, const int* cum,
                                            uint32_t ring, char* ring_ptr, float* rowm, float* sums, float*) {
  using C = Cfg<float, D>;
  constexpr int L = D / 4, KS = 32 / L;
  const int lane = threadIdx.x & 31, gl = lane % L, ks = lane / L;
  const int mine = blocks_of_warp<TW>(p);
  const char* vals = stream_of<float, D>(p, a.v, a.pv, a);
  const FetchValues<float, D, TW, F32> fetch(vals, p, a, lane);
  fetch.start(ring, mine, p.rows, !a.tc);
  // four lanes per row for phi: lane (g, t) takes rows g and g + 8, keys t, t + 4, ..
  const int g = lane >> 2, t = lane & 3;
  const bool w0 = g < p.rows, w1 = g + 8 < p.rows;
  part_maxima<TW>(rowm, p, cum, s, a);
  team_sync<TW>();
  const float m0 = rowm[g], m1 = rowm[g + 8];
  float acc[kRows][4];
#pragma unroll
  for (int r = 0; r < kRows; ++r) acc[r][0] = acc[r][1] = acc[r][2] = acc[r][3] = 0.0f;
  float t0 = 0.0f, t1 = 0.0f;
  for (int i = 0; i < mine; ++i) {
    copy_wait<C::kStages - 2>();
    __syncwarp();
    const int ahead = i + C::kStages - 1;
    if (ahead < mine) fetch(ring + ahead % C::kStages * C::kStageV, ahead, p.rows);
    copy_commit();
    const uint32_t stage = ring + i % C::kStages * C::kStageV;
    float* sc = reinterpret_cast<float*>(ring_ptr + i % C::kStages * C::kStageV + C::kBlockBytes);
#pragma unroll 2
    for (int k = 0; k < C::kKeys; k += 4) {
      if (w0) {
        float& x = sc[g * C::kScoreStride + k + t];
        x = phi_exact((m0 - x) * a.scale);
        t0 += x;
      }
      if (w1) {
        float& x = sc[(g + 8) * C::kScoreStride + k + t];
        x = phi_exact((m1 - x) * a.scale);
        t1 += x;
      }
    }
    __syncwarp();
#pragma unroll 2
    for (int kk = ks; kk < C::kKeys; kk += KS) {
      const uint4 u = lds128(stage + place<F32, C::kChunks>(kk, gl) * 16);
      const float4 v = make_float4(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z),
                                   __uint_as_float(u.w));
#pragma unroll
      for (int r0 = 0; r0 < kRows; r0 += 4) {
        if (r0 < p.rows) {
#pragma unroll
          for (int r = r0; r < r0 + 4; ++r) {   // rows past the last add what is never written out
            const float f = sc[r * C::kScoreStride + kk];
            acc[r][0] = fmaf(f, v.x, acc[r][0]);
            acc[r][1] = fmaf(f, v.y, acc[r][1]);
            acc[r][2] = fmaf(f, v.z, acc[r][2]);
            acc[r][3] = fmaf(f, v.w, acc[r][3]);
          }
        }
      }
    }
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    t0 += __shfl_xor_sync(0xffffffffu, t0, o);
    t1 += __shfl_xor_sync(0xffffffffu, t1, o);
  }
  if (t == 0) {
    sums[(threadIdx.x >> 5) * kRows + g] = t0;
    sums[(threadIdx.x >> 5) * kRows + g + 8] = t1;
  }
  __syncwarp();
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    if (r < p.rows) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int o = L; o < 32; o <<= 1) acc[r][e] += __shfl_xor_sync(0xffffffffu, acc[r][e], o);
      if (ks == 0)
        reinterpret_cast<float4*>(ring_ptr)[r * L + gl] = make_float4(acc[r][0], acc[r][1], acc[r][2], acc[r][3]);
    }
  }
}

template <typename T, int D, int TW>
__global__ void __launch_bounds__(kThreads, 4) decode_values_kernel(const DecodeArgs a) {
  extern __shared__ uint4 dyn[];
  constexpr int kRing = Cfg<T, D>::kStages * Cfg<T, D>::kStageV;
  static_assert(kRing >= kRows * D * 4, "a warp's partial sums fit its ring");
  int* cum = reinterpret_cast<int*>(reinterpret_cast<char*>(dyn) + kWarps * kRing);
  __shared__ float rowm_s[kWarps / TW * kRows], sums[kWarps * kRows];
  const int warp = threadIdx.x >> 5, team = warp / TW, tt = threadIdx.x % (32 * TW);
  char* ring = reinterpret_cast<char*>(dyn) + warp * kRing;
  const char* rings = reinterpret_cast<const char*>(dyn) + team * TW * kRing;   // the team's
  int longest;
  const Split s = make_split<Cfg<T, D>::kKeys>(cum, a, &longest);
  // The scores are awaited behind the first values' copies, unless, with the tensor cores, the kernel before the
  // previous one has written them, which all of the previous one had awaited when this one could start.
  each_part<TW>(team, cum, s, a, [&](const Part& p) {
    part_values<D, TW>(p, a, s, cum, smem_u32(ring), ring, rowm_s + team * kRows, sums, static_cast<T*>(nullptr));
    team_sync<TW>();
    if (tt < p.rows) {
      float f = sums[team * TW * kRows + tt];
#pragma unroll
      for (int w = 1; w < TW; ++w) f += sums[(team * TW + w) * kRows + tt];
      a.part_sum[static_cast<int64_t>(row_of(p, tt, a)) * a.slots + p.slot] = f;
    }
    for (int e = tt; e < p.rows * (D / 4); e += 32 * TW) {
      const int r = e / (D / 4), c = e % (D / 4);
      float4 f = reinterpret_cast<const float4*>(rings)[e];
#pragma unroll
      for (int w = 1; w < TW; ++w) {
        const float4 x = *reinterpret_cast<const float4*>(rings + w * kRing + e * 16);
        f.x += x.x;
        f.y += x.y;
        f.z += x.z;
        f.w += x.w;
      }
      reinterpret_cast<float4*>(a.part_o + (static_cast<int64_t>(row_of(p, r, a)) * a.slots + p.slot) * D)[c] = f;
    }
    team_sync<TW>();
  });
  release_dependents();
  // Whoever awaits this kernel awaits the tensor cores' part too: see the scores kernel.
  if (blockIdx.x == gridDim.x - 1) await_previous();
}

// ---------------------------------------------------------------------------------------------
// join
// ---------------------------------------------------------------------------------------------
constexpr int kWeightKeys = 4 * kThreads;   // keys a weight CTA takes at a time, four consecutive ones per thread
constexpr int kWeightRows = 8;              // rows whose scores a thread has in flight

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) decode_join_kernel(const DecodeArgs a, int row_warps, int weight_keys) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row_ctas = (a.B * a.Hq * row_warps + kWarps - 1) / kWarps;
  await_previous();
  const Split sp = decode_split(a, a.cum[a.B], a.cum[a.B + 1]);   // the counts that the scores kernel left
  if (static_cast<int>(blockIdx.x) < row_ctas) {   // one output row per warp, or per CTA
    constexpr int L = D / 4, KS = 32 / L;
    const bool whole = row_warps > 1;
    const int row = whole ? blockIdx.x : blockIdx.x * kWarps + warp;
    if (row >= a.B * a.Hq) return;
    const int b = row / a.Hq, kv = (row - b * a.Hq) / a.G;
    int shared, own;
    decode_row_slots(b, kv, row - b * a.Hq - kv * a.G, a.cum[b], a.cum[b + 1], sp, a, shared, own);
    const int gl = lane % L, ks = lane / L, step = KS * row_warps;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float total = 0.0f;
    for (int i0 = whole ? warp * KS + ks : ks; i0 < shared + own; i0 += 8 * step) {   // eight parts at a time in flight
      float f[8];
      float4 x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int i = i0 + j * step;
        const int64_t at = static_cast<int64_t>(row) * a.slots + (i < shared ? i : a.pslots + i - shared);
        const bool in = i < shared + own;
        f[j] = in ? __ldcg(a.part_sum + at) : 0.0f;
        x[j] = in ? __ldcg(reinterpret_cast<const float4*>(a.part_o + at * D) + gl) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (f[j] != 0.0f) {   // a part whose weights are all 0 may have written no output
          s.x += x[j].x;
          s.y += x[j].y;
          s.z += x[j].z;
          s.w += x[j].w;
          total += f[j];
        }
    }
#pragma unroll
    for (int o = L; o < 32; o <<= 1) {
      s.x += __shfl_xor_sync(0xffffffffu, s.x, o);
      s.y += __shfl_xor_sync(0xffffffffu, s.y, o);
      s.z += __shfl_xor_sync(0xffffffffu, s.z, o);
      s.w += __shfl_xor_sync(0xffffffffu, s.w, o);
      total += __shfl_xor_sync(0xffffffffu, total, o);
    }
    if (whole) {
      __shared__ float4 sums[kWarps][L];
      __shared__ float totals[kWarps];
      if (ks == 0) sums[warp][gl] = s;
      if (lane == 0) totals[warp] = total;
      __syncthreads();
      if (warp) return;
#pragma unroll
      for (int w = 1; w < kWarps; ++w) {
        const float4 x = sums[w][gl];
        s.x += x.x;
        s.y += x.y;
        s.z += x.z;
        s.w += x.w;
        total += totals[w];
      }
    }
    if (ks == 0) {
      const float inv = total != 0.0f ? 1.0f / total : 0.0f;   // no key at all: zeros
      T* o = static_cast<T*>(a.o) + static_cast<int64_t>(row) * D + gl * 4;
      if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(s.x * inv, s.y * inv), pack_bf16x2(s.z * inv, s.w * inv));
      } else {
        *reinterpret_cast<float4*>(o) = make_float4(s.x * inv, s.y * inv, s.z * inv, s.w * inv);
      }
    }
    return;
  }
  // the weights of weight_keys keys of one (sequence, key head)
  extern __shared__ float2 stat[];   // [G] maximum, 1 / sum
  const int splits = (a.C + weight_keys - 1) / weight_keys;
  const int item = blockIdx.x - row_ctas, bk = item / splits, b = bk / a.Hkv, kv = bk - b * a.Hkv;
  const int split0 = (item - bk * splits) * weight_keys, last = min(split0 + weight_keys, decode_own_length(a, b));
  if (split0 >= last) return;
  int first = split0 + threadIdx.x * 4;
  // the scores of the first rows and the weights are on their way while the statistics are gathered
  const float* sc = a.s_own + (static_cast<int64_t>(b) * a.Hq + kv * a.G) * a.own_width;
  float* w = a.weight + static_cast<int64_t>(bk) * a.C;
  float4 s[kWeightRows];
  auto load = [&](int g0) {   // a row of scores is padded to whole blocks
#pragma unroll
    for (int j = 0; j < kWeightRows; ++j)
      if (first < last && g0 + j < a.G)
        s[j] = __ldcg(reinterpret_cast<const float4*>(sc + static_cast<int64_t>(g0 + j) * a.own_width + first));
  };
  float old[4];
  auto load_old = [&]() {
#pragma unroll
    for (int i = 0; i < 4; ++i) old[i] = first + i < last ? w[first + i] : 0.0f;
  };
  load(0);
  load_old();
  // lanes per row: four, each with four of its parts in flight; more where parts are many and rows few
  const int lanes = a.slots <= 64 || a.G > 16 ? 4 : a.G > 8 ? 8 : a.G > 4 ? 16 : 32, t = threadIdx.x & (lanes - 1);
  for (int g0 = 0; g0 < a.G; g0 += kThreads / lanes) {
    const int g = g0 + threadIdx.x / lanes, gg = min(g, a.G - 1);
    int shared, own;
    decode_row_slots(b, kv, gg, a.cum[b], a.cum[b + 1], sp, a, shared, own);
    const int64_t at = (static_cast<int64_t>(b) * a.Hq + kv * a.G + gg) * a.slots;
    float m = -kInf, total = 0.0f;
    for (int i0 = t; i0 < shared + own; i0 += 4 * lanes) {
      float y[4], z[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = i0 + lanes * j;
        const bool in = i < shared + own;
        const int64_t slot = at + (i < shared ? i : a.pslots + i - shared);
        y[j] = in ? __ldcg(a.row_max + slot) : -kInf;
        z[j] = in ? __ldcg(a.part_sum + slot) : 0.0f;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        m = fmaxf(m, y[j]);
        total += z[j];
      }
    }
    for (int o = 1; o < lanes; o <<= 1) {
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      total += __shfl_xor_sync(0xffffffffu, total, o);
    }
    if (t == 0 && g < a.G) stat[g] = make_float2(m, 1.0f / total);
  }
  __syncthreads();
  while (first < last) {
    float add[4] = {};   // this call's weights first, then one addition to the running total
    for (int g0 = 0; g0 < a.G; g0 += kWeightRows) {
      if (g0) load(g0);
#pragma unroll
      for (int j = 0; j < kWeightRows; ++j) {
        if (g0 + j < a.G) {
          const float2 ms = stat[g0 + j];
          add[0] = fmaf(phi_t<T>((ms.x - s[j].x) * a.scale), ms.y, add[0]);
          add[1] = fmaf(phi_t<T>((ms.x - s[j].y) * a.scale), ms.y, add[1]);
          add[2] = fmaf(phi_t<T>((ms.x - s[j].z) * a.scale), ms.y, add[2]);
          add[3] = fmaf(phi_t<T>((ms.x - s[j].w) * a.scale), ms.y, add[3]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (first + i < last) w[first + i] = old[i] + add[i];
    first += kWeightKeys;
    load(0);
    load_old();
  }
}

template <typename T, int D, int TW>
cudaError_t go(const DecodeArgs& a, const PrefixMaps& maps, const LaunchCtx& ctx, cudaStream_t st) {
  using C = Cfg<T, D>;
  const int cum = (2 * a.B + 1) * 4;
  const int smem_scores = kWarps * C::kStages * C::kStageK + cum;
  const int smem_values = kWarps * C::kStages * C::kStageV + cum;
  // The most shared memory of an SM's carve-out also for kernels that would do with less: an SM changes
  // it only when it is empty, and the next kernel's CTAs, launched as dependents, come before that.
  constexpr int kMostCum = (2 * kDecodeMaxBatch + 1) * 4;
  cudaError_t e = set_up_kernel<decode_scores_kernel<T, D, TW>>(kWarps * C::kStages * C::kStageK + kMostCum, true);
  if (e == cudaSuccess)
    e = set_up_kernel<decode_values_kernel<T, D, TW>>(kWarps * C::kStages * C::kStageV + kMostCum, true);
  if (e == cudaSuccess) e = set_up_kernel<decode_join_kernel<T, D>>(0, true);
  if (e != cudaSuccess) return e;
  // CTAs for the runs that there can be
  const int64_t shared_streams = static_cast<int64_t>(a.Hkv) * a.shared_rowblocks,
                own_streams = static_cast<int64_t>(a.B) * a.Hkv * a.own_rowblocks, own = a.own_width / a.block;
  auto runs_of = [&](int64_t blocks) { return (blocks + TW - 1) / TW; };
  const int64_t ctas = TW == 1 ? runs_of(shared_streams * a.pblocks + own_streams * own)   // few runs: a CTA each
                               : shared_streams * runs_of(a.pblocks) + own_streams * runs_of(own);
  const int grid = static_cast<int>(ctas < kDecodeCtas ? ctas : kDecodeCtas);
  if (a.tc && (e = launch_decode_prefix(maps, a, false, ctx, st)) != cudaSuccess) return e;
  if (a.tc) {
    e = launch_dependent(decode_scores_kernel<T, D, TW>, grid, kThreads, smem_scores, st, a);
    if (e != cudaSuccess) return e;
  } else {
    decode_scores_kernel<T, D, TW><<<grid, kThreads, smem_scores, st>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;   // the next kernels read what this one leaves
  }
  if (a.tc && (e = launch_decode_prefix(maps, a, true, ctx, st)) != cudaSuccess) return e;
  e = launch_dependent(decode_values_kernel<T, D, TW>, grid, kThreads, smem_values, st, a);
  if (e != cudaSuccess) return e;
  // Few CTAs: a weight CTA takes as many keys, up to 4096, as leave about six per SM (starting the
  // 6144 CTAs of one row or 512 keys each took most of 15 us at B64 H32/8 C4096).
  // A CTA per row where rows are few and their partial results many.
  const int64_t rows = static_cast<int64_t>(a.B) * a.Hq;
  const int row_warps = rows <= 2 * kSms && a.slots > 8 * (128 / D) ? kWarps : 1;
  int64_t join = (rows * row_warps + kWarps - 1) / kWarps;
  int weight_keys = kWeightKeys;
  if (a.weight) {
    const int64_t streams = static_cast<int64_t>(a.B) * a.Hkv;
    while (weight_keys < 8 * kWeightKeys && streams * ((a.C + weight_keys - 1) / weight_keys) > 6 * kSms) weight_keys *= 2;
    join += streams * ((a.C + weight_keys - 1) / weight_keys);
  }
  return launch_dependent(decode_join_kernel<T, D>, static_cast<unsigned>(join), kThreads, a.weight ? a.G * 8 : 0, st, a,
                          row_warps, weight_keys);
}
template <typename T, int D>
cudaError_t go(const DecodeArgs& a, const PrefixMaps& maps, const LaunchCtx& ctx, cudaStream_t st) {
  return a.team == kWarps ? go<T, D, kWarps>(a, maps, ctx, st) : go<T, D, 1>(a, maps, ctx, st);
}

}  // namespace

// The split of the keys.  Shared keys of more than kTcRows rows per key head, and of more than two blocks (16
// keys by 16 rows) for every warp of the grid, go to the tensor cores, in whole tiles of 128, split so
// that one wave of CTAs takes them.  That costs two more launches, which few blocks do not pay back:
// bf16 D128 with them / without, B64 H32/8 P128 31.3 us / 24.8, P1024 35.0 / 38.0, B32 H32/8 P128 24.8 / 18.5,
// P2048 32.6 / 31.5, B128 H32/8 P256 31.5 / 28.1, P512 34.0 / 37.4.  Everything else is cut into runs:
// equal ones, one per warp, with many streams; one per CTA, each stream for itself, with fewer than 64, or
// up to 128 where a warp's equal run would be short.  `full`, the blocks of a run when the cache is
// full, one to eight per warp, bounds the partial results that a stream has places for; with shorter
// sequences runs are shorter (B64 H32/8 C4096 of 10 keys each: 39.9 us -> 11.8), but not beside the tensor
// cores' part, which fewer warps disturb less (B32 H32/8 C1024 P2048: 39.2 us with the shortest, 36.0).
// A short prefix counts for kShortPrefix blocks: what starting on its few keys costs (with P1, eight
// parts of one block to a warp took 62 us, B64 H32/8).
constexpr int64_t kTcRows = 32;
constexpr int kShortPrefix = 8;
size_t plan_decode(DecodeArgs* a, bool bf16, char* base) {
  const int64_t rows = static_cast<int64_t>(a->B) * a->Hq;
  a->G = a->Hq / a->Hkv;
  a->block = decode_block_keys(bf16, a->D);
  const int64_t shared_rows = static_cast<int64_t>(a->B) * a->G;
  a->own_rowblocks = (a->G + kRows - 1) / kRows;
  a->shared_rowblocks = static_cast<int>((shared_rows + kRows - 1) / kRows);
  const int own = (a->C + a->block - 1) / a->block;
  a->own_width = own * a->block;
  const int64_t shared = (a->P + a->block - 1) / a->block, shared_streams = static_cast<int64_t>(a->Hkv) * a->shared_rowblocks;
  a->tc = bf16 && shared_rows > kTcRows && shared * shared_streams > 2 * kDecodeCtas * kWarps;
  a->pblocks = a->tc || !a->P ? 0 : static_cast<int>(shared < kShortPrefix ? kShortPrefix : shared);
  a->pre_width = a->pblocks * a->block;
  const int64_t total = static_cast<int64_t>(a->B) * own * a->Hkv * a->own_rowblocks +
                        static_cast<int64_t>(a->pblocks) * a->Hkv * a->shared_rowblocks;
  const int64_t streams = static_cast<int64_t>(a->B) * a->Hkv * a->own_rowblocks +
                          (a->pblocks ? shared_streams : 0);
  if (total > INT_MAX / 2) return 0;
  a->team = streams < 64 || (streams <= 128 && total < 10 * kDecodeCtas * kWarps) ? kWarps : 1;
  a->runs = a->team == 1 ? kDecodeCtas * kWarps : kDecodeCtas - static_cast<int>(streams);
  const int64_t even = total / a->runs;
  const int64_t full = even < a->team ? a->team : even > 8 * a->team ? 8 * a->team : even;
  a->pchunk = a->pslots = 0;
  if (a->tc) {
    const int64_t per = a->Hkv * ((shared_rows + 127) / 128), tiles = (a->P + 127) / 128;
    int64_t n = kSms / per;
    n = n < 1 ? 1 : n > tiles ? tiles : n;
    a->pchunk = static_cast<int>((tiles + n - 1) / n * 128);
    a->pslots = (a->P + a->pchunk - 1) / a->pchunk;
  } else if (a->P > 0) {
    a->pslots = static_cast<int>((a->pblocks + full - 1) / full + 1);
  }
  // a stream of n blocks meets at most ceil(n / run) + 1 runs
  a->slots = a->pslots + static_cast<int>((own + full - 1) / full + 1);
  a->least = a->tc ? static_cast<int>(full) : 1;
  size_t at = 0;
  auto piece = [&](int64_t floats) {
    char* p = base + at;
    at += (static_cast<size_t>(floats) * 4 + 255) & ~static_cast<size_t>(255);
    return p;
  };
  a->s_own = reinterpret_cast<float*>(piece(rows * a->own_width));
  a->s_pre = reinterpret_cast<float*>(piece(rows * a->pre_width));
  a->row_max = reinterpret_cast<float*>(piece(rows * a->slots));
  a->part_sum = reinterpret_cast<float*>(piece(rows * a->slots));
  a->part_o = reinterpret_cast<float*>(piece(rows * a->slots * a->D));
  a->cum = reinterpret_cast<int*>(piece(a->B + 2));
  return at;
}

cudaError_t launch_decode(const DecodeArgs& a, bool bf16, const PrefixMaps& maps, const LaunchCtx& ctx,
                          cudaStream_t st) {
  if (bf16) return a.D == 64 ? go<__nv_bfloat16, 64>(a, maps, ctx, st) : go<__nv_bfloat16, 128>(a, maps, ctx, st);
  if (a.D == 16) return go<float, 16>(a, maps, ctx, st);
  if (a.D == 32) return go<float, 32>(a, maps, ctx, st);
  if (a.D == 64) return go<float, 64>(a, maps, ctx, st);
  return go<float, 128>(a, maps, ctx, st);
}

}  // namespace raattn
