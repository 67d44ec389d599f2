// Attention of one query token per sequence against a cache whose keys and values lie in pages, in 4 bits
// (paged.cuh): ra_attention_decode's mathematics on khat = lo + s u, vhat = lo + s u.
//
//   z_j = sum_g s_jg (sum_{d in g} q_d u_jd) + lo_jg (sum_{d in g} q_d)
//   phi_j as in decode.cu;  o_d = [sum_j (phi_j s_jg) u_jd + sum_j phi_j lo_jg] / sum_j phi_j,  g the group of d
//
// so the products run on the codes themselves and a scale is applied once per key and group (scores) or once per
// weight and group (values).  A code is an fp16 subnormal as it stands: the bits 0000 0000 0000 uuuu are u 2^-24, and
// four bits further left 16 u 2^-24, exactly.  So a mask makes an operand out of two codes: five integer instructions
// for eight codes, no conversion.  The factors 16 and 2^-24 are powers of two and go into the query (scores) and the end
// (values).  The tensor cores align products by their operands' exponent fields, so a subnormal's leading zeros cost
// up to six of the sum's 24 bits: nothing beside bf16's eight, but 2.6e-5 of an fp32 output.  fp32 calls make normal
// numbers of the codes (1024 + u in fp16, minus 1032) and count them from the middle, khat = (lo + 8 s) + s (u - 8): sums of
// s u and of lo cancel to the last of their bits where keys or values have no mean of their size.  They add each step's products
// to fp32 sums, since the tensor cores truncate theirs.  Errors against 64 bits over random calls: 1.4 times those of a
// plain 32-bit form before (3.0 at most), 0.7 times (1.2) now; B16 H32/8 C8192 38.1 us -> 38.7.
//   scores   m16n8k16: sixteen keys as M, eight query heads as N.  The query goes in as fp16 times a power of two of
//            its row (11 bits, bf16's 8 exactly, down to 2^-26 of the largest: it is below 2^14, every other dimension a sixteenth,
//            and fp16 ends at 2^-24); fp32 queries as two fp16 (22 bits).
//   values   m16n8k16: sixteen dimensions as M, eight heads as N, sixteen keys as K; two keys' words are put together
//            by byte.  phi s goes in as two fp16 (22 bits; with one, 11 bits, the errors of bf16 outputs against 64 bits
//            were 1.74e-3 of their size instead of the output's rounding alone, 1.66e-3; B64 H32/8 C16384 126.3 us with one, 129.4
//            with two) times a power of two that follows the largest phi s met so far, of each row and group: with one power for
//            all, a group or a key of much larger values, even one outside the support, took the others' bits (B64 H32/8 C16384
//            129.4 -> 132.0 us).
// A few rows of queries against many keys leave the fifth generation's products, 128 rows at a time, empty; their
// operands would have to be unpacked into shared memory first.
// Two launches, scores and values, around the rows' maxima; the last part of a row to be done joins them, or a third
// launch where they are many.  The scores of sixteen keys stand in the workspace as the value products want them: key t
// at 4 (t % 4) + t / 4.
//
// Bound: HBM, and behind it the latency of a warp's chain of loads, masks and products.  bf16 H32/8 D128, whole call in a
// graph: B64, up to 16384 keys each, 567 MB in 130.7 us, 4.3 TB/s (the scores kernel alone 5.2); B1, 131072 keys, 42.5 us, 3.6 TB/s.
// For 32 keys of 128 dimensions a warp issues 271 instructions in the scores and 392 in the values, about 100 of either to take codes
// apart, at 55 % of the issue slots.  Below that latency: B1 C512 7.3 us, two launches of a few dependent loads (lengths, page numbers, pages) each.
#include <algorithm>
#include <climits>
#include <cuda_fp16.h>

#include "decode_parts.cuh"
#include "paged.cuh"

namespace raattn {
namespace {

using namespace decode;
using namespace paged;

constexpr int kKeys = 32;                        // of a block: products' M, or K, of sixteen
constexpr int64_t kPrefetched = 1 << 18;          // numbers of a table that is fetched ahead: 1 MB
constexpr uint32_t kLow = 0x000f000fu, kHigh = 0x00f000f0u;

template <int D>
struct Cfg {
  static constexpr int G = D / kGroup;
  static constexpr int kTiles = kKeys / 16;
  static constexpr int kCodes = kKeys * D / 2;            // bytes of a block's codes
  static constexpr int kMeta = 4 * G;                     // bytes of a key's scales and minima
  static constexpr int kBlock = kKeys * row_bytes(D);
  static constexpr int kStages = 3;                       // of a warp's ring; four or five gave nothing
};
// CTAs of an SM.  More, with fewer registers each, lose more in spills and part starts than they hide (B64 H32/8 D128
// C16384, whole call, with one fp16 for a weight: 131 us with 4 and 128 registers, 152 with 4 and 96, 149 with 5; 96 for the scores with a CTA's runs alone,
// which leaves room for a CTA of the values beside them: B32 H32/8 C2048 21.2 us -> 21.6).  fp32's operands and sums, or
// sixteen rows, take more registers.
__host__ __device__ constexpr int resident(bool bf16, int tiles) { return bf16 && tiles == 1 ? 4 : 3; }
// A stage of the values: the block, then its rows of scores (FOLD: four at most).
template <int NT, bool FOLD>
__host__ __device__ constexpr int score_rows() { return FOLD ? 4 : 8 * NT; }
template <int D, int NT, bool FOLD>
__host__ __device__ constexpr int stage_values() { return Cfg<D>::kBlock + score_rows<NT, FOLD>() * kKeys * 4; }
// A warp's ring of them, and behind it a block's scales and minima in fp32.
template <int D, int NT, bool FOLD>
__host__ __device__ constexpr int ring_values() {
  return Cfg<D>::kStages * stage_values<D, NT, FOLD>() + kKeys * 2 * Cfg<D>::kMeta;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same with nothing to add to.
__device__ __forceinline__ void mma_f16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
// Loads that the compiler may move, unlike volatile ones: products and loads of neighbouring tiles mix.
template <typename V>
__device__ __forceinline__ V get(const char* p) { return *reinterpret_cast<const V*>(p); }
__device__ __forceinline__ uint32_t half2_bits(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// x and y as fp16 and, with TWO, what that loses as another.
template <bool TWO>
__device__ __forceinline__ void split_half2(float x, float y, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x, y);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  if constexpr (TWO) {
    const float2 f = __half22float2(h);
    lo = half2_bits(x - f.x, y - f.y);
  }
}
__device__ __forceinline__ float power_of_2(int e) {   // inf above fp32's range, 0 below
  return __uint_as_float(static_cast<uint32_t>(min(max(e + 127, 0), 255)) << 23);
}
__device__ __forceinline__ int exponent_of(float x) { return static_cast<int>(__float_as_uint(x) >> 23) - 127; }   // x >= 0

// Two codes as an operand: the fp16 of them times 2^-24 or, with TWO, of u - 8 (the higher ones: sixteen times that).
template <bool TWO>
__device__ __forceinline__ uint32_t codes2(uint32_t word, uint32_t mask) {
  if constexpr (!TWO) return word & mask;
  const uint32_t u = (word & mask) | 0x64006400u;
  const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&u), __float2half2_rn(mask == kLow ? 1032.0f : 1152.0f));
  return *reinterpret_cast<const uint32_t*>(&h);
}
// What a code's operand of 0 stands for.
template <bool TWO>
__device__ __forceinline__ float middle(float lo, float s) { return TWO ? fmaf(8.0f, s, lo) : lo; }
template <typename T>
__host__ __device__ constexpr float code_unit() { return sizeof(T) == 4 ? 1.0f : 0x1p-24f; }

// A key's scales and minima: (s, lo) of one group, or (s0, s1), (lo0, lo1) of two.
template <int G>
struct Meta {
  float s[G], lo[G];
  __device__ __forceinline__ explicit Meta(const char* p) {
    if constexpr (G == 2) {
      const uint2 u = get<uint2>(p);
      s[0] = bf16_low(u.x);
      s[1] = bf16_high(u.x);
      lo[0] = bf16_low(u.y);
      lo[1] = bf16_high(u.y);
    } else {
      const uint32_t u = get<uint32_t>(p);
      s[0] = bf16_low(u);
      lo[0] = bf16_high(u);
    }
  }
};

// ---------------------------------------------------------------------------------------------
// the split
// ---------------------------------------------------------------------------------------------
// A team (a warp, or a CTA's four) has a run of blocks for one key head and up to sixteen of its query rows.
// The blocks of all sequences, in order, are cut into runs of `per`, or with CUT each sequence for itself; every run
// has a team for each head, next to one another, since the heads' parts of a page lie together: a warp
// that moves from page to page on its own meets a new one for every 4.6 KB.
struct PagedPart {
  int b, kv, row0, rows;   // sequence, key head; rows within the head's G
  int first, count, keys;  // blocks of the sequence; its keys
  int slot, parts;         // its place among the sequence's parts
};
// CUT: of few sequences the least (a multiple of the team, so that its warps have as many each) with which their runs
// are a.runs in all, of eight; else what is enough whatever the lengths.
constexpr int kFewSequences = 64;
template <bool CUT>
__device__ __forceinline__ int blocks_per_run(const PagedDecodeArgs& p, const int* cum, int longest) {
  const DecodeArgs& a = p.a;
  const int least = (longest + a.slots - 2) / (a.slots - 1);   // a sequence of n blocks meets at most ceil(n / per) + 1 runs
  const int total = cum[a.B];
  if (!CUT) return max(max((total + a.runs - 1) / a.runs, least), 1);
  const auto whole = [&](int per) { return (max(per, 1) + a.team - 1) / a.team * a.team; };
  const int first = whole(max((total + a.runs - 1) / a.runs, least));
  const int enough = max(first, whole((total + a.runs - a.B - 1) / (a.runs - a.B)));   // one more run a sequence at most
  if (a.B > kFewSequences || total + first >= 1 << 20) return enough;
  if (total + a.B * (first - 1) <= a.runs * first) return first;   // it fits whatever the lengths
  // lane (c, g) counts candidate c's runs of every fourth sequence; the quotients are exact below 2^21
  const int lane = threadIdx.x & 31, mine = first + (lane & 7) * a.team;
  const float inv = 1.0f / mine;
  int runs = 0;
  for (int b = lane >> 3; b < a.B; b += 4) runs += static_cast<int>((static_cast<float>(cum[b + 1] - cum[b] + mine - 1) + 0.5f) * inv);
  runs += __shfl_xor_sync(0xffffffffu, runs, 8);
  runs += __shfl_xor_sync(0xffffffffu, runs, 16);
  const unsigned fits = __ballot_sync(0xffffffffu, runs <= a.runs) & 0xffu;
  return fits ? first + (__ffs(fits) - 1) * a.team : enough;
}
// Parts of a sequence whose blocks are c0 .. c1 - 1 of all.
template <bool CUT>
__device__ __forceinline__ int parts_of(int c0, int c1, int per) {
  return c0 == c1 ? 0 : CUT ? (c1 - c0 + per - 1) / per : (c1 - 1) / per - c0 / per + 1;
}
// f(part) for the parts of this team's run.  All lanes.
template <int TW, bool CUT, typename F>
__device__ __forceinline__ void each_paged_part(const PagedDecodeArgs& pa, const int* cum, int per, F f) {
  const DecodeArgs& a = pa.a;
  const int heads = a.Hkv * a.own_rowblocks;
  const int task = TW == 1 ? blockIdx.x * kWarps + (threadIdx.x >> 5) : blockIdx.x, run = task / heads, head = task - run * heads;
  PagedPart p;
  p.kv = a.own_rowblocks == 1 ? head : head / a.own_rowblocks;
  p.row0 = (head - p.kv * a.own_rowblocks) * kRows;
  p.rows = min(a.G - p.row0, kRows);
  if constexpr (CUT) {   // few sequences: 32 at a time
    const int lane = threadIdx.x & 31;
    int b = -1, i = run;
    for (int b0 = 0; b0 < a.B && b < 0; b0 += 32) {
      const int mine = b0 + lane < a.B ? (cum[b0 + lane + 1] - cum[b0 + lane] + per - 1) / per : 0;
      int upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
      }
      const unsigned past = __ballot_sync(0xffffffffu, upto > i);
      const int l = past ? __ffs(past) - 1 : 31;
      const int before = __shfl_sync(0xffffffffu, upto - mine, l), all = __shfl_sync(0xffffffffu, upto, 31);
      if (past) {
        b = b0 + l;
        i -= before;
      } else {
        i -= all;
      }
    }
    if (b < 0) return;
    const int blocks = cum[b + 1] - cum[b];
    p.b = b;
    p.keys = cum[a.B + 1 + b];
    p.first = i * per;
    p.count = min(blocks - p.first, per);
    p.slot = i;
    p.parts = parts_of<CUT>(cum[b], cum[b + 1], per);
    f(p);
  } else {
    const int total = cum[a.B], end = static_cast<int>(min(static_cast<int64_t>(run + 1) * per, static_cast<int64_t>(total)));
    for (int64_t u0 = static_cast<int64_t>(run) * per; u0 < end;) {
      const int u = static_cast<int>(u0);
      int lo = 0, hi = a.B - 1;   // the last b with cum[b] <= u: u lies in its blocks
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cum[mid] <= u) lo = mid; else hi = mid - 1;
      }
      const int c0 = cum[lo], c1 = cum[lo + 1];
      p.b = lo;
      p.keys = cum[a.B + 1 + lo];
      p.first = u - c0;
      p.count = min(c1, end) - u;
      p.slot = run - c0 / per;
      p.parts = parts_of<CUT>(c0, c1, per);
      u0 += p.count;
      f(p);
    }
  }
}
template <int TW>
__device__ __forceinline__ int blocks_of_warp(const PagedPart& p) { return (p.count - warp_of_team<TW>() + TW - 1) / TW; }
// Row r of a part (its last one for those past it) as an index into [B, H_q], and its scores.
__device__ __forceinline__ int row_of(const PagedPart& p, int r, const DecodeArgs& a) {
  return p.b * a.Hq + p.kv * a.G + p.row0 + min(r, p.rows - 1);
}
__device__ __forceinline__ float* score_row(int row, const DecodeArgs& a) { return a.s_own + static_cast<int64_t>(row) * a.own_width; }

// ---------------------------------------------------------------------------------------------
// a warp's blocks into its ring
// ---------------------------------------------------------------------------------------------
__device__ __forceinline__ void copy16_part(uint32_t dst, const void* src, int bytes, uint64_t policy) {   // zeros behind `bytes`
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(bytes), "l"(policy)
               : "memory");
}

// Blocks first, first + step, .. of a part.  The page numbers of their tiles (a page is at least sixteen keys) come
// through shared memory, half of kIds blocks at a time and that many ahead.  What no page holds and what lies behind the
// last key arrives as zeros: scales and minima of 0.
template <int D>
struct Fetch {
  using C = Cfg<D>;
  static constexpr int kIds = 2 * 32 / C::kTiles;    // blocks whose pages a warp has
  static constexpr int kLanesPerKey = D / 32;        // 16-byte chunks of a key's codes
  static constexpr int kKeysPerCopy = 32 / kLanesPerKey;
  static constexpr int kCopies = kKeys / kKeysPerCopy, kTileCopies = 16 / kKeysPerCopy;
  static constexpr int kMetaLanes = kKeys * C::kMeta / 16, kKeysPerChunk = 16 / C::kMeta;
  static_assert(kMetaLanes <= 32, "one copy");
  const PagePool& pool;
  const int32_t* row;
  const uint8_t* base;   // with this lane's place in a block's codes
  const int* ids;        // pages of block i's tiles: from (i % kIds) * kTiles on
  int first, step, blocks, keys, lane;
  uint64_t policy;       // keys and values leave L2 first: the scores had better stay

  // ids: of this warp's, which nobody reads any more.  await() comes before the first block.
  __device__ __forceinline__ Fetch(const PagedDecodeArgs& p, const PagedPart& part, int which, int warp, int warps, int blocks_,
                                   const int* ids_)
      : pool(p.pool), row(p.table + static_cast<int64_t>(part.b) * p.M), ids(ids_), first((part.first + warp) * kKeys),
        step(warps * kKeys), blocks(blocks_), keys(part.keys), lane(threadIdx.x & 31) {
    base = part_of(p.pool, 0, part.kv, which) + lane * 16;
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
    pages(0);
    pages(kIds / 2);
    copy_commit();
  }
  __device__ __forceinline__ void await() const {
    copy_wait<0>();
    __syncwarp();
  }
  __device__ __forceinline__ void pages(int i0) const {   // lane l: tile l % kTiles of block i0 + l / kTiles
    const int i = i0 + lane / C::kTiles, key = min(first + i * step + lane % C::kTiles * 16, keys - 1);
    if (i < blocks)
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(ids + i % kIds * C::kTiles + lane % C::kTiles)),
                   "l"(row + (key >> pool.shift))
                   : "memory");
  }
  __device__ __forceinline__ bool there(int id) const { return static_cast<unsigned>(id) < static_cast<unsigned>(pool.pages); }
  __device__ __forceinline__ void operator()(uint32_t stage, int i) {
    if ((i & (kIds / 2 - 1)) == 0 && i) pages(i + kIds / 2);   // the other half is in use
    stage += lane * 16;
    const int key0 = first + i * step, slot = key0 & (pool.page - 1);
    const int* id = ids + i % kIds * C::kTiles;
    if (pool.page >= kKeys && key0 + kKeys <= keys && there(id[0])) {
      const uint8_t* src = base + static_cast<int64_t>(id[0]) * pool.page_stride;
      const uint8_t* codes = src + slot * (D / 2);
#pragma unroll
      for (int c = 0; c < kCopies; ++c) copy16_once(stage + c * 512, codes + c * 512, policy);
      if (lane < kMetaLanes) copy16_once(stage + C::kCodes, src + pool.page * (D / 2) + slot * C::kMeta, policy);
    } else {
#pragma unroll 1
      for (int h = 0; h < C::kTiles; ++h) {
        const int at = id[h], in_page = (key0 + 16 * h) & (pool.page - 1);
        const bool in = there(at);
        const int left = in ? keys - key0 - 16 * h : 0;   // keys of the tile that there are
        const uint8_t* src = base + static_cast<int64_t>(in ? at : 0) * pool.page_stride;
#pragma unroll
        for (int c = 0; c < kTileCopies; ++c)
          copy16_part(stage + (h * kTileCopies + c) * 512, src + in_page * (D / 2) + c * 512,
                      c * kKeysPerCopy + lane / kLanesPerKey < left ? 16 : 0, policy);
        if (lane < kMetaLanes / C::kTiles)
          copy16_part(stage + C::kCodes + h * (kMetaLanes / C::kTiles) * 16, src + pool.page * (D / 2) + in_page * C::kMeta,
                      min(max((left - lane * kKeysPerChunk) * C::kMeta, 0), 16), policy);
      }
    }
  }
};

// ---------------------------------------------------------------------------------------------
// scores
// ---------------------------------------------------------------------------------------------
// Lane (r, j) = (lane / 4, lane % 4) reads, of keys r and r + 8 of sixteen, words 2 j and 2 j + 1 of every group
// (dimensions 16 j .. 16 j + 15): the A operand's rows.  Of query row r it holds the same dimensions, in the order of
// the codes' positions, as the B operand.
template <typename T, int D, int NT>
struct Query {
  static constexpr int G = D / kGroup;
  static constexpr bool TWO = sizeof(T) == 4;
  uint32_t b[NT][G][4][2], rest[NT][G][TWO ? 4 : 1][2];
  float sum[NT][G][2];   // of query rows 2 j, 2 j + 1: their sums over a group

  static constexpr int kWords = 16 * sizeof(T) / 16;   // 16-byte words of sixteen elements
  struct Raw {
    uint4 u[NT][G][kWords];
    __device__ __forceinline__ Raw(const PagedPart& p, const DecodeArgs& a) {
      const int lane = threadIdx.x & 31;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const T* q = static_cast<const T*>(a.q) + static_cast<int64_t>(row_of(p, t * 8 + (lane >> 2), a)) * D + 16 * (lane & 3);
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
          for (int i = 0; i < kWords; ++i) u[t][g][i] = __ldg(reinterpret_cast<const uint4*>(q + g * kGroup) + i);
      }
    }
  };

  // The rows' units go to `units`: what a score of 1 stands for, the same in all parts of a row.
  __device__ __forceinline__ Query(const Raw& raw, const PagedPart& p, const DecodeArgs& a, float* units) {
    const int lane = threadIdx.x & 31, r = lane >> 2, j = lane & 3;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float x[G][16], most = 0.0f;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        values(raw.u[t][g], x[g]);
#pragma unroll
        for (int i = 0; i < 16; ++i) most = fmaxf(most, fabsf(x[g][i]));
      }
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
      const int e = max(static_cast<int>(__float_as_uint(most) >> 23) - 126, -100);   // most < 2^e
      const float to = power_of_2(14 - e);
      if (j == 0 && t * 8 + r < p.rows) units[row_of(p, t * 8 + r, a)] = power_of_2(e - 14 + (TWO ? 0 : 24));
      float total[G];
#pragma unroll
      for (int g = 0; g < G; ++g) {
        total[g] = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          x[g][i] *= to;
          total[g] += x[g][i];
        }
        total[g] += __shfl_xor_sync(0xffffffffu, total[g], 1);
        total[g] += __shfl_xor_sync(0xffffffffu, total[g], 2);
        // step 2 w + f: nibbles (2 f, 2 f + 4) and, sixteen times as large, (2 f + 1, 2 f + 5) of word w
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int d = (k >> 1) * 8 + (k & 1) * 2;
          split_half2<TWO>(x[g][d], x[g][d + 4], b[t][g][k][0], rest[t][g][TWO ? k : 0][0]);
          split_half2<TWO>(x[g][d + 1] * 0.0625f, x[g][d + 5] * 0.0625f, b[t][g][k][1], rest[t][g][TWO ? k : 0][1]);
        }
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int from = 8 * j + 4 * c;
#pragma unroll
        for (int g = 0; g < G; ++g) sum[t][g][c] = __shfl_sync(0xffffffffu, total[g], from) * code_unit<T>();
      }
    }
  }
  static __device__ __forceinline__ void values(const uint4 (&u)[2], float (&x)[16]) {   // bf16
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        x[8 * i + 2 * k] = bf16_low(w[k]);
        x[8 * i + 2 * k + 1] = bf16_high(w[k]);
      }
    }
  }
  static __device__ __forceinline__ void values(const uint4 (&u)[4], float (&x)[16]) {   // fp32
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[4 * i] = __uint_as_float(u[i].x);
      x[4 * i + 1] = __uint_as_float(u[i].y);
      x[4 * i + 2] = __uint_as_float(u[i].z);
      x[4 * i + 3] = __uint_as_float(u[i].w);
    }
  }
};

template <typename T, int D, int TW, int NT>
__device__ __forceinline__ void part_scores(const PagedPart& p, const PagedDecodeArgs& pa, char* ring, const int* ids, float* best_s) {
  using C = Cfg<D>;
  constexpr int G = C::G;
  constexpr bool TWO = sizeof(T) == 4;
  const DecodeArgs& a = pa.a;
  const int lane = threadIdx.x & 31, r = lane >> 2, j = lane & 3;
  const int mine = blocks_of_warp<TW>(p);
  Fetch<D> fetch(pa, p, 0, warp_of_team<TW>(), TW, mine, ids);
  const typename Query<T, D, NT>::Raw raw(p, a);
  fetch.await();
#pragma unroll
  for (int i = 0; i < C::kStages - 1; ++i) {
    if (i < mine) fetch(smem_u32(ring) + i * C::kBlock, i);
    copy_commit();
  }
  const Query<T, D, NT> q(raw, p, a, pa.unit);
  const int first = (p.first + warp_of_team<TW>()) * kKeys, at = (r & 3) * 4 + (r >> 2);
  float* out[NT][2];   // sixteen keys' scores stand as the value products want them
  bool there[NT][2];
  float best[NT][2];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      out[t][c] = score_row(row_of(p, t * 8 + 2 * j + c, a), a) + first + at;
      there[t][c] = t * 8 + 2 * j + c < p.rows;
      best[t][c] = -kInf;
    }
  // this lane's 16 bytes (D = 128) or 8 of key r: the halves' order depends on the key's bit 1, which is r's
  const int chunk = r * (D / 2) + (G == 2 ? (16 * j) ^ ((r & 2) << 4) : 8 * j), meta = C::kCodes + r * C::kMeta;
  int left = p.keys - first;   // keys from the block's first on
  const char *stage = ring, *to = ring + (C::kStages - 1) * C::kBlock;
  for (int i = 0; i < mine; ++i, left -= TW * kKeys) {
    copy_wait<C::kStages - 2>();
    __syncwarp();   // block i has landed for all lanes, and all have read block i - 1
    if (i + C::kStages - 1 < mine) fetch(smem_u32(to), i + C::kStages - 1);
    copy_commit();
    to = to == ring + (C::kStages - 1) * C::kBlock ? ring : to + C::kBlock;
    float z[C::kTiles][NT][4];
#pragma unroll
    for (int tile = 0; tile < C::kTiles; ++tile) {
      uint32_t x[2][G][2];   // keys r, r + 8; words 2 j, 2 j + 1 of the groups
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const char* src = stage + chunk + (tile * 16 + h * 8) * (D / 2);
        if constexpr (G == 2) {
          const uint4 u = get<uint4>(src);
          x[h][0][0] = u.x;
          x[h][1][0] = u.y;
          x[h][0][1] = u.z;
          x[h][1][1] = u.w;
        } else {
          const uint2 u = get<uint2>(src);
          x[h][0][0] = u.x;
          x[h][0][1] = u.y;
        }
      }
      const Meta<G> m0(stage + meta + tile * 16 * C::kMeta), m1(stage + meta + (tile * 16 + 8) * C::kMeta);
#pragma unroll
      for (int g = 0; g < G; ++g) {
        float acc[NT][4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t u = x[0][g][k >> 1] >> (k & 1) * 8, v = x[1][g][k >> 1] >> (k & 1) * 8;
          const uint32_t a0 = codes2<TWO>(u, kLow), a1 = codes2<TWO>(v, kLow), a2 = codes2<TWO>(u, kHigh),
                         a3 = codes2<TWO>(v, kHigh);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            if constexpr (TWO) {
              float c[4];
              mma_f16_first(c, a0, a1, a2, a3, q.rest[t][g][k][0], q.rest[t][g][k][1]);
              mma_f16(c, a0, a1, a2, a3, q.b[t][g][k][0], q.b[t][g][k][1]);
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[t][e] = k ? acc[t][e] + c[e] : c[e];
            } else if (k == 0) {
              mma_f16_first(acc[t], a0, a1, a2, a3, q.b[t][g][k][0], q.b[t][g][k][1]);
            } else {
              mma_f16(acc[t], a0, a1, a2, a3, q.b[t][g][k][0], q.b[t][g][k][1]);
            }
          }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float s = e < 2 ? m0.s[g] : m1.s[g], lo = middle<TWO>(e < 2 ? m0.lo[g] : m1.lo[g], s), w = q.sum[t][g][e & 1];
            z[tile][t][e] = g ? fmaf(s, acc[t][e], fmaf(lo, w, z[tile][t][e])) : fmaf(s, acc[t][e], lo * w);
          }
      }
    }
    if (left < kKeys) {   // the last block may have fewer
#pragma unroll
      for (int tile = 0; tile < C::kTiles; ++tile)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (tile * 16 + r + 8 * (e >> 1) >= left) z[tile][t][e] = -kInf;
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int tile = 0; tile < C::kTiles; ++tile) {
          best[t][c] = fmaxf(best[t][c], fmaxf(z[tile][t][c], z[tile][t][2 + c]));
          if (there[t][c]) {
            out[t][c][tile * 16] = z[tile][t][c];
            out[t][c][tile * 16 + 2] = z[tile][t][2 + c];
          }
        }
      }
    stage = stage == ring + (C::kStages - 1) * C::kBlock ? ring : stage + C::kBlock;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int c = 0; c < 2; ++c) out[t][c] += TW * kKeys;
  }
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) best[t][c] = fmaxf(best[t][c], __shfl_xor_sync(0xffffffffu, best[t][c], o));
      if (r == 0) best_s[(threadIdx.x >> 5) * kRows + t * 8 + 2 * j + c] = best[t][c];
    }
}

template <typename T, int D, int TW, int NT, bool CUT>
__global__ void __launch_bounds__(kThreads, resident(sizeof(T) == 2, NT)) paged_scores_kernel(const PagedDecodeArgs pa) {
  extern __shared__ uint4 dyn[];
  constexpr int kRing = Cfg<D>::kStages * Cfg<D>::kBlock;
  const DecodeArgs& a = pa.a;
  int* cum = reinterpret_cast<int*>(reinterpret_cast<char*>(dyn) + kWarps * kRing);
  __shared__ float best[kWarps * kRows];
  __shared__ int ids[kWarps][64];
  const int warp = threadIdx.x >> 5, team = warp / TW, tt = threadIdx.x % (32 * TW);
  await_previous();
  release_dependents();   // the next kernel's first values are on their way while this one ends
  // the page numbers, if they are few, are on their way while the split is made
  const int64_t at = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) * 32, table = static_cast<int64_t>(a.B) * pa.M;
  if (at < table && table <= kPrefetched) asm volatile("prefetch.global.L2 [%0];" ::"l"(pa.table + at));
  const int per = blocks_per_run<CUT>(pa, cum, count_blocks<kKeys>(cum, a));
  for (int i = blockIdx.x * kThreads + threadIdx.x; i < a.B * a.Hkv * a.own_rowblocks; i += gridDim.x * kThreads) pa.done[i] = 0;
  if (pa.join && blockIdx.x == 0)   // for the join
    for (int b = threadIdx.x; b < a.B; b += kThreads) a.cum[b] = parts_of<CUT>(cum[b], cum[b + 1], per);
  each_paged_part<TW, CUT>(pa, cum, per, [&](const PagedPart& p) {
    part_scores<T, D, TW, NT>(p, pa, reinterpret_cast<char*>(dyn) + warp * kRing, ids[warp], best);
    team_sync<TW>();
    if (tt < p.rows) {
      float m = best[team * TW * kRows + tt];
#pragma unroll
      for (int w = 1; w < TW; ++w) m = fmaxf(m, best[(team * TW + w) * kRows + tt]);
      a.row_max[static_cast<int64_t>(row_of(p, tt, a)) * a.slots + p.slot] = m;
    }
    team_sync<TW>();   // the maxima are read, and the rings are free
  });
}

// ---------------------------------------------------------------------------------------------
// values
// ---------------------------------------------------------------------------------------------
// phi of four scores z, from their distances to the maximum m: w = (1 + u) / 2 by a saturating FMA, so that -inf gives
// w = 1; q = 1 / w - 1 with one reciprocal for two (phi.cuh).  c2: scale / 32 in units of the scores.
__device__ __forceinline__ void phi4(const float4& z, float m, float c2, float2& x, float2& y) {
  const float2 minus1 = make_float2(-1.0f, -1.0f), mm = make_float2(m, m);
  const float2 d = __ffma2_rn(make_float2(z.x, z.y), minus1, mm), e = __ffma2_rn(make_float2(z.z, z.w), minus1, mm);
  const float2 A = make_float2(fma_sat(d.x, c2, 0.5f), fma_sat(d.y, c2, 0.5f));
  const float2 B = make_float2(fma_sat(e.x, c2, 0.5f), fma_sat(e.y, c2, 0.5f));
  const float2 P = __fmul2_rn(A, B);
  const float2 R = make_float2(rcp_approx(P.x), rcp_approx(P.y));
  x = __ffma2_rn(R, B, minus1);
  y = __ffma2_rn(R, A, minus1);
  x = __fmul2_rn(x, x);
  y = __fmul2_rn(y, y);
  x = __fmul2_rn(x, x);
  y = __fmul2_rn(y, y);
  x = __fmul2_rn(x, x);
  y = __fmul2_rn(y, y);
}

// Where piece c (four keys) of row r's scores stands: the reads of eight lanes (two rows by four pieces) meet no
// bank conflict.
__device__ __forceinline__ int piece_of(int r, int c) { return c ^ ((r & 1) << 2); }

// Lane (r, j) reads, of keys j, j + 4, j + 8 and j + 12 of sixteen, word r of every group (dimensions 8 r .. 8 r + 7):
// rows r and r + 8 of the A operand of product n stand for dimensions 8 r + 2 n and 8 r + 2 n + 1, the latter sixteen times as
// large.  The weights of query row r at the same keys are the B operand.  FOLD, up to four rows: the lanes of columns 0 .. 3 form the
// weights at a block's first sixteen keys and those of columns 4 .. 7 the ones at its other sixteen, so that no lane forms weights for
// nothing, and where one half's columns take the first fp16 of its weights the other's take the second: no product more than with one
// fp16.  The columns are added at the end.
template <typename T, int D, int TW, int NT, bool FOLD>
__device__ __forceinline__ void part_values(const PagedPart& p, const PagedDecodeArgs& pa, char* ring, const int* ids, float* rowm,
                                            float* sums) {
  using C = Cfg<D>;
  constexpr int G = C::G, kStage = stage_values<D, NT, FOLD>(), S = C::kStages;
  constexpr bool TWO = sizeof(T) == 4;
  const DecodeArgs& a = pa.a;
  static_assert(!FOLD || (NT == 1 && C::kTiles == 2), "two tiles for eight columns");
  const int lane = threadIdx.x & 31, r = lane >> 2, j = lane & 3;
  const int row8 = FOLD ? r & 3 : r, half = r >> 2;   // this lane's row of eight (FOLD: of four), and of which tile
  const int mine = blocks_of_warp<TW>(p), first = (p.first + warp_of_team<TW>()) * kKeys;
  Fetch<D> fetch(pa, p, 1, warp_of_team<TW>(), TW, mine, ids);
  // the scores: kKeys / 4 pieces of a row; a warp copies kRowsPerCopy rows at a time
  constexpr int kPieces = kKeys / 4, kRowsPerCopy = 32 / kPieces;
  const int score_at = lane / kPieces, piece = lane % kPieces;
  const float* score = score_row(row_of(p, 0, a) + score_at, a) + first + piece * 4;
  const float* used = score_row(row_of(p, lane, a), a) + first;   // lanes below p.rows
  auto fetch_scores = [&](uint32_t stage, int i) {
    const float* src = score + i * (TW * kKeys);
#pragma unroll
    for (int k = 0; k < score_rows<NT, FOLD>() / kRowsPerCopy; ++k) {
      const int row = score_at + k * kRowsPerCopy;
      if (row < p.rows) copy16(stage + C::kBlock + (row * kPieces + piece_of(row, piece)) * 16, src, true);
      src += kRowsPerCopy * static_cast<int64_t>(a.own_width);
    }
  };
  fetch.await();
  // the first blocks of a part do not wait for the scores
#pragma unroll
  for (int i = 0; i < S - 1; ++i)
    if (i < mine) fetch(smem_u32(ring) + i * kStage, i);
  await_previous();
#pragma unroll
  for (int i = 0; i < S - 1; ++i) {
    if (i < mine) fetch_scores(smem_u32(ring) + i * kStage, i);
    copy_commit();
  }
  {   // the rows' maxima over all parts, each by 2 TW of the team's threads
    const int tt = threadIdx.x % (32 * TW), row = tt / (2 * TW);
    const float most = fold_slots<2 * TW>(a.row_max + static_cast<int64_t>(row_of(p, row, a)) * a.slots, 0, p.parts, 0,
                                          tt % (2 * TW), -kInf, [](float x, float y) { return fmaxf(x, y); });
    if (tt % (2 * TW) == 0) rowm[row] = most;
  }
  team_sync<TW>();
  float m[NT], c2[NT], total[NT], acc[NT][G][4][4];
  float unit[NT][G];   // the power of two of this lane's row and group: every weight met so far, times it, is below 2^15
  float2 low[NT];   // of the groups (D = 64: the first)
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    m[t] = rowm[t * 8 + row8];
    if (m[t] == -kInf) m[t] = 0.0f;
    c2[t] = a.scale * (TWO ? 1.0f : 0.03125f) * __ldcg(pa.unit + row_of(p, t * 8 + row8, a));
    total[t] = 0.0f;
    low[t] = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      unit[t][g] = 0x1p114f;
#pragma unroll
      for (int n = 0; n < 4; ++n) acc[t][g][n][0] = acc[t][g][n][1] = acc[t][g][n][2] = acc[t][g][n][3] = 0.0f;
    }
  }
  const int word = word_offset<G>(0, r, j);   // the halves' order: bit 1 of the key's slot is j's
  float* metas = reinterpret_cast<float*>(ring + S * kStage);
  const char *stage = ring, *to = ring + (S - 1) * kStage;
  for (int i = 0; i < mine; ++i) {
    copy_wait<S - 2>();
    __syncwarp();
    // nobody reads these scores again: a line of L2 less to be written back (B64 H32/8 D128 C16384 131 us -> 125.6)
    if (lane < p.rows) asm volatile("discard.global.L2 [%0], 128;" ::"l"(used + i * (TW * kKeys)) : "memory");
    if (i + S - 1 < mine) {
      fetch(smem_u32(to), i + S - 1);
      fetch_scores(smem_u32(to), i + S - 1);
    }
    copy_commit();
    to = to == ring + (S - 1) * kStage ? ring : to + kStage;
    {   // the keys' scales and minima, a lane for each of 32
      static_assert(kKeys == 32, "a lane for each key");
      const Meta<G> meta(stage + C::kCodes + lane * C::kMeta);
      if constexpr (G == 2)
        reinterpret_cast<float4*>(metas)[lane] =
            make_float4(meta.s[0], meta.s[1], middle<TWO>(meta.lo[0], meta.s[0]), middle<TWO>(meta.lo[1], meta.s[1]));
      else
        reinterpret_cast<float2*>(metas)[lane] = make_float2(meta.s[0], middle<TWO>(meta.lo[0], meta.s[0]));
      __syncwarp();
    }
    constexpr int FT = FOLD ? 1 : C::kTiles;   // tiles for which a lane forms weights
    float f[FT][NT][4];
    bool live = false;   // some weight that is not 0 (a NaN is not)
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int tile = 0; tile < FT; ++tile) {
        float* w = f[tile][t];
        w[0] = w[1] = w[2] = w[3] = 0.0f;
        if (t * 8 + row8 < p.rows) {
          const float4 z = get<float4>(stage + C::kBlock +
                                       ((t * 8 + row8) * kPieces + piece_of(row8, (FOLD ? half : tile) * 4 + j)) * 16);
          if constexpr (TWO) {
            w[0] = phi_exact((m[t] - z.x) * c2[t]);
            w[1] = phi_exact((m[t] - z.y) * c2[t]);
            w[2] = phi_exact((m[t] - z.z) * c2[t]);
            w[3] = phi_exact((m[t] - z.w) * c2[t]);
          } else {
            float2 x, y;
            phi4(z, m[t], c2[t], x, y);
            w[0] = x.x;
            w[1] = x.y;
            w[2] = y.x;
            w[3] = y.y;
          }
        }
        const float all = (w[0] + w[1]) + (w[2] + w[3]);
        total[t] += all;
        live |= all != 0.0f;
      }
    }
    // the weights times the scales and times the minima, which show a NaN whatever the weights
    float2 weight[FT][NT][4];   // of the groups (D = 64: the first)
#pragma unroll
    for (int tile = 0; tile < FT; ++tile)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int key = (FOLD ? half : tile) * 16 + j + 4 * k;
        if constexpr (G == 2) {
          const float4 meta = reinterpret_cast<const float4*>(metas)[key];
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const float2 ff = make_float2(f[tile][t][k], f[tile][t][k]);
            weight[tile][t][k] = __fmul2_rn(ff, make_float2(meta.x, meta.y));
            low[t] = __ffma2_rn(ff, make_float2(meta.z, meta.w), low[t]);
          }
        } else {
          const float2 meta = reinterpret_cast<const float2*>(metas)[key];
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            weight[tile][t][k].x = f[tile][t][k] * meta.x;
            low[t].x = fmaf(f[tile][t][k], meta.y, low[t].x);
          }
        }
      }
    // the rows' powers of two follow their largest weights, those of a group apart from the other's
    float most[NT][G];
    bool over = false;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int g = 0; g < G; ++g) {
        most[t][g] = 0.0f;
#pragma unroll
        for (int tile = 0; tile < FT; ++tile)
#pragma unroll
          for (int k = 0; k < 4; ++k) most[t][g] = fmaxf(most[t][g], g ? weight[tile][t][k].y : weight[tile][t][k].x);
        over |= most[t][g] * unit[t][g] >= 0x1p15f;
      }
    const unsigned state = __reduce_max_sync(0xffffffffu, over ? 2u : live ? 1u : 0u);
    if (state) {   // no products where all weights are 0: codes are finite
      if (state == 2) {   // a few times in a part
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int g = 0; g < G; ++g) {
            float w = most[t][g];
            w = fmaxf(w, __shfl_xor_sync(0xffffffffu, w, 1));
            w = fmaxf(w, __shfl_xor_sync(0xffffffffu, w, 2));
            if constexpr (FOLD) w = fmaxf(w, __shfl_xor_sync(0xffffffffu, w, 16));
            const int now = exponent_of(unit[t][g]), e = w * unit[t][g] >= 0x1p15f ? 13 - exponent_of(w) : now;
            unit[t][g] = power_of_2(e);
            const float by = power_of_2(e - now);
            const float f0 = __shfl_sync(0xffffffffu, by, 8 * j), f1 = __shfl_sync(0xffffffffu, by, 8 * j + 4);   // of the sums' columns
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              acc[t][g][n][0] *= f0;
              acc[t][g][n][1] *= f1;
              acc[t][g][n][2] *= f0;
              acc[t][g][n][3] *= f1;
            }
          }
      }
      uint32_t wb[FT][NT][G][2], rest[FT][NT][G][2];   // as operands
#pragma unroll
      for (int tile = 0; tile < FT; ++tile)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int g = 0; g < G; ++g) {
            const float2* w = weight[tile][t];
            const float u = unit[t][g];
            split_half2<true>((g ? w[0].y : w[0].x) * u, (g ? w[1].y : w[1].x) * u, wb[tile][t][g][0], rest[tile][t][g][0]);
            split_half2<true>((g ? w[2].y : w[2].x) * u, (g ? w[3].y : w[3].x) * u, wb[tile][t][g][1], rest[tile][t][g][1]);
          }
      if constexpr (FOLD) {   // the other half's second fp16 of the same row
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
          for (int h = 0; h < 2; ++h) rest[0][0][g][h] = __shfl_xor_sync(0xffffffffu, rest[0][0][g][h], 16);
      }
#pragma unroll
      for (int tile = 0; tile < C::kTiles; ++tile) {
        uint32_t x[4][G];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const char* src = stage + (tile * 16 + j + 4 * k) * (D / 2) + word;
          if constexpr (G == 2) {
            const uint2 u = get<uint2>(src);
            x[k][0] = u.x;
            x[k][1] = u.y;
          } else {
            x[k][0] = get<uint32_t>(src);
          }
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
          uint32_t b[NT][2];
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              b[t][h] = FOLD ? half == tile ? wb[0][t][g][h] : rest[0][t][g][h] : wb[FOLD ? 0 : tile][t][g][h];
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            const uint32_t sel = n < 2 ? 0x5410u : 0x7632u;
            const uint32_t u = __byte_perm(x[0][g], x[1][g], sel) >> (n & 1) * 8;
            const uint32_t v = __byte_perm(x[2][g], x[3][g], sel) >> (n & 1) * 8;
            const uint32_t a0 = codes2<TWO>(u, kLow), a1 = codes2<TWO>(u, kHigh), a2 = codes2<TWO>(v, kLow),
                           a3 = codes2<TWO>(v, kHigh);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              const uint32_t* second = rest[FOLD ? 0 : tile][t][g];
              if constexpr (TWO) {
                float c[4];
                if constexpr (FOLD) {
                  mma_f16_first(c, a0, a1, a2, a3, b[t][0], b[t][1]);
                } else {
                  mma_f16_first(c, a0, a1, a2, a3, second[0], second[1]);
                  mma_f16(c, a0, a1, a2, a3, b[t][0], b[t][1]);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[t][g][n][k] += c[k];
              } else {
                if constexpr (!FOLD) mma_f16(acc[t][g][n], a0, a1, a2, a3, second[0], second[1]);
                mma_f16(acc[t][g][n], a0, a1, a2, a3, b[t][0], b[t][1]);
              }
            }
          }
        }
      }
    }
    stage = stage == ring + (S - 1) * kStage ? ring : stage + kStage;
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      total[t] += __shfl_xor_sync(0xffffffffu, total[t], o);
      low[t].x += __shfl_xor_sync(0xffffffffu, low[t].x, o);
      if (G == 2) low[t].y += __shfl_xor_sync(0xffffffffu, low[t].y, o);
    }
    if constexpr (FOLD) {   // rows r and r + 4, columns c and c + 4 are one
      total[t] += __shfl_xor_sync(0xffffffffu, total[t], 16);
      low[t].x += __shfl_xor_sync(0xffffffffu, low[t].x, 16);
      if (G == 2) low[t].y += __shfl_xor_sync(0xffffffffu, low[t].y, 16);
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[t][g][n][k] += __shfl_xor_sync(0xffffffffu, acc[t][g][n][k], 2);
    }
    if (j == 0) sums[(threadIdx.x >> 5) * kRows + t * 8 + r] = total[t];
  }
  __syncwarp();   // this warp's blocks have been read: its sums into their place
  float* out = reinterpret_cast<float*>(ring);
  constexpr float undo = 0x1p-14f / code_unit<T>();
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int row = t * 8 + 2 * j + c;
        const float lo = __shfl_sync(0xffffffffu, g ? low[t].y : low[t].x, 8 * j + 4 * c);
        const float back = power_of_2(14 - exponent_of(__shfl_sync(0xffffffffu, unit[t][g], 8 * j + 4 * c)));
        float y[8];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          y[2 * n] = fmaf(acc[t][g][n][c] * undo, back, lo);
          y[2 * n + 1] = fmaf(acc[t][g][n][2 + c] * (undo * 0.0625f), back, lo);
        }
        if (row < p.rows) {   // FOLD: lanes with j < 2
          float4* o = reinterpret_cast<float4*>(out + row * D + g * kGroup + r * 8);
          o[0] = make_float4(y[0], y[1], y[2], y[3]);
          o[1] = make_float4(y[4], y[5], y[6], y[7]);
        }
      }
}

template <typename T>
__device__ __forceinline__ void put4(void* o, int64_t at, const float4& f, float inv) {
  if constexpr (sizeof(T) == 2)
    static_cast<uint2*>(o)[at] = make_uint2(pack_bf16x2(f.x * inv, f.y * inv), pack_bf16x2(f.z * inv, f.w * inv));
  else
    static_cast<float4*>(o)[at] = make_float4(f.x * inv, f.y * inv, f.z * inv, f.w * inv);
}
__device__ __forceinline__ float4 add4(const float4& x, const float4& y) {
  return make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
}

// The output rows of a stream from its parts' sums, in their order, by the team of the last part to be done.
template <typename T, int D, int TW>
__device__ __forceinline__ void join_rows(const PagedPart& p, const DecodeArgs& a, int parts) {
  constexpr int kRowThreads = D / 4;   // of a row
  const int tt = threadIdx.x % (32 * TW);
  for (int e = tt; e < p.rows * kRowThreads; e += 32 * TW) {
    const int row = row_of(p, e / kRowThreads, a), c = e % kRowThreads;
    const int64_t at = static_cast<int64_t>(row) * a.slots;
    const float4* x = reinterpret_cast<const float4*>(a.part_o + at * D) + c;
    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float total = 0.0f;
    for (int i0 = 0; i0 < parts; i0 += 8) {   // eight parts at a time in flight
      float4 y[8];
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool in = i0 + i < parts;
        y[i] = in ? __ldcg(x + static_cast<int64_t>(i0 + i) * kRowThreads) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        f[i] = in ? __ldcg(a.part_sum + at + i0 + i) : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sum = add4(sum, y[i]);
        total += f[i];
      }
    }
    put4<T>(a.o, static_cast<int64_t>(row) * kRowThreads + c, sum, total != 0.0f ? 1.0f / total : 0.0f);
  }
}

template <typename T, int D, int TW, int NT, bool CUT, bool FOLD>
__global__ void __launch_bounds__(kThreads, resident(sizeof(T) == 2, NT)) paged_values_kernel(const PagedDecodeArgs pa) {
  extern __shared__ uint4 dyn[];
  constexpr int kRing = ring_values<D, NT, FOLD>();
  static_assert(kRing >= score_rows<NT, FOLD>() * D * 4, "a warp's partial sums fit its ring");
  const DecodeArgs& a = pa.a;
  int* cum = reinterpret_cast<int*>(reinterpret_cast<char*>(dyn) + kWarps * kRing);
  __shared__ float rowm_s[kWarps / TW * kRows], sums[kWarps * kRows];
  __shared__ int ids[kWarps][64];
  const int warp = threadIdx.x >> 5, team = warp / TW, tt = threadIdx.x % (32 * TW);
  char* ring = reinterpret_cast<char*>(dyn) + warp * kRing;
  const char* rings = reinterpret_cast<const char*>(dyn) + team * TW * kRing;   // the team's
  const int per = blocks_per_run<CUT>(pa, cum, count_blocks<kKeys>(cum, a));
  __shared__ int last_s[kWarps / TW];
  each_paged_part<TW, CUT>(pa, cum, per, [&](const PagedPart& p) {
    part_values<T, D, TW, NT, FOLD>(p, pa, ring, ids[warp], rowm_s + team * kRows, sums);
    const int parts = p.parts;
    team_sync<TW>();
    const auto sum_of = [&](int row) {
      float f = sums[team * TW * kRows + row];
#pragma unroll
      for (int w = 1; w < TW; ++w) f += sums[(team * TW + w) * kRows + row];
      return f;
    };
    if (parts > 1 && tt < p.rows) a.part_sum[static_cast<int64_t>(row_of(p, tt, a)) * a.slots + p.slot] = sum_of(tt);
    for (int e = tt; e < p.rows * (D / 4); e += 32 * TW) {
      const int row = e / (D / 4), c = e % (D / 4);
      float4 f = reinterpret_cast<const float4*>(rings)[e];
#pragma unroll
      for (int w = 1; w < TW; ++w) f = add4(f, *reinterpret_cast<const float4*>(rings + w * kRing + e * 16));
      if (parts == 1) {
        const float total = sum_of(row);
        put4<T>(a.o, static_cast<int64_t>(row_of(p, row, a)) * (D / 4) + c, f, total != 0.0f ? 1.0f / total : 0.0f);
      } else {
        reinterpret_cast<float4*>(a.part_o + (static_cast<int64_t>(row_of(p, row, a)) * a.slots + p.slot) * D)[c] = f;
      }
    }
    if (parts > 1 && !pa.join) {
      __threadfence();   // this thread's sums are there before the part counts as done
      team_sync<TW>();
      if (tt == 0)
        last_s[team] = atomicAdd(pa.done + (p.b * a.Hkv + p.kv) * a.own_rowblocks + p.row0 / kRows, 1) == parts - 1;
      team_sync<TW>();
      if (last_s[team]) {
        __threadfence();
        join_rows<T, D, TW>(p, a, parts);
      }
    }
    team_sync<TW>();
  });
  for (int b = blockIdx.x; b < a.B; b += gridDim.x)   // sequences without any key
    if (cum[a.B + 1 + b] == 0)
      for (int i = threadIdx.x; i < a.Hq * (D / 4); i += kThreads)
        put4<T>(a.o, static_cast<int64_t>(b) * a.Hq * (D / 4) + i, make_float4(0.0f, 0.0f, 0.0f, 0.0f), 0.0f);
  release_dependents();
  // Whoever awaits this kernel awaits the scores too: a CTA without a part sees to it.
  if (blockIdx.x == gridDim.x - 1) await_previous();
}

// A CTA per row: D / 4 threads across, the others over the parts.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) paged_join_kernel(const DecodeArgs a) {
  constexpr int L = D / 4, KS = kThreads / L;
  __shared__ float4 sums[KS][L];
  __shared__ float totals[KS];
  const int row = blockIdx.x, c = threadIdx.x % L, ks = threadIdx.x / L;
  await_previous();
  const int parts = __ldcg(a.cum + row / a.Hq);
  if (parts <= 1) return;   // written already
  const int64_t at = static_cast<int64_t>(row) * a.slots;
  float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  float total = 0.0f;
  for (int i0 = ks; i0 < parts; i0 += 8 * KS) {   // eight parts at a time in flight
    float4 x[8];
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bool in = i0 + i * KS < parts;
      x[i] = in ? __ldcg(reinterpret_cast<const float4*>(a.part_o + (at + i0 + i * KS) * D) + c) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      f[i] = in ? __ldcg(a.part_sum + at + i0 + i * KS) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      sum = add4(sum, x[i]);
      total += f[i];
    }
  }
  sums[ks][c] = sum;
  if (c == 0) totals[ks] = total;
  __syncthreads();
  if (ks) return;
#pragma unroll
  for (int i = 1; i < KS; ++i) {
    sum = add4(sum, sums[i][c]);
    total += totals[i];
  }
  put4<T>(a.o, static_cast<int64_t>(row) * L + c, sum, total != 0.0f ? 1.0f / total : 0.0f);
}

template <typename T, int D, int TW, int NT, bool FOLD, bool CUT>
cudaError_t go(const PagedDecodeArgs& p, cudaStream_t st) {
  const DecodeArgs& a = p.a;
  constexpr int kScores = kWarps * Cfg<D>::kStages * Cfg<D>::kBlock;
  constexpr int kValues = kWarps * ring_values<D, NT, FOLD>();
  constexpr int kMostCum = (2 * kDecodeMaxBatch + 1) * 4;
  const int cum = (2 * a.B + 1) * 4;
  cudaError_t e = set_up_kernel<paged_scores_kernel<T, D, TW, NT, CUT>>(kScores + kMostCum, true);
  if (e == cudaSuccess) e = set_up_kernel<paged_values_kernel<T, D, TW, NT, CUT, FOLD>>(kValues + kMostCum, true);
  if (e != cudaSuccess) return e;
  // teams for the runs that there can be, one for each head
  const int64_t heads = static_cast<int64_t>(a.Hkv) * a.own_rowblocks, blocks = static_cast<int64_t>(a.B) * (a.own_width / a.block);
  const int64_t runs = std::min<int64_t>(a.runs, blocks);
  const unsigned grid = static_cast<unsigned>((runs * heads + kWarps / TW - 1) / (kWarps / TW));
  e = launch_dependent(paged_scores_kernel<T, D, TW, NT, CUT>, grid, kThreads, kScores + cum, st, p);
  if (e != cudaSuccess) return e;   // the next kernel reads what this one leaves
  e = launch_dependent(paged_values_kernel<T, D, TW, NT, CUT, FOLD>, grid, kThreads, kValues + cum, st, p);
  if (e != cudaSuccess || !p.join) return e;
  return launch_dependent(paged_join_kernel<T, D>, static_cast<unsigned>(a.B) * a.Hq, kThreads, 0, st, a);
}
template <typename T, int D, int NT, bool FOLD>
cudaError_t go(const PagedDecodeArgs& p, cudaStream_t st) {
  if (p.a.team == kWarps) return p.cut ? go<T, D, kWarps, NT, FOLD, true>(p, st) : go<T, D, kWarps, NT, FOLD, false>(p, st);
  return p.cut ? go<T, D, 1, NT, FOLD, true>(p, st) : go<T, D, 1, NT, FOLD, false>(p, st);
}
template <typename T, int D>
cudaError_t go(const PagedDecodeArgs& p, cudaStream_t st) {
  return p.a.G > 8 ? go<T, D, 2, false>(p, st) : p.a.G > 4 ? go<T, D, 1, false>(p, st) : go<T, D, 1, true>(p, st);
}

}  // namespace

// The split: `runs` runs for every head, as many as teams that are resident at a time.  Where streams are few, and a warp
// would have few blocks, a run belongs to a CTA, whose warps' sums meet in shared memory: a row then has a quarter of the
// parts.  That is so up to half as many streams as CTAs, where each sequence can still be cut for itself and no CTA starts twice
// (a CTA's runs / a warp's, H32/8 D128, us: B16 C2048 15.1 / 15.4, B32 19.6 / 21.5, B36 21.1 / 22.2; B40, 320 streams for 608
// CTAs, 30.1 / 26.2, B50 31.0 / 27.7; fp32, 456 CTAs: B28 22.2 / 24.2, B32 31.9 / 28.9).  kFewBlocks of a warp: B32 C6144, 20 of
// them, 38.3 by CTAs and 38.2 by warps that are not cut, C10240, 34, 53.4 / 52.0.
// With a warp's runs too each sequence is cut for itself if that leaves enough of them and blocks are few (cut / not: B64 H32/8
// C512 17.2 / 21.5, C2048, 13 blocks a warp, 28.9 / 32.9, C6144, 40, 58.4 / 59.5; B128, 1024 streams: C512 24.6 / 26.6, C1536, 20,
// 46.5 / 41.1, C2048, 27, 57.1 / 46.2; B64 C16384, 108, 130.5 / 130.7).
// Rows of more than kMostJoined parts, when sequences are full, are joined by CTAs of their own: the team of the last part
// takes eight parts at a time (by it / by a kernel: B64 H8 C2048, 5 parts, 25.8 us / 28.4; B16 H32/8 C16384, 19 parts, 47.0 /
// 39.6; B2 H24/1 D64 C131072, 100 parts, 29.3 / 20.0).
constexpr int kMostJoined = 8;
constexpr int kMostCutStreams = 1024, kFewBlocks = 24;
size_t plan_decode_paged(PagedDecodeArgs* p, bool bf16, char* base) {
  DecodeArgs* a = &p->a;
  const int64_t rows = static_cast<int64_t>(a->B) * a->Hq;
  a->G = a->Hq / a->Hkv;
  a->block = kKeys;
  a->own_rowblocks = (a->G + kRows - 1) / kRows;
  const int own = (a->C + a->block - 1) / a->block;
  a->own_width = own * a->block;
  const int64_t heads = static_cast<int64_t>(a->Hkv) * a->own_rowblocks, streams = heads * a->B, blocks = static_cast<int64_t>(a->B) * own;
  if (streams * own > INT_MAX / 2) return 0;
  const int64_t ctas = kSms * resident(bf16, a->G > 8 ? 2 : 1);
  const bool few = streams * own < kFewBlocks * ctas * kWarps;
  a->team = streams < 64 || (2 * streams <= ctas && few) ? kWarps : 1;
  int64_t runs = (a->team == 1 ? ctas * kWarps : ctas) / heads;   // of each head
  p->cut = runs >= 2 * a->B && (a->team > 1 || (streams <= kMostCutStreams && few));
  a->runs = static_cast<int>(std::max<int64_t>(runs, 1));
  // the most parts of a sequence: as if a run had eight blocks a warp at most
  const int64_t even = blocks / a->runs, full = std::min<int64_t>(std::max<int64_t>(even, a->team), 8 * a->team);
  a->slots = static_cast<int>((own + full - 1) / full + 2);
  p->join = own > kMostJoined * std::max<int64_t>(even, a->team);   // a full sequence's parts
  // whole lines, since scores are discarded by the line: up to a line of the workspace in front, too
  size_t at = static_cast<size_t>(-reinterpret_cast<intptr_t>(base)) & 127;
  auto piece = [&](int64_t floats) {
    char* q = base + at;
    at += (static_cast<size_t>(floats) * 4 + 255) & ~static_cast<size_t>(255);
    return q;
  };
  a->s_own = reinterpret_cast<float*>(piece(rows * a->own_width));
  a->s_pre = nullptr;
  a->row_max = reinterpret_cast<float*>(piece(rows * a->slots));
  a->part_sum = reinterpret_cast<float*>(piece(rows * a->slots));
  a->part_o = reinterpret_cast<float*>(piece(rows * a->slots * a->D));
  a->cum = reinterpret_cast<int*>(piece(a->B + 2));
  p->unit = reinterpret_cast<float*>(piece(rows));
  p->done = reinterpret_cast<int*>(piece(streams));
  return base ? at : at + 128;
}

cudaError_t launch_decode_paged(const PagedDecodeArgs& p, bool bf16, cudaStream_t st) {
  if (bf16) return p.a.D == 64 ? go<__nv_bfloat16, 64>(p, st) : go<__nv_bfloat16, 128>(p, st);
  return p.a.D == 64 ? go<float, 64>(p, st) : go<float, 128>(p, st);
}

}  // namespace raattn
