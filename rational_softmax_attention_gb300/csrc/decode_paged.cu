// Attention of one query token per sequence against a cache whose keys and values lie in pages, in 4 bits
// (paged.cuh): ra_attention_decode's mathematics on khat = lo + s u, vhat = lo + s u.
//
//   z_j = sum_g s_jg (sum_{d in g} q_d u_jd) + lo_jg (sum_{d in g} q_d)
//   phi_j as in decode.cu;  o_d = [sum_j (phi_j s_jg) u_jd + sum_j phi_j lo_jg] / sum_j phi_j,  g the group of d
//
// so the products run on the codes themselves and a scale is applied once per key and group (scores) or once per
// weight and group (values).  A code is an fp16 subnormal as it stands: the bits 0000 0000 0000 uuuu are u 2^-24, and four
// bits further left 16 u 2^-24, exactly.  So a mask makes an operand out of two codes: five integer instructions for
// eight codes, no conversion.  The factors 16 and 2^-24 are powers of two and go into the query (scores) and the end
// (values).  The tensor cores align products by their operands' exponent fields, so a subnormal's leading zeros cost
// up to six of the sum's 24 bits: nothing beside bf16's eight.  fp32 calls make normal numbers of the codes (1024 + u in fp16, minus
// 1024), and add the products of each block of keys to fp32 sums: the tensor cores truncate theirs.
//   scores   m16n8k16: sixteen keys as M, eight query heads as N.  The query goes in as fp16 times a power of two of
//            its row (11 bits, bf16's 8 exactly, down to 2^-28 of the largest); fp32 queries as two fp16 (22 bits).
//   values   m16n8k16: sixteen dimensions as M, eight heads as N, sixteen keys as K; two keys' words are put together
//            by byte.  phi s goes in as fp16 times a power of two that follows the largest scale met so far (11 bits: 2^-11 of a weight
//            at most, an eighth of what the output's rounding to bf16 costs, and the weights' errors differ); fp32 as two fp16.
// Three launches, as in decode.cu, whose split, join and partial results these kernels share.  The scores of sixteen
// keys stand in the workspace as the value products want them: key t at 4 (t % 4) + t / 4.
#include <climits>
#include <cuda_fp16.h>

#include "decode_parts.cuh"
#include "paged.cuh"

namespace raattn {
namespace {

using namespace decode;
using namespace paged;

constexpr int kCtasPerSm = 5, kCtas = kSms * kCtasPerSm;
constexpr int kKeys = 32;                        // of a block: two products' M, or K
constexpr uint32_t kLow = 0x000f000fu, kHigh = 0x00f000f0u;

template <int D>
struct Cfg {
  static constexpr int G = D / kGroup;
  static constexpr int kCodes = kKeys * D / 2;            // bytes of a block's codes
  static constexpr int kMeta = 4 * G;                     // bytes of a key's scales and minima
  static constexpr int kBlock = kKeys * row_bytes(D);
  static constexpr int kStagesK = 4, kStagesV = 3;
};
// CTAs of an SM that the registers have to leave room for: two fp16 for each weight or sixteen rows take more.
template <typename T, int NT>
__host__ __device__ constexpr int resident() { return sizeof(T) == 2 && NT == 1 ? kCtasPerSm : 3; }
// A stage of the values: the block, then eight or sixteen rows of scores.
template <int D, int NT>
__host__ __device__ constexpr int stage_values() { return Cfg<D>::kBlock + 8 * NT * kKeys * 4; }

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t u;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(u) : "r"(addr));
  return u;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 u;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(u.x), "=r"(u.y) : "r"(addr));
  return u;
}
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

// Two codes as an operand: the fp16 of them times 2^-24 or, with TWO, themselves.
template <bool TWO>
__device__ __forceinline__ uint32_t codes2(uint32_t word, uint32_t mask) {
  if constexpr (!TWO) return word & mask;
  const uint32_t u = (word & mask) | 0x64006400u;
  const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&u), __float2half2_rn(1024.0f));
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <typename T>
__host__ __device__ constexpr float code_unit() { return sizeof(T) == 4 ? 1.0f : 0x1p-24f; }

// A key's scales and minima: (s, lo) of one group, or (s0, s1), (lo0, lo1) of two.
template <int G>
struct Meta {
  float s[G], lo[G];
  __device__ __forceinline__ explicit Meta(uint32_t addr) {
    if constexpr (G == 2) {
      const uint2 u = lds64(addr);
      s[0] = bf16_low(u.x);
      s[1] = bf16_high(u.x);
      lo[0] = bf16_low(u.y);
      lo[1] = bf16_high(u.y);
    } else {
      const uint32_t u = lds32(addr);
      s[0] = bf16_low(u);
      lo[0] = bf16_high(u);
    }
  }
};

// ---------------------------------------------------------------------------------------------
// a warp's blocks into its ring
// ---------------------------------------------------------------------------------------------
__device__ __forceinline__ void copy16_part(uint32_t dst, const void* src, int bytes) {   // zeros behind `bytes`
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// Blocks first, first + step, .. of a part.  A page is at least sixteen keys, so a block's halves lie in a page
// each: lane l holds the page of half l % 2 of block i0 + l / 2, and those of the next sixteen blocks are on
// their way.  What no page holds and what lies behind the last key arrives as zeros: scales and minima of 0.
template <int D>
struct Fetch {
  static constexpr int kLanesPerKey = D / 32;        // 16-byte chunks of a key's codes
  static constexpr int kKeysPerCopy = 32 / kLanesPerKey;
  static constexpr int kCopies = kKeys / kKeysPerCopy;
  static constexpr int kMetaLanes = kKeys * Cfg<D>::kMeta / 16, kKeysPerChunk = 16 / Cfg<D>::kMeta;
  const PagePool& pool;
  const int32_t* row;
  const uint8_t* base;
  int first, step, blocks, keys, lane;
  int now, next;

  __device__ __forceinline__ Fetch(const PagedDecodeArgs& p, const Part& part, int which, int warp, int warps, int blocks_)
      : pool(p.pool), row(p.table + static_cast<int64_t>(part.b) * p.M), base(part_of(p.pool, 0, part.kv, which)),
        first((part.first + warp) * kKeys), step(warps * kKeys), blocks(blocks_), keys(part.keys), lane(threadIdx.x & 31) {
    now = pages(0);
    next = pages(16);
  }
  __device__ __forceinline__ int pages(int i0) const {
    const int i = i0 + (lane >> 1), key = first + i * step + (lane & 1) * 16;
    return i < blocks && key < keys ? page_at(pool, row, key >> pool.shift) : -1;
  }
  __device__ __forceinline__ void operator()(uint32_t stage, int i) {
    if ((i & 15) == 0 && i) {
      now = next;
      next = pages(i + 16);
    }
    const int key0 = first + i * step, mask = pool.page - 1;
    const uint8_t* src[2];
    int slot[2], left[2];   // the half's first slot in its page; keys of it that there are
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int id = __shfl_sync(0xffffffffu, now, 2 * (i & 15) + h);
      src[h] = base + max(id, 0) * pool.page_stride;
      slot[h] = (key0 + 16 * h) & mask;
      left[h] = id < 0 ? 0 : keys - key0 - 16 * h;
    }
#pragma unroll
    for (int c = 0; c < kCopies; ++c) {
      constexpr int kPerHalf = kCopies / 2;
      const int h = c / kPerHalf, key = c % kPerHalf * kKeysPerCopy + lane / kLanesPerKey;
      copy16_part(stage + (c * 32 + lane) * 16, src[h] + slot[h] * (D / 2) + (c % kPerHalf * 32 + lane) * 16,
                  key < left[h] ? 16 : 0);
    }
    if (lane < kMetaLanes) {
      const int h = lane >= kMetaLanes / 2, key = (lane - h * (kMetaLanes / 2)) * kKeysPerChunk;
      const int bytes = min(max(((h ? left[1] : left[0]) - key) * Cfg<D>::kMeta, 0), 16);
      copy16_part(stage + Cfg<D>::kCodes + lane * 16,
                  (h ? src[1] : src[0]) + pool.page * (D / 2) + ((h ? slot[1] : slot[0]) + key) * Cfg<D>::kMeta, bytes);
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
  float sum[NT][G][2], unit[NT][2];   // of query rows 2 j, 2 j + 1: their sums over a group, and a score's unit

  __device__ __forceinline__ Query(const Part& p, const DecodeArgs& a) {
    const int lane = threadIdx.x & 31, r = lane >> 2, j = lane & 3;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const T* q = static_cast<const T*>(a.q) + static_cast<int64_t>(row_of(p, t * 8 + r, a)) * D + 16 * j;
      float x[G][16], most = 0.0f;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        load(q + g * kGroup, x[g]);
#pragma unroll
        for (int i = 0; i < 16; ++i) most = fmaxf(most, fabsf(x[g][i]));
      }
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
      const int e = max(static_cast<int>(__float_as_uint(most) >> 23) - 126, -100);   // most < 2^e
      const float to = power_of_2(14 - e), of = power_of_2(e - 14 + (TWO ? 0 : 24));
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
        unit[t][c] = __shfl_sync(0xffffffffu, of, from);
#pragma unroll
        for (int g = 0; g < G; ++g) sum[t][g][c] = __shfl_sync(0xffffffffu, total[g], from) * code_unit<T>();
      }
    }
  }
  static __device__ __forceinline__ void load(const __nv_bfloat16* q, float (&x)[16]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 u = reinterpret_cast<const uint4*>(q)[i];
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        x[8 * i + 2 * k] = bf16_low(w[k]);
        x[8 * i + 2 * k + 1] = bf16_high(w[k]);
      }
    }
  }
  static __device__ __forceinline__ void load(const float* q, float (&x)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 u = reinterpret_cast<const float4*>(q)[i];
      x[4 * i] = u.x;
      x[4 * i + 1] = u.y;
      x[4 * i + 2] = u.z;
      x[4 * i + 3] = u.w;
    }
  }
};

template <typename T, int D, int TW, int NT>
__device__ __forceinline__ void part_scores(const Part& p, const PagedDecodeArgs& pa, uint32_t ring, float* best_s) {
  using C = Cfg<D>;
  constexpr int G = C::G;
  constexpr bool TWO = sizeof(T) == 4;
  const DecodeArgs& a = pa.a;
  const int lane = threadIdx.x & 31, r = lane >> 2, j = lane & 3;
  const int mine = blocks_of_warp<TW>(p);
  Fetch<D> fetch(pa, p, 0, warp_of_team<TW>(), TW, mine);
#pragma unroll
  for (int i = 0; i < C::kStagesK - 1; ++i) {
    if (i < mine) fetch(ring + i * C::kBlock, i);
    copy_commit();
  }
  const Query<T, D, NT> q(p, a);
  const int first = (p.first + warp_of_team<TW>()) * kKeys, at = (r & 3) * 4 + (r >> 2);
  float* out[NT][2];
  float best[NT][2];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      out[t][c] = score_row(p, row_of(p, t * 8 + 2 * j + c, a), a) + at;
      best[t][c] = -kInf;
    }
  // this lane's 16 bytes (D = 128) or 8 of key r: the halves' order depends on the key's bit 1, which is r's
  const int chunk = r * (D / 2) + (G == 2 ? (16 * j) ^ ((r & 2) << 4) : 8 * j), meta = C::kCodes + r * C::kMeta;
  for (int i = 0; i < mine; ++i) {
    copy_wait<C::kStagesK - 2>();
    __syncwarp();   // block i has landed for all lanes, and all have read block i - 1
    const int ahead = i + C::kStagesK - 1;
    if (ahead < mine) fetch(ring + ahead % C::kStagesK * C::kBlock, ahead);
    copy_commit();
    const uint32_t stage = ring + i % C::kStagesK * C::kBlock;
    const int key0 = first + i * (TW * kKeys);
#pragma unroll
    for (int tile = 0; tile < kKeys / 16; ++tile) {
      uint32_t x[2][G][2];   // keys r, r + 8; words 2 j, 2 j + 1 of the groups
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t src = stage + chunk + (tile * 16 + h * 8) * (D / 2);
        if constexpr (G == 2) {
          const uint4 u = lds128(src);
          x[h][0][0] = u.x;
          x[h][1][0] = u.y;
          x[h][0][1] = u.z;
          x[h][1][1] = u.w;
        } else {
          const uint2 u = lds64(src);
          x[h][0][0] = u.x;
          x[h][0][1] = u.y;
        }
      }
      const Meta<G> m0(stage + meta + tile * 16 * C::kMeta), m1(stage + meta + (tile * 16 + 8) * C::kMeta);
      float z[NT][4];
#pragma unroll
      for (int g = 0; g < G; ++g) {
        float acc[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.0f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t u = x[0][g][k >> 1] >> (k & 1) * 8, v = x[1][g][k >> 1] >> (k & 1) * 8;
          const uint32_t a0 = codes2<TWO>(u, kLow), a1 = codes2<TWO>(v, kLow), a2 = codes2<TWO>(u, kHigh),
                         a3 = codes2<TWO>(v, kHigh);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            mma_f16(acc[t], a0, a1, a2, a3, q.b[t][g][k][0], q.b[t][g][k][1]);
            if constexpr (TWO) mma_f16(acc[t], a0, a1, a2, a3, q.rest[t][g][k][0], q.rest[t][g][k][1]);
          }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float lo = e < 2 ? m0.lo[g] : m1.lo[g], s = e < 2 ? m0.s[g] : m1.s[g], w = q.sum[t][g][e & 1];
            z[t][e] = g ? fmaf(s, acc[t][e], fmaf(lo, w, z[t][e])) : fmaf(s, acc[t][e], lo * w);
          }
      }
      const int key = key0 + tile * 16;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int c = e & 1, h = e >> 1;
          const float s = key + r + 8 * h < p.keys ? z[t][e] * q.unit[t][c] : -kInf;
          best[t][c] = fmaxf(best[t][c], s);
          if (t * 8 + 2 * j + c < p.rows) out[t][c][key + 2 * h] = s;
        }
    }
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

template <typename T, int D, int TW, int NT>
__global__ void __launch_bounds__(kThreads, resident<T, NT>()) paged_scores_kernel(const PagedDecodeArgs pa) {
  extern __shared__ uint4 dyn[];
  constexpr int kRing = Cfg<D>::kStagesK * Cfg<D>::kBlock;
  const DecodeArgs& a = pa.a;
  int* cum = reinterpret_cast<int*>(reinterpret_cast<char*>(dyn) + kWarps * kRing);
  __shared__ float best[kWarps * kRows];
  const int warp = threadIdx.x >> 5, team = warp / TW, tt = threadIdx.x % (32 * TW);
  release_dependents();   // the next kernel's first values are on their way while this one ends
  int longest;
  const Split s = make_split<kKeys>(cum, a, &longest);
  if (blockIdx.x == 0) {   // for the join
    for (int b = threadIdx.x; b <= a.B; b += kThreads) a.cum[b] = cum[b];
    if (threadIdx.x == 0) a.cum[a.B + 1] = longest;
  }
  each_part<TW>(team, cum, s, a, [&](const Part& p) {
    part_scores<T, D, TW, NT>(p, pa, smem_u32(dyn) + warp * kRing, best);
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
// phi of four scores, from their distances to the maximum: w = (1 + u) / 2 by a saturating FMA, so that -inf gives
// w = 1; q = 1 / w - 1 with one reciprocal for two (phi.cuh).
__device__ __forceinline__ void phi4(const float4& z, float m, float c2, float (&f)[4]) {
  const float2 A = make_float2(fma_sat(m - z.x, c2, 0.5f), fma_sat(m - z.y, c2, 0.5f));
  const float2 B = make_float2(fma_sat(m - z.z, c2, 0.5f), fma_sat(m - z.w, c2, 0.5f));
  const float2 P = __fmul2_rn(A, B);
  const float2 R = make_float2(rcp_approx(P.x), rcp_approx(P.y)), minus1 = make_float2(-1.0f, -1.0f);
  float2 x = __ffma2_rn(R, B, minus1), y = __ffma2_rn(R, A, minus1);
  x = __fmul2_rn(x, x);
  y = __fmul2_rn(y, y);
  x = __fmul2_rn(x, x);
  y = __fmul2_rn(y, y);
  x = __fmul2_rn(x, x);
  y = __fmul2_rn(y, y);
  f[0] = x.x;
  f[1] = x.y;
  f[2] = y.x;
  f[3] = y.y;
}

// Where piece c (four keys) of row r's scores stands: the reads of eight lanes (two rows by four pieces) meet no
// bank conflict.
__device__ __forceinline__ int piece_of(int r, int c) { return c ^ ((r & 1) << 2); }

// Lane (r, j) reads, of keys j, j + 4, j + 8 and j + 12 of sixteen, word r of every group (dimensions 8 r .. 8 r + 7):
// rows r and r + 8 of the A operand of product n stand for dimensions 8 r + 2 n and 8 r + 2 n + 1, the latter sixteen times as
// large.  The weights of query row r at the same keys are the B operand.
template <typename T, int D, int TW, int NT>
__device__ __forceinline__ void part_values(const Part& p, const PagedDecodeArgs& pa, const Split& s, const int* cum,
                                            uint32_t ring, char* ring_ptr, float* rowm, float* sums) {
  using C = Cfg<D>;
  constexpr int G = C::G, kStage = stage_values<D, NT>(), S = C::kStagesV;
  constexpr bool TWO = sizeof(T) == 4;
  const DecodeArgs& a = pa.a;
  const int lane = threadIdx.x & 31, r = lane >> 2, j = lane & 3;
  const int mine = blocks_of_warp<TW>(p), first = (p.first + warp_of_team<TW>()) * kKeys;
  Fetch<D> fetch(pa, p, 1, warp_of_team<TW>(), TW, mine);
  const float* score[2 * NT];   // lane's piece of rows lane / 8 + 4 i
#pragma unroll
  for (int i = 0; i < 2 * NT; ++i) score[i] = score_row(p, row_of(p, (lane >> 3) + 4 * i, a), a) + first + (lane & 7) * 4;
  auto fetch_scores = [&](uint32_t stage, int i) {
#pragma unroll
    for (int k = 0; k < 2 * NT; ++k) {
      const int row = (lane >> 3) + 4 * k;
      if (row < p.rows)
        copy16_part(stage + C::kBlock + (row * 8 + piece_of(row, lane & 7)) * 16, score[k] + i * (TW * kKeys), 16);
    }
  };
  // the first blocks of a part do not wait for the scores
#pragma unroll
  for (int i = 0; i < S - 1; ++i)
    if (i < mine) fetch(ring + i * kStage, i);
  await_previous();
#pragma unroll
  for (int i = 0; i < S - 1; ++i) {
    if (i < mine) fetch_scores(ring + i * kStage, i);
    copy_commit();
  }
  part_maxima<TW>(rowm, p, cum, s, a);
  team_sync<TW>();
  float m[NT], total[NT], low[NT][G], acc[NT][G][4][4];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    m[t] = rowm[t * 8 + r];
    if (m[t] == -kInf) m[t] = 0.0f;
    total[t] = 0.0f;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      low[t][g] = 0.0f;
#pragma unroll
      for (int n = 0; n < 4; ++n) acc[t][g][n][0] = acc[t][g][n][1] = acc[t][g][n][2] = acc[t][g][n][3] = 0.0f;
    }
  }
  const float c2 = a.scale * 0.03125f;
  int exponent = -100;   // every scale met so far is below 2^exponent
  float unit = power_of_2(14 - exponent);
  const int word = word_offset<G>(0, r, j);   // the halves' order: bit 1 of the key's slot is j's
  for (int i = 0; i < mine; ++i) {
    copy_wait<S - 2>();
    __syncwarp();
    const int ahead = i + S - 1;
    if (ahead < mine) {
      fetch(ring + ahead % S * kStage, ahead);
      fetch_scores(ring + ahead % S * kStage, ahead);
    }
    copy_commit();
    const uint32_t stage = ring + i % S * kStage;
    {   // bits of bf16 scales, which are not negative, are in their order
      const uint32_t w = lds32(stage + C::kCodes + lane * C::kMeta);
      const uint32_t most = __reduce_max_sync(0xffffffffu, G == 2 ? max(w & 0xffffu, w >> 16) : w & 0xffffu);
      const int e = static_cast<int>(most >> 7) - 126;
      if (e > exponent) {
        const float f = power_of_2(exponent - e);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int g = 0; g < G; ++g)
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
              for (int k = 0; k < 4; ++k) acc[t][g][n][k] *= f;
        exponent = e;
        unit = power_of_2(14 - e);
      }
    }
#pragma unroll
    for (int tile = 0; tile < kKeys / 16; ++tile) {
      float f[NT][4];
      bool live = false;   // some weight that is not 0 (a NaN is not)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if (t * 8 + r < p.rows) {
          const uint4 u = lds128(stage + C::kBlock + ((t * 8 + r) * 8 + piece_of(r, tile * 4 + j)) * 16);
          const float4 z = make_float4(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w));
          if constexpr (TWO) {
            f[t][0] = phi_exact((m[t] - z.x) * a.scale);
            f[t][1] = phi_exact((m[t] - z.y) * a.scale);
            f[t][2] = phi_exact((m[t] - z.z) * a.scale);
            f[t][3] = phi_exact((m[t] - z.w) * a.scale);
          } else {
            phi4(z, m[t], c2, f[t]);
          }
        } else {
          f[t][0] = f[t][1] = f[t][2] = f[t][3] = 0.0f;
        }
        const float all = (f[t][0] + f[t][1]) + (f[t][2] + f[t][3]);
        total[t] += all;
        live |= all != 0.0f;
      }
      if (!__any_sync(0xffffffffu, live)) continue;
      uint32_t x[4][G];
      float weight[NT][G][4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int key = tile * 16 + j + 4 * k;
        const uint32_t src = stage + key * (D / 2) + word;
        if constexpr (G == 2) {
          const uint2 u = lds64(src);
          x[k][0] = u.x;
          x[k][1] = u.y;
        } else {
          x[k][0] = lds32(src);
        }
        const Meta<G> meta(stage + C::kCodes + key * C::kMeta);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const float fu = f[t][k] * unit;
#pragma unroll
          for (int g = 0; g < G; ++g) {
            weight[t][g][k] = fu * meta.s[g];
            low[t][g] = fmaf(f[t][k], meta.lo[g], low[t][g]);
          }
        }
      }
#pragma unroll
      for (int g = 0; g < G; ++g) {
        uint32_t b[NT][2], rest[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          split_half2<TWO>(weight[t][g][0], weight[t][g][1], b[t][0], rest[t][0]);
          split_half2<TWO>(weight[t][g][2], weight[t][g][3], b[t][1], rest[t][1]);
        }
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const uint32_t sel = n < 2 ? 0x5410u : 0x7632u;
          const uint32_t u = __byte_perm(x[0][g], x[1][g], sel) >> (n & 1) * 8;
          const uint32_t v = __byte_perm(x[2][g], x[3][g], sel) >> (n & 1) * 8;
          const uint32_t a0 = codes2<TWO>(u, kLow), a1 = codes2<TWO>(u, kHigh), a2 = codes2<TWO>(v, kLow),
                         a3 = codes2<TWO>(v, kHigh);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            if constexpr (TWO) {
              float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
              mma_f16(c, a0, a1, a2, a3, rest[t][0], rest[t][1]);
              mma_f16(c, a0, a1, a2, a3, b[t][0], b[t][1]);
#pragma unroll
              for (int k = 0; k < 4; ++k) acc[t][g][n][k] += c[k];
            } else {
              mma_f16(acc[t][g][n], a0, a1, a2, a3, b[t][0], b[t][1]);
            }
          }
        }
      }
    }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      total[t] += __shfl_xor_sync(0xffffffffu, total[t], o);
#pragma unroll
      for (int g = 0; g < G; ++g) low[t][g] += __shfl_xor_sync(0xffffffffu, low[t][g], o);
    }
    if (j == 0) sums[(threadIdx.x >> 5) * kRows + t * 8 + r] = total[t];
  }
  __syncwarp();   // this warp's blocks have been read: its sums into their place
  float* out = reinterpret_cast<float*>(ring_ptr);
  const float back = power_of_2(exponent), undo = 0x1p-14f / code_unit<T>();
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int row = t * 8 + 2 * j + c;
        const float lo = __shfl_sync(0xffffffffu, low[t][g], 8 * j + 4 * c);
        float y[8];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          y[2 * n] = fmaf(acc[t][g][n][c] * undo, back, lo);
          y[2 * n + 1] = fmaf(acc[t][g][n][2 + c] * (undo * 0.0625f), back, lo);
        }
        if (row < p.rows) {
          float4* o = reinterpret_cast<float4*>(out + row * D + g * kGroup + r * 8);
          o[0] = make_float4(y[0], y[1], y[2], y[3]);
          o[1] = make_float4(y[4], y[5], y[6], y[7]);
        }
      }
}

template <typename T, int D, int TW, int NT>
__global__ void __launch_bounds__(kThreads, resident<T, NT>()) paged_values_kernel(const PagedDecodeArgs pa) {
  extern __shared__ uint4 dyn[];
  constexpr int kRing = Cfg<D>::kStagesV * stage_values<D, NT>();
  static_assert(kRing >= 8 * NT * D * 4, "a warp's partial sums fit its ring");
  const DecodeArgs& a = pa.a;
  int* cum = reinterpret_cast<int*>(reinterpret_cast<char*>(dyn) + kWarps * kRing);
  __shared__ float rowm_s[kWarps / TW * kRows], sums[kWarps * kRows];
  const int warp = threadIdx.x >> 5, team = warp / TW, tt = threadIdx.x % (32 * TW);
  char* ring = reinterpret_cast<char*>(dyn) + warp * kRing;
  const char* rings = reinterpret_cast<const char*>(dyn) + team * TW * kRing;   // the team's
  int longest;
  const Split s = make_split<kKeys>(cum, a, &longest);
  each_part<TW>(team, cum, s, a, [&](const Part& p) {
    part_values<T, D, TW, NT>(p, pa, s, cum, smem_u32(ring), ring, rowm_s + team * kRows, sums);
    team_sync<TW>();
    if (tt < p.rows) {
      float f = sums[team * TW * kRows + tt];
#pragma unroll
      for (int w = 1; w < TW; ++w) f += sums[(team * TW + w) * kRows + tt];
      a.part_sum[static_cast<int64_t>(row_of(p, tt, a)) * a.slots + p.slot] = f;
    }
    for (int e = tt; e < p.rows * (D / 4); e += 32 * TW) {
      const int row = e / (D / 4), c = e % (D / 4);
      float4 f = reinterpret_cast<const float4*>(rings)[e];
#pragma unroll
      for (int w = 1; w < TW; ++w) {
        const float4 x = *reinterpret_cast<const float4*>(rings + w * kRing + e * 16);
        f.x += x.x;
        f.y += x.y;
        f.z += x.z;
        f.w += x.w;
      }
      reinterpret_cast<float4*>(a.part_o + (static_cast<int64_t>(row_of(p, row, a)) * a.slots + p.slot) * D)[c] = f;
    }
    team_sync<TW>();
  });
  release_dependents();
  // Whoever awaits this kernel awaits the scores too: a CTA without a part sees to it.
  if (blockIdx.x == gridDim.x - 1) await_previous();
}

template <typename T, int D, int TW, int NT>
cudaError_t go(const PagedDecodeArgs& p, cudaStream_t st) {
  const DecodeArgs& a = p.a;
  constexpr int kScores = kWarps * Cfg<D>::kStagesK * Cfg<D>::kBlock;
  constexpr int kValues = kWarps * Cfg<D>::kStagesV * stage_values<D, NT>();
  constexpr int kMostCum = (2 * kDecodeMaxBatch + 1) * 4;
  const int cum = (2 * a.B + 1) * 4;
  cudaError_t e = set_up_kernel<paged_scores_kernel<T, D, TW, NT>>(kScores + kMostCum, true);
  if (e == cudaSuccess) e = set_up_kernel<paged_values_kernel<T, D, TW, NT>>(kValues + kMostCum, true);
  if (e != cudaSuccess) return e;
  // CTAs for the runs that there can be
  const int64_t streams = static_cast<int64_t>(a.B) * a.Hkv * a.own_rowblocks, own = a.own_width / a.block;
  const int64_t ctas = TW == 1 ? streams * own : streams * ((own + TW - 1) / TW);
  const int grid = static_cast<int>(ctas < kCtas ? ctas : kCtas);
  paged_scores_kernel<T, D, TW, NT><<<grid, kThreads, kScores + cum, st>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;   // the next kernels read what this one leaves
  e = launch_dependent(paged_values_kernel<T, D, TW, NT>, grid, kThreads, kValues + cum, st, p);
  if (e != cudaSuccess) return e;
  return launch_decode_join(a, sizeof(T) == 2, st);
}
template <typename T, int D>
cudaError_t go(const PagedDecodeArgs& p, cudaStream_t st) {
  if (p.a.G > 8) return p.a.team == kWarps ? go<T, D, kWarps, 2>(p, st) : go<T, D, 1, 2>(p, st);
  return p.a.team == kWarps ? go<T, D, kWarps, 1>(p, st) : go<T, D, 1, 1>(p, st);
}

}  // namespace

// The split of decode.cu without shared keys: equal runs, one per warp, with many streams; one per CTA, each stream
// for itself, with few.
size_t plan_decode_paged(PagedDecodeArgs* p, char* base) {
  DecodeArgs* a = &p->a;
  const int64_t rows = static_cast<int64_t>(a->B) * a->Hq;
  a->G = a->Hq / a->Hkv;
  a->block = kKeys;
  a->own_rowblocks = (a->G + kRows - 1) / kRows;
  a->shared_rowblocks = 1;
  const int own = (a->C + kKeys - 1) / kKeys;
  a->own_width = own * kKeys;
  a->tc = a->pblocks = a->pre_width = a->pchunk = a->pslots = 0;
  const int64_t streams = static_cast<int64_t>(a->B) * a->Hkv * a->own_rowblocks, total = streams * own;
  if (total > INT_MAX / 2) return 0;
  a->team = streams < 64 || (streams <= 128 && total < 10 * kCtas * kWarps) ? kWarps : 1;
  a->runs = a->team == 1 ? kCtas * kWarps : kCtas - static_cast<int>(streams);
  const int64_t even = total / a->runs;
  const int64_t full = even < a->team ? a->team : even > 8 * a->team ? 8 * a->team : even;
  a->slots = static_cast<int>((own + full - 1) / full + 1);
  a->least = 1;
  size_t at = 0;
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
  return at;
}

cudaError_t launch_decode_paged(const PagedDecodeArgs& p, bool bf16, cudaStream_t st) {
  if (bf16) return p.a.D == 64 ? go<__nv_bfloat16, 64>(p, st) : go<__nv_bfloat16, 128>(p, st);
  return p.a.D == 64 ? go<float, 64>(p, st) : go<float, 128>(p, st);
}

}  // namespace raattn
