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
//   scores   the keys are read once; scores go to the workspace in fp32 (4 bytes per query head
//            against the key's 2 D), with each item's maximum;
//   values   phi from the scores and the final maximum; the values are read once, and not at
//            all where every phi of a block is 0; partial sums (fp32) per item.  Sums need no
//            rescaling: all items share one maximum;
//   join     adds an output row's partial sums in a fixed order, and the weights.
// An item is a range of keys for a block of up to 16 query rows that share them: the query
// heads of a key head (own keys), or the whole batch's rows of a key head (shared keys).
// Every CTA forms the list of items from the lengths by itself: no host copy of them is needed,
// and a cache much larger than what it holds costs nothing.
//
// Bound: HBM, K and V once.  bf16: m16n8k16 products with rows as M; K fragments come
// straight from global memory (a lane's 16-byte vector is the operand of two products, the
// query's dimensions permuted alike), V fragments by interleaving two keys' vectors, so
// neither passes through shared memory.  fp32: FFMA.
#include "kernels.cuh"

namespace raattn {
namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;
constexpr int kRows = 16;        // query rows of an item
constexpr int kBlock = 32;       // keys a warp takes at a time; score rows are padded to whole blocks
constexpr float kInf = __builtin_huge_valf();

__device__ __forceinline__ float phi_fast(float d) {   // bf16 inputs: 2 ulp reciprocal, exact 1 at d = 0
  const float q = fmaxf(16.0f - d, 0.0f) * rcp_approx(16.0f + d);
  const float q2 = q * q, q4 = q2 * q2;
  return q4 * q4;
}
__device__ __forceinline__ float phi_exact(float d) {        // fp32 inputs: IEEE division
  const float q = d < 16.0f ? (16.0f - d) / (16.0f + d) : 0.0f;
  const float q2 = q * q, q4 = q2 * q2;
  return q4 * q4;
}
template <typename T>
__device__ __forceinline__ float phi_t(float d) {
  return sizeof(T) == 2 ? phi_fast(d) : phi_exact(d);
}

struct Item {
  int first, last;      // keys [first, last)
  int slot;             // its place among a row's partial results
  int kv;               // key head
  int b;                // sequence, or -1: shared keys
  int row0, rows;       // rows of the block: within the head's G (own) or the batch's B G (shared)
};

// cum[b] = own chunks of the sequences before b, for b <= B.  All threads.
__device__ void count_chunks(int* cum, const DecodeArgs& a) {
  __shared__ int sums[kWarps];
  const int per = (a.B + kThreads - 1) / kThreads, b0 = threadIdx.x * per;
  int mine = 0;
  for (int i = 0; i < per && b0 + i < a.B; ++i) mine += (decode_own_length(a, b0 + i) + a.chunk - 1) / a.chunk;
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
  for (int i = 0; i < per && b0 + i < a.B; ++i) {
    cum[b0 + i] = run;
    run += (decode_own_length(a, b0 + i) + a.chunk - 1) / a.chunk;
  }
  if (b0 < a.B && b0 + per >= a.B) cum[a.B] = run;
  __syncthreads();
}

// Row blocks of the shared keys' items: none where the tensor cores take them.
__device__ __forceinline__ int shared_blocks(const DecodeArgs& a) { return a.tc ? 0 : (a.B * a.G + kRows - 1) / kRows; }

__device__ __forceinline__ int64_t item_count(const int* cum, const DecodeArgs& a) {
  return static_cast<int64_t>(a.Hkv) * a.pchunks * shared_blocks(a) + static_cast<int64_t>(cum[a.B]) * a.Hkv * ((a.G + kRows - 1) / kRows);
}

// Item i: the shared keys' items first (a key range's row blocks together, so that they find it
// in L2), then the sequences' in order.
__device__ __forceinline__ Item get_item(int64_t i, const int* cum, const DecodeArgs& a) {
  Item it;
  const int blocks = shared_blocks(a);
  const int64_t shared = static_cast<int64_t>(a.Hkv) * a.pchunks * blocks;
  if (i < shared) {
    const int rb = static_cast<int>(i % blocks), rest = static_cast<int>(i / blocks);
    it.b = -1;
    it.kv = rest % a.Hkv;
    it.slot = rest / a.Hkv;
    it.first = it.slot * a.pchunk;
    it.last = min(it.first + a.pchunk, a.P);
    it.row0 = rb * kRows;
    it.rows = min(a.B * a.G - it.row0, kRows);
    return it;
  }
  i -= shared;
  const int own_blocks = (a.G + kRows - 1) / kRows;
  const int rb = static_cast<int>(i % own_blocks);
  i /= own_blocks;
  it.kv = static_cast<int>(i % a.Hkv);
  const int c = static_cast<int>(i / a.Hkv);
  int lo = 0, hi = a.B - 1;   // the last b with cum[b] <= c
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cum[mid] <= c) lo = mid; else hi = mid - 1;
  }
  it.b = lo;
  const int k = c - cum[lo];
  it.slot = a.pchunks + k;
  it.first = k * a.chunk;
  it.last = min(it.first + a.chunk, decode_own_length(a, lo));
  it.row0 = rb * kRows;
  it.rows = min(a.G - it.row0, kRows);
  return it;
}

// Row r of an item as an index into [B, H_q].
__device__ __forceinline__ int row_of(const Item& it, int r, const DecodeArgs& a) {
  const int x = it.row0 + r;
  if (it.b >= 0) return it.b * a.Hq + it.kv * a.G + x;
  return x / a.G * a.Hq + it.kv * a.G + x % a.G;
}
__device__ __forceinline__ float* score_row(const Item& it, int row, const DecodeArgs& a) {
  return it.b >= 0 ? a.s_own + static_cast<int64_t>(row) * a.own_width
                   : a.s_pre + static_cast<int64_t>(row) * a.pre_width;
}
template <typename T>
__device__ __forceinline__ const T* keys_of(const Item& it, const void* own, const void* pre, const DecodeArgs& a) {
  return it.b >= 0 ? static_cast<const T*>(own) + (static_cast<int64_t>(it.b) * a.Hkv + it.kv) * a.C * a.D
                   : static_cast<const T*>(pre) + static_cast<int64_t>(it.kv) * a.P * a.D;
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 load_stream(const void* p) {   // read once: past L1
  uint4 u;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
               : "l"(p));
  return u;
}

// ---------------------------------------------------------------------------------------------
// scores
// ---------------------------------------------------------------------------------------------
// bf16.  Lane (g, t) = (lane / 4, lane % 4) loads, of key g of a block of eight, the vectors
// t, t + 4, .. of its row: words 0, 1 of vector c are the B operand of product 2 c, words 2, 3 of
// product 2 c + 1, and the query's vectors give the A operand in the same order.
template <int D>
__device__ __forceinline__ void item_scores(const Item& it, const DecodeArgs& a, __nv_bfloat16*, float* smax) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  constexpr int NV = D / 32;   // vectors of a lane per key
  const __nv_bfloat16* keys = keys_of<__nv_bfloat16>(it, a.k, a.pk, a);
  uint4 q0[NV], q1[NV];
  const int r0 = row_of(it, min(g, it.rows - 1), a), r1 = row_of(it, min(g + 8, it.rows - 1), a);
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q);
#pragma unroll
  for (int c = 0; c < NV; ++c) {
    q0[c] = *reinterpret_cast<const uint4*>(q + static_cast<int64_t>(r0) * D + c * 32 + t * 8);
    q1[c] = *reinterpret_cast<const uint4*>(q + static_cast<int64_t>(r1) * D + c * 32 + t * 8);
  }
  float* s0 = score_row(it, r0, a);
  float* s1 = score_row(it, r1, a);
  const bool w0 = g < it.rows, w1 = g + 8 < it.rows;
  float m0 = -kInf, m1 = -kInf;
  for (int k0 = it.first + warp * kBlock; k0 < it.last; k0 += kWarps * kBlock) {
    uint4 kv[4][NV];
#pragma unroll
    for (int nb = 0; nb < 4; ++nb) {
      const int key = k0 + nb * 8 + g;
      const __nv_bfloat16* p = keys + static_cast<int64_t>(key) * D + t * 8;
#pragma unroll
      for (int c = 0; c < NV; ++c) kv[nb][c] = key < it.last ? load_stream(p + c * 32) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int nb = 0; nb < 4; ++nb) {
      float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int c = 0; c < NV; ++c) {
        mma_bf16(s, q0[c].x, q1[c].x, q0[c].y, q1[c].y, kv[nb][c].x, kv[nb][c].y);
        mma_bf16(s, q0[c].z, q1[c].z, q0[c].w, q1[c].w, kv[nb][c].z, kv[nb][c].w);
      }
      const int key = k0 + nb * 8 + 2 * t;
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] = key + (i & 1) < it.last ? s[i] : -kInf;
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
    smax[warp * kRows + g] = m0;
    smax[warp * kRows + g + 8] = m1;
  }
}

// fp32: a key across D / 4 lanes, the block's queries in shared memory.
template <int D>
__device__ __forceinline__ void item_scores(const Item& it, const DecodeArgs& a, float*, float* smax) {
  constexpr int L = D / 4, KS = kThreads / L;
  __shared__ float4 qs[kRows][L];
  const int gl = threadIdx.x % L, ks = threadIdx.x / L;
  for (int i = threadIdx.x; i < it.rows * L; i += kThreads)
    qs[i / L][i % L] = reinterpret_cast<const float4*>(
        static_cast<const float*>(a.q) + static_cast<int64_t>(row_of(it, i / L, a)) * D)[i % L];
  for (int i = threadIdx.x; i < kWarps * kRows; i += kThreads) smax[i] = -kInf;
  __syncthreads();
  const float* keys = keys_of<float>(it, a.k, a.pk, a);
  const int end = it.first + (it.last - it.first + kBlock - 1) / kBlock * kBlock;   // whole blocks: -inf past the last
  float best[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) best[r] = -kInf;
  for (int k0 = it.first; k0 < end; k0 += KS) {
    const int key = k0 + ks;
    const bool in = key < it.last;
    const float4 kv = in ? reinterpret_cast<const float4*>(keys + static_cast<int64_t>(key) * D)[gl]
                         : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if (r < it.rows) {
        const float4 q = qs[r][gl];
        float s = fmaf(q.x, kv.x, fmaf(q.y, kv.y, fmaf(q.z, kv.z, q.w * kv.w)));
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        s = in ? s : -kInf;
        best[r] = fmaxf(best[r], s);
        if (gl == 0 && key < end) score_row(it, row_of(it, r, a), a)[key] = s;
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    float v = best[r];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    if ((threadIdx.x & 31) == 0) smax[(threadIdx.x >> 5) * kRows + r] = v;
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) decode_scores_kernel(const DecodeArgs a) {
  extern __shared__ int cum[];
  __shared__ float smax[kWarps * kRows];
  count_chunks(cum, a);
  const int64_t items = item_count(cum, a);
  for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
    const Item it = get_item(i, cum, a);
    item_scores<D>(it, a, static_cast<T*>(nullptr), smax);
    __syncthreads();
    if (threadIdx.x < static_cast<unsigned>(it.rows)) {
      float m = smax[threadIdx.x];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) m = fmaxf(m, smax[w * kRows + threadIdx.x]);
      a.row_max[static_cast<int64_t>(row_of(it, threadIdx.x, a)) * a.slots + it.slot] = m;
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------------------------
// values
// ---------------------------------------------------------------------------------------------
// A row's maximum over its shared and own items.  A whole warp.
__device__ __forceinline__ float row_maximum(const DecodeArgs& a, int row) {
  const int b = row / a.Hq;
  const int n = a.pchunks + (decode_own_length(a, b) + a.chunk - 1) / a.chunk;
  float m = -kInf;
  for (int i = threadIdx.x & 31; i < n; i += 32) m = fmaxf(m, a.row_max[static_cast<int64_t>(row) * a.slots + i]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

// bf16.  Lane (g, t) loads, of keys 2 t, 2 t + 1, 2 t + 8 and 2 t + 9 of sixteen, the dimensions
// 8 g .. 8 g + 7 of every 64: words of two keys, interleaved, are the B operand of the product
// whose column g stands for dimension 8 g + j.  phi of scores at the same keys is the A operand.
template <int D>
__device__ __forceinline__ void item_values(const Item& it, const DecodeArgs& a, __nv_bfloat16*, const float* rowm,
                                            float* sums, float* acc_s) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  constexpr int NC = D / 64;
  const __nv_bfloat16* vals = keys_of<__nv_bfloat16>(it, a.v, a.pv, a);
  const bool w0 = g < it.rows, w1 = g + 8 < it.rows;
  const float* s0 = score_row(it, row_of(it, min(g, it.rows - 1), a), a);
  const float* s1 = score_row(it, row_of(it, min(g + 8, it.rows - 1), a), a);
  const float m0 = rowm[g], m1 = rowm[g + 8];
  float acc[NC][8][4];
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[c][j][0] = acc[c][j][1] = acc[c][j][2] = acc[c][j][3] = 0.0f;
  float t0 = 0.0f, t1 = 0.0f;
  for (int k0 = it.first + warp * kBlock; k0 < it.last; k0 += kWarps * kBlock) {
    uint32_t p[2][4];
    bool live = false;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int key = k0 + h * 16 + e * 8 + 2 * t;
        float2 x = w0 ? *reinterpret_cast<const float2*>(s0 + key) : make_float2(-kInf, -kInf);
        float2 y = w1 ? *reinterpret_cast<const float2*>(s1 + key) : make_float2(-kInf, -kInf);
        x.x = phi_fast((m0 - x.x) * a.scale);
        x.y = phi_fast((m0 - x.y) * a.scale);
        y.x = phi_fast((m1 - y.x) * a.scale);
        y.y = phi_fast((m1 - y.y) * a.scale);
        t0 += x.x + x.y;
        t1 += y.x + y.y;
        live |= x.x > 0.0f || x.y > 0.0f || y.x > 0.0f || y.y > 0.0f;
        // V is bf16, so phi goes into the product as bf16: 2^-8 relative at most per weight,
        // like the rounding of the output; the sums above keep all 32 bits
        p[h][2 * e] = pack_bf16x2(x.x, x.y);
        p[h][2 * e + 1] = pack_bf16x2(y.x, y.y);
      }
    }
    if (!__any_sync(0xffffffffu, live)) continue;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint4 v[4][NC];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = k0 + h * 16 + (i >> 1) * 8 + 2 * t + (i & 1);
        const __nv_bfloat16* src = vals + static_cast<int64_t>(key) * D + g * 8;
#pragma unroll
        for (int c = 0; c < NC; ++c) v[i][c] = key < it.last ? load_stream(src + c * 64) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const uint32_t x0[4] = {v[0][c].x, v[0][c].y, v[0][c].z, v[0][c].w};
        const uint32_t x1[4] = {v[1][c].x, v[1][c].y, v[1][c].z, v[1][c].w};
        const uint32_t x2[4] = {v[2][c].x, v[2][c].y, v[2][c].z, v[2][c].w};
        const uint32_t x3[4] = {v[3][c].x, v[3][c].y, v[3][c].z, v[3][c].w};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t sel = j & 1 ? 0x7632u : 0x5410u;
          mma_bf16(acc[c][j], p[h][0], p[h][1], p[h][2], p[h][3], __byte_perm(x0[j >> 1], x1[j >> 1], sel),
                   __byte_perm(x2[j >> 1], x3[j >> 1], sel));
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
    sums[warp * kRows + g] = t0;
    sums[warp * kRows + g + 8] = t1;
  }
  // accumulator columns 2 t, 2 t + 1 stand for dimensions 16 t + j and 16 t + 8 + j
  float* out = acc_s + warp * kRows * D;
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int j = 0; j < 8; j += 4)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *reinterpret_cast<float4*>(out + (g + (e >> 1) * 8) * D + c * 64 + t * 16 + (e & 1) * 8 + j) =
            make_float4(acc[c][j][e], acc[c][j + 1][e], acc[c][j + 2][e], acc[c][j + 3][e]);
}

// fp32: D / 4 lanes across the dimensions; each of the kThreads / (D / 4) lane groups takes every
// so many keys of a tile whose phi stands in shared memory.
template <int D>
__device__ __forceinline__ void item_values(const Item& it, const DecodeArgs& a, float*, const float* rowm,
                                            float* sums, float* acc_s) {
  constexpr int L = D / 4, KS = kThreads / L, TK = 64;
  __shared__ float ph[kRows][TK];
  const int gl = threadIdx.x % L, ks = threadIdx.x / L;
  const float* vals = keys_of<float>(it, a.v, a.pv, a);
  float acc[kRows][4];
#pragma unroll
  for (int r = 0; r < kRows; ++r) acc[r][0] = acc[r][1] = acc[r][2] = acc[r][3] = 0.0f;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float tot[kRows / kWarps] = {};
  for (int k0 = it.first; k0 < it.last; k0 += TK) {
    __syncthreads();
#pragma unroll
    for (int rr = 0; rr < kRows / kWarps; ++rr) {
      const int r = warp + rr * kWarps;
      if (r < it.rows) {
        const float* s = score_row(it, row_of(it, r, a), a);
        for (int i = lane; i < TK; i += 32) {
          const float f = k0 + i < it.last ? phi_exact((rowm[r] - s[k0 + i]) * a.scale) : 0.0f;
          ph[r][i] = f;
          tot[rr] += f;
        }
      }
    }
    __syncthreads();
    const int n = min(TK, it.last - k0);
    for (int i = ks; i < n; i += KS) {
      const float4 v = reinterpret_cast<const float4*>(vals + static_cast<int64_t>(k0 + i) * D)[gl];
#pragma unroll
      for (int r = 0; r < kRows; ++r)
        if (r < it.rows) {
          const float f = ph[r][i];
          acc[r][0] = fmaf(f, v.x, acc[r][0]);
          acc[r][1] = fmaf(f, v.y, acc[r][1]);
          acc[r][2] = fmaf(f, v.z, acc[r][2]);
          acc[r][3] = fmaf(f, v.w, acc[r][3]);
        }
    }
  }
#pragma unroll
  for (int rr = 0; rr < kRows / kWarps; ++rr) {
    float f = tot[rr];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) f += __shfl_xor_sync(0xffffffffu, f, o);
    if (lane < kWarps) sums[lane * kRows + warp + rr * kWarps] = lane == 0 ? f : 0.0f;
  }
  // lane groups of one warp first, so that kWarps partial sums remain
#pragma unroll
  for (int r = 0; r < kRows; ++r)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float f = acc[r][e];
#pragma unroll
      for (int o = L; o < 32; o <<= 1) f += __shfl_xor_sync(0xffffffffu, f, o);
      if (lane < L) acc_s[(warp * kRows + r) * D + gl * 4 + e] = f;
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) decode_values_kernel(const DecodeArgs a) {
  extern __shared__ float4 dyn4[];
  float* acc_s = reinterpret_cast<float*>(dyn4);                    // [kWarps][kRows][D]
  int* cum = reinterpret_cast<int*>(acc_s + kWarps * kRows * D);
  __shared__ float rowm[kRows], sums[kWarps * kRows];
  __shared__ int live;
  count_chunks(cum, a);
  const int64_t items = item_count(cum, a);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
    const Item it = get_item(i, cum, a);
    if (threadIdx.x == 0) live = 0;
    __syncthreads();
    for (int r = warp; r < kRows; r += kWarps) {
      if (r < it.rows) {
        const int row = row_of(it, r, a);
        const float m = row_maximum(a, row);
        if (lane == 0) {
          rowm[r] = m;
          if ((m - a.row_max[static_cast<int64_t>(row) * a.slots + it.slot]) * a.scale < 16.0f) live = 1;
        }
      } else if (lane == 0) {
        rowm[r] = 0.0f;
      }
    }
    __syncthreads();
    if (!live) {   // every phi of the item is 0
      if (threadIdx.x < static_cast<unsigned>(it.rows))
        a.part_sum[static_cast<int64_t>(row_of(it, threadIdx.x, a)) * a.slots + it.slot] = 0.0f;
      __syncthreads();
      continue;
    }
    item_values<D>(it, a, static_cast<T*>(nullptr), rowm, sums, acc_s);
    __syncthreads();
    if (threadIdx.x < static_cast<unsigned>(it.rows)) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) s += sums[w * kRows + threadIdx.x];
      a.part_sum[static_cast<int64_t>(row_of(it, threadIdx.x, a)) * a.slots + it.slot] = s;
    }
    for (int e = threadIdx.x; e < it.rows * (D / 4); e += kThreads) {
      const int r = e / (D / 4), c = e % (D / 4);
      float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 x = reinterpret_cast<const float4*>(acc_s + (w * kRows + r) * D)[c];
        s.x += x.x;
        s.y += x.y;
        s.z += x.z;
        s.w += x.w;
      }
      reinterpret_cast<float4*>(a.part_o + (static_cast<int64_t>(row_of(it, r, a)) * a.slots + it.slot) * D)[c] = s;
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------------------------
// join
// ---------------------------------------------------------------------------------------------
// A row's sum of phi over its items, in a fixed order.  A whole warp.
__device__ __forceinline__ float row_total(const DecodeArgs& a, int row) {
  const int b = row / a.Hq;
  const int n = a.pchunks + (decode_own_length(a, b) + a.chunk - 1) / a.chunk;
  float s = 0.0f;
  for (int i = threadIdx.x & 31; i < n; i += 32) s += a.part_sum[static_cast<int64_t>(row) * a.slots + i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

constexpr int kWeightKeys = 1024;   // keys of a weight CTA

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) decode_join_kernel(const DecodeArgs a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t rows = static_cast<int64_t>(a.B) * a.Hq;
  if (blockIdx.x < rows) {   // one output row
    constexpr int L = D / 4, KS = kThreads / L;
    __shared__ float4 part[KS][L];
    const int row = blockIdx.x, b = row / a.Hq;
    const int n = a.pchunks + (decode_own_length(a, b) + a.chunk - 1) / a.chunk;
    const float total = row_total(a, row);
    const int gl = threadIdx.x % L, ks = threadIdx.x / L;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int i = ks; i < n; i += KS) {
      const int64_t at = static_cast<int64_t>(row) * a.slots + i;
      if (a.part_sum[at] > 0.0f) {   // 0: the item was skipped and wrote no partial output
        const float4 x = reinterpret_cast<const float4*>(a.part_o + at * D)[gl];
        s.x += x.x;
        s.y += x.y;
        s.z += x.z;
        s.w += x.w;
      }
    }
    part[ks][gl] = s;
    __syncthreads();
    if (ks == 0) {
#pragma unroll
      for (int i = 1; i < KS; ++i) {
        const float4 x = part[i][gl];
        s.x += x.x;
        s.y += x.y;
        s.z += x.z;
        s.w += x.w;
      }
      const float inv = total > 0.0f ? 1.0f / total : 0.0f;   // no key at all: zeros
      T* o = static_cast<T*>(a.o) + static_cast<int64_t>(row) * D + gl * 4;
      if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(s.x * inv, s.y * inv), pack_bf16x2(s.z * inv, s.w * inv));
      } else {
        *reinterpret_cast<float4*>(o) = make_float4(s.x * inv, s.y * inv, s.z * inv, s.w * inv);
      }
    }
    return;
  }
  // weights of kWeightKeys keys of one (sequence, key head)
  extern __shared__ float2 ms[];   // [G] maximum and 1 / sum
  const int splits = (a.C + kWeightKeys - 1) / kWeightKeys;
  const int64_t x = blockIdx.x - rows;
  const int split = static_cast<int>(x % splits);
  const int bk = static_cast<int>(x / splits), b = bk / a.Hkv, kv = bk - b * a.Hkv;
  const int first = split * kWeightKeys, last = min(first + kWeightKeys, decode_own_length(a, b));
  if (first >= last) return;
  for (int g = warp; g < a.G; g += kWarps) {
    const int row = b * a.Hq + kv * a.G + g;
    const float m = row_maximum(a, row), s = row_total(a, row);
    if (lane == 0) ms[g] = make_float2(m, s);
  }
  __syncthreads();
  float* w = a.weight + static_cast<int64_t>(bk) * a.C;
  for (int key = first + threadIdx.x; key < last; key += kThreads) {
    float sum = 0.0f;
    for (int g = 0; g < a.G; ++g) {
      const float s = a.s_own[(static_cast<int64_t>(b) * a.Hq + kv * a.G + g) * a.own_width + key];
      sum += phi_t<T>((ms[g].x - s) * a.scale) / ms[g].y;
    }
    w[key] += sum;
  }
}

template <typename T, int D>
cudaError_t go(const DecodeArgs& a, const PrefixMaps& maps, const LaunchCtx& ctx, cudaStream_t st) {
  const int cum = (a.B + 1) * 4;
  const int smem_values = kWarps * kRows * D * 4 + cum;
  cudaError_t e = cudaSuccess;
  if (smem_values > 40 * 1024) {   // many sequences: 32 KB of partial sums and up to 32 KB of chunk counts
    e = cudaFuncSetAttribute(decode_values_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_values);
    if (e != cudaSuccess) return e;
  }
  const int64_t shared = a.tc ? 0 : static_cast<int64_t>(a.Hkv) * a.pchunks * ((a.B * a.G + kRows - 1) / kRows);
  const int64_t own = static_cast<int64_t>(a.B) * ((a.C + a.chunk - 1) / a.chunk) * a.Hkv *
                      ((a.G + kRows - 1) / kRows);
  const int64_t most = shared + own;
  const int grid = static_cast<int>(most < 3 * kSms ? most : 3 * kSms);
  if (a.tc && (e = launch_decode_prefix(maps, a, false, ctx, st)) != cudaSuccess) return e;
  decode_scores_kernel<T, D><<<grid, kThreads, cum, st>>>(a);
  if (a.tc && (e = launch_decode_prefix(maps, a, true, ctx, st)) != cudaSuccess) return e;
  decode_values_kernel<T, D><<<grid, kThreads, smem_values, st>>>(a);
  const int64_t join = static_cast<int64_t>(a.B) * a.Hq +
                       (a.weight ? static_cast<int64_t>(a.B) * a.Hkv * ((a.C + kWeightKeys - 1) / kWeightKeys) : 0);
  decode_join_kernel<T, D><<<static_cast<unsigned>(join), kThreads, a.weight ? a.G * 8 : 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

// The split of the keys.  Own items of 256 keys, or of 128 where that would leave SMs without an
// item.  Shared keys of more than kTcRows rows per key head go to the tensor cores, in whole
// tiles of 128, split so that one wave of CTAs takes them; otherwise in as many items as give
// every SM three, of at least 128 keys.
constexpr int64_t kTcRows = 32;
size_t plan_decode(DecodeArgs* a, bool bf16, char* base) {
  const int64_t rows = static_cast<int64_t>(a->B) * a->Hq;
  a->G = a->Hq / a->Hkv;
  const int64_t shared_rows = static_cast<int64_t>(a->B) * a->G;
  const int64_t own_blocks = (a->G + kRows - 1) / kRows;
  a->chunk = static_cast<int64_t>(a->B) * a->Hkv * own_blocks * ((a->C + 255) / 256) < 2 * kSms ? 128 : 256;
  const int own = (a->C + a->chunk - 1) / a->chunk;
  a->own_width = own * a->chunk;
  a->pchunk = a->pchunks = a->pre_width = 0;
  a->tc = bf16 && a->P > 0 && shared_rows > kTcRows;
  if (a->P > 0) {
    const int64_t per = a->Hkv * (a->tc ? (shared_rows + 255) / 256 : (shared_rows + kRows - 1) / kRows);
    const int64_t tiles = (a->P + 127) / 128;
    int64_t n = a->tc ? kSms / per : (3 * kSms + per - 1) / per;
    n = n < 1 ? 1 : n > tiles ? tiles : n;
    a->pchunk = static_cast<int>((tiles + n - 1) / n * 128);
    a->pchunks = (a->P + a->pchunk - 1) / a->pchunk;
    a->pre_width = a->tc ? 0 : a->pchunks * a->pchunk;
  }
  a->slots = a->pchunks + own;
  size_t at = 0;
  auto piece = [&](int64_t floats) {
    float* p = reinterpret_cast<float*>(base + at);
    at += (static_cast<size_t>(floats) * 4 + 255) & ~static_cast<size_t>(255);
    return p;
  };
  a->s_own = piece(rows * a->own_width);
  a->s_pre = piece(rows * a->pre_width);
  a->row_max = piece(rows * a->slots);
  a->part_sum = piece(rows * a->slots);
  a->part_o = piece(rows * a->slots * a->D);
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
