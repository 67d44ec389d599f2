// The shared prefix of ra_attention_decode on the tensor cores (tcgen05 + TMEM + TMA): the query
// rows of a whole batch against the keys and values they share, bf16, D = 64 or 128.
//
// All B G rows of a key head see the same keys, so this part is GEMM-shaped: rows as the M of
// 128-row products, 128 keys per tile.  The rational map needs the row maximum before any phi
// (see decode.cu), so it comes as two kernels around the maxima of the sequences' own keys:
//   max     S = Q K^T per tile into TMEM, each row's maximum over the CTA's keys;
//   values  S again, phi on the FMA pipe, P (bf16) to shared memory, O += P V in TMEM; partial
//           sums and outputs (fp32) per CTA to the workspace.
// Forming S twice costs a third more products, but 256 rows of scores in fp32 would be four times
// the bytes of the keys.
//
// A CTA takes up to 256 rows (two tiles A and B, so every K and V tile loaded serves both) of one
// key head and a run of key tiles; the keys are split so that one wave of CTAs, one per SM, covers
// heads x row pairs x splits.  Roles as in the attention forward: warp 8 feeds a ring of K (and V)
// tiles by TMA; warps 9 and 10 issue the products of tile A and B, one thread each; warps 0-3 and
// 4-7 own the rows of A and B, thread = row.  Query rows are gathered by their own threads (a head's
// rows are G at a time in memory) into the 128-byte-swizzled operand layout.
//
// Bound: HBM for K and V while rows are few, the products from about 256 rows per key head on.
#include "decode_split.cuh"
#include "phi.cuh"

namespace raattn {
namespace {

constexpr int BM = 128, BN = 128;
constexpr int NGROUP = 2, GROUP_WARPS = 4, SOFTMAX_WARPS = NGROUP * GROUP_WARPS;
constexpr int PRODUCER_WARP = SOFTMAX_WARPS, MMA_WARP = SOFTMAX_WARPS + 1;
constexpr int THREADS = 32 * (SOFTMAX_WARPS + 1 + NGROUP);
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t TMEM_O = 256;          // S of tile g at column 128 g (max: also at 256 + 128 g), O at 256 + 128 g
constexpr int BOX_BYTES = 128 * 64 * 2;   // one TMA box: 128 rows x 64 values

template <int D, bool VALUES>
struct Cfg {
  static constexpr int TILE_BYTES = BN * D * 2;
  static constexpr int NSTAGE = D == 128 ? (VALUES ? 3 : 4) : 6;
  static constexpr int P_BYTES = VALUES ? BM * BN * 2 : 0;
  static constexpr int OFF_RING = NGROUP * TILE_BYTES;
  static constexpr int OFF_P = OFF_RING + NSTAGE * TILE_BYTES;
  static constexpr int OFF_BAR = OFF_P + NGROUP * P_BYTES;
  // q_full, ring_full[], ring_empty[], s_full[2][2], s_empty[2][2], p_full[2], p_empty[2], o_full[2], drain[2]
  static constexpr int NUM_BARS = 1 + 2 * NSTAGE + 8 * NGROUP;
  static constexpr int OFF_MISC = (OFF_BAR + NUM_BARS * 8 + 15) / 16 * 16;
  static constexpr int USED = OFF_MISC + 16 + SOFTMAX_WARPS * 4;
  static constexpr int SLACK = USED + 1024 <= 232448 ? 1024 : 0;   // else the base has to be aligned already
  static constexpr int SMEM_BYTES = USED + SLACK;
  static_assert(SMEM_BYTES <= 232448, "shared memory per CTA");
};

// phi of 64 columns of a row: d = m - s is exact 0 at the maximum; columns from `n` on are not keys.
template <bool RAGGED>
__device__ __forceinline__ float2 phi_half(const uint32_t (&h)[2][32], uint32_t (&pk)[32], int n, float c2, float m) {
  float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int c8 = 0; c8 < 8; ++c8) {
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = c8 * 8 + e;
      x[e] = u2f(h[c >> 5][c & 31]) - m;
      if (RAGGED && c >= n) x[e] = -INFINITY;
    }
    float2 p0, p1, p2, p3;
    phi_quad(x[0], x[1], x[2], x[3], c2, 0.5f, p0, p1);
    phi_quad(x[4], x[5], x[6], x[7], c2, 0.5f, p2, p3);
    sum = __fadd2_rn(sum, __fadd2_rn(__fadd2_rn(p0, p1), __fadd2_rn(p2, p3)));
    // V is bf16, so P is: half a step, 2^-8 relative at most per weight; the sum keeps fp32
    pk[4 * c8 + 0] = pack_bf16x2(p0.x, p0.y);
    pk[4 * c8 + 1] = pack_bf16x2(p1.x, p1.y);
    pk[4 * c8 + 2] = pack_bf16x2(p2.x, p2.y);
    pk[4 * c8 + 3] = pack_bf16x2(p3.x, p3.y);
  }
  return sum;
}

__device__ __forceinline__ void store_p_half(const uint32_t (&pk)[32], uint8_t* row, int row_local) {
#pragma unroll
  for (int c = 0; c < 8; ++c)
    *reinterpret_cast<uint4*>(row + ((c ^ (row_local & 7)) << 4)) =
        make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
}

// The maximum of a row over all its parts, read by one thread.
__device__ __forceinline__ float row_maximum(const DecodeArgs& a, int row, int b, int kv, int g) {
  int shared, own;
  decode_row_slots(b, kv, g, a.cum[b], a.cum[b + 1], decode_split(a, a.cum[a.B]), a, shared, own);
  const float* p = a.row_max + static_cast<int64_t>(row) * a.slots;
  float m = -INFINITY;
#pragma unroll 8
  for (int i = 0; i < shared; ++i) m = fmaxf(m, __ldcg(p + i));
#pragma unroll 4
  for (int i = 0; i < own; ++i) m = fmaxf(m, __ldcg(p + a.pslots + i));
  return m;
}

template <int D, bool VALUES>
__global__ void __launch_bounds__(THREADS, 1)
    decode_prefix_kernel(const __grid_constant__ PrefixMaps maps, const DecodeArgs a, const LaunchCtx ctx) {
  using C = Cfg<D, VALUES>;
  constexpr int NST = C::NSTAGE;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t mis = smem_u32(smem_raw) & 1023u;
  if (C::SLACK == 0 && mis != 0) {   // uniform over the CTA: nothing has started
    if (threadIdx.x == 0) atomicOr(ctx.status, kStatusBadSmem);
    return;
  }
  uint8_t* smem = smem_raw + ((1024u - mis) & 1023u);
  uint8_t* sQ = smem;
  uint8_t* sRing = smem + C::OFF_RING;
  uint8_t* sP = smem + C::OFF_P;
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* ring_full = q_full + 1;
  uint64_t* ring_empty = ring_full + NST;
  uint64_t* s_full = ring_empty + NST;   // score buffer b of tile g at 2 g + b
  uint64_t* s_empty = s_full + 2 * NGROUP;
  uint64_t* p_full = s_empty + 2 * NGROUP;
  uint64_t* p_empty = p_full + NGROUP;
  uint64_t* o_full = p_empty + NGROUP;
  uint64_t* drain = o_full + NGROUP;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  volatile int* live = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 16);   // votes of the softmax warps

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // item: key head fastest (its neighbours read other keys), then row pair, then key split
  const int rows = a.B * a.G;
  const int pairs = (rows + NGROUP * BM - 1) / (NGROUP * BM);
  const int kv = blockIdx.x % a.Hkv, rest = blockIdx.x / a.Hkv;
  const int x0 = rest % pairs * (NGROUP * BM), split = rest / pairs;
  const int tps = a.pchunk / BN;
  const int t0 = split * tps, nt = min(t0 + tps, (a.P + BN - 1) / BN) - t0;   // this CTA's key tiles, at least one
  const int groups = x0 + BM < rows ? 2 : 1;                                   // row tiles with rows

  if (threadIdx.x == 0) {
    mbar_init(q_full, groups * GROUP_WARPS);
    for (int i = 0; i < NST; ++i) {
      mbar_init(&ring_full[i], 1);
      mbar_init(&ring_empty[i], groups);   // one commit per issuer at work
    }
    for (int g = 0; g < NGROUP; ++g) {
      for (int b = 0; b < 2; ++b) {
        mbar_init(&s_full[2 * g + b], 1);
        mbar_init(&s_empty[2 * g + b], GROUP_WARPS);
      }
      mbar_init(&p_full[g], GROUP_WARPS);
      mbar_init(&p_empty[g], 1);
      mbar_init(&o_full[g], 1);
      mbar_init(&drain[g], 1);
    }
    *abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == MMA_WARP) {
    tmem_alloc(tmem_slot, TMEM_COLS);
    tmem_relinquish();
  }
  if constexpr (VALUES) await_previous();   // all maxima
  release_dependents();                     // the sequences' own values need no more than that either
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == PRODUCER_WARP) {
    if (lane == 0) {
      tma_prefetch_desc(&maps.k);
      if (VALUES) tma_prefetch_desc(&maps.v);
      uint32_t it = 0;
      uint32_t last_par[NST];
      bool issued[NST];
#pragma unroll
      for (int i = 0; i < NST; ++i) {
        issued[i] = false;
        last_par[i] = 0;
      }
      auto issue = [&](const CUtensorMap* map, int j) -> bool {
        const int st = it % NST;
        const uint32_t par = (it / NST) & 1u;
        if (!mbar_wait(&ring_empty[st], par ^ 1u, abort_flag, ctx)) return false;
        mbar_arrive_expect_tx(&ring_full[st], C::TILE_BYTES);
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
          tma_load_3d(sRing + st * C::TILE_BYTES + c * BOX_BYTES, map, &ring_full[st], c * 64, (t0 + j) * BN, kv);
        issued[st] = true;
        last_par[st] = par;
        ++it;
        return true;
      };
      bool ok = true;
      for (int j = 0; j < nt && ok; ++j) {   // values: K_0, then K_j and V_(j-1), then the last V
        ok = issue(&maps.k, j);
        if (VALUES && ok && j > 0) ok = issue(&maps.v, j - 1);
      }
      if (VALUES && ok) issue(&maps.v, nt - 1);
      for (int i = 0; i < NST; ++i)
        if (issued[i]) drain_wait(&ring_full[i], last_par[i], ctx);
    }
  } else if (warp >= MMA_WARP) {
    const int g = warp - MMA_WARP;
    if (lane == 0 && g < groups) {
      constexpr uint32_t idesc_qk = idesc_bf16_f32(BM, BN, 0, 0);
      constexpr uint32_t idesc_pv = idesc_bf16_f32(BM, D, 0, 1);
      constexpr uint32_t HI = sdesc_hi_sw128(1024);
      const uint32_t ring = smem_u32(sRing);
      const uint32_t qlo = sdesc_lo(smem_u32(sQ) + g * C::TILE_BYTES, 16);
      const uint32_t plo = sdesc_lo(smem_u32(sP) + g * C::P_BYTES, 16);
      uint32_t pos = 0, used[2] = {0, 0};
      bool o_started = false;
      auto ring_wait = [&](uint32_t p, uint32_t& addr) -> bool {
        const int st = p % NST;
        if (!mbar_wait(&ring_full[st], (p / NST) & 1u, abort_flag, ctx)) return false;
        tc_fence_after();
        addr = ring + st * C::TILE_BYTES;
        return true;
      };
      auto mma_s = [&](uint32_t kaddr, int b) -> bool {   // S = Q K^T into score buffer b
        if (!mbar_wait(&s_empty[2 * g + b], (used[b] & 1u) ^ 1u, abort_flag, ctx)) return false;
        tc_fence_after();
        const uint32_t klo = sdesc_lo(kaddr, 16), col = tmem + 128 * g + 256 * b;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * BOX_BYTES + (kk & 3) * 32) >> 4;
          tc_mma_f16(col, sdesc(qlo + off, HI), sdesc(klo + off, HI), idesc_qk, kk > 0 ? 1u : 0u);
        }
        tc_commit(&s_full[2 * g + b]);
        ++used[b];
        return true;
      };
      auto mma_pv = [&](uint32_t c, uint32_t vaddr) -> bool {   // O += P V of the c-th tile, unless P is 0
        if (!mbar_wait(&p_full[g], c & 1u, abort_flag, ctx)) return false;
        tc_fence_after();
        int any = 0;
#pragma unroll
        for (int w = 0; w < GROUP_WARPS; ++w) any |= live[g * GROUP_WARPS + w];
        if (any) {
          const uint32_t vlo = sdesc_lo(vaddr, BOX_BYTES), col = tmem + TMEM_O + 128 * g;
#pragma unroll
          for (int kk = 0; kk < BN / 16; ++kk) {
            const uint32_t aoff = ((kk >> 2) * BOX_BYTES + (kk & 3) * 32) >> 4;   // P: K-major
            const uint32_t boff = (kk * 16 * 128) >> 4;                            // V: MN-major, 16 key rows
            tc_mma_f16(col, sdesc(plo + aoff, HI), sdesc(vlo + boff, HI), idesc_pv, kk > 0 || o_started ? 1u : 0u);
          }
          o_started = true;
        }
        tc_commit(&p_empty[g]);
        return true;
      };
      bool ok = mbar_wait(q_full, 0, abort_flag, ctx);
      // test knob: nothing is committed to `drain` yet, so this wait can only time out
      if (ok && ctx.force_timeout) ok = mbar_wait(&drain[g], 0, abort_flag, ctx);
      tc_fence_after();
      uint32_t addr = 0;
      for (int j = 0; j < nt && ok; ++j) {
        const uint32_t kpos = pos++;
        ok = ring_wait(kpos, addr) && mma_s(addr, VALUES ? 0 : j & 1);
        if (ok) tc_commit(&ring_empty[kpos % NST]);
        if (VALUES && ok && j > 0) {
          const uint32_t vpos = pos++;
          ok = ring_wait(vpos, addr) && mma_pv(j - 1, addr);
          if (ok) tc_commit(&ring_empty[vpos % NST]);
        }
      }
      if (VALUES && ok) {
        ok = ring_wait(pos, addr) && mma_pv(nt - 1, addr);
        if (ok) tc_commit(&ring_empty[pos % NST]);
      }
      if (ok) tc_commit(&o_full[g]);
      tc_commit(&drain[g]);
      drain_wait(&drain[g], 0, ctx);
    }
  } else if (warp / GROUP_WARPS < groups) {
    const int g = warp / GROUP_WARPS, quarter = warp % GROUP_WARPS;
    const int row_local = quarter * 32 + lane, x = x0 + g * BM + row_local;
    const bool row_ok = x < rows;
    const int row = row_ok ? x / a.G * a.Hq + kv * a.G + x % a.G : 0;
    auto warp_wait = [&](uint64_t* bar, uint32_t par) -> bool {
      int r = 1;
      if (lane == 0) r = mbar_wait(bar, par, abort_flag, ctx) ? 1 : 0;
      return __shfl_sync(0xffffffffu, r, 0) != 0;
    };
    {   // this row of Q
      const uint4* q = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + static_cast<int64_t>(row) * D);
      uint8_t* dst = sQ + g * C::TILE_BYTES + row_local * 128;
      uint4 v[D / 8];
#pragma unroll
      for (int c = 0; c < D / 8; ++c) v[c] = row_ok ? q[c] : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int c = 0; c < D / 8; ++c)
        *reinterpret_cast<uint4*>(dst + (c >> 3) * BOX_BYTES + (((c & 7) ^ (row_local & 7)) << 4)) = v[c];
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
    }
    const uint32_t scol = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + 128 * g;
    const int tail = a.P - t0 * BN;   // keys from this CTA's first on
    bool ok = true;
    if constexpr (!VALUES) {
      float m = -INFINITY;
      for (int j = 0; j < nt && ok; ++j) {
        const int b = j & 1;
        ok = warp_wait(&s_full[2 * g + b], (j >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        uint32_t s[4][32];
#pragma unroll
        for (int k = 0; k < 4; ++k) tmem_ld32(scol + 256 * b + 32 * k, s[k]);
        tc_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_empty[2 * g + b]);
        float u0 = -INFINITY, u1 = -INFINITY;
        if ((j + 1) * BN <= tail) {
#pragma unroll
          for (int c = 0; c < 128; c += 4) {
            u0 = max3f(u0, u2f(s[c >> 5][c & 31]), u2f(s[c >> 5][(c & 31) + 1]));
            u1 = max3f(u1, u2f(s[c >> 5][(c & 31) + 2]), u2f(s[c >> 5][(c & 31) + 3]));
          }
        } else {
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (j * BN + c < tail) u0 = fmaxf(u0, u2f(s[c >> 5][c & 31]));
        }
        m = fmaxf(m, fmaxf(u0, u1));
      }
      if (ok && row_ok) a.row_max[static_cast<int64_t>(row) * a.slots + split] = m;
    } else {
      const float m = row_ok ? row_maximum(a, row, x / a.G, kv, x % a.G) : 0.0f;
      const float c2 = a.scale * (1.0f / 32.0f);
      uint8_t* prow = sP + g * C::P_BYTES + row_local * 128;
      float total = 0.0f;
      for (int j = 0; j < nt && ok; ++j) {
        ok = warp_wait(&s_full[2 * g], j & 1);
        if (!ok) break;
        tc_fence_after();
        const int n = tail - j * BN;
        uint32_t h[2][32], pk[32];
        tmem_ld32(scol, h[0]);
        tmem_ld32(scol + 32, h[1]);
        tc_wait_ld();
        float2 sum = n < BN ? phi_half<true>(h, pk, n, c2, m) : phi_half<false>(h, pk, n, c2, m);
        tmem_ld32(scol + 64, h[0]);
        tmem_ld32(scol + 96, h[1]);
        tc_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_empty[2 * g]);
        ok = warp_wait(&p_empty[g], (j & 1) ^ 1);   // the previous product has read the P tile
        if (!ok) break;
        store_p_half(pk, prow, row_local);
        const float2 sum2 = n < BN ? phi_half<true>(h, pk, n - 64, c2, m) : phi_half<false>(h, pk, n - 64, c2, m);
        store_p_half(pk, prow + BOX_BYTES, row_local);
        fence_proxy_async_smem();
        const float t = (sum.x + sum.y) + (sum2.x + sum2.y);
        total += t;
        const unsigned any = __any_sync(0xffffffffu, t > 0.0f);
        if (lane == 0) live[g * GROUP_WARPS + quarter] = any ? 1 : 0;
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[g]);
      }
      if (ok) ok = warp_wait(&o_full[g], 0);
      if (ok) {
        tc_fence_after();
        // through this tile's P buffer (its last product has read it), 4 KB per warp, so that
        // whole 128-byte row segments leave
        uint8_t* stage = sP + g * C::P_BYTES + quarter * 4096;
        const int64_t out = row_ok && total > 0.0f ? (static_cast<int64_t>(row) * a.slots + split) * D : -1;
#pragma unroll
        for (int c0 = 0; c0 < D; c0 += 32) {
          uint32_t ov[32];
          tmem_ld32(tmem + (static_cast<uint32_t>(quarter * 32) << 16) + TMEM_O + 128 * g + c0, ov);
          tc_wait_ld();
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 8; ++k)
            *reinterpret_cast<uint4*>(stage + lane * 128 + ((k ^ (lane & 7)) << 4)) =
                make_uint4(ov[4 * k], ov[4 * k + 1], ov[4 * k + 2], ov[4 * k + 3]);
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = i * 4 + (lane >> 3), k = lane & 7;
            const uint4 u = *reinterpret_cast<const uint4*>(stage + r * 128 + ((k ^ (r & 7)) << 4));
            const int64_t o = __shfl_sync(0xffffffffu, out, r);   // -1: no row, or a sum of 0 (nothing to add)
            if (o >= 0) *reinterpret_cast<uint4*>(a.part_o + o + c0 + k * 4) = u;
          }
        }
        if (row_ok) a.part_sum[static_cast<int64_t>(row) * a.slots + split] = total;
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == MMA_WARP) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

template <int D, bool VALUES>
cudaError_t go(const PrefixMaps& maps, const DecodeArgs& a, const LaunchCtx& ctx, cudaStream_t st) {
  auto kernel = decode_prefix_kernel<D, VALUES>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             Cfg<D, VALUES>::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  const int pairs = (a.B * a.G + NGROUP * BM - 1) / (NGROUP * BM);
  const unsigned grid = static_cast<unsigned>(a.Hkv) * pairs * a.pslots;
  if constexpr (VALUES) return launch_dependent(kernel, grid, THREADS, Cfg<D, VALUES>::SMEM_BYTES, st, maps, a, ctx);
  kernel<<<grid, THREADS, Cfg<D, VALUES>::SMEM_BYTES, st>>>(maps, a, ctx);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decode_prefix(const PrefixMaps& maps, const DecodeArgs& a, bool values, const LaunchCtx& ctx,
                                 cudaStream_t st) {
  if (a.D == 64) return values ? go<64, true>(maps, a, ctx, st) : go<64, false>(maps, a, ctx, st);
  return values ? go<128, true>(maps, a, ctx, st) : go<128, false>(maps, a, ctx, st);
}

}  // namespace raattn
