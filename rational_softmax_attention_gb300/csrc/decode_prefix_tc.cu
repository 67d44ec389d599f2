// The shared prefix of ra_attention_decode on the tensor cores (tcgen05 + TMEM + TMA): the query
// rows of a whole batch against the keys and values they share, bf16, D = 64 or 128.
//
// All B G rows of a key head see the same keys, so this part is GEMM-shaped: rows as the M of
// 128-row products, 128 keys per tile.  The rational map needs the row maximum before any phi
// (see decode.cu), so it comes as two kernels around the maxima of the sequences' own keys:
//   max     S = Q K^T per tile into TMEM, each row's maximum over the CTA's keys;
//   values  S again, phi on the FMA pipe, P (bf16) over S's own columns in TMEM, O += P V with A read
//           from there; partial sums and outputs (fp32) per CTA to the workspace.
// Forming S twice costs a third more products, but 128 rows of scores in fp32 would be twice the
// bytes of the keys.
//
// V is bf16, so P is, rounded: 2^-8 relative at most per weight, like the output.  Up
// to 128 rows a key head P goes in as two bf16 instead, itself and what that leaves, for little (whole call,
// B32 H32/8 C1024 P8192: 46.5 us -> 48.3).  With more rows it costs more: prefix alone, P32768, B64 72.7 -> 86.6 us, B128
// 130 -> 158; whole call, full caches, B64 H32/8 C4096 P32768 242 -> 251, B40 H32/8 C1024 P8192 57.8 -> 62.0, B128 H16/4 D64
// C512 P16384 52.3 -> 59.2.  So the error there is 0.0023 of the output instead of 0.0017, its own rounding.  The
// tensor pipe is 29 to 32% busy then: what the second product lengthens is the chain of a tile, load, S, phi,
// hand-off and P V.
//
// A CTA takes 128 rows of one key head and a run of key tiles; the keys are split so that one wave of
// CTAs, one per SM, covers heads x row tiles x splits.  Roles: warp 8 feeds a ring of K (and V) tiles
// by TMA; a thread of warp 9 issues the products; warps 0-3 and 4-7 own the 128 rows, thread = row,
// for the lower and the upper 64 keys of a tile.  Two score buffers: S of the next tile is formed under
// phi of this one, and the thread that issues the products needs one hand-off per tile, "P is
// written", since products run in the order of their issue (P V of tile j, then S of tile j + 2 into
// the same columns).  Query rows are gathered by their own threads (a head's rows are G at a time in
// memory) into tensor memory, from where the products read them: shared memory is all ring.
//
// One row tile per CTA leaves registers and shared memory for a CTA of the kernels that stream the
// sequences' own keys (decode.cu), which are launched behind these as dependents and run beside
// them: this part is bound by the tile loads into an SM and the chain of its steps, that one by HBM.
#include "decode_split.cuh"
#include "phi.cuh"

namespace raattn {
namespace {

constexpr int BM = 128, BN = 128;
constexpr int SOFTMAX_WARPS = 8, PRODUCER_WARP = 8, MMA_WARP = 9;
constexpr int THREADS = 32 * 10;
// score buffer b at column 128 b, O behind both, then Q (bf16 pairs), in all that there is
constexpr uint32_t TMEM_O = 256, TMEM_Q = 384, TMEM_COLS = 512;
constexpr int SPLIT_BATCH = 512;          // up to so many sequences' block counts are kept in shared memory
constexpr int BOX_BYTES = 128 * 64 * 2;   // one TMA box: 128 rows x 64 values

template <int D, bool VALUES>
struct Cfg {
  static constexpr int TILE_BYTES = BN * D * 2;
  static constexpr int NSTAGE = D == 128 ? 5 : 8;
  static constexpr int OFF_BAR = NSTAGE * TILE_BYTES;
  // q_full, ring_full[], ring_empty[], s_full[2], handed[2], o_full, drain
  static constexpr int NUM_BARS = 1 + 2 * NSTAGE + 6;
  static constexpr int OFF_MISC = (OFF_BAR + NUM_BARS * 8 + 15) / 16 * 16;   // tmem base, abort flag, votes [2][8]
  static constexpr int OFF_HALF = OFF_MISC + 16 + 2 * SOFTMAX_WARPS * 4;     // the upper halves' row results
  static constexpr int OFF_CUM = OFF_HALF + BM * 4;
  static constexpr int SMEM_BYTES = OFF_CUM + (VALUES ? (SPLIT_BATCH + 2) * 4 : 0);
  // beside it, on one SM, a CTA of decode_values_kernel of 63.5 KB
  static_assert(SMEM_BYTES + 1024 + 65024 <= 233472, "shared memory per SM");
  static_assert(NSTAGE * TILE_BYTES >= SOFTMAX_WARPS * 4096, "the output leaves through the ring");
};

// phi of 32 columns of a row, as bf16 or (TWO) as two of them; d = m - s is exact 0 at the maximum; columns
// from `n` on are not keys.
template <bool RAGGED, bool TWO>
__device__ __forceinline__ float phi_chunk(const uint32_t (&h)[32], uint32_t (&pk)[16], uint32_t (&lo)[16],
                                           int n, float c2, float m) {
  float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int c = 0; c < 32; c += 4) {
    float x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[e] = u2f(h[c + e]) - m;
      if (RAGGED && c + e >= n) x[e] = -INFINITY;
    }
    float2 p0, p1;
    phi_quad(x[0], x[1], x[2], x[3], c2, 0.5f, p0, p1);
    sum = __fadd2_rn(sum, __fadd2_rn(p0, p1));
    if constexpr (TWO) {
      split_bf16x2(p0.x, p0.y, pk[c / 2], lo[c / 2]);
      split_bf16x2(p1.x, p1.y, pk[c / 2 + 1], lo[c / 2 + 1]);
    } else {
      pk[c / 2] = pack_bf16x2(p0.x, p0.y);
      pk[c / 2 + 1] = pack_bf16x2(p1.x, p1.y);
    }
  }
  return sum.x + sum.y;
}

// The maximum of every second part of a row from part `first` on; cum: own blocks per stream of
// the sequences before each.
__device__ __forceinline__ float half_maximum(const DecodeArgs& a, const int* cum, int row, int b, int kv, int g,
                                              int first) {
  int shared, own;
  decode_row_slots(b, kv, g, cum[b], cum[b + 1], decode_split(a, cum[a.B], cum[a.B + 1]), a, shared, own);
  const float* p = a.row_max + static_cast<int64_t>(row) * a.slots;
  float m = -INFINITY;
  for (int i0 = first; i0 < shared + own; i0 += 16) {   // eight loads at a time in flight
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = i0 + 2 * j;
      y[j] = i < shared + own ? __ldcg(p + (i < shared ? i : a.pslots + i - shared)) : -INFINITY;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) m = fmaxf(m, y[j]);
  }
  return m;
}

__device__ __forceinline__ void softmax_barrier() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// Bounded as for 640 threads, that is 96 registers each: the 320 leave 34,816 of an SM's, enough
// for two CTAs of the kernels that run beside this one.
template <int D, bool VALUES, bool TWO>
__global__ void __launch_bounds__(640, 1)
    decode_prefix_kernel(const __grid_constant__ PrefixMaps maps, const DecodeArgs a, const LaunchCtx ctx) {
  using C = Cfg<D, VALUES>;
  constexpr int NST = C::NSTAGE;
  extern __shared__ uint8_t smem_raw[];
  if (smem_u32(smem_raw) & 1023u) {   // uniform over the CTA: nothing has started
    if (threadIdx.x == 0) atomicOr(ctx.status, kStatusBadSmem);
    return;
  }
  uint8_t* smem = smem_raw;
  uint8_t* sRing = smem;
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* ring_full = q_full + 1;
  uint64_t* ring_empty = ring_full + NST;
  uint64_t* s_full = ring_empty + NST;   // [2] per score buffer: S is formed
  uint64_t* handed = s_full + 2;         // [2] max: its scores are in registers; values: P is written over them
  uint64_t* o_full = handed + 2;
  uint64_t* drain = o_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  volatile int* live = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 16);   // [2][8] the softmax warps' votes
  float* half = reinterpret_cast<float*>(smem + C::OFF_HALF);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // item: key head fastest (its neighbours read other keys), then row tile, then key split
  const int rows = a.B * a.G, row_tiles = (rows + BM - 1) / BM;
  const int kv = blockIdx.x % a.Hkv, rest = blockIdx.x / a.Hkv;
  const int x0 = rest % row_tiles * BM, split = rest / row_tiles;
  const int tps = a.pchunk / BN, t0 = split * tps;
  const int nt = min(t0 + tps, (a.P + BN - 1) / BN) - t0;   // this CTA's key tiles, at least one

  if (threadIdx.x == 0) {
    mbar_init(q_full, SOFTMAX_WARPS);
    for (int i = 0; i < NST; ++i) {
      mbar_init(&ring_full[i], 1);
      mbar_init(&ring_empty[i], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&s_full[b], 1);
      mbar_init(&handed[b], SOFTMAX_WARPS);
    }
    mbar_init(o_full, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == MMA_WARP) {
    tmem_alloc(tmem_slot, TMEM_COLS);
    tmem_relinquish();
  }
  if constexpr (!VALUES) release_dependents();
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
      // values: the last use of K and the only one of V in this call (B64 C4096 P32768 150.8 us -> 148.7)
      uint64_t policy;
      asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
      auto issue = [&](const CUtensorMap* map, int j) -> bool {
        const int st = it % NST;
        const uint32_t par = (it / NST) & 1u;
        if (!mbar_wait(&ring_empty[st], par ^ 1u, abort_flag, ctx)) return false;
        mbar_arrive_expect_tx(&ring_full[st], C::TILE_BYTES);
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          void* box = sRing + st * C::TILE_BYTES + c * BOX_BYTES;
          if (VALUES) tma_load_3d(box, map, &ring_full[st], c * 64, (t0 + j) * BN, kv, policy);
          else tma_load_3d(box, map, &ring_full[st], c * 64, (t0 + j) * BN, kv);
        }
        issued[st] = true;
        last_par[st] = par;
        ++it;
        return true;
      };
      bool ok = true;
      ok = issue(&maps.k, 0);   // values: K_0, then K_(j+1) and V_j
      for (int j = 0; j < nt && ok; ++j) {
        if (j + 1 < nt) ok = issue(&maps.k, j + 1);
        if (VALUES && ok) ok = issue(&maps.v, j);
      }
      for (int i = 0; i < NST; ++i)
        if (issued[i]) drain_wait(&ring_full[i], last_par[i], ctx);
    }
  } else if (warp == MMA_WARP) {
    if (lane == 0) {
      constexpr uint32_t idesc_qk = idesc_bf16_f32(BM, BN, 0, 0);
      constexpr uint32_t idesc_pv = idesc_bf16_f32(BM, D, 0, 1);
      constexpr uint32_t HI = sdesc_hi_sw128(1024);
      const uint32_t ring = smem_u32(sRing);
      uint32_t pos = 0;
      bool o_started = false;
      auto ring_wait = [&](uint32_t p, uint32_t& addr) -> bool {
        const int st = p % NST;
        if (!mbar_wait(&ring_full[st], (p / NST) & 1u, abort_flag, ctx)) return false;
        tc_fence_after();
        addr = ring + st * C::TILE_BYTES;
        return true;
      };
      auto mma_s = [&](int j) -> bool {   // S of tile j into its buffer, and its ring stage back
        uint32_t kaddr;
        const uint32_t p = pos++;
        if (!ring_wait(p, kaddr)) return false;
        const uint32_t klo = sdesc_lo(kaddr, 16), col = tmem + 128 * (j & 1);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * BOX_BYTES + (kk & 3) * 32) >> 4;
          tc_mma_f16_ts(col, tmem + TMEM_Q + kk * 8, sdesc(klo + off, HI), idesc_qk, kk > 0 ? 1u : 0u);
        }
        tc_commit(&s_full[j & 1]);
        tc_commit(&ring_empty[p % NST]);
        return true;
      };
      // scores of tile j taken (max), or P of it written (values)
      auto handed_over = [&](int j) -> bool {
        if (!mbar_wait(&handed[j & 1], (j >> 1) & 1, abort_flag, ctx)) return false;
        tc_fence_after();
        return true;
      };
      auto mma_pv = [&](int j) -> bool {   // O += P V of tile j, unless P is 0
        uint32_t vaddr;
        const uint32_t p = pos++;
        if (!ring_wait(p, vaddr) || !handed_over(j)) return false;
        int any = 0;
#pragma unroll
        for (int w = 0; w < SOFTMAX_WARPS; ++w) any |= live[(j & 1) * SOFTMAX_WARPS + w];
        if (any) {
          const uint32_t vlo = sdesc_lo(vaddr, BOX_BYTES), col = tmem + TMEM_O, pcol = tmem + 128 * (j & 1);
#pragma unroll
          for (int kk = 0; kk < BN / 16; ++kk) {
            const uint32_t acol = pcol + (kk >> 1) * 32 + (kk & 1) * 8;   // P over its own scores, 32 keys at a time
            const uint32_t boff = (kk * 16 * 128) >> 4;                    // V: MN-major, 16 key rows
            tc_mma_f16_ts(col, acol, sdesc(vlo + boff, HI), idesc_pv, kk > 0 || o_started ? 1u : 0u);
            if constexpr (TWO) tc_mma_f16_ts(col, acol + 16, sdesc(vlo + boff, HI), idesc_pv, 1u);
          }
          o_started = true;
        }
        tc_commit(&ring_empty[p % NST]);
        return true;
      };
      bool ok = mbar_wait(q_full, 0, abort_flag, ctx);
      // test knob: nothing is committed to `drain` yet, so this wait can only time out
      if (ok && ctx.force_timeout) ok = mbar_wait(drain, 0, abort_flag, ctx);
      tc_fence_after();
      ok = ok && mma_s(0);
      for (int j = 0; j < nt && ok; ++j) {
        if constexpr (VALUES) {   // S(j + 1) goes where P(j - 1) was, whose product has been issued
          if (j + 1 < nt) ok = mma_s(j + 1);
          ok = ok && mma_pv(j);
        } else if (j + 1 < nt) {   // S(j + 1) goes where S(j - 1) was
          ok = (j == 0 || handed_over(j - 1)) && mma_s(j + 1);
        }
      }
      if (ok) tc_commit(o_full);
      tc_commit(drain);
      drain_wait(drain, 0, ctx);
    }
  } else {
    const int quarter = warp & 3, upper = warp >> 2;   // rows 32 quarter .., keys 64 upper .. of a tile
    const int row_local = quarter * 32 + lane, x = x0 + row_local;
    const bool row_ok = x < rows;
    const int b = row_ok ? x / a.G : 0, g = row_ok ? x - b * a.G : 0;
    const int row = b * a.Hq + kv * a.G + g;
    auto warp_wait = [&](uint64_t* bar, uint32_t par) -> bool {
      int r = 1;
      if (lane == 0) r = mbar_wait(bar, par, abort_flag, ctx) ? 1 : 0;
      return __shfl_sync(0xffffffffu, r, 0) != 0;
    };
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    {   // this row's half of Q
      const uint4* q = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + static_cast<int64_t>(row) * D) +
                       upper * (D / 16);
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 v = row_ok ? q[c * 4 + i] : make_uint4(0, 0, 0, 0);
          w[4 * i] = v.x;
          w[4 * i + 1] = v.y;
          w[4 * i + 2] = v.z;
          w[4 * i + 3] = v.w;
        }
        tmem_st16(lanes + TMEM_Q + upper * (D / 4) + c * 16, w);
      }
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
    }
    const int tail = a.P - t0 * BN - 64 * upper;   // keys from this half's first on
    bool ok = true;
    uint32_t h[32];
    // 32 columns of this half's scores of tile j into registers
    auto take = [&](int j, int c) {
      tmem_ld32(lanes + 128 * (j & 1) + 64 * upper + c, h);
      tc_wait_ld();
    };
    auto formed = [&](int j) -> bool {
      if (!warp_wait(&s_full[j & 1], (j >> 1) & 1)) return false;
      tc_fence_after();
      return true;
    };
    auto hand = [&](int j) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&handed[j & 1]);
    };
    if constexpr (!VALUES) {
      float m = -INFINITY;
      for (int j = 0; j < nt; ++j) {
        ok = formed(j);
        if (!ok) break;
        float u0 = -INFINITY, u1 = -INFINITY;
#pragma unroll
        for (int c0 = 0; c0 < 64; c0 += 32) {
          take(j, c0);
          if (c0) hand(j);
          if (j * BN + c0 + 32 <= tail) {
#pragma unroll
            for (int c = 0; c < 32; c += 4) {
              u0 = max3f(u0, u2f(h[c]), u2f(h[c + 1]));
              u1 = max3f(u1, u2f(h[c + 2]), u2f(h[c + 3]));
            }
          } else {
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (j * BN + c0 + c < tail) u0 = fmaxf(u0, u2f(h[c]));
          }
        }
        m = fmaxf(m, fmaxf(u0, u1));
      }
      if (upper) half[row_local] = m;
      softmax_barrier();
      if (!upper && ok && row_ok) a.row_max[static_cast<int64_t>(row) * a.slots + split] = fmaxf(m, half[row_local]);
    } else {
      // While the maxima are still being formed: where this row's parts are, from the lengths.
      int* cum = reinterpret_cast<int*>(smem + C::OFF_CUM);
      if (warp == 0 && a.B <= SPLIT_BATCH) {
        int run = 0, longest = 0;
        for (int i = 0; i < a.B; i += 32) {
          int n = i + lane < a.B ? (decode_own_length(a, i + lane) + a.block - 1) / a.block : 0;
          longest = max(longest, n);
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, n, o);
            if (lane >= o) n += v;
          }
          if (i + lane < a.B) cum[i + lane + 1] = run + n;
          run += __shfl_sync(0xffffffffu, n, 31);
        }
        longest = __reduce_max_sync(0xffffffffu, longest);
        if (lane == 0) {
          cum[0] = 0;
          cum[a.B + 1] = longest;
        }
      }
      // All maxima, which the sequences' own values, the next kernel, need no less; the first tiles are
      // on their way, and the first scores formed, meanwhile.
      await_previous();
      release_dependents();
      softmax_barrier();
      float m = row_ok ? half_maximum(a, a.B <= SPLIT_BATCH ? cum : a.cum, row, b, kv, g, upper) : 0.0f;
      if (upper) half[row_local] = m;
      softmax_barrier();
      if (!upper) half[row_local] = m = fmaxf(m, half[row_local]);
      softmax_barrier();
      m = half[row_local];
      const float c2 = a.scale * (1.0f / 32.0f);
      float total = 0.0f;
      for (int j = 0; j < nt; ++j) {
        ok = formed(j);
        if (!ok) break;
        float t = 0.0f;
#pragma unroll
        for (int c0 = 0; c0 < 64; c0 += 32) {
          take(j, c0);
          const int n = tail - j * BN - c0;
          uint32_t pk[16], lo[16];
          t += n < 32 ? phi_chunk<true, TWO>(h, pk, lo, n, c2, m) : phi_chunk<false, TWO>(h, pk, lo, n, c2, m);
          // P over its own scores, which only this thread reads: two keys per column, 16 columns of
          // P and 16 of what its rounding left
          tmem_st16(lanes + 128 * (j & 1) + 64 * upper + c0, pk);
          if constexpr (TWO) tmem_st16(lanes + 128 * (j & 1) + 64 * upper + c0 + 16, lo);
        }
        tc_wait_st();
        total += t;
        const unsigned any = __any_sync(0xffffffffu, t > 0.0f);
        if (lane == 0) live[(j & 1) * SOFTMAX_WARPS + warp] = any ? 1 : 0;
        hand(j);
      }
      if (ok) ok = warp_wait(o_full, 0);
      softmax_barrier();   // both halves have read the row's maximum
      if (upper) half[row_local] = total;
      softmax_barrier();
      if (!upper) half[row_local] = total += half[row_local];
      softmax_barrier();
      total = half[row_local];
      if (ok) {
        tc_fence_after();
        // through the ring (every tile has been read), 4 KB per warp, so that whole 128-byte row
        // segments leave; the two halves take the output's columns in turn
        uint8_t* stage = sRing + warp * 4096;
        const int64_t out = row_ok && total > 0.0f ? (static_cast<int64_t>(row) * a.slots + split) * D : -1;
#pragma unroll
        for (int c0 = 32 * upper; c0 < D; c0 += 64) {
          uint32_t ov[32];
          tmem_ld32(lanes + TMEM_O + c0, ov);
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
        if (row_ok && !upper) a.part_sum[static_cast<int64_t>(row) * a.slots + split] = total;
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

template <int D, bool VALUES, bool TWO = false>
cudaError_t go(const PrefixMaps& maps, const DecodeArgs& a, const LaunchCtx& ctx, cudaStream_t st) {
  auto kernel = decode_prefix_kernel<D, VALUES, TWO>;
  const cudaError_t e = set_up_kernel<decode_prefix_kernel<D, VALUES, TWO>>(Cfg<D, VALUES>::SMEM_BYTES, true);
  if (e != cudaSuccess) return e;
  const unsigned grid = static_cast<unsigned>(a.Hkv) * ((a.B * a.G + BM - 1) / BM) * a.pslots;
  if constexpr (VALUES) return launch_dependent(kernel, grid, THREADS, Cfg<D, VALUES>::SMEM_BYTES, st, maps, a, ctx);
  kernel<<<grid, THREADS, Cfg<D, VALUES>::SMEM_BYTES, st>>>(maps, a, ctx);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decode_prefix(const PrefixMaps& maps, const DecodeArgs& a, bool values, const LaunchCtx& ctx,
                                 cudaStream_t st) {
  if (!values) return a.D == 64 ? go<64, false>(maps, a, ctx, st) : go<128, false>(maps, a, ctx, st);
  if (a.B * a.G <= BM) return a.D == 64 ? go<64, true, true>(maps, a, ctx, st) : go<128, true, true>(maps, a, ctx, st);
  return a.D == 64 ? go<64, true>(maps, a, ctx, st) : go<128, true>(maps, a, ctx, st);
}

}  // namespace raattn
