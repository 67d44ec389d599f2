// The forward of the per-head normalisation and rotation (the mathematics: norm_rope.cuh).
// bf16 B4 N8192 H16/8 D128, RMS norm: 537 MB in 86.5 us, 6.2 TB/s; fp32, the same, 1.07 GB in 176 us, 6.1 TB/s.  Four rows
// ahead per lane group: what is in flight then covers the latency at two CTAs per SM.
#include "norm_rope.cuh"

namespace raattn {
namespace {

using namespace norm_rope;

constexpr int kAhead = 4;   // rows of a lane group in flight: 32 KB per CTA

template <typename T, int D, int NORM>
__global__ void __launch_bounds__(kThreads, 2) norm_rope_fwd_kernel(const NormRopeShape a, const NormRopeFwd io) {
  constexpr int E = Vec<T>::E, P = E / 2, L = D / E / 2, NG = kThreads / L;
  __shared__ Tables tb;
  __shared__ uint4 ring[kAhead][2][kThreads];
  const int tile_tokens = a.tiles[0];
  const int g = threadIdx.x / L, gl = threadIdx.x % L;
  const int tl = g % tile_tokens, hs = g / tile_tokens, hstep = NG / tile_tokens;
  // rows of every lane group, query and key or value heads; some may be no head
  const int q_rows = (a.Hq + hstep - 1) / hstep, kv_rows = (a.Hkv + hstep - 1) / hstep;
  const LaneMap lm = lane_map<E, L>(a, gl);
  const int tokens = a.B * a.N;   // fits, and so does a tile past the last
  const int tiles = (tokens - 1) / tile_tokens + 1;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const bool turns = a.pairs > 0, whole = 2 * a.pairs == D;
  if (turns) init_turns(tb, a);
  int buf = 0;
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x, buf ^= 1) {
    const int tok = tile * tile_tokens + tl;
    const bool there = tok < tokens;
    const int b = there ? tok / a.N : 0, n = there ? tok - b * a.N : 0;
    const T* row = static_cast<const T*>(a.qkv) + b * a.batch_stride + n * a.token_stride + hs * D;
    // the rows in order: query heads, key heads, value heads
    const T* src = row;
    int f_kind = 0, f_row = 0, fetched = 0, used = 0;
    auto fetch = [&]() {
      if (f_kind < 3) {   // nothing past the tile's rows: every copy is waited for before its slot is used again
        const bool in = there && hs + f_row * hstep < (f_kind ? a.Hkv : a.Hq);
        uint4* slot = &ring[fetched % kAhead][0][threadIdx.x];
        copy_own(slot, in ? src + lm.v0 * E : a.qkv, in);
        copy_own(slot + kThreads, in ? src + lm.v1 * E : a.qkv, in);
        src += hstep * D;
        if (++f_row == (f_kind ? kv_rows : q_rows)) {
          f_row = 0;
          src = row + (++f_kind == 1 ? a.Hq : a.Hq + a.Hkv) * D;
        }
      }
      copy_commit();
      ++fetched;
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch();
    // keys and values go to a slot of the cache, if it is one
    bool kv_writes = there;
    int64_t slot = n;
    if (io.start) {
      slot += io.start[b];
      if (slot < 0 || slot >= io.capacity || (io.count && n >= io.count[b])) kv_writes = false;
    }
    const int64_t kv_at = (static_cast<int64_t>(b) * a.Hkv + hs) * io.capacity + slot;
    if (turns) {   // under the first rows' copies
      fill_table<sizeof(T) == 2>(tb, buf, a, tile * tile_tokens, tile_tokens);
      __syncthreads();
    }
#pragma unroll 1
    for (int kind = 0; kind < 2; ++kind) {
      float2 A0[P], B0[P], C0[P], A1[P], B1[P], C1[P];
      if (turns) {
        float cs[E], sn[E];
        load_turn<E>(cs, sn, tb, buf, tl, lm, a, whole);
        factors<E>(cs, sn, a.interleaved, A0, B0, A1, B1);
      }
      if (NORM != RA_NORM_NONE) {
        const uint4* w = reinterpret_cast<const uint4*>(kind ? a.kw : a.qw);
        const uint4* bias = NORM == RA_NORM_LAYER ? reinterpret_cast<const uint4*>(kind ? a.kb : a.qb) : nullptr;
        float2 w0[P], w1[P], wp0[P], wp1[P];
        if (NORM == RA_NORM_LAYER) {   // C: the bias, turned by the factors alone
          Vec<T>::get(bias ? bias[lm.v0] : zero, C0);
          Vec<T>::get(bias ? bias[lm.v1] : zero, C1);
          if (turns) {
            partners<P>(C0, C1, wp0, wp1, lm, a.interleaved, whole);
#pragma unroll
            for (int k = 0; k < P; ++k) {
              C0[k] = __ffma2_rn(wp0[k], B0[k], __fmul2_rn(C0[k], A0[k]));
              C1[k] = __ffma2_rn(wp1[k], B1[k], __fmul2_rn(C1[k], A1[k]));
            }
          }
        }
        Vec<T>::get(w[lm.v0], w0);
        Vec<T>::get(w[lm.v1], w1);
        partners<P>(w0, w1, wp0, wp1, lm, a.interleaved, whole);
#pragma unroll
        for (int k = 0; k < P; ++k) {
          A0[k] = turns ? __fmul2_rn(A0[k], w0[k]) : w0[k];
          A1[k] = turns ? __fmul2_rn(A1[k], w1[k]) : w1[k];
          if (turns) {
            B0[k] = __fmul2_rn(B0[k], wp0[k]);
            B1[k] = __fmul2_rn(B1[k], wp1[k]);
          }
        }
      }
      const int heads = kind ? a.Hkv : a.Hq, rows = kind ? kv_rows : q_rows;
      const bool writes = kind ? kv_writes : there;
      T* out = static_cast<T*>(kind ? io.k : io.q) +
               (kind ? kv_at : (static_cast<int64_t>(b) * a.Hq + hs) * a.N + n) * D;
      const int64_t out_step = static_cast<int64_t>(hstep) * (kind ? io.capacity : a.N) * D;
#pragma unroll 1
      for (int i = 0; i < rows; ++i, ++used) {
        copy_wait<kAhead - 1>();
        float2 x0[P], x1[P], p0[P], p1[P];
        Vec<T>::get(ring[used % kAhead][0][threadIdx.x], x0);
        Vec<T>::get(ring[used % kAhead][1][threadIdx.x], x1);
        if (NORM == RA_NORM_LAYER) {
          const float2 m = f2(-row_sum<P, L>(x0, x1) * (1.0f / D));
#pragma unroll
          for (int k = 0; k < P; ++k) {
            x0[k] = __fadd2_rn(x0[k], m);
            x1[k] = __fadd2_rn(x1[k], m);
          }
        }
        float2 r = f2(1.0f);
        if (NORM != RA_NORM_NONE) r = f2(inverse_rms(row_dot<P, L>(x0, x1, x0, x1) * (1.0f / D), a.eps));
        if (turns) {
          partners<P>(x0, x1, p0, p1, lm, a.interleaved, whole);
#pragma unroll
          for (int k = 0; k < P; ++k) {
            x0[k] = __ffma2_rn(p0[k], B0[k], __fmul2_rn(x0[k], A0[k]));
            x1[k] = __ffma2_rn(p1[k], B1[k], __fmul2_rn(x1[k], A1[k]));
          }
        } else if (NORM != RA_NORM_NONE) {
#pragma unroll
          for (int k = 0; k < P; ++k) {
            x0[k] = __fmul2_rn(x0[k], A0[k]);
            x1[k] = __fmul2_rn(x1[k], A1[k]);
          }
        }
#pragma unroll
        for (int k = 0; k < P; ++k) {
          if (NORM == RA_NORM_LAYER) {
            x0[k] = __ffma2_rn(x0[k], r, C0[k]);
            x1[k] = __ffma2_rn(x1[k], r, C1[k]);
          } else if (NORM == RA_NORM_RMS) {
            x0[k] = __fmul2_rn(x0[k], r);
            x1[k] = __fmul2_rn(x1[k], r);
          }
        }
        if (writes && hs + i * hstep < heads) {
          reinterpret_cast<uint4*>(out)[lm.v0] = Vec<T>::put(x0);
          reinterpret_cast<uint4*>(out)[lm.v1] = Vec<T>::put(x1);
        }
        out += out_step;
        fetch();   // into the slot just read: after the stores, which needed what it held
      }
    }
    T* out = static_cast<T*>(io.v) + kv_at * D;
    const int64_t out_step = static_cast<int64_t>(hstep) * io.capacity * D;
#pragma unroll 1
    for (int i = 0; i < kv_rows; ++i, ++used) {
      copy_wait<kAhead - 1>();
      if (kv_writes && hs + i * hstep < a.Hkv) {
        reinterpret_cast<uint4*>(out)[lm.v0] = ring[used % kAhead][0][threadIdx.x];
        reinterpret_cast<uint4*>(out)[lm.v1] = ring[used % kAhead][1][threadIdx.x];
      }
      out += out_step;
      fetch();
    }
  }
}

template <typename T, int D>
void go(const NormRopeShape& a, const NormRopeFwd& io, cudaStream_t st) {
  const int grid = a.ctas[0];
  if (a.norm == RA_NORM_NONE) norm_rope_fwd_kernel<T, D, RA_NORM_NONE><<<grid, kThreads, 0, st>>>(a, io);
  else if (a.norm == RA_NORM_RMS) norm_rope_fwd_kernel<T, D, RA_NORM_RMS><<<grid, kThreads, 0, st>>>(a, io);
  else norm_rope_fwd_kernel<T, D, RA_NORM_LAYER><<<grid, kThreads, 0, st>>>(a, io);
}

}  // namespace

cudaError_t launch_norm_rope_fwd(NormRopeShape a, const NormRopeFwd& io, bool bf16, cudaStream_t st) {
  const int groups = kThreads / (a.D * (bf16 ? 2 : 4) / 32), tokens = a.B * a.N, most = 2 * kSms;
  const int t = best_tile(tokens, groups, most, 2, [&](int step) {
    return (a.Hq + step - 1) / step + 2 * ((a.Hkv + step - 1) / step);
  });
  const int tiles = (tokens - 1) / t + 1;
  a.tiles[0] = t;
  a.ctas[0] = tiles < most ? tiles : most;
  if (bf16) {
    if (a.D == 16) go<__nv_bfloat16, 16>(a, io, st);
    if (a.D == 32) go<__nv_bfloat16, 32>(a, io, st);
    if (a.D == 64) go<__nv_bfloat16, 64>(a, io, st);
    if (a.D == 128) go<__nv_bfloat16, 128>(a, io, st);
  } else {
    if (a.D == 16) go<float, 16>(a, io, st);
    if (a.D == 32) go<float, 32>(a, io, st);
    if (a.D == 64) go<float, 64>(a, io, st);
    if (a.D == 128) go<float, 128>(a, io, st);
  }
  return cudaGetLastError();
}

}  // namespace raattn
