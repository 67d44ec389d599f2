// The forward of the per-head normalisation and rotation (the mathematics: norm_rope.cuh).
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
  const Work wk = work_of(a);
  const int g = threadIdx.x / L, gl = threadIdx.x % L;
  const int tl = g % wk.tile, hs = g / wk.tile, hstep = NG / wk.tile;
  const int rows = (wk.heads + hstep - 1) / hstep;   // of every lane group; some may be no head
  const LaneMap lm = lane_map<E, L>(a, gl);
  const int tokens = a.B * a.N;   // fits, and so does a tile past the last
  const int tiles = (tokens - 1) / wk.tile + 1;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const bool turns = a.pairs > 0 && wk.kind < 2, whole = 2 * a.pairs == D;
  if (turns) init_turns(tb, a);
  int buf = 0;
  for (int tile = wk.first; tile < tiles; tile += wk.step, buf ^= 1) {
    const int tok = tile * wk.tile + tl;
    const bool there = tok < tokens;
    const int b = there ? tok / a.N : 0, n = there ? tok - b * a.N : 0;
    const T* src = static_cast<const T*>(a.qkv) + b * a.batch_stride + n * a.token_stride + (wk.head0 + hs) * D;
    int ahead = 0;
    auto fetch = [&]() {
      if (ahead < rows) {   // nothing past the tile's rows: every copy is waited for before its slot is used again
        const bool in = there && hs + ahead * hstep < wk.heads;
        uint4* slot = &ring[ahead % kAhead][0][threadIdx.x];
        copy_own(slot, in ? src + lm.v0 * E : a.qkv, in);
        copy_own(slot + kThreads, in ? src + lm.v1 * E : a.qkv, in);
      }
      copy_commit();
      ++ahead;
      src += hstep * D;
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch();
    // where this token's rows go; keys and values to a slot of the cache, if it is one
    bool writes = there;
    int64_t out_row, out_step;
    if (wk.kind == 0) {
      out_row = static_cast<int64_t>(b) * a.Hq * a.N + n;
      out_step = a.N;
    } else {
      int64_t slot = n;
      if (io.start) {
        slot += io.start[b];
        if (slot < 0 || slot >= io.capacity || (io.count && n >= io.count[b])) writes = false;
      }
      out_row = static_cast<int64_t>(b) * a.Hkv * io.capacity + slot;
      out_step = io.capacity;
    }
    T* out = static_cast<T*>(wk.kind == 0 ? io.q : wk.kind == 1 ? io.k : io.v) + (out_row + hs * out_step) * D;
    out_step *= static_cast<int64_t>(hstep) * D;
    float2 A0[P], B0[P], C0[P], A1[P], B1[P], C1[P];
    if (wk.kind < 2) {
      if (turns) {   // under the first rows' copies
        fill_table(tb, buf, a, tile * wk.tile, wk.tile);
        __syncthreads();
        float cs[E], sn[E];
        load_turn<E>(cs, sn, tb, buf, tl, lm, a, whole);
        factors<E>(cs, sn, a.interleaved, A0, B0, A1, B1);
      }
      if (NORM != RA_NORM_NONE) {
        const uint4* w = reinterpret_cast<const uint4*>(wk.kind ? a.kw : a.qw);
        const uint4* bias = NORM == RA_NORM_LAYER ? reinterpret_cast<const uint4*>(wk.kind ? a.kb : a.qb) : nullptr;
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
    }
#pragma unroll 1
    for (int i = 0; i < rows; ++i) {
      copy_wait<kAhead - 1>();
      uint4 u0 = ring[i % kAhead][0][threadIdx.x], u1 = ring[i % kAhead][1][threadIdx.x];
      if (wk.kind < 2) {
        float2 x0[P], x1[P], p0[P], p1[P];
        Vec<T>::get(u0, x0);
        Vec<T>::get(u1, x1);
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
        u0 = Vec<T>::put(x0);
        u1 = Vec<T>::put(x1);
      }
      if (writes && hs + i * hstep < wk.heads) {
        reinterpret_cast<uint4*>(out)[lm.v0] = u0;
        reinterpret_cast<uint4*>(out)[lm.v1] = u1;
      }
      out += out_step;
      fetch();   // into the slot just read: after the stores, which needed what it held
    }
  }
}

template <typename T, int D>
void go(const NormRopeShape& a, const NormRopeFwd& io, cudaStream_t st) {
  const int grid = a.ctas[0] + a.ctas[1] + a.ctas[2];
  if (a.norm == RA_NORM_NONE) norm_rope_fwd_kernel<T, D, RA_NORM_NONE><<<grid, kThreads, 0, st>>>(a, io);
  else if (a.norm == RA_NORM_RMS) norm_rope_fwd_kernel<T, D, RA_NORM_RMS><<<grid, kThreads, 0, st>>>(a, io);
  else norm_rope_fwd_kernel<T, D, RA_NORM_LAYER><<<grid, kThreads, 0, st>>>(a, io);
}

}  // namespace

cudaError_t launch_norm_rope_fwd(NormRopeShape a, const NormRopeFwd& io, bool bf16, cudaStream_t st) {
  plan_work(&a, bf16 ? 2 : 4, 2 * kSms, {1, 1, 1});
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
