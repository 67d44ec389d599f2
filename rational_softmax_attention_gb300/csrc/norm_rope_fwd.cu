// The forward of the per-head normalisation and rotation (the mathematics: norm_rope.cuh).
#include "norm_rope.cuh"

namespace raattn {
namespace {

using namespace norm_rope;

constexpr int U = 2;       // rows a lane group works on together
constexpr int kAhead = 4;  // batches of U rows in flight: 32 KB per CTA

template <typename T, int D, int NORM>
__global__ void __launch_bounds__(kThreads, 2) norm_rope_fwd_kernel(const NormRopeShape a, const NormRopeFwd io) {
  constexpr int E = Vec<T>::E, P = E / 2, L = D / E, NG = kThreads / L;
  __shared__ Tables tb;
  __shared__ uint4 ring[kAhead * U][kThreads];
  const int g = threadIdx.x / L, gl = threadIdx.x % L, lane = threadIdx.x & 31;
  const int tl = g % a.tile;
  const Walk walk = make_walk<U>(a, g, NG);
  const Partner pt = find_partner<E>(a, gl, lane);
  const int64_t tokens = static_cast<int64_t>(a.B) * a.N;
  const int64_t tiles = (tokens + a.tile - 1) / a.tile;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  if (a.pairs) init_turns(tb, a);
  int buf = 0;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x, buf ^= 1) {
    const int64_t tok = tile * a.tile + tl;
    const bool there = tok < tokens;
    const int b = there ? static_cast<int>(tok / a.N) : 0;
    const int n = there ? static_cast<int>(tok - static_cast<int64_t>(b) * a.N) : 0;
    const T* row = static_cast<const T*>(a.qkv) + b * a.batch_stride + n * a.token_stride + gl * E;
    auto fetch = [&](int i) {
      int kind, h, heads;
      batch_of<U>(walk, i, a, kind, h, heads);
      const T* src = row + (kind == 0 ? 0 : kind == 1 ? a.Hq : a.Hq + a.Hkv) * D;
#pragma unroll
      for (int j = 0; j < U; ++j, h += walk.hstep) {
        const bool in = there && i < walk.all && h < heads;
        copy_own(&ring[i % kAhead * U + j][threadIdx.x], in ? src + h * D : a.qkv, in);
      }
      copy_commit();
    };
#pragma unroll 1
    for (int i = 0; i < kAhead; ++i) fetch(i);
    // the slot of this token's keys and values, or -1 where they are not to be written
    int slot = n;
    if (io.start) {
      const int64_t s = static_cast<int64_t>(io.start[b]) + n;
      slot = s < 0 || s >= io.capacity || (io.count && n >= io.count[b]) ? -1 : static_cast<int>(s);
    }
    const int64_t q_at = (static_cast<int64_t>(b) * a.Hq * a.N + n) * D + gl * E;
    const int64_t kv_at = (static_cast<int64_t>(b) * a.Hkv * io.capacity + slot) * D + gl * E;
    if (a.pairs) {   // under the first rows' copies
      fill_table(tb, buf, a, tile * a.tile);
      __syncthreads();
    }
    float2 A[P], Bp[P], C[P];
#pragma unroll 1
    for (int i = 0; i < walk.all; ++i) {
      copy_wait<kAhead - 1>();
      uint4 u[U];
#pragma unroll
      for (int j = 0; j < U; ++j) u[j] = ring[i % kAhead * U + j][threadIdx.x];
      int kind, h, heads;
      batch_of<U>(walk, i, a, kind, h, heads);
      T* out = static_cast<T*>(kind == 0 ? io.q : kind == 1 ? io.k : io.v) + (kind == 0 ? q_at : kv_at);
      const int64_t step = static_cast<int64_t>(kind == 0 ? a.N : io.capacity) * D;
      const bool writes = there && (kind == 0 || slot >= 0);
      if (kind < 2) {
        if (i == 0 || i == walk.q) {   // the factors of this kind at this token
          Turn<P> t;
          if (a.pairs) load_turn<E>(t, tb, buf, tl, gl, pt, a);
          uint4 wu = zero, bu = zero;
          if (NORM != RA_NORM_NONE) wu = reinterpret_cast<const uint4*>(kind ? a.kw : a.qw)[gl];
          const void* bias = kind ? a.kb : a.qb;
          if (NORM == RA_NORM_LAYER && bias) bu = reinterpret_cast<const uint4*>(bias)[gl];
          float2 w[P], wp[P], c[P], cp[P];
          Vec<T>::get(wu, w);
          Vec<T>::get(bu, c);
          if (a.pairs) {
            partners<T>(wu, w, wp, pt, a.interleaved);
            partners<T>(bu, c, cp, pt, a.interleaved);
          }
#pragma unroll
          for (int k = 0; k < P; ++k) {
            if (NORM == RA_NORM_NONE) w[k] = wp[k] = f2(1.0f);
            A[k] = a.pairs ? __fmul2_rn(w[k], t.cs[k]) : w[k];
            Bp[k] = a.pairs ? __fmul2_rn(wp[k], t.sn[k]) : f2(0.0f);
            if (NORM == RA_NORM_LAYER) C[k] = a.pairs ? __ffma2_rn(cp[k], t.sn[k], __fmul2_rn(c[k], t.cs[k])) : c[k];
          }
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
          float2 x[P], p[P];
          Vec<T>::get(u[j], x);
          if (a.pairs) partners<T>(u[j], x, p, pt, a.interleaved);
          if (NORM == RA_NORM_LAYER) {
            const float2 m = f2(-row_sum<P, L>(x) * (1.0f / D));
#pragma unroll
            for (int k = 0; k < P; ++k) {
              x[k] = __fadd2_rn(x[k], m);
              p[k] = __fadd2_rn(p[k], m);
            }
          }
          const float r = NORM != RA_NORM_NONE ? inverse_rms(row_dot<P, L>(x, x) * (1.0f / D), a.eps) : 1.0f;
#pragma unroll
          for (int k = 0; k < P; ++k) {
            x[k] = __fmul2_rn(x[k], A[k]);
            if (a.pairs) x[k] = __ffma2_rn(p[k], Bp[k], x[k]);
            if (NORM == RA_NORM_LAYER) x[k] = __ffma2_rn(x[k], f2(r), C[k]);
            if (NORM == RA_NORM_RMS) x[k] = __fmul2_rn(x[k], f2(r));
          }
          u[j] = Vec<T>::put(x);
        }
      }
#pragma unroll
      for (int j = 0; j < U; ++j, h += walk.hstep)
        if (writes && h < heads) *reinterpret_cast<uint4*>(out + h * step) = u[j];
      fetch(i + kAhead);
    }
  }
}

template <typename T, int D>
void go(const NormRopeShape& a, const NormRopeFwd& io, int grid, cudaStream_t st) {
  if (a.norm == RA_NORM_NONE) norm_rope_fwd_kernel<T, D, RA_NORM_NONE><<<grid, kThreads, 0, st>>>(a, io);
  else if (a.norm == RA_NORM_RMS) norm_rope_fwd_kernel<T, D, RA_NORM_RMS><<<grid, kThreads, 0, st>>>(a, io);
  else norm_rope_fwd_kernel<T, D, RA_NORM_LAYER><<<grid, kThreads, 0, st>>>(a, io);
}

}  // namespace

cudaError_t launch_norm_rope_fwd(NormRopeShape a, const NormRopeFwd& io, bool bf16, cudaStream_t st) {
  a.tile = tile_for(a, bf16 ? 2 : 4);
  const int64_t tiles = (static_cast<int64_t>(a.B) * a.N + a.tile - 1) / a.tile;
  const int grid = static_cast<int>(tiles < 4 * kSms ? tiles : 4 * kSms);
  if (bf16) {
    if (a.D == 16) go<__nv_bfloat16, 16>(a, io, grid, st);
    if (a.D == 32) go<__nv_bfloat16, 32>(a, io, grid, st);
    if (a.D == 64) go<__nv_bfloat16, 64>(a, io, grid, st);
    if (a.D == 128) go<__nv_bfloat16, 128>(a, io, grid, st);
  } else {
    if (a.D == 16) go<float, 16>(a, io, grid, st);
    if (a.D == 32) go<float, 32>(a, io, grid, st);
    if (a.D == 64) go<float, 64>(a, io, grid, st);
    if (a.D == 128) go<float, 128>(a, io, grid, st);
  }
  return cudaGetLastError();
}

}  // namespace raattn
