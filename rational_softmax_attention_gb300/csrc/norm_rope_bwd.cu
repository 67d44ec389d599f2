// The gradient of the per-head normalisation and rotation (the mathematics: norm_rope.cuh).
#include "norm_rope.cuh"

namespace raattn {
namespace {

using namespace norm_rope;

constexpr int U = 2;       // rows a lane group works on together
constexpr int kAhead = 3;  // batches of U rows, gradient and projection, in flight: 48 KB per CTA

// Each lane keeps its elements' sums of the four parameter gradients over all rows that it meets; a
// CTA adds its lane groups' sums in a fixed order and writes them to its own place of the
// workspace, and norm_rope_param_kernel adds the CTAs', so results do not depend on the order in
// which CTAs run.
template <typename T, int D, int NORM>
__global__ void __launch_bounds__(kThreads, 2) norm_rope_bwd_kernel(const NormRopeShape a, const NormRopeBwd io) {
  constexpr int E = Vec<T>::E, P = E / 2, L = D / E, NG = kThreads / L;
  extern __shared__ uint4 ring[];   // [kAhead][U][gradient, projection][kThreads]; the CTA's sums at the end
  __shared__ Tables tb;
  const int g = threadIdx.x / L, gl = threadIdx.x % L, lane = threadIdx.x & 31;
  const int tl = g % a.tile;
  const Walk walk = make_walk<U>(a, g, NG);
  const Partner pt = find_partner<E>(a, gl, lane);
  const int64_t tokens = static_cast<int64_t>(a.B) * a.N;
  const int64_t tiles = (tokens + a.tile - 1) / a.tile;
  if (a.pairs) init_turns(tb, a);
  float2 acc[4][P];   // q weight, q bias, k weight, k bias
#pragma unroll
  for (int j = 0; j < P; ++j) acc[0][j] = acc[1][j] = acc[2][j] = acc[3][j] = f2(0.0f);
  int buf = 0;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x, buf ^= 1) {
    const int64_t tok = tile * a.tile + tl;
    const bool there = tok < tokens;
    const int b = there ? static_cast<int>(tok / a.N) : 0;
    const int n = there ? static_cast<int>(tok - static_cast<int64_t>(b) * a.N) : 0;
    const T* row = static_cast<const T*>(a.qkv) + b * a.batch_stride + n * a.token_stride + gl * E;
    T* out_row = static_cast<T*>(io.dqkv) + tok * static_cast<int64_t>(a.Hq + 2 * a.Hkv) * D + gl * E;
    const int64_t step = static_cast<int64_t>(a.N) * D;
    const int64_t q_at = (static_cast<int64_t>(b) * a.Hq * a.N + n) * D + gl * E;
    const int64_t kv_at = (static_cast<int64_t>(b) * a.Hkv * a.N + n) * D + gl * E;
    auto slot_of = [&](int i, int j, int which) { return &ring[((i % kAhead * U + j) * 2 + which) * kThreads + threadIdx.x]; };
    // the incoming gradient, and the projection's row where the norm needs it
    auto fetch = [&](int i) {
      int kind, h, heads;
      batch_of<U>(walk, i, a, kind, h, heads);
      const T* src = static_cast<const T*>(kind == 0 ? io.dq : kind == 1 ? io.dk : io.dv) + (kind == 0 ? q_at : kv_at);
      const T* from = row + (kind == 0 ? 0 : a.Hq) * D;
#pragma unroll
      for (int j = 0; j < U; ++j, h += walk.hstep) {
        const bool in = there && i < walk.all && h < heads;
        copy_own(slot_of(i, j, 0), in ? src + h * step : io.dq, in);
        if (NORM != RA_NORM_NONE && kind < 2) copy_own(slot_of(i, j, 1), in ? from + h * D : a.qkv, in);
      }
      copy_commit();
    };
#pragma unroll 1
    for (int i = 0; i < kAhead; ++i) fetch(i);
    Turn<P> t;
    if (a.pairs) {
      fill_table(tb, buf, a, tile * a.tile);
      __syncthreads();
      load_turn<E>(t, tb, buf, tl, gl, pt, a);
#pragma unroll
      for (int k = 0; k < P; ++k) t.sn[k] = make_float2(-t.sn[k].x, -t.sn[k].y);   // back by the angle
    }
    // the rows of one kind
    auto rows = [&](int i, int end, const void* weight, float2 (&dw)[P], float2 (&db)[P]) {
      float2 w[P];
      if (NORM != RA_NORM_NONE) Vec<T>::get(reinterpret_cast<const uint4*>(weight)[gl], w);
#pragma unroll 1
      for (; i < end; ++i) {
        copy_wait<kAhead - 1>();
        int kind, h, heads;
        batch_of<U>(walk, i, a, kind, h, heads);
        T* out = out_row + (kind == 0 ? h : a.Hq + h) * D;
        uint4 u[U], v[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
          u[j] = *slot_of(i, j, 0);
          if (NORM != RA_NORM_NONE) v[j] = *slot_of(i, j, 1);
        }
#pragma unroll
        for (int j = 0; j < U; ++j, h += walk.hstep, out += walk.hstep * D) {
          float2 d[P], p[P];
          Vec<T>::get(u[j], d);
          if (a.pairs) {
            partners<T>(u[j], d, p, pt, a.interleaved);
#pragma unroll
            for (int k = 0; k < P; ++k) d[k] = __ffma2_rn(p[k], t.sn[k], __fmul2_rn(d[k], t.cs[k]));
          }
          if (NORM != RA_NORM_NONE) {
            float2 x[P];
            Vec<T>::get(v[j], x);
            if (NORM == RA_NORM_LAYER) {
              const float2 m = f2(-row_sum<P, L>(x) * (1.0f / D));
#pragma unroll
              for (int k = 0; k < P; ++k) x[k] = __fadd2_rn(x[k], m);
            }
            const float r = inverse_rms(row_dot<P, L>(x, x) * (1.0f / D), a.eps);
#pragma unroll
            for (int k = 0; k < P; ++k) {
              x[k] = __fmul2_rn(x[k], f2(r));
              dw[k] = __ffma2_rn(d[k], x[k], dw[k]);   // a row that is not there has d = 0 and adds nothing
              if (NORM == RA_NORM_LAYER) db[k] = __fadd2_rn(db[k], d[k]);
              d[k] = __fmul2_rn(d[k], w[k]);
            }
            const float s2 = row_dot<P, L>(d, x) * (-1.0f / D);
            const float s1 = NORM == RA_NORM_LAYER ? row_sum<P, L>(d) * (-1.0f / D) : 0.0f;
#pragma unroll
            for (int k = 0; k < P; ++k) {
              const float2 c = NORM == RA_NORM_LAYER ? __ffma2_rn(x[k], f2(s2), f2(s1)) : __fmul2_rn(x[k], f2(s2));
              d[k] = __fmul2_rn(__fadd2_rn(d[k], c), f2(r));
            }
          }
          if (there && h < heads) *reinterpret_cast<uint4*>(out) = Vec<T>::put(d);
        }
        fetch(i + kAhead);
      }
    };
    rows(0, walk.q, a.qw, acc[0], acc[1]);
    rows(walk.q, walk.k, a.kw, acc[2], acc[3]);
#pragma unroll 1
    for (int i = walk.k; i < walk.all; ++i) {   // dv as it is
      copy_wait<kAhead - 1>();
      int kind, h, heads;
      batch_of<U>(walk, i, a, kind, h, heads);
#pragma unroll
      for (int j = 0; j < U; ++j, h += walk.hstep)
        if (there && h < heads) *reinterpret_cast<uint4*>(out_row + (a.Hq + a.Hkv + h) * D) = *slot_of(i, j, 0);
      fetch(i + kAhead);
    }
  }
  if (NORM == RA_NORM_NONE) return;
  copy_wait<0>();
  float* part = reinterpret_cast<float*>(ring);   // [NG][D]
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < P; ++j) *reinterpret_cast<float2*>(&part[g * D + gl * E + 2 * j]) = acc[k][j];
    __syncthreads();
    for (int e = threadIdx.x; e < D; e += kThreads) {
      float s = 0.0f;
      for (int i = 0; i < NG; ++i) s += part[i * D + e];
      io.partial[(static_cast<int64_t>(blockIdx.x) * 4 + k) * D + e] = s;
    }
  }
}

// dparams[4][D] = the sum over CTAs of partial[cta][4][D]: a CTA per 16 columns, 64 partial sums
// per column, whose loads are in flight together.
constexpr int kParamCols = 16, kParamSlices = 64;
__global__ void __launch_bounds__(kParamCols * kParamSlices)
    norm_rope_param_kernel(const float* partial, float* dparams, int ctas, int cols) {
  __shared__ float part[kParamSlices][kParamCols];
  const int c = threadIdx.x % kParamCols, s = threadIdx.x / kParamCols, col = blockIdx.x * kParamCols + c;
  float v = 0.0f;
#pragma unroll 8
  for (int i = s; i < ctas; i += kParamSlices) v += partial[static_cast<int64_t>(i) * cols + col];
  part[s][c] = v;
  __syncthreads();
  for (int o = kParamSlices / 2; o > 0; o >>= 1) {
    if (s < o) part[s][c] += part[s + o][c];
    __syncthreads();
  }
  if (s == 0) dparams[col] = part[0][c];
}

constexpr int kRingBytes = kAhead * U * 2 * kThreads * 16;
static_assert(kRingBytes >= kThreads * 8 * 4, "the lane groups' sums fit the ring");

template <typename T, int D, int NORM>
cudaError_t go(const NormRopeShape& a, const NormRopeBwd& io, int grid, cudaStream_t st) {
  auto kernel = norm_rope_bwd_kernel<T, D, NORM>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
  if (e != cudaSuccess) return e;
  kernel<<<grid, kThreads, kRingBytes, st>>>(a, io);
  if (NORM != RA_NORM_NONE)
    norm_rope_param_kernel<<<4 * D / kParamCols, kParamCols * kParamSlices, 0, st>>>(io.partial, io.dparams, grid,
                                                                                     4 * D);
  return cudaGetLastError();
}
template <typename T, int D>
cudaError_t go(const NormRopeShape& a, const NormRopeBwd& io, int grid, cudaStream_t st) {
  if (a.norm == RA_NORM_NONE) return go<T, D, RA_NORM_NONE>(a, io, grid, st);
  return a.norm == RA_NORM_RMS ? go<T, D, RA_NORM_RMS>(a, io, grid, st) : go<T, D, RA_NORM_LAYER>(a, io, grid, st);
}

}  // namespace

int norm_rope_bwd_ctas() { return 2 * kSms; }

cudaError_t launch_norm_rope_bwd(NormRopeShape a, const NormRopeBwd& io, bool bf16, cudaStream_t st) {
  a.tile = tile_for(a, bf16 ? 2 : 4);
  const int64_t tiles = (static_cast<int64_t>(a.B) * a.N + a.tile - 1) / a.tile;
  const int most = norm_rope_bwd_ctas();
  const int grid = static_cast<int>(tiles < most ? tiles : most);
  if (bf16) {
    if (a.D == 16) return go<__nv_bfloat16, 16>(a, io, grid, st);
    if (a.D == 32) return go<__nv_bfloat16, 32>(a, io, grid, st);
    if (a.D == 64) return go<__nv_bfloat16, 64>(a, io, grid, st);
    return go<__nv_bfloat16, 128>(a, io, grid, st);
  }
  if (a.D == 16) return go<float, 16>(a, io, grid, st);
  if (a.D == 32) return go<float, 32>(a, io, grid, st);
  if (a.D == 64) return go<float, 64>(a, io, grid, st);
  return go<float, 128>(a, io, grid, st);
}

}  // namespace raattn
