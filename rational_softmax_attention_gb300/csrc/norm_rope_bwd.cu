// The gradient of the per-head normalisation and rotation (the mathematics: norm_rope.cuh).
// bf16 B4 N8192 H16 D128, layer norm with biases: 1.07 GB in 201 us, 5.3 TB/s; issue slots 52% busy.  fp32 B4 N8192
// H16/8: 1.48 GB in 249 us, 5.9 TB/s.  Small ones (fp32 B3 N1001 H6/2 D64: 12.7 us) are two launches, the second of
// which starts when the first has ended.
#include "norm_rope.cuh"

namespace raattn {
namespace {

using namespace norm_rope;

constexpr int kAhead = 4;   // rows of a lane group, gradient and projection, in flight: 64 KB per CTA

// Each lane keeps its elements' sums of the weight's and the bias's gradient over all rows that it
// meets; a CTA adds its lane groups' sums in a fixed order (in short chains: one after the other, the 128 groups of
// D16 in fp32 had twice the plain form's error) and writes them to its own place of the
// workspace, and norm_rope_param_kernel adds the CTAs', so results do not depend on the order in
// which CTAs run.
template <typename T, int D, int NORM>
__global__ void __launch_bounds__(kThreads, 2) norm_rope_bwd_kernel(const NormRopeShape a, const NormRopeBwd io) {
  constexpr int E = Vec<T>::E, P = E / 2, L = D / E / 2, NG = kThreads / L;
  extern __shared__ uint4 ring[];   // [kAhead][gradient v0, v1, projection v0, v1][kThreads]; the sums at the end
  __shared__ Tables tb;
  const Work wk = work_of(a);
  const int g = threadIdx.x / L, gl = threadIdx.x % L;
  const int tl = g % wk.tile, hs = g / wk.tile, hstep = NG / wk.tile;
  const int rows = (wk.heads + hstep - 1) / hstep;
  const LaneMap lm = lane_map<E, L>(a, gl);
  const int tokens = a.B * a.N;   // fits, and so does a tile past the last
  const int tiles = (tokens - 1) / wk.tile + 1;
  const bool turns = a.pairs > 0 && wk.kind < 2, whole = 2 * a.pairs == D;
  const bool norm = NORM != RA_NORM_NONE && wk.kind < 2;
  if (turns) init_turns(tb, a);
  uint4 wu0 = make_uint4(0, 0, 0, 0), wu1 = wu0;
  if (norm) {
    wu0 = reinterpret_cast<const uint4*>(wk.kind ? a.kw : a.qw)[lm.v0];
    wu1 = reinterpret_cast<const uint4*>(wk.kind ? a.kw : a.qw)[lm.v1];
  }
  float2 dw0[P], dw1[P], db0[P], db1[P];
#pragma unroll
  for (int k = 0; k < P; ++k) dw0[k] = dw1[k] = db0[k] = db1[k] = f2(0.0f);
  int buf = 0;
  for (int tile = wk.first; tile < tiles; tile += wk.step, buf ^= 1) {
    const int tok = tile * wk.tile + tl;
    const bool there = tok < tokens;
    const int b = there ? tok / a.N : 0, n = there ? tok - b * a.N : 0;
    const T* x_src = static_cast<const T*>(a.qkv) + b * a.batch_stride + n * a.token_stride + (wk.head0 + hs) * D;
    const T* d_src = static_cast<const T*>(wk.kind == 0 ? io.dq : wk.kind == 1 ? io.dk : io.dv) +
                     ((static_cast<int64_t>(b) * wk.heads + hs) * a.N + n) * D;
    const int64_t d_step = static_cast<int64_t>(hstep) * a.N * D;
    T* out = static_cast<T*>(io.dqkv) + (static_cast<int64_t>(tok) * (a.Hq + 2 * a.Hkv) + wk.head0 + hs) * D;
    int ahead = 0;
    auto fetch = [&]() {   // the incoming gradient, and the projection's row where the norm needs it
      if (ahead < rows) {   // nothing past the tile's rows: every copy is waited for before its slot is used again
        const bool in = there && hs + ahead * hstep < wk.heads;
        uint4* slot = &ring[ahead % kAhead * 4 * kThreads + threadIdx.x];
        copy_own(slot, in ? d_src + lm.v0 * E : io.dq, in);
        copy_own(slot + kThreads, in ? d_src + lm.v1 * E : io.dq, in);
        if (norm) {
          copy_own(slot + 2 * kThreads, in ? x_src + lm.v0 * E : a.qkv, in);
          copy_own(slot + 3 * kThreads, in ? x_src + lm.v1 * E : a.qkv, in);
        }
      }
      copy_commit();
      ++ahead;
      d_src += d_step;
      x_src += hstep * D;
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch();
    float cs[E], sn[E];
    if (turns) {
      fill_table<sizeof(T) == 2>(tb, buf, a, tile * wk.tile, wk.tile);
      __syncthreads();
      load_turn<E>(cs, sn, tb, buf, tl, lm, a, whole);
#pragma unroll
      for (int j = 0; j < E; ++j) sn[j] = -sn[j];   // back by the angle
    }
#pragma unroll 1
    for (int i = 0; i < rows; ++i) {
      copy_wait<kAhead - 1>();
      const uint4* slot = &ring[i % kAhead * 4 * kThreads + threadIdx.x];
      uint4 u0 = slot[0], u1 = slot[kThreads], v0 = u0, v1 = u1;
      if (norm) {
        v0 = slot[2 * kThreads];
        v1 = slot[3 * kThreads];
      }
      if (wk.kind < 2) {
        float2 d0[P], d1[P];
        Vec<T>::get(u0, d0);
        Vec<T>::get(u1, d1);
        if (turns) {
          float2 a0[P], b0[P], a1[P], b1[P], p0[P], p1[P];
          factors<E>(cs, sn, a.interleaved, a0, b0, a1, b1);
          partners<P>(d0, d1, p0, p1, lm, a.interleaved, whole);
#pragma unroll
          for (int k = 0; k < P; ++k) {
            d0[k] = __ffma2_rn(p0[k], b0[k], __fmul2_rn(d0[k], a0[k]));
            d1[k] = __ffma2_rn(p1[k], b1[k], __fmul2_rn(d1[k], a1[k]));
          }
        }
        if (NORM != RA_NORM_NONE) {
          float2 x0[P], x1[P], w0[P], w1[P];
          Vec<T>::get(v0, x0);
          Vec<T>::get(v1, x1);
          if (NORM == RA_NORM_LAYER) {
            const float2 m = f2(-row_sum<P, L>(x0, x1) * (1.0f / D));
#pragma unroll
            for (int k = 0; k < P; ++k) {
              x0[k] = __fadd2_rn(x0[k], m);
              x1[k] = __fadd2_rn(x1[k], m);
            }
          }
          const float2 r = f2(inverse_rms(row_dot<P, L>(x0, x1, x0, x1) * (1.0f / D), a.eps));
          Vec<T>::get(wu0, w0);
          Vec<T>::get(wu1, w1);
#pragma unroll
          for (int k = 0; k < P; ++k) {   // a row that is not there has d = 0 and adds nothing
            x0[k] = __fmul2_rn(x0[k], r);
            x1[k] = __fmul2_rn(x1[k], r);
            dw0[k] = __ffma2_rn(d0[k], x0[k], dw0[k]);
            dw1[k] = __ffma2_rn(d1[k], x1[k], dw1[k]);
            if (NORM == RA_NORM_LAYER) {
              db0[k] = __fadd2_rn(db0[k], d0[k]);
              db1[k] = __fadd2_rn(db1[k], d1[k]);
            }
            d0[k] = __fmul2_rn(d0[k], w0[k]);
            d1[k] = __fmul2_rn(d1[k], w1[k]);
          }
          const float2 s2 = f2(row_dot<P, L>(d0, d1, x0, x1) * (-1.0f / D));
          const float2 s1 = f2(NORM == RA_NORM_LAYER ? row_sum<P, L>(d0, d1) * (-1.0f / D) : 0.0f);
#pragma unroll
          for (int k = 0; k < P; ++k) {
            d0[k] = __ffma2_rn(x0[k], s2, NORM == RA_NORM_LAYER ? __fadd2_rn(d0[k], s1) : d0[k]);
            d1[k] = __ffma2_rn(x1[k], s2, NORM == RA_NORM_LAYER ? __fadd2_rn(d1[k], s1) : d1[k]);
            d0[k] = __fmul2_rn(d0[k], r);
            d1[k] = __fmul2_rn(d1[k], r);
          }
        }
        u0 = Vec<T>::put(d0);
        u1 = Vec<T>::put(d1);
      }
      if (there && hs + i * hstep < wk.heads) {
        reinterpret_cast<uint4*>(out)[lm.v0] = u0;
        reinterpret_cast<uint4*>(out)[lm.v1] = u1;
      }
      out += hstep * D;
      fetch();   // into the slot just read: after the stores, which needed what it held
    }
  }
  if (!norm) return;   // uniform over the CTA
  copy_wait<0>();
  float* part = reinterpret_cast<float*>(ring);   // [NG][D]
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    __syncthreads();
#pragma unroll
    for (int k = 0; k < P; ++k) {
      *reinterpret_cast<float2*>(&part[g * D + lm.v0 * E + 2 * k]) = s ? db0[k] : dw0[k];
      *reinterpret_cast<float2*>(&part[g * D + lm.v1 * E + 2 * k]) = s ? db1[k] : dw1[k];
    }
    __syncthreads();
    // SLICES threads per column, each adding every SLICES-th lane group, then theirs by halves
    constexpr int SLICES = kThreads / D;
    float f = 0.0f;
#pragma unroll
    for (int i = 0; i < NG / SLICES; ++i) f += part[threadIdx.x + i * kThreads];
    __syncthreads();
    part[threadIdx.x] = f;
    __syncthreads();
    if (threadIdx.x < D) {
      float v[SLICES];
#pragma unroll
      for (int i = 0; i < SLICES; ++i) v[i] = part[i * D + threadIdx.x];
#pragma unroll
      for (int o = SLICES / 2; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < o; ++i) v[i] += v[i + o];
      io.partial[(static_cast<int64_t>(wk.place) * 2 + s) * D + threadIdx.x] = v[0];
    }
  }
}

// dparams[4][D]: the query weight's and bias's gradients are the sum over the query CTAs of
// partial[cta][2][D], the key's over the key CTAs.  A CTA per 16 columns, 64 partial sums per
// column, whose loads are in flight together.
constexpr int kParamCols = 16, kParamSlices = 64;
__global__ void __launch_bounds__(kParamCols * kParamSlices)
    norm_rope_param_kernel(const float* partial, float* dparams, int q_ctas, int k_ctas, int cols) {
  __shared__ float part[kParamSlices][kParamCols];
  const int c = threadIdx.x % kParamCols, s = threadIdx.x / kParamCols, col = blockIdx.x * kParamCols + c;
  await_previous();
  const bool key = col >= cols;   // cols = 2 D
  const int first = key ? q_ctas : 0, last = key ? q_ctas + k_ctas : q_ctas;
  float v = 0.0f;
#pragma unroll 8
  for (int i = first + s; i < last; i += kParamSlices) v += partial[static_cast<int64_t>(i) * cols + col % cols];
  part[s][c] = v;
  __syncthreads();
  for (int o = kParamSlices / 2; o > 0; o >>= 1) {
    if (s < o) part[s][c] += part[s + o][c];
    __syncthreads();
  }
  if (s == 0) dparams[col] = part[0][c];
}

constexpr int kRingBytes = kAhead * 4 * kThreads * 16;
static_assert(kRingBytes >= kThreads * 16 * 4, "the lane groups' sums fit the ring");

template <typename T, int D, int NORM>
cudaError_t go(const NormRopeShape& a, const NormRopeBwd& io, cudaStream_t st) {
  cudaError_t e = set_up_kernel<norm_rope_bwd_kernel<T, D, NORM>>(kRingBytes, false);
  if (e != cudaSuccess) return e;
  norm_rope_bwd_kernel<T, D, NORM><<<a.ctas[0] + a.ctas[1] + a.ctas[2], kThreads, kRingBytes, st>>>(a, io);
  if (NORM == RA_NORM_NONE) return cudaGetLastError();
  e = cudaGetLastError();
  return e != cudaSuccess ? e
                          : launch_dependent(norm_rope_param_kernel, 4 * D / kParamCols, kParamCols * kParamSlices, 0,
                                             st, io.partial, io.dparams, a.ctas[0], a.ctas[1], 2 * D);
}
template <typename T, int D>
cudaError_t go(const NormRopeShape& a, const NormRopeBwd& io, cudaStream_t st) {
  if (a.norm == RA_NORM_NONE) return go<T, D, RA_NORM_NONE>(a, io, st);
  return a.norm == RA_NORM_RMS ? go<T, D, RA_NORM_RMS>(a, io, st) : go<T, D, RA_NORM_LAYER>(a, io, st);
}

}  // namespace

int norm_rope_bwd_ctas() { return 2 * kSms + 2; }   // a kind has at least one

cudaError_t launch_norm_rope_bwd(NormRopeShape a, const NormRopeBwd& io, bool bf16, cudaStream_t st) {
  // By measurement: bytes alone, 3, 3 and 2 per head, gave 214 us at B4 N8192 H16 D128 against 200, and
  // 184 against 115 with 8 query heads on one key head, where a tile's start counts for more.
  plan_work(&a, bf16 ? 2 : 4, 2 * kSms, {5, 5, 2}, {6, 8, 6});
  if (bf16) {
    if (a.D == 16) return go<__nv_bfloat16, 16>(a, io, st);
    if (a.D == 32) return go<__nv_bfloat16, 32>(a, io, st);
    if (a.D == 64) return go<__nv_bfloat16, 64>(a, io, st);
    return go<__nv_bfloat16, 128>(a, io, st);
  }
  if (a.D == 16) return go<float, 16>(a, io, st);
  if (a.D == 32) return go<float, 32>(a, io, st);
  if (a.D == 64) return go<float, 64>(a, io, st);
  return go<float, 128>(a, io, st);
}

}  // namespace raattn
