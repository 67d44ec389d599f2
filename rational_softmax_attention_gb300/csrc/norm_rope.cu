// Per-head normalisation of queries and keys with the position rotation in the same pass, from
// the packed projection [B, N, (H_q + 2 H_kv) D] to q [B, H_q, N, D], k and v [B, H_kv, N, D]
// (or k and v straight into a key/value cache), and the gradient of that step.
//
// Forward, per (token, head) row x of q or k:
//   layer:  xhat = (x - mean) r, r = 1 / sqrt(mean((x - mean)^2) + eps);   y = xhat w + b
//   rms:    xhat = x r,          r = 1 / sqrt(mean(x^2) + eps);            y = xhat w
//   none:   y = x
//   pair i of the first 2 R dimensions ((i, i + R), or (2i, 2i + 1) when interleaved) turned
//   by the angle position[axis(i)] * frequency[i]; the other dimensions stay.
// v rows are copied.  Backward: the incoming gradient turned back by the same angle gives g;
//   dw = sum g xhat, db = sum g, t = g w,  dx = r (t - xhat mean(t xhat) - [layer] mean(t)).
// xhat and r are formed again from the projection, whose row the backward would have to read
// for xhat anyway, so the forward saves nothing else.
//
// Bound: HBM (about 10 operations per element forward, 20 backward).  A row lies across
// D * size / 16 lanes, one 16-byte vector each, so every access is a whole vector and the
// row sums are a few shuffles.  A CTA takes a tile of tokens; a lane group stays with one
// token and walks its heads, so the cosines and sines of its elements are read from shared
// memory once per token, not once per row.
#include "kernels.cuh"

namespace raattn {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTile = 16;   // tokens of a CTA's tile
constexpr int kMaxPairs = 64;

template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int E = 4;
  static __device__ __forceinline__ void get(const uint4& u, float (&x)[4]) {
    x[0] = __uint_as_float(u.x);
    x[1] = __uint_as_float(u.y);
    x[2] = __uint_as_float(u.z);
    x[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 put(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int E = 8;
  static __device__ __forceinline__ void get(const uint4& u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  // the one rounding of a bf16 output: half a step, 2^-8 relative at most
  static __device__ __forceinline__ uint4 put(const float (&x)[8]) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
  }
};

template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// position * turns as a fraction of a turn in about [-0.5, 0.5]: the position is split into two
// parts that fp32 holds exactly, each product into its rounded value (whose whole turns leave
// exactly) and its rounding error, so far positions lose nothing.
__device__ __forceinline__ float turn_fraction(int pos, float2 turns) {
  const float lo = static_cast<float>(pos & 0xfff), hi = static_cast<float>(pos & ~0xfff);
  const float a = lo * turns.x, b = hi * turns.x;
  const float c = hi * turns.y;
  float f = (a - rintf(a)) + (b - rintf(b));
  f += (c - rintf(c)) + fmaf(lo, turns.y, fmaf(lo, turns.x, -a) + (fmaf(hi, turns.x, -b) + fmaf(hi, turns.y, -c)));
  return f - rintf(f);
}

struct Tables {
  float2 turns[kMaxPairs];              // frequency / (2 pi) as the sum of two floats
  float cs[2][kMaxTile][kMaxPairs];     // double-buffered by tile: one barrier per tile
  float sn[2][kMaxTile][kMaxPairs];
};

__device__ __forceinline__ void init_turns(Tables& tb, const NormRopeShape& a) {
  for (int p = threadIdx.x; p < a.pairs; p += kThreads) {
    const double t = a.freq[p] * 0.15915494309189533577;   // 1 / (2 pi)
    const float hi = static_cast<float>(t);
    tb.turns[p] = make_float2(hi, static_cast<float>(t - static_cast<double>(hi)));
  }
  __syncthreads();
}

__device__ __forceinline__ void fill_table(Tables& tb, int buf, const NormRopeShape& a, int64_t tok0) {
  const int64_t tokens = static_cast<int64_t>(a.B) * a.N;
  for (int i = threadIdx.x; i < a.tile * a.pairs; i += kThreads) {
    const int tl = i / a.pairs, p = i - tl * a.pairs;
    const int64_t tok = tok0 + tl;
    if (tok < tokens) {
      const int b = static_cast<int>(tok / a.N), n = static_cast<int>(tok - static_cast<int64_t>(b) * a.N);
      const int axis = (p >= a.end[0]) + (p >= a.end[1]) + (p >= a.end[2]);
      const int pos = a.pos[axis * a.pos_axis_stride + b * a.pos_batch_stride + n];
      float s, c;
      sincospif(2.0f * turn_fraction(pos, tb.turns[p]), &s, &c);
      tb.cs[buf][tl][p] = c;
      tb.sn[buf][tl][p] = s;
    }
  }
}

// The lane's part of a token's rotation: out[j] = x[j] cs[j] + partner[j] sn[j] for the first
// `count` of its elements, the partner being its neighbour (interleaved) or the same element
// of lane `from` of the warp.
template <int E>
struct Turn {
  float cs[E], sn[E];
  int count;
  int from;
};

template <int E>
__device__ __forceinline__ void load_turn(Turn<E>& t, const Tables& tb, int buf, int tl, int gl, int lane,
                                          const NormRopeShape& a) {
  const int e0 = gl * E;
  if (a.interleaved) {
    t.count = min(max(2 * a.pairs - e0, 0), E);
    t.from = lane;
#pragma unroll
    for (int j = 0; j < E; j += 2) {
      const int p = (e0 + j) >> 1;
      const bool in = j < t.count;
      const float c = in ? tb.cs[buf][tl][p] : 1.0f, s = in ? tb.sn[buf][tl][p] : 0.0f;
      t.cs[j] = t.cs[j + 1] = c;
      t.sn[j] = -s;
      t.sn[j + 1] = s;
    }
  } else {   // pairs is a multiple of 8, so a vector lies in one half and its partner is a whole lane away
    const bool first = e0 < a.pairs, second = !first && e0 < 2 * a.pairs;
    t.count = first || second ? E : 0;
    t.from = first ? lane + a.pairs / E : second ? lane - a.pairs / E : lane;
    const int p = second ? e0 - a.pairs : e0;
#pragma unroll
    for (int j = 0; j < E; ++j) {
      t.cs[j] = t.count ? tb.cs[buf][tl][p + j] : 1.0f;
      const float s = t.count ? tb.sn[buf][tl][p + j] : 0.0f;
      t.sn[j] = first ? -s : s;
    }
  }
}

// BACK: by the opposite angle.
template <int E, bool BACK>
__device__ __forceinline__ void rotate(float (&x)[E], const Turn<E>& t, int interleaved) {
  float p[E];
  if (interleaved) {
#pragma unroll
    for (int j = 0; j < E; j += 2) {
      p[j] = x[j + 1];
      p[j + 1] = x[j];
    }
  } else {
#pragma unroll
    for (int j = 0; j < E; ++j) p[j] = __shfl_sync(0xffffffffu, x[j], t.from);
  }
#pragma unroll
  for (int j = 0; j < E; ++j)
    if (j < t.count) x[j] = fmaf(p[j], BACK ? -t.sn[j] : t.sn[j], x[j] * t.cs[j]);
}

// x becomes xhat; returns r (1 where there is no norm).
template <int E, int L>
__device__ __forceinline__ float normalise(float (&x)[E], int norm, float eps) {
  constexpr float kInv = 1.0f / (E * L);
  if (norm == RA_NORM_NONE) return 1.0f;
  if (norm == RA_NORM_LAYER) {
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < E; ++j) s += x[j];
    const float mean = group_sum<L>(s) * kInv;
#pragma unroll
    for (int j = 0; j < E; ++j) x[j] -= mean;
  }
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < E; ++j) s = fmaf(x[j], x[j], s);
  const float r = rsqrtf(fmaf(group_sum<L>(s), kInv, eps));
#pragma unroll
  for (int j = 0; j < E; ++j) x[j] *= r;
  return r;
}

__device__ __forceinline__ uint4 load_vec(const void* p) {
  uint4 u;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
               : "l"(p));
  return u;
}

constexpr int kRowsAhead = 4;   // rows a lane group loads before it works on the first

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) norm_rope_fwd_kernel(const NormRopeShape a, const NormRopeFwd io) {
  constexpr int E = Vec<T>::E, L = D / E, NG = kThreads / L;
  __shared__ Tables tb;
  const int g = threadIdx.x / L, gl = threadIdx.x % L, lane = threadIdx.x & 31;
  const int tl = g % a.tile, hs = g / a.tile, hstep = NG / a.tile;
  const int heads = a.Hq + 2 * a.Hkv, rounds = (heads + hstep - 1) / hstep;
  const int64_t tokens = static_cast<int64_t>(a.B) * a.N;
  const int64_t tiles = (tokens + a.tile - 1) / a.tile;
  uint4 qw = make_uint4(0, 0, 0, 0), qb = qw, kw = qw, kb = qw;
  if (a.norm != RA_NORM_NONE) {
    qw = reinterpret_cast<const uint4*>(a.qw)[gl];
    kw = reinterpret_cast<const uint4*>(a.kw)[gl];
    if (a.qb) qb = reinterpret_cast<const uint4*>(a.qb)[gl];
    if (a.kb) kb = reinterpret_cast<const uint4*>(a.kb)[gl];
  }
  if (a.pairs) init_turns(tb, a);
  int buf = 0;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x, buf ^= 1) {
    const int64_t tok = tile * a.tile + tl;
    const bool there = tok < tokens;
    const int b = there ? static_cast<int>(tok / a.N) : 0;
    const int n = there ? static_cast<int>(tok - static_cast<int64_t>(b) * a.N) : 0;
    const T* row = static_cast<const T*>(a.qkv) + b * a.batch_stride + n * a.token_stride + gl * E;
    // the slot of this token's keys and values, or -1 where they are not to be written
    int slot = n;
    if (io.start) {
      const int64_t s = static_cast<int64_t>(io.start[b]) + n;
      slot = s < 0 || s >= io.capacity || (io.count && n >= io.count[b]) ? -1 : static_cast<int>(s);
    }
    Turn<E> t;
    uint4 u[kRowsAhead];
    for (int r0 = 0; r0 < rounds; r0 += kRowsAhead) {
#pragma unroll
      for (int i = 0; i < kRowsAhead; ++i) {
        const int h = hs + (r0 + i) * hstep;
        u[i] = there && h < heads ? load_vec(row + static_cast<int64_t>(h) * D) : make_uint4(0, 0, 0, 0);
      }
      if (r0 == 0 && a.pairs) {   // under the first rows' loads
        fill_table(tb, buf, a, tile * a.tile);
        __syncthreads();
        load_turn<E>(t, tb, buf, tl, gl, lane, a);
      }
#pragma unroll
      for (int i = 0; i < kRowsAhead; ++i) {
        const int h = hs + (r0 + i) * hstep;
        const bool is_q = h < a.Hq, is_v = h >= a.Hq + a.Hkv;
        uint4 out = u[i];
        if (!__all_sync(0xffffffffu, is_v)) {
          float x[E];
          Vec<T>::get(u[i], x);
          normalise<E, L>(x, a.norm, a.eps);
          if (a.norm != RA_NORM_NONE) {
            float w[E], c[E];
            Vec<T>::get(is_q ? qw : kw, w);
            Vec<T>::get(is_q ? qb : kb, c);
#pragma unroll
            for (int j = 0; j < E; ++j) x[j] = fmaf(x[j], w[j], c[j]);
          }
          if (a.pairs) rotate<E, false>(x, t, a.interleaved);
          if (!is_v) out = Vec<T>::put(x);
        }
        if (there && h < heads) {
          T* dst;
          if (is_q) {
            dst = static_cast<T*>(io.q) + ((static_cast<int64_t>(b) * a.Hq + h) * a.N + n) * D;
          } else {
            const int hk = is_v ? h - a.Hq - a.Hkv : h - a.Hq;
            dst = static_cast<T*>(is_v ? io.v : io.k) +
                  ((static_cast<int64_t>(b) * a.Hkv + hk) * io.capacity + slot) * D;
          }
          if (is_q || slot >= 0) *reinterpret_cast<uint4*>(dst + gl * E) = out;
        }
      }
    }
  }
}

// The gradient.  Each lane keeps its elements' sums of the four parameter gradients over all
// rows that it meets; a CTA adds its lane groups' sums in a fixed order and writes them to
// its own place of the workspace, and norm_rope_param_kernel adds the CTAs', so results do
// not depend on the order in which CTAs run.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) norm_rope_bwd_kernel(const NormRopeShape a, const NormRopeBwd io) {
  constexpr int E = Vec<T>::E, L = D / E, NG = kThreads / L;
  __shared__ Tables tb;
  __shared__ float part[NG][D];
  const int g = threadIdx.x / L, gl = threadIdx.x % L, lane = threadIdx.x & 31;
  const int tl = g % a.tile, hs = g / a.tile, hstep = NG / a.tile;
  const int heads = a.Hq + 2 * a.Hkv, rounds = (heads + hstep - 1) / hstep;
  const int64_t tokens = static_cast<int64_t>(a.B) * a.N;
  const int64_t tiles = (tokens + a.tile - 1) / a.tile;
  uint4 qw = make_uint4(0, 0, 0, 0), kw = qw;
  if (a.norm != RA_NORM_NONE) {
    qw = reinterpret_cast<const uint4*>(a.qw)[gl];
    kw = reinterpret_cast<const uint4*>(a.kw)[gl];
  }
  if (a.pairs) init_turns(tb, a);
  float acc[4][E];
#pragma unroll
  for (int j = 0; j < E; ++j) acc[0][j] = acc[1][j] = acc[2][j] = acc[3][j] = 0.0f;
  constexpr int kAhead = 2;
  int buf = 0;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x, buf ^= 1) {
    const int64_t tok = tile * a.tile + tl;
    const bool there = tok < tokens;
    const int b = there ? static_cast<int>(tok / a.N) : 0;
    const int n = there ? static_cast<int>(tok - static_cast<int64_t>(b) * a.N) : 0;
    const T* row = static_cast<const T*>(a.qkv) + b * a.batch_stride + n * a.token_stride + gl * E;
    T* out_row = static_cast<T*>(io.dqkv) + tok * static_cast<int64_t>(heads) * D + gl * E;
    Turn<E> t;
    uint4 u[kAhead], v[kAhead];
    for (int r0 = 0; r0 < rounds; r0 += kAhead) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int h = hs + (r0 + i) * hstep;
        const bool is_q = h < a.Hq, is_v = h >= a.Hq + a.Hkv;
        u[i] = v[i] = make_uint4(0, 0, 0, 0);
        if (there && h < heads) {
          const T* src;
          if (is_q) {
            src = static_cast<const T*>(io.dq) + ((static_cast<int64_t>(b) * a.Hq + h) * a.N + n) * D;
          } else {
            const int hk = is_v ? h - a.Hq - a.Hkv : h - a.Hq;
            src = static_cast<const T*>(is_v ? io.dv : io.dk) + ((static_cast<int64_t>(b) * a.Hkv + hk) * a.N + n) * D;
          }
          v[i] = load_vec(src + gl * E);
          if (!is_v && a.norm != RA_NORM_NONE) u[i] = load_vec(row + static_cast<int64_t>(h) * D);
        }
      }
      if (r0 == 0 && a.pairs) {
        fill_table(tb, buf, a, tile * a.tile);
        __syncthreads();
        load_turn<E>(t, tb, buf, tl, gl, lane, a);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int h = hs + (r0 + i) * hstep;
        const bool is_q = h < a.Hq, is_v = h >= a.Hq + a.Hkv;
        uint4 out = v[i];
        if (!__all_sync(0xffffffffu, is_v)) {
          float d[E];
          Vec<T>::get(v[i], d);
          if (a.pairs) rotate<E, true>(d, t, a.interleaved);
          if (a.norm != RA_NORM_NONE) {
            float x[E], w[E];
            Vec<T>::get(u[i], x);
            const float r = normalise<E, L>(x, a.norm, a.eps);
            Vec<T>::get(is_q ? qw : kw, w);
            float s1 = 0.0f, s2 = 0.0f;
            const bool count = there && !is_v;   // rows past the last head hold zeros
#pragma unroll
            for (int j = 0; j < E; ++j) {
              if (count && is_q) {
                acc[0][j] = fmaf(d[j], x[j], acc[0][j]);
                acc[1][j] += d[j];
              } else if (count) {
                acc[2][j] = fmaf(d[j], x[j], acc[2][j]);
                acc[3][j] += d[j];
              }
              d[j] *= w[j];
              s1 += d[j];
              s2 = fmaf(d[j], x[j], s2);
            }
            s2 = group_sum<L>(s2) * (1.0f / D);
            s1 = a.norm == RA_NORM_LAYER ? group_sum<L>(s1) * (1.0f / D) : 0.0f;
#pragma unroll
            for (int j = 0; j < E; ++j) d[j] = r * (d[j] - fmaf(x[j], s2, s1));
          }
          if (!is_v) out = Vec<T>::put(d);
        }
        if (there && h < heads) *reinterpret_cast<uint4*>(out_row + static_cast<int64_t>(h) * D) = out;
      }
    }
  }
  if (a.norm == RA_NORM_NONE) return;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < E; ++j) part[g][gl * E + j] = acc[k][j];
    __syncthreads();
    for (int e = threadIdx.x; e < D; e += kThreads) {
      float s = 0.0f;
      for (int i = 0; i < NG; ++i) s += part[i][e];
      io.partial[(static_cast<int64_t>(blockIdx.x) * 4 + k) * D + e] = s;
    }
  }
}

// dparams[4][D] = the sum over CTAs of partial[cta][4][D]: one CTA per parameter, eight partial
// sums per element.
__global__ void __launch_bounds__(1024) norm_rope_param_kernel(const float* partial, float* dparams, int ctas, int D) {
  __shared__ float part[1024];
  const int slices = 1024 / D, e = threadIdx.x % D, s = threadIdx.x / D;
  float v = 0.0f;
  for (int c = s; c < ctas; c += slices) v += partial[(static_cast<int64_t>(c) * 4 + blockIdx.x) * D + e];
  part[threadIdx.x] = v;
  __syncthreads();
  if (s == 0) {
    for (int i = 1; i < slices; ++i) v += part[i * D + e];
    dparams[blockIdx.x * D + e] = v;
  }
}

// Tokens of a tile: enough tiles for two CTAs on every SM first, then as many tokens as leave a
// lane group five to eight heads of one token (its cosines and sines are loaded once per token).
int tile_for(const NormRopeShape& a, int es) {
  const int groups = kThreads / (a.D * es / 16), heads = a.Hq + 2 * a.Hkv;
  const int64_t tokens = static_cast<int64_t>(a.B) * a.N;
  int t = 1;
  while (t < kMaxTile && 2 * t <= groups && tokens / (2 * t) >= 2 * kSms && heads * 2 * t <= 8 * groups) t *= 2;
  return t;
}

}  // namespace

int norm_rope_bwd_ctas() { return 3 * kSms; }

cudaError_t launch_norm_rope_fwd(NormRopeShape a, const NormRopeFwd& io, bool bf16, cudaStream_t st) {
  a.tile = tile_for(a, bf16 ? 2 : 4);
  const int64_t tiles = (static_cast<int64_t>(a.B) * a.N + a.tile - 1) / a.tile;
  const int grid = static_cast<int>(tiles < 6 * kSms ? tiles : 6 * kSms);
#define RA_GO(T, DD) norm_rope_fwd_kernel<T, DD><<<grid, kThreads, 0, st>>>(a, io)
  if (bf16) {
    if (a.D == 16) RA_GO(__nv_bfloat16, 16);
    if (a.D == 32) RA_GO(__nv_bfloat16, 32);
    if (a.D == 64) RA_GO(__nv_bfloat16, 64);
    if (a.D == 128) RA_GO(__nv_bfloat16, 128);
  } else {
    if (a.D == 16) RA_GO(float, 16);
    if (a.D == 32) RA_GO(float, 32);
    if (a.D == 64) RA_GO(float, 64);
    if (a.D == 128) RA_GO(float, 128);
  }
#undef RA_GO
  return cudaGetLastError();
}

cudaError_t launch_norm_rope_bwd(NormRopeShape a, const NormRopeBwd& io, bool bf16, cudaStream_t st) {
  a.tile = tile_for(a, bf16 ? 2 : 4);
  const int64_t tiles = (static_cast<int64_t>(a.B) * a.N + a.tile - 1) / a.tile;
  const int most = norm_rope_bwd_ctas();
  const int grid = static_cast<int>(tiles < most ? tiles : most);
#define RA_GO(T, DD) norm_rope_bwd_kernel<T, DD><<<grid, kThreads, 0, st>>>(a, io)
  if (bf16) {
    if (a.D == 16) RA_GO(__nv_bfloat16, 16);
    if (a.D == 32) RA_GO(__nv_bfloat16, 32);
    if (a.D == 64) RA_GO(__nv_bfloat16, 64);
    if (a.D == 128) RA_GO(__nv_bfloat16, 128);
  } else {
    if (a.D == 16) RA_GO(float, 16);
    if (a.D == 32) RA_GO(float, 32);
    if (a.D == 64) RA_GO(float, 64);
    if (a.D == 128) RA_GO(float, 128);
  }
#undef RA_GO
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.norm == RA_NORM_NONE) return e;
  norm_rope_param_kernel<<<4, 1024, 0, st>>>(io.partial, io.dparams, grid, a.D);
  return cudaGetLastError();
}

}  // namespace raattn
