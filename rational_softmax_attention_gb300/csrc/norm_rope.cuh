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
// Bound: HBM, with the issue slots close behind: a row lies across D * size / 16 lanes, one 16-byte
// vector each, so every access is a whole vector and the row sums are a few shuffles.  A CTA takes
// a tile of tokens; a lane group stays with one token and walks its heads, so what depends on the
// token alone is formed once and not per row: the norm's weight w and the rotation fold into
// two factors and an addend,
//   y_j = r (x_j A_j + x_partner B_j) + C_j,  A = w cos, B = +-w_partner sin, C = the rotated bias,
// and the arithmetic runs as packed pairs of floats.  The half-split form's partners are fetched
// from the other lanes as the raw 16-byte vector, four words and not eight floats.  Each thread copies
// the next rows' vectors asynchronously into shared-memory slots of its own, which costs no
// registers and needs no barrier.
#pragma once

#include "kernels.cuh"

namespace raattn {
namespace norm_rope {

constexpr int kThreads = 256;
constexpr int kMaxTile = 16;   // tokens of a CTA's tile
constexpr int kMaxPairs = 64;

__device__ __forceinline__ float2 f2(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 swap(float2 x) { return make_float2(x.y, x.x); }

// A lane's vector as pairs of floats.
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int E = 4;
  static __device__ __forceinline__ void get(const uint4& u, float2 (&x)[2]) {
    x[0] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
    x[1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
  }
  static __device__ __forceinline__ uint4 put(const float2 (&x)[2]) {
    return make_uint4(__float_as_uint(x[0].x), __float_as_uint(x[0].y), __float_as_uint(x[1].x),
                      __float_as_uint(x[1].y));
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int E = 8;
  static __device__ __forceinline__ float2 pair(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  static __device__ __forceinline__ void get(const uint4& u, float2 (&x)[4]) {
    x[0] = pair(u.x);
    x[1] = pair(u.y);
    x[2] = pair(u.z);
    x[3] = pair(u.w);
  }
  // the one rounding of a bf16 output: half a step, 2^-8 relative at most
  static __device__ __forceinline__ uint4 put(const float2 (&x)[4]) {
    return make_uint4(pack_bf16x2(x[0].x, x[0].y), pack_bf16x2(x[1].x, x[1].y), pack_bf16x2(x[2].x, x[2].y),
                      pack_bf16x2(x[3].x, x[3].y));
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

// The lane's part of a token's rotation, out = x cs + partner sn; a pair (j, j + 1) of its elements
// is turned or not as a whole (pairs are even numbers of elements).
template <int P>
struct Turn {
  float2 cs[P], sn[P];   // 1 and 0 where not turned
};

// What does not depend on the token: where a lane's partners are.
struct Partner {
  int from;         // lane of the warp that holds them (half-split), or this lane
  uint32_t keep;    // half-split: all ones, or 0 where the lane's elements are not turned
  int count;        // interleaved: how many of the lane's elements are turned
};
template <int E>
__device__ __forceinline__ Partner find_partner(const NormRopeShape& a, int gl, int lane) {
  Partner p;
  const int e0 = gl * E;
  const bool first = e0 < a.pairs, second = !first && e0 < 2 * a.pairs;   // pairs is a multiple of 8 then
  p.from = a.interleaved ? lane : first ? lane + a.pairs / E : second ? lane - a.pairs / E : lane;
  p.keep = first || second ? ~0u : 0u;
  p.count = min(max(2 * a.pairs - e0, 0), E);
  return p;
}

template <int E>
__device__ __forceinline__ void load_turn(Turn<E / 2>& t, const Tables& tb, int buf, int tl, int gl,
                                          const Partner& pt, const NormRopeShape& a) {
  const int e0 = gl * E;
  if (a.interleaved) {
#pragma unroll
    for (int j = 0; j < E / 2; ++j) {
      const bool in = 2 * j < pt.count;
      const float c = in ? tb.cs[buf][tl][e0 / 2 + j] : 1.0f, s = in ? tb.sn[buf][tl][e0 / 2 + j] : 0.0f;
      t.cs[j] = f2(c);
      t.sn[j] = make_float2(-s, s);
    }
  } else {
    const bool first = e0 < a.pairs;
    const int p = pt.keep ? (first ? e0 : e0 - a.pairs) : 0;
#pragma unroll
    for (int j = 0; j < E / 2; ++j) {
      const float2 c = *reinterpret_cast<const float2*>(&tb.cs[buf][tl][p + 2 * j]);
      const float2 s = *reinterpret_cast<const float2*>(&tb.sn[buf][tl][p + 2 * j]);
      t.cs[j] = pt.keep ? c : f2(1.0f);
      t.sn[j] = !pt.keep ? f2(0.0f) : first ? make_float2(-s.x, -s.y) : s;
    }
  }
}

// The partners of a lane's vector (zeros where an element is not turned, so that nothing of it,
// an infinity say, meets a factor 0).
template <typename T>
__device__ __forceinline__ void partners(const uint4& u, const float2 (&x)[Vec<T>::E / 2], float2 (&p)[Vec<T>::E / 2],
                                         const Partner& pt, int interleaved) {
  constexpr int E = Vec<T>::E;
  if (interleaved) {
#pragma unroll
    for (int j = 0; j < E / 2; ++j) p[j] = 2 * j < pt.count ? swap(x[j]) : f2(0.0f);
  } else {
    uint4 w;
    w.x = __shfl_sync(0xffffffffu, u.x, pt.from) & pt.keep;
    w.y = __shfl_sync(0xffffffffu, u.y, pt.from) & pt.keep;
    w.z = __shfl_sync(0xffffffffu, u.z, pt.from) & pt.keep;
    w.w = __shfl_sync(0xffffffffu, u.w, pt.from) & pt.keep;
    Vec<T>::get(w, p);
  }
}

// Over a row's lanes.
template <int P, int L>
__device__ __forceinline__ float row_sum(const float2 (&x)[P]) {
  float2 s = x[0];
#pragma unroll
  for (int j = 1; j < P; ++j) s = __fadd2_rn(s, x[j]);
  return group_sum<L>(s.x + s.y);
}
template <int P, int L>
__device__ __forceinline__ float row_dot(const float2 (&x)[P], const float2 (&y)[P]) {
  float2 s = __fmul2_rn(x[0], y[0]);
#pragma unroll
  for (int j = 1; j < P; ++j) s = __ffma2_rn(x[j], y[j], s);
  return group_sum<L>(s.x + s.y);
}
// 1 / sqrt(mean square + eps); a row of zeros stays finite with eps = 0 too.
__device__ __forceinline__ float inverse_rms(float mean_square, float eps) {
  return rsqrtf(fmaxf(mean_square + eps, 1e-37f));
}

// A tile's rows in the order in which a lane group walks them: its share of the token's query
// heads, then of its key heads, then of its value heads, in batches of U heads of one kind.
struct Walk {
  int hs, hstep;    // heads hs, hs + hstep, ..
  int q, k, all;    // batches of query heads; of query and key heads; of all
};
template <int U>
__device__ __forceinline__ Walk make_walk(const NormRopeShape& a, int g, int groups) {
  Walk w;
  w.hs = g / a.tile;
  w.hstep = groups / a.tile;
  const int per = U * w.hstep;
  w.q = (a.Hq + per - 1) / per;
  w.k = w.q + (a.Hkv + per - 1) / per;
  w.all = w.k + (a.Hkv + per - 1) / per;
  return w;
}
// Kind of batch i (0 query, 1 key, 2 value), its first head for this group, and the kind's heads.
template <int U>
__device__ __forceinline__ void batch_of(const Walk& w, int i, const NormRopeShape& a, int& kind, int& h, int& heads) {
  kind = i < w.q ? 0 : i < w.k ? 1 : 2;
  h = w.hs + (i - (kind == 0 ? 0 : kind == 1 ? w.q : w.k)) * U * w.hstep;
  heads = kind == 0 ? a.Hq : a.Hkv;
}

// A thread's asynchronous 16-byte copies into its own slots (zeros when not `in`).
__device__ __forceinline__ void copy_own(uint4* slot, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(slot)), "l"(src), "r"(in ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Tokens of a tile: what a token's rotation costs is shared by the heads that one lane group walks,
// so as many tokens as lane groups are best, short of leaving SMs without tiles or the last round
// of tiles half empty: up to half of the groups, and at least six tiles per SM.
inline int tile_for(const NormRopeShape& a, int es) {
  const int groups = kThreads / (a.D * es / 16);
  const int64_t tokens = static_cast<int64_t>(a.B) * a.N;
  int t = 1;
  while (t < kMaxTile && 4 * t <= groups && tokens / (2 * t) >= 6 * kSms) t *= 2;
  return t;
}

}  // namespace norm_rope
}  // namespace raattn
