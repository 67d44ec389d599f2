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
// Bound: HBM, with the issue slots close behind.  A lane holds two 16-byte vectors of a row (a row
// lies across D * size / 32 lanes), chosen so that in the half-split form it holds both members of
// its pairs: the rotation needs no exchange between lanes, and the row sums are a few shuffles.  A
// CTA takes a tile of tokens at a time; a lane group stays with one token and walks its heads, so what
// depends on the token alone is formed once and not per row.  (In the backward a CTA works on one
// kind of row, queries, keys or values, so that a lane holds one kind's sums.)  In the forward the norm's weight w and
// the rotation fold into two factors and an addend,
//   y_j = r (x_j A_j + x_partner B_j) + C_j,  A = w cos, B = +-w_partner sin, C = the rotated bias,
// and all arithmetic runs as packed pairs of floats.  Each thread copies the next rows' vectors
// asynchronously into shared-memory slots of its own, which costs no registers and no barrier.
#pragma once

#include "kernels.cuh"

namespace raattn {
namespace norm_rope {

constexpr int kThreads = 256;
constexpr int kMaxTile = 32;   // tokens of a CTA's tile
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

struct Tables {
  unsigned long long turns[kMaxPairs];  // frequency / (2 pi) without its whole turns, in units of 2^-64
  float cs[2][kMaxTile][kMaxPairs];     // double-buffered by tile: one barrier per tile
  float sn[2][kMaxTile][kMaxPairs];
};

// frequency / (2 pi) to about 2^-64 turns: 1 / (2 pi) as the sum of two doubles, the first product with its
// rounding error.
__device__ __forceinline__ void init_turns(Tables& tb, const NormRopeShape& a) {
  constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18;
  for (int p = threadIdx.x; p < a.pairs; p += kThreads) {
    const double f = a.freq[p], t = f * kHi, rest = fma(f, kHi, -t) + f * kLo;
    tb.turns[p] = static_cast<unsigned long long>(__double2ll_rn((t - rint(t)) * 0x1p64)) +
                  static_cast<unsigned long long>(__double2ll_rn(rest * 0x1p64));
  }
  __syncthreads();
}

// The cosine and sine of position * turns.  The product wraps at a whole turn, so every position's angle is within
// its 2^-64 of turns times the position, 2^-33 at most.  FAST (bf16): the approximate functions, off by 2^-21 at most
// within half a turn, far below bf16's 2^-8.  Else the angle from the nearest quarter turn, which fp32 holds
// to 2^-28 turns.
template <bool FAST>
__device__ __forceinline__ void turn(unsigned long long turns, int pos, float& c, float& s) {
  const unsigned long long x = turns * static_cast<unsigned long long>(static_cast<long long>(pos));
  if (FAST) {
    __sincosf(static_cast<float>(static_cast<int>(x >> 32)) * 1.46291808e-9f, &s, &c);   // 2 pi / 2^32
  } else {
    const unsigned q = static_cast<unsigned>((x + (1ull << 61)) >> 62);
    float c0, s0;
    sincospif(static_cast<float>(static_cast<long long>(x - (static_cast<unsigned long long>(q) << 62))) * 0x1p-63f, &s0, &c0);
    c = q & 1 ? s0 : c0;
    s = q & 1 ? c0 : s0;
    if (q == 1 || q == 2) c = -c;
    if (q & 2) s = -s;
  }
}

// The cosines and sines of a tile's tokens.  Threads are laid out with the pairs (a power of two
// of them) fastest; token numbers fit 32 bits, where a division is cheap.
template <bool FAST>
__device__ __forceinline__ void fill_table(Tables& tb, int buf, const NormRopeShape& a, int tok0, int tile) {
  const int lg = 32 - __clz(a.pairs - 1), p = threadIdx.x & ((1 << lg) - 1);   // pairs = 1: lg = 0
  if (p >= a.pairs) return;
  const int axis = (p >= a.end[0]) + (p >= a.end[1]) + (p >= a.end[2]);
  const int* pos = a.pos + axis * a.pos_axis_stride;
  const unsigned long long turns = tb.turns[p];
  const int tokens = a.B * a.N;
  for (int tl = threadIdx.x >> lg; tl < tile; tl += kThreads >> lg) {
    const int tok = tok0 + tl;
    float s = 0.0f, c = 1.0f;   // a token past the last: what its rows of zeros meet has to be finite
    if (tok < tokens) {
      const int b = tok / a.N, n = tok - b * a.N;
      turn<FAST>(turns, pos[b * a.pos_batch_stride + n], c, s);
    }
    tb.cs[buf][tl][p] = c;
    tb.sn[buf][tl][p] = s;
  }
}

// Which vectors of a row a lane holds, and how they are turned.
struct LaneMap {
  int v0, v1;       // vectors of E elements
  int pair;         // half-split: first of the lane's E pairs (v0 holds their first members)
  bool turned;      // half-split: whether they are turned
  int n0, n1;       // interleaved: turned pairs of v0 and of v1
};
template <int E, int L>
__device__ __forceinline__ LaneMap lane_map(const NormRopeShape& a, int gl) {
  LaneMap m;
  const int half = a.pairs / E;   // half-split: pairs is a multiple of 8, so whole vectors
  if (a.interleaved || gl >= half) {
    // interleaved, or a lane of the part that is not turned: that part's vectors, two by two
    m.v0 = a.interleaved ? gl : 2 * gl;
    m.v1 = a.interleaved ? gl + L : 2 * gl + 1;
    m.turned = false;
    m.pair = 0;
  } else {
    m.v0 = gl;
    m.v1 = gl + half;
    m.turned = true;
    m.pair = gl * E;
  }
  m.n0 = min(max(a.pairs - m.v0 * (E / 2), 0), E / 2);
  m.n1 = min(max(a.pairs - m.v1 * (E / 2), 0), E / 2);
  return m;
}

// A token's cosines and sines of a lane's pairs: half-split E pairs, v0 the first members; interleaved
// E / 2 pairs of v0, then of v1.  1 and 0 where not turned (whole: everywhere turned).
template <int E>
__device__ __forceinline__ void load_turn(float (&cs)[E], float (&sn)[E], const Tables& tb, int buf, int tl,
                                          const LaneMap& m, const NormRopeShape& a, bool whole) {
  const int p0 = a.interleaved ? m.v0 * (E / 2) : m.pair, p1 = a.interleaved ? m.v1 * (E / 2) : m.pair + E / 2;
  const float* c = tb.cs[buf][tl];
  const float* s = tb.sn[buf][tl];
#pragma unroll
  for (int j = 0; j < E / 2; j += 2) {
    const float2 x = *reinterpret_cast<const float2*>(c + p0 + j), y = *reinterpret_cast<const float2*>(c + p1 + j);
    const float2 u = *reinterpret_cast<const float2*>(s + p0 + j), v = *reinterpret_cast<const float2*>(s + p1 + j);
    cs[j] = x.x;
    cs[j + 1] = x.y;
    cs[E / 2 + j] = y.x;
    cs[E / 2 + j + 1] = y.y;
    sn[j] = u.x;
    sn[j + 1] = u.y;
    sn[E / 2 + j] = v.x;
    sn[E / 2 + j + 1] = v.y;
  }
  if (!whole) {
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const bool in = a.interleaved ? (j < E / 2 ? j < m.n0 : j - E / 2 < m.n1) : m.turned;
      cs[j] = in ? cs[j] : 1.0f;
      sn[j] = in ? sn[j] : 0.0f;
    }
  }
}

// The rotation's factors on a row x0, x1: y0 = x0 a0 + p0 b0, y1 = x1 a1 + p1 b1 with the partners
// p0, p1 of partners().
template <int E>
__device__ __forceinline__ void factors(const float (&cs)[E], const float (&sn)[E], int interleaved,
                                        float2 (&a0)[E / 2], float2 (&b0)[E / 2], float2 (&a1)[E / 2],
                                        float2 (&b1)[E / 2]) {
#pragma unroll
  for (int k = 0; k < E / 2; ++k) {
    if (interleaved) {
      a0[k] = f2(cs[k]);
      b0[k] = make_float2(-sn[k], sn[k]);
      a1[k] = f2(cs[E / 2 + k]);
      b1[k] = make_float2(-sn[E / 2 + k], sn[E / 2 + k]);
    } else {
      a0[k] = a1[k] = make_float2(cs[2 * k], cs[2 * k + 1]);
      b1[k] = make_float2(sn[2 * k], sn[2 * k + 1]);
      b0[k] = make_float2(-b1[k].x, -b1[k].y);
    }
  }
}
// The partners of x0 and x1: zero where a pair is not turned, so that nothing of it, an infinity
// say, meets a factor 0.  whole: every pair of every lane is turned (no selection needed).
template <int P>
__device__ __forceinline__ void partners(const float2 (&x0)[P], const float2 (&x1)[P], float2 (&p0)[P],
                                         float2 (&p1)[P], const LaneMap& m, int interleaved, bool whole) {
#pragma unroll
  for (int k = 0; k < P; ++k) {
    p0[k] = interleaved ? swap(x0[k]) : x1[k];
    p1[k] = interleaved ? swap(x1[k]) : x0[k];
  }
  if (!whole) {
#pragma unroll
    for (int k = 0; k < P; ++k) {
      if (!(interleaved ? k < m.n0 : m.turned)) p0[k] = f2(0.0f);
      if (!(interleaved ? k < m.n1 : m.turned)) p1[k] = f2(0.0f);
    }
  }
}

// Over a row's lanes.
template <int P, int L>
__device__ __forceinline__ float row_sum(const float2 (&x0)[P], const float2 (&x1)[P]) {
  float2 s = __fadd2_rn(x0[0], x1[0]);
#pragma unroll
  for (int j = 1; j < P; ++j) s = __fadd2_rn(s, __fadd2_rn(x0[j], x1[j]));
  return group_sum<L>(s.x + s.y);
}
template <int P, int L>
__device__ __forceinline__ float row_dot(const float2 (&x0)[P], const float2 (&x1)[P], const float2 (&y0)[P],
                                         const float2 (&y1)[P]) {
  float2 s = __fmul2_rn(x0[0], y0[0]), s2 = __fmul2_rn(x1[0], y1[0]);
#pragma unroll
  for (int j = 1; j < P; ++j) {
    s = __ffma2_rn(x0[j], y0[j], s);
    s2 = __ffma2_rn(x1[j], y1[j], s2);
  }
  s = __fadd2_rn(s, s2);
  return group_sum<L>(s.x + s.y);
}
// 1 / sqrt(mean square + eps); a row of zeros stays finite with eps = 0 too, and a NaN in the row (which a
// maximum would drop) makes all of it NaN.
__device__ __forceinline__ float inverse_rms(float mean_square, float eps) {
  const float s = mean_square + eps;
  float r;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s < 1e-37f ? 1e-37f : s));   // 2 ulp
  return r;
}

// What a CTA works on.
struct Work {
  int kind;             // 0 queries, 1 keys, 2 values
  int heads, head0;     // its heads, the first of them in a token of the projection
  int tile;             // tokens of a tile
  int first, step;      // tiles first, first + step, ..
  int place;            // among all CTAs, those of a kind together
};
__device__ __forceinline__ Work work_of(const NormRopeShape& a) {
  Work w;
  const int all = a.ctas[0] + a.ctas[1] + a.ctas[2];
  int x = blockIdx.x * a.stride % all;   // a permutation: an SM's CTAs are seldom of one kind
  w.place = x;
  w.kind = x < a.ctas[0] ? 0 : x < a.ctas[0] + a.ctas[1] ? 1 : 2;
  if (w.kind > 0) x -= a.ctas[0];
  if (w.kind > 1) x -= a.ctas[1];
  w.heads = w.kind == 0 ? a.Hq : a.Hkv;
  w.head0 = w.kind == 0 ? 0 : w.kind == 1 ? a.Hq : a.Hq + a.Hkv;
  w.tile = a.tiles[w.kind];
  w.first = x;
  w.step = a.ctas[w.kind];
  return w;
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

// The tokens of a tile for which the CTA with most tiles is done first: a tile takes its rows per lane group and
// `start` more (the token's factors, the refilled ring).  rows(step): rows of a lane group that takes
// every step-th head.  Forward, bf16 B4 N8192: 16 tokens, 7 tiles and 18 rows each for the longest CTA, 86 us
// with H16/8 D128, against 94 with 8 tokens and 92 with 32; with H8/1, 32 tokens 39 us against 46 with 16.
template <typename F>
int best_tile(int64_t tokens, int groups, int64_t ctas, int start, F rows) {
  int best = 1;
  int64_t least = 0;
  for (int t = 1; t <= groups && t <= kMaxTile; t *= 2) {
    const int64_t tiles = (tokens + t - 1) / t;
    if (t > 1 && 4 * tiles < 3 * ctas) break;   // loads in flight on every SM count for more
    const int64_t time = (tiles + ctas - 1) / ctas * (rows(groups / t) + start);
    if (t == 1 || 33 * time < 32 * least) {   // near ties to the smaller
      least = time;
      best = t;
    }
  }
  return best;
}

// Shares `most` CTAs among the kinds by their cost per head and per token, and sets the tiles' tokens.
inline void plan_work(NormRopeShape* a, int es, int most, const int (&head_cost)[3], const int (&token_cost)[3]) {
  const int groups = kThreads / (a->D * es / 32);
  const int64_t tokens = static_cast<int64_t>(a->B) * a->N;
  const int heads[3] = {a->Hq, a->Hkv, a->Hkv};
  int64_t cost[3], all = 0;
  for (int k = 0; k < 3; ++k) all += cost[k] = static_cast<int64_t>(head_cost[k]) * heads[k] + token_cost[k];
  for (int k = 0; k < 3; ++k) {
    const int64_t share = most * cost[k] / all;
    const int64_t ctas = share < 1 ? 1 : share;
    const int t = best_tile(tokens, groups, ctas, 1, [&](int step) { return (heads[k] + step - 1) / step; });
    const int64_t tiles = (tokens + t - 1) / t;
    a->tiles[k] = t;
    a->ctas[k] = static_cast<int>(tiles < ctas ? tiles : ctas);
  }
  // a step of about three eighths of the grid that has no divisor in common with it
  const int grid = a->ctas[0] + a->ctas[1] + a->ctas[2];
  auto common = [](int x, int y) {
    while (y) {
      const int r = x % y;
      x = y;
      y = r;
    }
    return x;
  };
  a->stride = grid * 3 / 8 + 1;
  while (common(a->stride, grid) != 1) ++a->stride;
}

}  // namespace norm_rope
}  // namespace raattn
