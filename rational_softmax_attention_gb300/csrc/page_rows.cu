// Keys and values into pages held in 4 bits, and out of them (the layout and its mathematics: paged.cuh).
//
// The unit of work is a group of a row, 64 dimensions on eight lanes: a lane's eight elements are one word of codes,
// and minimum and maximum take three shuffles each.  The nearest code is found without a division: u' =
// rint((x - lo) (1 / s)) is at most one off, next to the middle between two codes, and the remainder (x - lo) - s u', which an
// FMA gives exactly, says whether it is.  Bound: HBM; each lane has several groups' 16-byte loads in flight.
#include <climits>

#include "paged.cuh"

namespace raattn {
namespace {

using namespace paged;

constexpr int kThreads = 256, kAhead = 4;   // groups of a thread in flight

struct RowsArgs {
  PageRows a;
  FastDiv groups, N, Hkv, B;   // unit = (((which B + b) Hkv + h) N + n) G + g
  int units;                   // of keys and values
};

struct Place {
  int which, b, h, n, g;
};
template <int G>
__device__ __forceinline__ Place place_of(uint32_t unit, const RowsArgs& ra) {
  Place p;
  p.g = unit % G;
  uint32_t x = unit / G, y = div_by(x, ra.N);
  p.n = x - y * ra.N.d;
  x = div_by(y, ra.Hkv);
  p.h = y - x * ra.Hkv.d;
  p.which = x >= ra.B.d;
  p.b = x - p.which * ra.B.d;
  return p;
}

// A lane's eight elements.
template <typename T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = bf16_low(w[i]);
      x[2 * i + 1] = bf16_high(w[i]);
    }
  }
  // the one rounding of a bf16 output: half a step, 2^-8 relative at most
  static __device__ __forceinline__ void put(__nv_bfloat16* p, const float (&x)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                                              pack_bf16x2(x[6], x[7]));
  }
};
template <>
struct Eight<float> {
  float4 u, v;
  __device__ __forceinline__ void load(const float* p) {
    u = __ldcs(reinterpret_cast<const float4*>(p));
    v = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = u.x;
    x[1] = u.y;
    x[2] = u.z;
    x[3] = u.w;
    x[4] = v.x;
    x[5] = v.y;
    x[6] = v.z;
    x[7] = v.w;
  }
  static __device__ __forceinline__ void put(float* p, const float (&x)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
};

// Minimum and maximum that a NaN does not get lost in.
__device__ __forceinline__ float min_nan(float x, float y) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float max_nan(float x, float y) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}

// What x - y loses when it is rounded to d (the exact difference is d plus this).
__device__ __forceinline__ float lost(float x, float y, float d) {
  const float v = __fsub_rn(d, x);   // about -y
  return __fadd_rn(__fsub_rn(x, __fsub_rn(d, v)), __fsub_rn(-y, v));
}

struct Held {
  uint32_t word;
  float s, lo;
};
// Eight lanes' elements as they are held.  All arithmetic below is exact or its error is accounted for, so that the codes are
// those of the definition whatever the inputs.
__device__ __forceinline__ Held quantise(const float (&x)[8]) {
  float low = x[0], high = x[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    low = min_nan(low, x[i]);
    high = max_nan(high, x[i]);
  }
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    low = min_nan(low, __shfl_xor_sync(0xffffffffu, low, o));
    high = max_nan(high, __shfl_xor_sync(0xffffffffu, high, o));
  }
  Held q;
  // 16 bits, rounded down (towards -infinity); no minus zero
  const uint32_t lb = __float_as_uint(__fadd_rn(low, 0.0f));
  q.lo = __uint_as_float((lb >> 31 ? lb + 0xffffu : lb) & 0xffff0000u);
  // the least s of 16 bits with 15 s >= high - lo = span + rest
  const float span = __fsub_rn(high, q.lo), rest = lost(high, q.lo, span);
  uint32_t sb = (__float_as_uint(__fmul_rn(span, 1.0f / 15.0f)) + 0xffffu) & 0xffff0000u;
  const auto covers = [&](uint32_t bits) {   // the product has 12 bits; the difference of near numbers is exact
    return __fsub_rn(__fmul_rn(15.0f, __uint_as_float(bits)), span) >= rest;
  };
  if (sb >= 0x10000u && covers(sb - 0x10000u)) sb -= 0x10000u;
  else if (!covers(sb)) sb += 0x10000u;
  q.s = __uint_as_float(sb);
  const float kInf = __uint_as_float(0x7f800000u);
  const bool good = span < kInf && q.s < kInf;   // a NaN is not
  if (!good) q.lo = __uint_as_float(0x7fc00000u);
  if (!good || q.s < 0x1p-100f) q.s = 0.0f;
  const float inv = q.s > 0.0f ? 1.0f / q.s : 0.0f, half = 0.5f * q.s;
  q.word = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float d = __fsub_rn(x[i], q.lo);
    float u = rintf(__fmul_rn(d, inv));   // 0 to 15, one off at most
    const float r = fmaf(-q.s, u, d);     // exact
    // beyond the middle, or in it with an odd code: the next one; where d itself was rounded that decides
    float over = fabsf(r) - half;
    if (over == 0.0f) over = copysignf(1.0f, r) * lost(x[i], q.lo, d);
    const bool odd = static_cast<int>(u) & 1;
    if (over > 0.0f || (over == 0.0f && odd)) u += copysignf(1.0f, r);
    q.word |= (q.s > 0.0f ? static_cast<uint32_t>(static_cast<int>(u)) & 15u : 0u) << (4 * i);
  }
  return q;
}
__device__ __forceinline__ void values_of(const Held& q, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = fmaf(q.s, static_cast<float>(q.word >> (4 * i) & 15u), q.lo);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) page_write_kernel(const RowsArgs ra) {
  constexpr int G = D / kGroup;
  const PageRows& a = ra.a;
  const int lane8 = threadIdx.x & 7, per = gridDim.x * (kThreads / 8);
  for (int64_t u0 = blockIdx.x * (kThreads / 8) + (threadIdx.x >> 3); u0 - (threadIdx.x >> 3 & 3) < ra.units;
       u0 += static_cast<int64_t>(kAhead) * per) {   // a warp's four groups together: the shuffles are the warp's
    Eight<T> in[kAhead];
    Place p[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t u = u0 + static_cast<int64_t>(i) * per;
      p[i] = place_of<G>(static_cast<uint32_t>(u < ra.units ? u : 0), ra);
      const int64_t* st = p[i].which ? a.v_stride : a.k_stride;
      const T* x = static_cast<const T*>(p[i].which ? a.v : a.k) + p[i].b * st[0] + p[i].h * st[1] + p[i].n * st[2] +
                   p[i].g * kGroup + lane8 * 8;
      in[i].load(x);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t u = u0 + static_cast<int64_t>(i) * per;
      float x[8];
      in[i].get(x);
      const Held q = quantise(x);
      if (u >= ra.units) continue;
      const int64_t slot = static_cast<int64_t>(a.start ? a.start[p[i].b] : 0) + p[i].n;
      const bool wanted = slot >= 0 && slot < static_cast<int64_t>(a.M) << a.pool.shift &&
                          (!a.limit || p[i].n < a.limit[p[i].b]);
      const int page = wanted ? page_at(a.pool, a.table + static_cast<int64_t>(p[i].b) * a.M, static_cast<int>(slot >> a.pool.shift)) : -1;
      if (page >= 0) {
        const int in_page = static_cast<int>(slot) & (a.pool.page - 1);
        uint8_t* part = part_of(a.pool, page, p[i].h, p[i].which);
        *reinterpret_cast<uint32_t*>(part + in_page * (D / 2) + word_offset<G>(p[i].g, lane8, in_page)) = q.word;
        // the first lane the scale, the second the minimum
        uint16_t* meta = reinterpret_cast<uint16_t*>(part + a.pool.page * (D / 2) + in_page * (4 * G));
        if (lane8 < 2) meta[lane8 * G + p[i].g] = static_cast<uint16_t>(__float_as_uint(lane8 ? q.lo : q.s) >> 16);
      }
      if (a.k_out) {
        values_of(q, x);
        const int64_t row = (static_cast<int64_t>(p[i].b) * a.pool.Hkv + p[i].h) * a.N + p[i].n;
        Eight<T>::put(static_cast<T*>(p[i].which ? a.v_out : a.k_out) + row * D + p[i].g * kGroup + lane8 * 8, x);
      }
    }
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) page_read_kernel(const RowsArgs ra) {
  constexpr int G = D / kGroup;
  const PageRows& a = ra.a;
  const int lane8 = threadIdx.x & 7, per = gridDim.x * (kThreads / 8);
  for (int64_t u0 = blockIdx.x * (kThreads / 8) + (threadIdx.x >> 3); u0 < ra.units; u0 += static_cast<int64_t>(kAhead) * per) {
    Held q[kAhead];
    Place p[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t u = u0 + static_cast<int64_t>(i) * per;
      p[i] = place_of<G>(static_cast<uint32_t>(u < ra.units ? u : 0), ra);
      const int64_t slot = static_cast<int64_t>(a.start ? a.start[p[i].b] : 0) + p[i].n;
      const bool wanted = slot >= 0 && slot < static_cast<int64_t>(a.M) << a.pool.shift &&
                          (!a.limit || slot < a.limit[p[i].b]);
      const int page = wanted ? page_at(a.pool, a.table + static_cast<int64_t>(p[i].b) * a.M, static_cast<int>(slot >> a.pool.shift)) : -1;
      q[i] = Held{0u, 0.0f, 0.0f};
      if (page >= 0) {
        const int in_page = static_cast<int>(slot) & (a.pool.page - 1);
        const uint8_t* part = part_of(a.pool, page, p[i].h, p[i].which);
        q[i].word = __ldcs(reinterpret_cast<const uint32_t*>(part + in_page * (D / 2) + word_offset<G>(p[i].g, lane8, in_page)));
        const uint16_t* meta = reinterpret_cast<const uint16_t*>(part + a.pool.page * (D / 2) + in_page * (4 * G));
        q[i].s = bf16_low(meta[p[i].g]);
        q[i].lo = bf16_low(meta[G + p[i].g]);
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (u0 + static_cast<int64_t>(i) * per >= ra.units) break;
      float x[8];
      values_of(q[i], x);
      const int64_t row = (static_cast<int64_t>(p[i].b) * a.pool.Hkv + p[i].h) * a.N + p[i].n;
      Eight<T>::put(static_cast<T*>(p[i].which ? a.v_out : a.k_out) + row * D + p[i].g * kGroup + lane8 * 8, x);
    }
  }
}

template <bool WRITE, typename T, int D>
cudaError_t go(const RowsArgs& ra, cudaStream_t st) {
  const int64_t most = 8 * kSms, need = (ra.units + kThreads / 8 - 1) / (kThreads / 8);
  const int grid = static_cast<int>(need < most ? need : most);
  if constexpr (WRITE) page_write_kernel<T, D><<<grid, kThreads, 0, st>>>(ra);
  else page_read_kernel<T, D><<<grid, kThreads, 0, st>>>(ra);
  return cudaGetLastError();
}
template <bool WRITE>
cudaError_t launch(const PageRows& a, bool bf16, cudaStream_t st) {
  const int G = a.pool.D / kGroup;
  RowsArgs ra{a, fast_div(G), fast_div(a.N), fast_div(a.pool.Hkv), fast_div(a.B), 2 * a.B * a.pool.Hkv * a.N * G};
  if (bf16) return G == 1 ? go<WRITE, __nv_bfloat16, 64>(ra, st) : go<WRITE, __nv_bfloat16, 128>(ra, st);
  return G == 1 ? go<WRITE, float, 64>(ra, st) : go<WRITE, float, 128>(ra, st);
}

}  // namespace

cudaError_t launch_page_write(const PageRows& a, bool bf16, cudaStream_t st) { return launch<true>(a, bf16, st); }
cudaError_t launch_page_read(const PageRows& a, bool bf16, cudaStream_t st) { return launch<false>(a, bf16, st); }

}  // namespace raattn
