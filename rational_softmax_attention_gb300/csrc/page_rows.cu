// Keys and values into pages held in 4 bits, and out of them (the layout and its mathematics: paged.cuh).
//
// A warp takes sixteen neighbouring slots of one head's keys or values, which lie in one page: what depends on the
// place is formed once for 2048 elements (D = 128).  Eight lanes have a token's row, a lane eight dimensions, one word of
// codes, of each group, four tokens at a time.
//
// Codes of bf16 rows.  fma(x - lo, 1 / s, 3 2^22) has the nearest integer in its low bits.  With the reciprocal's
// neighbours on either side the two results differ only next to the middle between two codes; there the even one is right
// if x - lo is the middle exactly.  Numbers of eight bits that are not far below s cannot come closer without meeting it:
// with (2 k + 1) s / 2 in steps of 2^(e_s - 8) and x - lo in steps of 2^(e_x - 7), e the exponents, a distance is 0 or
// at least 2^-19 s from |x| >= 2^-10 s on, and the reciprocals' neighbours part at 15 2^-23.  A lane with a smaller x takes
// the way of fp32 rows: u' = rint((x - lo) (1 / s)) is one off at most, and the remainder (x - lo) - s u', which an FMA
// gives exactly, with what x - lo itself has lost, says whether it is.
// Minimum and maximum of a group, as bf16 pairs (min x, min -x): the 32 (D = 128) groups of a warp's tokens are reduced
// over their eight lanes each so that every lane ends with one group, and forms that group's lo and s for all.
//
// Bound: HBM, with the issue slots close behind in the write (about twelve instructions an element).  bf16 H8 D128: write with
// the held values B4 N4096, 153 MB in 30.7 us, 5.0 TB/s (six CTAs per SM; 35.5 with the registers of four); read B4 N16384,
// 344 MB in 57 us, 6.05 TB/s.
#include <climits>

#include "paged.cuh"

namespace raattn {
namespace {

using namespace paged;

constexpr int kThreads = 128;
constexpr int kSlots = 16, kSteps = 4;   // slots of a warp at a time, four in a step

struct RowsArgs {
  PageRows a;
  FastDiv chunks, Hkv, B;   // item = ((which B + b) Hkv + h) chunks + chunk
  int items;
};

// A warp's sixteen slots.
struct Chunk {
  int which, b, h;
  int n;           // token of the call in the first slot (negative: the first ones lie in later slots)
  int slot;        // of the first one in its page
  int page;        // -1: none
  __device__ __forceinline__ Chunk(const RowsArgs& ra, int item) {
    const PageRows& a = ra.a;
    uint32_t x = div_by(item, ra.chunks);
    const int chunk = item - x * ra.chunks.d;
    uint32_t y = div_by(x, ra.Hkv);
    h = x - y * ra.Hkv.d;
    which = y >= ra.B.d;
    b = y - which * ra.B.d;
    const int64_t start = a.start ? a.start[b] : 0, first = (start & ~static_cast<int64_t>(kSlots - 1)) + kSlots * static_cast<int64_t>(chunk);
    n = static_cast<int>(first - start);   // at most N + 15: 32 bits hold it
    const bool in = first >= 0 && first < static_cast<int64_t>(a.M) << a.pool.shift;
    page = in ? page_at(a.pool, a.table + static_cast<int64_t>(b) * a.M, static_cast<int>(first >> a.pool.shift)) : -1;
    slot = static_cast<int>(first) & (a.pool.page - 1);
  }
};

// A lane's eight elements.
template <typename T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p, bool in) {
    u = in ? __ldcs(reinterpret_cast<const uint4*>(p)) : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = bf16_low(w[i]);
      x[2 * i + 1] = bf16_high(w[i]);
    }
  }
  // a bf16 output's rounding, after the fp32 of lo + s u: half a step, 2^-8 relative at most
  static __device__ __forceinline__ void put(__nv_bfloat16* p, const float (&x)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                                              pack_bf16x2(x[6], x[7]));
  }
};
template <>
struct Eight<float> {
  float4 u, v;
  __device__ __forceinline__ void load(const float* p, bool in) {
    u = in ? __ldcs(reinterpret_cast<const float4*>(p)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    v = in ? __ldcs(reinterpret_cast<const float4*>(p) + 1) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
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

constexpr float kRound = 12582912.0f;   // 3 2^22: a sum with it has the nearest integer in its low bits

// A group's minimum and maximum as it is held.  All arithmetic is exact or its error is accounted for, so that lo, s and the
// codes are those of the definition whatever the inputs.
struct Scale {
  float s, lo;
  __device__ __forceinline__ Scale(float low, float high) {
    // 16 bits, rounded down (towards -infinity); no minus zero
    const uint32_t lb = __float_as_uint(__fadd_rn(low, 0.0f));
    lo = __uint_as_float((lb >> 31 ? lb + 0xffffu : lb) & 0xffff0000u);
    // the least s of 16 bits with 15 s >= high - lo = span + rest
    const float span = __fsub_rn(high, lo), rest = lost(high, lo, span);
    uint32_t sb = (__float_as_uint(__fmul_rn(span, 1.0f / 15.0f)) + 0xffffu) & 0xffff0000u;
    const auto covers = [&](uint32_t bits) {   // the product has 12 bits; the difference of near numbers is exact
      return __fsub_rn(__fmul_rn(15.0f, __uint_as_float(bits)), span) >= rest;
    };
    if (sb >= 0x10000u && covers(sb - 0x10000u)) sb -= 0x10000u;
    else if (!covers(sb)) sb += 0x10000u;
    s = __uint_as_float(sb);
    const float kInf = __uint_as_float(0x7f800000u);
    const bool good = span < kInf && s < kInf;   // a NaN is not
    if (!good) lo = __uint_as_float(0x7fc00000u);
    if (!good || s < 0x1p-100f) s = 0.0f;
  }
  __device__ __forceinline__ Scale(uint32_t bits) : s(bf16_low(bits)), lo(bf16_high(bits)) {}
  __device__ __forceinline__ uint32_t bits() const { return __float_as_uint(s) >> 16 | __float_as_uint(lo); }
};

// A word of codes of any eight numbers.
__device__ __noinline__ uint32_t codes_of(const Scale q, float x0, float x1, float x2, float x3, float x4, float x5, float x6,
                                          float x7) {
  const float x[8] = {x0, x1, x2, x3, x4, x5, x6, x7};
  const float inv = q.s > 0.0f ? 1.0f / q.s : 0.0f, half = 0.5f * q.s;
  uint32_t word = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float d = __fsub_rn(x[i], q.lo);
    const float t = __fmaf_rn(d, inv, kRound);
    float u = __fsub_rn(t, kRound);           // 0 to 15, one off at most
    const float r = fmaf(-q.s, u, d);         // exact
    // beyond the middle, or in it with an odd code: the next one; where d itself was rounded that decides
    float over = fabsf(r) - half;
    if (over == 0.0f) over = copysignf(1.0f, r) * lost(x[i], q.lo, d);
    int c = __float_as_int(t);
    if (over > 0.0f || (over == 0.0f && (c & 1))) c += r < 0.0f ? -1 : 1;
    word |= (q.s > 0.0f ? static_cast<uint32_t>(c) & 15u : 0u) << (4 * i);
  }
  return word;
}

// The values that a word of codes stands for: a byte with one code and zeros above becomes the float 2^23 + u.
__device__ __forceinline__ void values_of(uint32_t word, const Scale& q, float (&x)[8]) {
  const uint32_t low = word & 0x0f0f0f0fu, high = (word >> 4) & 0x0f0f0f0fu;
  const float2 s = make_float2(q.s, q.s), lo = make_float2(q.lo, q.lo), back = make_float2(-8388608.0f, -8388608.0f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 u = make_float2(__uint_as_float(__byte_perm(low, 0x4b000000u, 0x7440 + i)),
                                 __uint_as_float(__byte_perm(high, 0x4b000000u, 0x7440 + i)));
    const float2 v = __ffma2_rn(s, __fadd2_rn(u, back), lo);
    x[2 * i] = v.x;
    x[2 * i + 1] = v.y;
  }
}

__device__ __forceinline__ uint32_t min2_nan(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ uint32_t max2_nan(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}

// The scales of a warp's groups, and its words of codes.  in[i][g]: group g of step i's token of this lane's eight.
template <int G>
__device__ __forceinline__ void quantise(const Eight<__nv_bfloat16> (&in)[kSteps][G], uint32_t (&scale)[kSteps][G],
                                         uint32_t (&word)[kSteps][G]) {
  const int lane8 = threadIdx.x & 7;
  // (min x, min -x) of this lane's eight
  uint32_t m[kSteps * G];
#pragma unroll
  for (int i = 0; i < kSteps; ++i)
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const uint4& u = in[i][g].u;
      const uint32_t low = min2_nan(min2_nan(u.x, u.y), min2_nan(u.z, u.w)), high = max2_nan(max2_nan(u.x, u.y), max2_nan(u.z, u.w));
      // the halves' minima, and the maxima with the sign turned
      const uint32_t a = __byte_perm(low, high ^ 0x80008000u, 0x5410), b = __byte_perm(low, high ^ 0x80008000u, 0x7632);
      m[i * G + g] = min2_nan(a, b);
    }
  // over the eight lanes: in each step a lane keeps half of its groups and gives the others away
#pragma unroll
  for (int left = kSteps * G, o = 4; o > 0; o >>= 1) {
    if (left > 1) {
      left >>= 1;
      const bool up = lane8 & o;
#pragma unroll
      for (int k = 0; k < left; ++k) {
        const uint32_t give = up ? m[k] : m[k + left], keep = up ? m[k + left] : m[k];
        m[k] = min2_nan(keep, __shfl_xor_sync(0xffffffffu, give, o));
      }
    } else {
      m[0] = min2_nan(m[0], __shfl_xor_sync(0xffffffffu, m[0], o));
    }
  }
  const Scale mine(bf16_low(m[0]), -bf16_high(m[0]));
  // the reciprocal; negative: a group whose numbers may come closer to a middle than they can in the fast way
  const float near = 0x1p-10f * mine.s;
  const bool far = mine.lo == 0.0f || fabsf(mine.lo) >= near;   // a NaN is not
  const float inv = mine.s > 0.0f ? 1.0f / mine.s : 0.0f;
  const uint32_t bits = mine.bits();
  const float inv_mine = far ? inv : -1.0f;
  const int base = threadIdx.x & 24;
  constexpr int kShare = 8 / (kSteps * G);   // lanes with the same group
#pragma unroll
  for (int i = 0; i < kSteps; ++i)
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int from = base + (i * G + g) * kShare;
      scale[i][g] = __shfl_sync(0xffffffffu, bits, from);
      const float r = __shfl_sync(0xffffffffu, inv_mine, from);
      const Scale q(scale[i][g]);
      float x[8];
      in[i][g].get(x);
      const uint4& u = in[i][g].u;
      // the smallest magnitude
      const uint32_t k = 0x7fff7fffu;
      const uint32_t least = min2_nan(min2_nan(u.x & k, u.y & k), min2_nan(u.z & k, u.w & k));
      const float smallest = fminf(bf16_low(least), bf16_high(least));
      if (r >= 0.0f && smallest >= 0x1p-10f * q.s) {
        const float2 lo = make_float2(-q.lo, -q.lo), round = make_float2(kRound, kRound);
        const float down = __uint_as_float(__float_as_uint(r) - (r > 0.0f)), up = __uint_as_float(__float_as_uint(r) + (r > 0.0f));
        uint32_t pair[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 d = __fadd2_rn(make_float2(x[2 * e], x[2 * e + 1]), lo);
          const float2 s0 = __ffma2_rn(d, make_float2(down, down), round), s1 = __ffma2_rn(d, make_float2(up, up), round);
          const uint32_t a0 = __float_as_uint(s0.x), a1 = __float_as_uint(s1.x), b0 = __float_as_uint(s0.y), b1 = __float_as_uint(s1.y);
          const uint32_t first = a0 + ((a0 ^ a1) & a0 & 1u), second = b0 + ((b0 ^ b1) & b0 & 1u);   // the even one of two
          pair[e] = second * 16u + first;   // its low byte
        }
        word[i][g] = __byte_perm(__byte_perm(pair[0], pair[1], 0x0040), __byte_perm(pair[2], pair[3], 0x0040), 0x5410);
      } else {
        word[i][g] = codes_of(q, x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7]);
      }
    }
}
template <int G>
__device__ __forceinline__ void quantise(const Eight<float> (&in)[kSteps][G], uint32_t (&scale)[kSteps][G],
                                         uint32_t (&word)[kSteps][G]) {
#pragma unroll
  for (int i = 0; i < kSteps; ++i)
#pragma unroll
    for (int g = 0; g < G; ++g) {
      float x[8];
      in[i][g].get(x);
      float low = x[0], high = x[0];
#pragma unroll
      for (int e = 1; e < 8; ++e) {
        low = min_nan(low, x[e]);
        high = max_nan(high, x[e]);
      }
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) {
        low = min_nan(low, __shfl_xor_sync(0xffffffffu, low, o));
        high = max_nan(high, __shfl_xor_sync(0xffffffffu, high, o));
      }
      const Scale q(low, high);
      scale[i][g] = q.bits();
      word[i][g] = codes_of(q, x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7]);
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 6) page_write_kernel(const RowsArgs ra) {
  constexpr int G = D / kGroup;
  const PageRows& a = ra.a;
  const int w = threadIdx.x & 7, token = (threadIdx.x & 31) >> 3, warps = gridDim.x * (kThreads / 32);
  await_previous();
  release_dependents();
  for (int64_t item = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); item < ra.items; item += warps) {
    const Chunk c(ra, static_cast<int>(item));
    if (c.n >= a.N) continue;
    const int64_t* st = c.which ? a.v_stride : a.k_stride;
    const T* src = static_cast<const T*>(c.which ? a.v : a.k) + c.b * st[0] + c.h * st[1] + w * 8;
    Eight<T> in[kSteps][G];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int n = c.n + 4 * i + token;
      const bool there = n >= 0 && n < a.N;
#pragma unroll
      for (int g = 0; g < G; ++g) in[i][g].load(src + (there ? n : 0) * st[2] + g * kGroup, there);
    }
    uint32_t scale[kSteps][G], word[kSteps][G];
    quantise<G>(in, scale, word);
    const int last = a.limit ? min(a.limit[c.b], a.N) : a.N;
    uint8_t* part = part_of(a.pool, max(c.page, 0), c.h, c.which);
    uint8_t* meta = part + a.pool.page * (D / 2);
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int n = c.n + 4 * i + token, slot = c.slot + 4 * i + token;
      if (c.page >= 0 && n >= 0 && n < last) {
        if constexpr (G == 2) {
          *reinterpret_cast<uint2*>(part + slot * (D / 2) + word_offset<G>(0, w, slot)) = make_uint2(word[i][0], word[i][1]);
          if (w == 0)
            *reinterpret_cast<uint2*>(meta + slot * 8) =
                make_uint2(__byte_perm(scale[i][0], scale[i][1], 0x5410), __byte_perm(scale[i][0], scale[i][1], 0x7632));
        } else {
          *reinterpret_cast<uint32_t*>(part + slot * (D / 2) + w * 4) = word[i][0];
          if (w == 0) *reinterpret_cast<uint32_t*>(meta + slot * 4) = scale[i][0];
        }
      }
      if (a.k_out && n >= 0 && n < a.N) {
        T* out = static_cast<T*>(c.which ? a.v_out : a.k_out) + ((static_cast<int64_t>(c.b) * a.pool.Hkv + c.h) * a.N + n) * D + w * 8;
#pragma unroll
        for (int g = 0; g < G; ++g) {
          float x[8];
          values_of(word[i][g], Scale(scale[i][g]), x);
          Eight<T>::put(out + g * kGroup, x);
        }
      }
    }
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) page_read_kernel(const RowsArgs ra) {
  constexpr int G = D / kGroup;
  const PageRows& a = ra.a;
  const int w = threadIdx.x & 7, token = (threadIdx.x & 31) >> 3, warps = gridDim.x * (kThreads / 32);
  await_previous();
  release_dependents();
  for (int64_t item = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); item < ra.items; item += warps) {
    const Chunk c(ra, static_cast<int>(item));
    if (c.n >= a.N) continue;
    // tokens whose slots are below the length
    const int64_t last = a.limit ? static_cast<int64_t>(a.limit[c.b]) - (a.start ? a.start[c.b] : 0) : a.N;
    const uint8_t* part = part_of(a.pool, max(c.page, 0), c.h, c.which);
    const uint8_t* meta = part + a.pool.page * (D / 2);
    uint32_t word[kSteps][G], scale[kSteps][G];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int n = c.n + 4 * i + token, slot = c.slot + 4 * i + token;
#pragma unroll
      for (int g = 0; g < G; ++g) word[i][g] = scale[i][g] = 0u;
      if (c.page >= 0 && n >= 0 && n < a.N && n < last) {
        if constexpr (G == 2) {
          const uint2 u = __ldcs(reinterpret_cast<const uint2*>(part + slot * (D / 2) + word_offset<G>(0, w, slot)));
          const uint2 q = __ldcs(reinterpret_cast<const uint2*>(meta + slot * 8));
          word[i][0] = u.x;
          word[i][1] = u.y;
          scale[i][0] = __byte_perm(q.x, q.y, 0x5410);
          scale[i][1] = __byte_perm(q.x, q.y, 0x7632);
        } else {
          word[i][0] = __ldcs(reinterpret_cast<const uint32_t*>(part + slot * (D / 2) + w * 4));
          scale[i][0] = __ldcs(reinterpret_cast<const uint32_t*>(meta + slot * 4));
        }
      }
    }
    T* out = static_cast<T*>(c.which ? a.v_out : a.k_out) + ((static_cast<int64_t>(c.b) * a.pool.Hkv + c.h) * a.N) * D + w * 8;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int n = c.n + 4 * i + token;
      if (n >= 0 && n < a.N) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
          float x[8];
          values_of(word[i][g], Scale(scale[i][g]), x);
          Eight<T>::put(out + static_cast<int64_t>(n) * D + g * kGroup, x);
        }
      }
    }
  }
}

template <bool WRITE, typename T, int D>
cudaError_t go(const RowsArgs& ra, cudaStream_t st) {
  const int need = (ra.items - 1) / (kThreads / 32) + 1, most = 32 * kSms, grid = need < most ? need : most;
  if constexpr (WRITE) return launch_dependent(page_write_kernel<T, D>, grid, kThreads, 0, st, ra);
  else return launch_dependent(page_read_kernel<T, D>, grid, kThreads, 0, st, ra);
}
template <bool WRITE>
cudaError_t launch(const PageRows& a, bool bf16, cudaStream_t st) {
  const int chunks = (a.N + kSlots - 2) / kSlots + 1;   // sixteen slots each, wherever the first token falls
  const RowsArgs ra{a, fast_div(chunks), fast_div(a.pool.Hkv), fast_div(a.B), 2 * a.B * a.pool.Hkv * chunks};
  if (bf16) return a.pool.D == 64 ? go<WRITE, __nv_bfloat16, 64>(ra, st) : go<WRITE, __nv_bfloat16, 128>(ra, st);
  return a.pool.D == 64 ? go<WRITE, float, 64>(ra, st) : go<WRITE, float, 128>(ra, st);
}

}  // namespace

cudaError_t launch_page_write(const PageRows& a, bool bf16, cudaStream_t st) { return launch<true>(a, bf16, st); }
cudaError_t launch_page_read(const PageRows& a, bool bf16, cudaStream_t st) { return launch<false>(a, bf16, st); }

}  // namespace raattn
