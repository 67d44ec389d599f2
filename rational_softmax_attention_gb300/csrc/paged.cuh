// Pages of a key/value cache held in 4 bits, and what the page operators need of them.
//
// A token's row of D keys (or values) of one head is cut into groups of 64 dimensions.  A group is held as
//   lo  the largest 16-bit (bfloat16) number that is not above the group's minimum,
//   s   the least 16-bit number whose fifteenfold covers maximum - lo,
//   u   64 codes of 4 bits, the nearest integers to (x - lo) / s, ties to even,
// and stands for lo + s u, at most s / 2 away from x.  A group with a NaN, an infinity or a span that fp32 does
// not hold has lo = NaN; a span below 15 * 2^-100 has s = 0.
//
// A pool is [pages][key heads][keys, values] parts of page * row bytes, row = D / 2 + D / 16; a part is its tokens'
// codes, then their scales and minima: (s of each group, lo of each group).  D = 128: 72 bytes for the 256 of bfloat16.
// Dimension 64 g + 8 w + n is nibble n of a token's 32-bit word w G + g, G = D / 64: 16 bytes of a row hold two
// words of every group, as a lane of the score products wants them, and 8 bytes one word of every group, as a lane
// of the value products does.  With D = 128 tokens with bit 1 of their slot set hold their two 32-byte halves in
// the other order: the 8-byte reads of four neighbouring tokens then meet no bank conflict in shared memory.
#pragma once

#include "kernels.cuh"

namespace raattn {
namespace paged {

constexpr int kGroup = 64;

__host__ __device__ constexpr int row_bytes(int D) { return D / 2 + D / 16; }

// The part of head h (which: 0 keys, 1 values) of a page.
__device__ __forceinline__ uint8_t* part_of(const PagePool& p, int64_t page, int h, int which) {
  return p.base + page * p.page_stride + (2 * h + which) * p.part;   // a page's bytes fit 32 bits
}
// Page `at` of a table row, or -1: none, or no page of the pool.
__device__ __forceinline__ int page_at(const PagePool& p, const int32_t* row, int at) {
  const int id = row[at];
  return static_cast<unsigned>(id) < static_cast<unsigned>(p.pages) ? id : -1;
}
// Byte of word w G + g of a token's codes.
template <int G>
__device__ __forceinline__ int word_offset(int g, int w, int slot) {
  const int at = (w * G + g) * 4;
  return G == 2 ? at ^ ((slot & 2) << 4) : at;
}

__device__ __forceinline__ float bf16_low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Division by a number that the host knows: n / d for n, d < 2^31.
struct FastDiv {
  uint32_t d, mul, shift;
};
inline FastDiv fast_div(int64_t d) {
  FastDiv f{static_cast<uint32_t>(d), 0, 0};
  while ((1ll << f.shift) < d) ++f.shift;
  f.mul = static_cast<uint32_t>(((1ull << 32) * ((1ull << f.shift) - static_cast<uint64_t>(d))) / static_cast<uint64_t>(d) + 1);
  return f;
}
__device__ __forceinline__ uint32_t div_by(uint32_t n, const FastDiv& f) {
  return (__umulhi(n, f.mul) + n) >> f.shift;   // n < 2^31: the sum fits
}

}  // namespace paged
}  // namespace raattn
