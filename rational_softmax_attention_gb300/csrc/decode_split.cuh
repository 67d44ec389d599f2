// Where the decode kernels find a row's partial results (decode.cu, decode_prefix_tc.cu).
#pragma once

#include "kernels.cuh"

namespace raattn {

constexpr int kDecodeThreads = 128, kDecodeCtasPerSm = 3;
constexpr int kDecodeCtas = kSms * kDecodeCtasPerSm;   // a grid that fills every SM
constexpr int kDecodeRows = 16;                                               // query rows of a stream

struct DecodeSplit {
  int64_t total;   // blocks of all streams
  int64_t own0;    // blocks of the shared keys' streams, which come first
  int per;         // blocks of a run
};

// own: blocks per stream of all sequences together (cum[B]).
__device__ __forceinline__ DecodeSplit decode_split(const DecodeArgs& a, int own) {
  DecodeSplit s;
  s.own0 = a.tc ? 0 : static_cast<int64_t>(a.Hkv) * a.pblocks * a.shared_rowblocks;
  s.total = s.own0 + static_cast<int64_t>(own) * a.Hkv * a.own_rowblocks;
  const int64_t even = (s.total + a.runs - 1) / a.runs;
  s.per = static_cast<int>(even > a.min_run ? even : a.min_run);
  return s;
}

// The slots of a row: [0, shared) of the shared keys, [pslots, pslots + own) of its own; cum0 and
// cum1 are cum[b] and cum[b + 1] of its sequence.
__device__ __forceinline__ int decode_slots_of(int64_t stream0, int blocks, int per) {
  return blocks ? static_cast<int>((stream0 + blocks - 1) / per - stream0 / per) + 1 : 0;
}
__device__ __forceinline__ void decode_row_slots(int row, int cum0, int cum1, const DecodeSplit& s,
                                                 const DecodeArgs& a, int& shared, int& own) {
  const int b = row / a.Hq, h = row - b * a.Hq, kv = h / a.G, g = h - kv * a.G;
  if (a.tc) {
    shared = a.pslots;
  } else {
    const int64_t st = static_cast<int64_t>(kv) * a.shared_rowblocks + (b * a.G + g) / kDecodeRows;
    shared = decode_slots_of(st * a.pblocks, a.pblocks, s.per);
  }
  const int n = cum1 - cum0;
  const int64_t seq0 = s.own0 + static_cast<int64_t>(cum0) * a.Hkv * a.own_rowblocks;
  own = decode_slots_of(seq0 + static_cast<int64_t>(kv * a.own_rowblocks + g / kDecodeRows) * n, n, s.per);
}

}  // namespace raattn
