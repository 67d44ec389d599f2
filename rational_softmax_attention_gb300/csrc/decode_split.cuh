// Where the decode kernels find a row's partial results (decode.cu, decode_prefix_tc.cu).
#pragma once

#include "kernels.cuh"

namespace raattn {

constexpr int kDecodeThreads = 128, kDecodeCtasPerSm = 3;
constexpr int kDecodeCtas = kSms * kDecodeCtasPerSm;   // a grid that fills every SM
constexpr int kDecodeRows = 16;                                               // query rows of a stream

// All in 32 bits (plan_decode refuses more blocks): divisions are on every kernel's way.
struct DecodeSplit {
  int total;   // blocks of all streams
  int own0;    // blocks of the shared keys' streams, which come first
  int per;     // blocks of a run
};

// own: blocks per stream of all sequences together (cum[B]); longest: the most of one.  A run is as short
// as the grid allows, and long enough for the streams' partial results to find their places.  With a
// run per warp the runs are equal parts of all blocks.  With one per CTA each stream is cut for itself,
// into runs of `per` blocks that are few enough for one grid: no more than total / per and one for each
// of the (few) streams.
__device__ __forceinline__ DecodeSplit decode_split(const DecodeArgs& a, int own, int longest) {
  DecodeSplit s;
  s.own0 = a.Hkv * a.pblocks * a.shared_rowblocks;   // 0 with tc
  s.total = s.own0 + own * a.Hkv * a.own_rowblocks;
  s.per = max((s.total + a.runs - 1) / a.runs, a.least);
  const int own_places = a.slots - a.pslots - 1;   // a stream of n blocks meets at most ceil(n / per) + 1 runs
  s.per = max(s.per, (longest + own_places - 1) / own_places);
  if (a.pblocks) s.per = max(s.per, (a.pblocks + a.pslots - 2) / (a.pslots - 1));
  if (a.team > 1) s.per = (s.per + a.team - 1) / a.team * a.team;   // as many for each warp
  return s;
}

// The slots of a row: [0, shared) of the shared keys, [pslots, pslots + own) of its own; cum0 and
// cum1 are cum[b] and cum[b + 1] of its sequence.
__device__ __forceinline__ int decode_slots_of(int stream0, int blocks, int per) {
  return blocks ? (stream0 + blocks - 1) / per - stream0 / per + 1 : 0;
}
__device__ __forceinline__ void decode_row_slots(int b, int kv, int g, int cum0, int cum1, const DecodeSplit& s,
                                                 const DecodeArgs& a, int& shared, int& own) {
  const int n = cum1 - cum0;
  if (a.team > 1) {
    shared = a.tc ? a.pslots : (a.pblocks + s.per - 1) / s.per;
    own = (n + s.per - 1) / s.per;
    return;
  }
  shared = a.tc ? a.pslots
                : decode_slots_of((kv * a.shared_rowblocks + (b * a.G + g) / kDecodeRows) * a.pblocks, a.pblocks, s.per);
  own = decode_slots_of(s.own0 + cum0 * a.Hkv * a.own_rowblocks + (kv * a.own_rowblocks + g / kDecodeRows) * n, n,
                        s.per);
}

}  // namespace raattn
