// The order in which the prompt kernels take their units: rows of packed sequences, those
// with the most keys first.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace medusa {

// A sequence is cut into tiles of 2^shift rows; units are (tile number, sequence), by tile
// number from the last one down, then by sequence, so that the longest units start first and
// the shortest fill the end. A whole warp calls every function; units asked for in ascending
// order cost little. Sequences whose bounds leave [0, T] have no tiles, and neither have those
// from the first decrease of the bounds on: the others do not overlap, so that there are
// rows / 2^shift + B units at most (a grid holds no more). Each lane keeps the tiles of one of the
// first 32 sequences (a short call is a chain of such latencies).
struct PromptWalk {
  const int32_t* cu;
  int B, T, shift;        // B: sequences; past 32, those ahead of the first decrease
  int mine;               // tiles of sequence `lane`
  int t, before, count;   // `count` units have tile number t; `before` come ahead of them

  __device__ __forceinline__ int lane() const { return threadIdx.x & 31; }
  __device__ __forceinline__ int tiles_between(int c0, int c1) const {
    return (c0 >= 0 && c1 >= c0 && c1 <= T) ? (int)(((unsigned)(c1 - c0) + (1u << shift) - 1) >> shift) : 0;
  }
  __device__ __forceinline__ int tiles(int b) const { return b < B ? tiles_between(cu[b], cu[b + 1]) : 0; }
  __device__ __forceinline__ int above() const {   // sequences with more than t tiles
    if (B <= 32) return __popc(__ballot_sync(0xffffffffu, mine > t));
    int c = mine > t;
    for (int b = 32 + lane(); b < B; b += 32) c += tiles(b) > t;
    return __reduce_add_sync(0xffffffffu, c);
  }
  __device__ void begin(const int32_t* cu_, int B_, int T_, int shift_) {
    cu = cu_;
    B = B_;
    T = T_;
    shift = shift_;
    const int c0 = lane() < B ? cu[lane()] : 0, c1 = lane() < B ? cu[lane() + 1] : 0;
    const unsigned falls = __ballot_sync(0xffffffffu, c1 < c0);
    // (lanes from the first fall on have none)
    mine = lane() < B && !(falls & ((2u << lane()) - 1)) ? tiles_between(c0, c1) : 0;
    int most = mine;
    if (B > 32) {
      if (falls) B = 32;
      for (int b0 = 32; b0 < B; b0 += 32) {
        const int b = b0 + lane(), d0 = b < B ? cu[b] : 0, d1 = b < B ? cu[b + 1] : 0;
        const unsigned f = __ballot_sync(0xffffffffu, d1 < d0);
        if (f) B = b0 + __ffs(f) - 1;
        if (b < B) most = max(most, tiles_between(d0, d1));
      }
    }
    t = __reduce_max_sync(0xffffffffu, most) - 1;
    before = 0;
    count = t >= 0 ? above() : 0;
  }
  // Sequence of unit u (t: its tile number), or -1 past the last unit.
  __device__ int find(int u) {
    if (u < before) begin(cu, B, T, shift);
    while (t >= 0 && u >= before + count) {
      before += count;
      --t;
      count = t >= 0 ? above() : 0;
    }
    if (t < 0) return -1;
    int rank = u - before;
    for (int b0 = 0; b0 < B; b0 += 32) {
      const unsigned votes = __ballot_sync(0xffffffffu, (b0 == 0 ? mine : tiles(b0 + lane())) > t);
      const int c = __popc(votes);
      if (rank < c) {   // the rank-th of the votes
        const bool it = ((votes >> lane()) & 1u) && __popc(votes & ((1u << lane()) - 1u)) == rank;
        return b0 + __ffs(__ballot_sync(0xffffffffu, it)) - 1;
      }
      rank -= c;
    }
    return -1;
  }
};

}  // namespace medusa
