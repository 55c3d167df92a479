// The order in which the prompt kernels take their units: rows of packed sequences, those
// with the most keys first.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace medusa {

// A sequence is cut into tiles of 2^shift rows; units are (tile number, sequence), by tile
// number from the last one down, then by sequence, so that the longest units start first and
// the shortest fill the end. A whole warp calls every function. Sequences whose bounds leave
// [0, T] have no tiles, and neither have those from the first decrease of the bounds on: the
// others do not overlap, so that there are rows / 2^shift + B units at most (a grid holds no more).
// Up to 32 sequences each lane keeps the tiles of one and tile numbers are passed one by one (a
// short call is a chain of such latencies). Past 32 the bounds are read again for every tile
// number that is looked at, so those are found by doubling steps and halving intervals, and a
// sequence is looked for from where the last one was found: units asked for in ascending order
// cost little (4096 prompts of 1 to 60 rows, 8 heads, bf16: 322 us, 1815 with a scan for every unit).
struct PromptWalk {
  const int32_t* cu;
  int B, T, shift;
  bool many;              // more than 32 sequences: B is then the number of those ahead of the first decrease
  int mine;               // tiles of sequence `lane`
  int top;                // where t begins
  int t, before, count;   // `count` units have tile number t; `before` come ahead of them
  int at, passed;         // past 32: `passed` of those belong to sequences ahead of `at`

  __device__ __forceinline__ int lane() const { return threadIdx.x & 31; }
  __device__ __forceinline__ int tiles_between(int c0, int c1) const {
    return (c0 >= 0 && c1 >= c0 && c1 <= T) ? (int)(((unsigned)(c1 - c0) + (1u << shift) - 1) >> shift) : 0;
  }
  __device__ __forceinline__ int tiles(int b) const { return b < B ? tiles_between(cu[b], cu[b + 1]) : 0; }
  // the lane of the rank-th vote
  __device__ __forceinline__ int pick(unsigned votes, int rank) const {
    const bool it = ((votes >> lane()) & 1u) && __popc(votes & ((1u << lane()) - 1u)) == rank;
    return __ffs(__ballot_sync(0xffffffffu, it)) - 1;
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
    many = B > 32;
    if (!many) {
      top = __reduce_max_sync(0xffffffffu, most) - 1;
      restart();
      return;
    }
    int fall = falls ? __ffs(falls) - 1 : B;
#pragma unroll 4
    for (int b = 32 + lane(); b < B; b += 32) {
      const int d0 = cu[b], d1 = cu[b + 1];
      if (d1 < d0) fall = min(fall, b);
      most = max(most, tiles_between(d0, d1));
    }
    B = __reduce_min_sync(0xffffffffu, fall);
    top = __reduce_max_sync(0xffffffffu, most);   // no unit has this tile number
    restart();
  }
  __device__ __forceinline__ void restart() {
    t = top;
    before = at = passed = 0;
    count = many || t < 0 ? 0 : __popc(__ballot_sync(0xffffffffu, mine > t));
  }
  // Sequence of unit u (t: its tile number), or -1 past the last unit.
  __device__ int find(int u) {
    if (u < before) restart();
    if (many) return find_many(u);
    while (t >= 0 && u >= before + count) {
      before += count;
      --t;
      count = t >= 0 ? __popc(__ballot_sync(0xffffffffu, mine > t)) : 0;
    }
    if (t < 0) return -1;
    const int rank = u - before;
    return pick(__ballot_sync(0xffffffffu, mine > t), rank);
  }
  __device__ __forceinline__ int find_many(int u) {
    if (u >= before + count) {   // the largest tile number `lo` that more than u units have or exceed
      int hi = t, units_hi = before + count, lo = -1, units_lo = 0, step = 1;
      while (lo < 0 || hi - lo > 1) {
        if (hi == 0) {   // there are no more
          t = count = 0;
          before = units_hi;
          return -1;
        }
        const int x = lo < 0 ? max(0, hi - step) : (lo + hi) >> 1;
        int n = 0;
#pragma unroll 4
        for (int b = lane(); b < B; b += 32) n += max(0, tiles_between(cu[b], cu[b + 1]) - x);
        n = __reduce_add_sync(0xffffffffu, n);   // units with tile number x or more
        if (n > u) {
          lo = x;
          units_lo = n;
        } else {
          hi = x;
          units_hi = n;
          step *= 2;
        }
      }
      t = lo;
      before = units_hi;
      count = units_lo - units_hi;
      at = passed = 0;
    }
    const int rank = u - before;
    if (rank < passed) at = passed = 0;
    while (at < B) {
      constexpr int X = 4;   // groups of 32 sequences that are fetched together
      int n[X];
#pragma unroll
      for (int x = 0; x < X; ++x) n[x] = tiles(at + 32 * x + lane());
#pragma unroll
      for (int x = 0; x < X; ++x) {
        const unsigned votes = __ballot_sync(0xffffffffu, n[x] > t);
        const int c = __popc(votes);
        if (rank - passed < c) return at + pick(votes, rank - passed);
        passed += c;
        at += 32;
      }
    }
    return -1;
  }
};

}  // namespace medusa
