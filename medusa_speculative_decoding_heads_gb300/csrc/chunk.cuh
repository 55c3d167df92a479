// Attention of new tokens over the pages of a cache: what its kernels share.
//
// Work. A unit is a block of query rows (the query heads of one KV head that share a tile, times
// positions) of one sequence; it takes the key tiles that any of its rows sees, the first rows' ones
// ahead of the window's. All units' tiles, one after another, are cut into equal ranges, one for each
// stream (a CTA), wherever the cuts fall: lengths differ from sequence to sequence and are on the device
// only, and so are the cuts. A unit that is cut leaves partial
// results, at most two per stream (of the unit that was begun ahead of its range, and of the one that
// ends behind it), which chunk_merge_kernel joins.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/medusa.h"

namespace medusa {

constexpr int kChunkStreams = 152;   // one CTA per SM

struct ChunkArgs {
  const int32_t* cu;      // [B + 1]
  const int32_t* start;   // [B], or NULL: 0
  const int32_t* table;   // [B][max_pages]
  int B, T, Hq, Hkv;
  int L_cap, page_rows, max_pages, num_pages;
  int window, sinks;      // row p sees keys j <= p with j > p - window or j < sinks
  int64_t q_stride;
  float scale_log2;
};

// A unit that begins in a stream's range and ends behind it; parts: how many further streams have a
// part of it (0: there is no such unit).
struct ChunkCut {
  int pos0, left, h0, parts;   // first packed row, positions from it on, first query head
};

// Partial results. Two classes of units: `pairs`, two tiles of npos positions over the same keys, of
// sequences with more than npos rows; `singles`, one tile, of the others. (float32: one tile, of
// sequences with more than one row, and up to 4 heads of single tokens.)
struct ChunkSpace {
  int gp_shift, npos;          // query heads of a tile (log2), positions of a tile
  int pair_streams, pair_rows; // streams, and rows of one partial result
  int streams, single_rows, single_npos, single_shift;   // the same of single tiles, their positions and heads (log2)
  size_t ml, cuts, total;      // where maxima and sums begin, and the cuts, in bytes
  __host__ __device__ int64_t pair_part(int stream, int second) const { return ((int64_t)2 * stream + second) * pair_rows; }
  __host__ __device__ int64_t single_part(int stream, int second) const {
    return (int64_t)2 * pair_streams * pair_rows + ((int64_t)2 * stream + second) * single_rows;
  }
};

// The tiles that units take. kShift: log2 of the keys of a tile.
template <int kShift>
struct ChunkTiles {
  int window, sink_tiles;
  __device__ __forceinline__ void begin(int window_, int sinks) {
    window = window_;
    sink_tiles = (int)(((unsigned)sinks + ((1u << kShift) - 1)) >> kShift);
  }
  // key tiles between the first rows and the window of row p, which nothing of a unit that begins with p sees
  __device__ __forceinline__ int skip(int p) const { return max(0, (max(0, p - window + 1) >> kShift) - sink_tiles); }
  // tiles of a unit of the logical rows p0 .. p1
  __device__ __forceinline__ int count(int p0, int p1) const { return (p1 >> kShift) + 1 - skip(p0); }
  // key tile that is number j of a unit
  __device__ __forceinline__ int tile(int j, int skipped) const { return j < sink_tiles ? j : j + skipped; }
};

// A part of a unit: `m` of its `all` tiles, from number `off` on.
struct ChunkPart {
  int b, s, n, c0;        // the sequence, its first logical row, rows, first packed row
  int row, hg;            // the unit's first row of them, its group of query heads
  int off, m, all, x;     // x: where among all tiles it begins
  __device__ __forceinline__ bool cut() const { return m < all; }   // (a unit that is cut writes partial results)
};

// A stream's units of one class, one after another; a whole warp calls every function. (What it does ahead
// of the first unit is time without any: its code is short, and counted in 32 bits, which the host has checked.)
template <int kShift>
struct ChunkWalk {
  ChunkTiles<kShift> tiles;
  const int32_t *cu, *start;
  int B, T, L_cap, HG;
  int r, least, most;   // rows per unit (log2); sequences of least .. most rows
  int extra;            // tiles that a unit counts for beside its own, ahead of them: what it costs to go to the next one
  int x, end, range;    // of all tiles: the next one, one past the stream's last, tiles of a stream
  int group, my_n, my_s, my_c0, my_w;   // the lanes' sequences group .. group + 31, and their tiles
  int b, n, s, c0, t, units, hg, off;   // the current unit, and its first tile that is this stream's (extra ones first)

  __device__ __forceinline__ int lane() const { return threadIdx.x & 31; }
  __device__ __forceinline__ bool mine() const { return my_n >= least && my_n <= most; }
  struct Bounds {
    int first, end, start;
  };
  __device__ __forceinline__ Bounds fetch(int g) const {   // of sequence g + lane
    const int i = g + lane();
    if (i >= B) return {0, 0, 0};
    return {cu[i], cu[i + 1], start ? start[i] : 0};
  }
  // The lanes' sequences; those that leave [0, T] or the cache have no rows, nor have any from a decrease on.
  __device__ __forceinline__ void settle(int g, const Bounds& q) {
    group = g;
    my_n = my_s = my_c0 = 0;
    const unsigned falls = __ballot_sync(0xffffffffu, q.end < q.first);
    if (!(falls & ((2u << lane()) - 1)) && q.first >= 0 && q.end > q.first && q.end <= T && q.start >= 0 &&
        q.start <= L_cap - (q.end - q.first)) {
      my_n = q.end - q.first;
      my_s = q.start;
      my_c0 = q.first;
    }
  }
  __device__ __forceinline__ void load(int g) { settle(g, fetch(g)); }
  __device__ __forceinline__ void begin(const ChunkArgs& a, int gp_shift) {
    tiles.begin(a.window, a.sinks);
    cu = a.cu;
    start = a.start;
    B = a.B;
    T = a.T;
    L_cap = a.L_cap;
    HG = a.Hq >> gp_shift;
    if (B > 32) {   // B becomes the number of those ahead of the first decrease of the offsets
#pragma unroll 4
      for (int i = lane(); i < a.B; i += 32)
        if (cu[i + 1] < cu[i]) B = min(B, i);
      B = __reduce_min_sync(0xffffffffu, B);
    }
    if (B <= 32) load(0);   // (once for all; more are read again wherever they are looked at)
  }
  __device__ __forceinline__ int units_of(int n_) const { return (int)(((unsigned)n_ + ((1u << r) - 1)) >> r); }
  // all heads' tiles of units number t_ of n_ rows from logical row s_ on
  __device__ __forceinline__ int all_heads(int t_, int s_, int n_) const {
    const int a = t_ << r, e = n_ - a > (1 << r) ? a + (1 << r) : n_;
    return HG * (tiles.count(s_ + a, s_ + e - 1) + extra);
  }
  __device__ __forceinline__ void take(int from) {   // the sequence of a lane
    b = group + from;
    n = __shfl_sync(0xffffffffu, my_n, from);
    s = __shfl_sync(0xffffffffu, my_s, from);
    c0 = __shfl_sync(0xffffffffu, my_c0, from);
    units = units_of(n);
    t = hg = 0;
  }
  // Inclusive sums over the lanes.
  __device__ __forceinline__ int scan(int v) const {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane() >= o) v += u;
    }
    return v;
  }
  // The stream's range of the class's tiles and its first unit; false: it has none. (Little work is cut as thin as
  // one tile: with four at least 333 rows behind 1000 in a window of 201 took 30 us instead of 24.)
  __device__ __forceinline__ bool open(int r_, int least_, int most_, int extra_, int stream, int streams) {
    r = r_;
    least = least_;
    most = most_;
    extra = extra_;
    int all = 0;
    x = end = 0;
    for (int pass = 0;; ++pass) {   // the sum of all; then the sequence with tile x
      int y = x;
      Bounds ahead[3];   // of the next groups: they arrive while one is worked on
#pragma unroll
      for (int k = 0; k < 3; ++k) ahead[k] = B > 32 ? fetch(32 * k) : Bounds{0, 0, 0};
#pragma unroll 1
      for (int g = 0; g < B; g += 32) {
        if (pass == 0 || B > 32) {
          if (B > 32) {
            settle(g, ahead[0]);
            ahead[0] = ahead[1];
            ahead[1] = ahead[2];
            ahead[2] = fetch(g + 96);
          }
          const int m = mine() ? units_of(my_n) : 0;
          my_w = m == 1 ? all_heads(0, my_s, my_n) : 0;
          for (unsigned many = __ballot_sync(0xffffffffu, m > 1); many; many &= many - 1) {
            const int from = __ffs(many) - 1;
            take(from);
            int w = 0;
            for (int i = lane(); i < units; i += 32) w += all_heads(i, s, n);
            w = __reduce_add_sync(0xffffffffu, w);
            if (lane() == from) my_w = w;
          }
        }
        const int sum = __reduce_add_sync(0xffffffffu, my_w);
        if (pass == 0) {
          all += sum;
        } else if (y < sum) {
          const int upto = scan(my_w), from = __ffs(__ballot_sync(0xffffffffu, upto > y)) - 1;
          y -= __shfl_sync(0xffffffffu, upto - my_w, from);
          take(from);
          break;
        } else {
          y -= sum;
        }
      }
      if (pass == 0) {
        range = max(1, (int)(((unsigned)all + (streams - 1)) / (unsigned)streams));
        const int64_t first = (int64_t)stream * range;
        if (first >= all) return false;
        x = (int)first;
        end = min(all, x + min(range, all - x));
        continue;
      }
      for (; units > 1; t += 32) {   // the unit with that tile
        const int w = t + lane() < units ? all_heads(t + lane(), s, n) : 0, upto = scan(w);
        const unsigned past = __ballot_sync(0xffffffffu, upto > y);
        if (past) {
          const int from = __ffs(past) - 1;
          y -= __shfl_sync(0xffffffffu, upto - w, from);
          t += from;
          break;
        }
        y -= __shfl_sync(0xffffffffu, upto, 31);
      }
      const int each = count() + extra;
      hg = y / each;
      off = y - hg * each;
      return true;
    }
  }
  __device__ __forceinline__ int first_row() const { return t << r; }
  __device__ __forceinline__ int end_row() const { return n - first_row() > (1 << r) ? first_row() + (1 << r) : n; }
  __device__ __forceinline__ int count() const { return tiles.count(s + first_row(), s + end_row() - 1); }
  // The current unit's part in this range; false: none (the range ends among what the unit counts for beside). x is
  // then the part's first tile.
  __device__ __forceinline__ bool part(ChunkPart& p) {
    p.all = count();
    const int ahead = max(0, extra - off);
    p.off = max(0, off - extra);
    x += ahead;
    p.x = x;
    p.m = min(p.all - p.off, end - x);
    p.b = b;
    p.s = s;
    p.n = n;
    p.c0 = c0;
    p.row = first_row();
    p.hg = hg;
    return p.m > 0;
  }
  // On to the next unit, behind a part of m tiles; false: the range is at its end.
  __device__ __forceinline__ bool next(int m) {
    x += m;
    off = 0;
    if (x >= end) return false;
    if (++hg < HG) return true;
    hg = 0;
    if (++t < units) return true;
    unsigned left = __ballot_sync(0xffffffffu, mine() && group + lane() > b);
    while (!left && group + 32 < B) {
      load(group + 32);
      left = __ballot_sync(0xffffffffu, mine());
    }
    if (!left) return false;   // (there is one)
    take(__ffs(left) - 1);
    return true;
  }
};

size_t chunk_workspace(const medusa_cfg& c, int T);
bool chunk_countable(const medusa_cfg& c, int T);   // key tiles of any lengths stay within 32 bits
ChunkSpace chunk_space(const medusa_cfg& c, int T);
cudaError_t launch_chunk_f32(const medusa_cfg& c, const void* Q, const void* Kp, const void* Vp, void* O, const ChunkArgs& a,
                             const ChunkSpace& sp, void* ws, cudaStream_t st);
cudaError_t launch_chunk_tc(const medusa_cfg& c, const void* Q, const void* Kp, const void* Vp, void* O, const ChunkArgs& a,
                            const ChunkSpace& sp, void* ws, cudaStream_t st);
cudaError_t launch_chunk_attention(const medusa_cfg& c, const void* Q, const void* Kp, const void* Vp, void* O, const ChunkArgs& a,
                                   void* ws, cudaStream_t st);

}  // namespace medusa
