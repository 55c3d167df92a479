// Attention of new tokens over the pages of a cache: what its kernels share.
//
// Work. A unit is a block of query rows (the query heads of one KV head that share a tile, times
// positions) of one sequence; it takes the key tiles that any of its rows sees, the first rows' ones
// ahead of the window's. All units' tiles, one after another, are cut into equal ranges, one for each
// stream (a CTA, or one of a CTA's two tiles of rows), wherever the cuts fall: lengths differ from
// sequence to sequence and are on the device only, and so are the cuts. A unit that is cut leaves partial
// results, at most two per stream (of the unit that was begun ahead of its range, and of the one that
// ends behind it), which chunk_merge_kernel joins. Where a unit lies among the tiles is known in closed
// form: rows per unit and keys per tile are powers of two.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/medusa.h"

namespace medusa {

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
// sequences with more than npos rows; `singles`, one tile, of the others. (float32: one class.)
struct ChunkSpace {
  int gp_shift, npos;          // query heads of a tile (log2), positions of a tile
  int pair_streams, pair_rows; // streams, and rows of one partial result
  int streams, single_rows, single_npos;   // the same of single tiles, and their positions
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
  __device__ __forceinline__ void begin(const ChunkArgs& a) {
    window = a.window;
    sink_tiles = (int)(((unsigned)a.sinks + ((1u << kShift) - 1)) >> kShift);
  }
  // key tiles between the first rows and the window of row p, which nothing of a unit that begins with p sees
  __device__ __forceinline__ int skip(int p) const { return max(0, (max(0, p - window + 1) >> kShift) - sink_tiles); }
  // tiles of a unit of the logical rows p0 .. p1
  __device__ __forceinline__ int count(int p0, int p1) const { return (p1 >> kShift) + 1 - skip(p0); }
  // key tile that is number j of a unit
  __device__ __forceinline__ int tile(int j, int skipped) const { return j < sink_tiles ? j : j + skipped; }

  // sum over t < m of floor((a + t 2^r) / 2^kShift), a >= 0
  static __device__ __forceinline__ int64_t floors(int64_t m, int64_t a, int r) {
    if (r >= kShift) return m * (a >> kShift) + ((m * (m - 1) / 2) << (r - kShift));
    const int q = kShift - r;
    auto upto = [&](int64_t k) {   // sum over i < k of floor(i / 2^q)
      const int64_t j = k >> q;
      return ((j * (j - 1) / 2) << q) + (k - (j << q)) * j;
    };
    return upto((a >> r) + m) - upto(a >> r);
  }
  // tiles of the first m of a sequence's units of 2^r rows (n rows from logical row s on)
  __device__ __forceinline__ int64_t upto(int m, int s, int n, int r) const {
    const int64_t R = (int64_t)1 << r;
    int64_t sum = floors(m, s + R - 1, r) + m;
    const int64_t over = s + m * R;   // one past the last of those units' rows, if it is whole
    if (over > (int64_t)s + n) sum += ((s + n - 1) >> kShift) - ((over - 1) >> kShift);
    const int64_t a = (int64_t)s - window + 1 - ((int64_t)sink_tiles << kShift);
    const int64_t t = a >= 0 ? 0 : (-a + R - 1) >> r;   // the first unit that skips any
    if (t < m) sum -= floors(m - t, a + t * R, r);
    return sum;
  }
};

// Finds and follows units of one class; a whole warp calls every function.
template <int kShift>
struct ChunkWalk {
  ChunkTiles<kShift> tiles;
  const int32_t *cu, *start;
  int B, T, L_cap, HG;
  int r, least, most;   // rows per unit (log2); sequences of least .. most rows
  // the lanes' sequences, group .. group + 31
  int group, my_n, my_s, my_c0;
  // the current unit
  int b, n, s, c0, t, units, hg;

  __device__ __forceinline__ int lane() const { return threadIdx.x & 31; }
  // Sequences from the first decrease of the offsets on have no rows; those that leave [0, T] or the cache neither.
  __device__ __forceinline__ void load(int g, int& n_, int& s_, int& c0_) const {
    const int i = g + lane();
    n_ = s_ = c0_ = 0;
    if (i >= B) return;
    const int a = cu[i], e = cu[i + 1], f = start ? start[i] : 0;
    if (a < 0 || e <= a || e > T || f < 0 || f > L_cap - (e - a)) return;
    n_ = e - a;
    s_ = f;
    c0_ = a;
  }
  __device__ __forceinline__ bool in_class(int rows) const { return rows >= least && rows <= most; }
  __device__ __forceinline__ int64_t work(int n_, int s_) const {
    return in_class(n_) ? HG * tiles.upto((int)(((int64_t)n_ + (1 << r) - 1) >> r), s_, n_, r) : 0;
  }
  static __device__ __forceinline__ int64_t sum(int64_t v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }
  __device__ __forceinline__ void begin(const ChunkArgs& a, int gp_shift) {
    tiles.begin(a);
    cu = a.cu;
    start = a.start;
    B = a.B;
    T = a.T;
    L_cap = a.L_cap;
    HG = a.Hq >> gp_shift;
    // (B ends ahead of the first decrease)
    for (int g = 0; g < B; g += 32) {
      const int i = g + lane();
      const unsigned falls = __ballot_sync(0xffffffffu, i < B && cu[i + 1] < cu[i]);
      if (falls) B = g + __ffs(falls) - 1;
    }
    group = 0;
    load(0, my_n, my_s, my_c0);
  }
  __device__ __forceinline__ void choose(int r_, int least_, int most_) {
    r = r_;
    least = least_;
    most = most_;
  }
  // Tiles of all units of the class.
  __device__ int64_t total() {
    int64_t w = 0;
    if (B <= 32) return sum(work(my_n, my_s));
#pragma unroll 2
    for (int g = 0; g < B; g += 32) {
      int n_, s_, c_;
      load(g, n_, s_, c_);
      w += work(n_, s_);
    }
    return sum(w);
  }
  __device__ __forceinline__ void take(int from) {   // the sequence of a lane
    b = group + from;
    n = __shfl_sync(0xffffffffu, my_n, from);
    s = __shfl_sync(0xffffffffu, my_s, from);
    c0 = __shfl_sync(0xffffffffu, my_c0, from);
    units = (int)(((int64_t)n + (1 << r) - 1) >> r);
    t = hg = 0;
  }
  // The unit with tile x of all (x < total()); returns which of its tiles that is.
  __device__ int seek(int64_t x) {
    for (group = 0;; group += 32) {
      if (B > 32) load(group, my_n, my_s, my_c0);
      const int64_t w = work(my_n, my_s);
      int64_t upto = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane() >= o) upto += v;
      }
      const int64_t all = __shfl_sync(0xffffffffu, upto, 31);
      if (x >= all && group + 32 < B) {
        x -= all;
        continue;
      }
      const unsigned past = __ballot_sync(0xffffffffu, upto > x);
      const int from = past ? __ffs(past) - 1 : 31;   // (x < total(): there is one)
      x -= __shfl_sync(0xffffffffu, upto - w, from);
      take(from);
      break;
    }
    int lo = 0, hi = units;   // unit lo begins at or ahead of x, unit hi behind it
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) >> 5, at = lo + (lane() + 1) * step;
      const bool ahead = at < hi && HG * tiles.upto(at, s, n, r) <= x;
      lo += __popc(__ballot_sync(0xffffffffu, ahead)) * step;
      hi = min(hi, lo + step);
    }
    t = lo;
    x -= HG * tiles.upto(t, s, n, r);
    const int each = count();
    hg = (int)(x / each);
    return (int)(x - (int64_t)hg * each);
  }
  __device__ __forceinline__ int first_row() const { return t << r; }
  __device__ __forceinline__ int last_row() const { return (int)min((int64_t)n, ((int64_t)t + 1) << r) - 1; }
  __device__ __forceinline__ int count() const { return tiles.count(s + first_row(), s + last_row()); }
  // The next unit (there is one).
  __device__ void next() {
    if (++hg < HG) return;
    hg = 0;
    if (++t < units) return;
    unsigned left = __ballot_sync(0xffffffffu, in_class(my_n) && group + lane() > b);
    while (!left && group + 32 < B) {
      group += 32;
      load(group, my_n, my_s, my_c0);
      left = __ballot_sync(0xffffffffu, in_class(my_n));
    }
    if (left) take(__ffs(left) - 1);
  }
};

size_t chunk_workspace(const medusa_cfg& c, int T);
ChunkSpace chunk_space(const medusa_cfg& c, int T);
cudaError_t launch_chunk_tc(const medusa_cfg& c, const void* Q, const void* Kp, const void* Vp, void* O, const ChunkArgs& a,
                            const ChunkSpace& sp, void* ws, cudaStream_t st);
cudaError_t launch_chunk_attention(const medusa_cfg& c, const void* Q, const void* Kp, const void* Vp, void* O, const ChunkArgs& a,
                                   void* ws, cudaStream_t st);

}  // namespace medusa
