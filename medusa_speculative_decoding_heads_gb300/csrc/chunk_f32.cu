// Attention of new tokens over the pages of a cache in float32 on the CUDA cores, with the running maximum
// and sum of "최적화 2편" (beengineer500), section 3.3; everything float32. One CTA per SM takes its ranges
// of the work (chunk.cuh):
//   sequences of two rows and more   64 rows (query heads of a KV head times positions) against tiles of 64
//                                    keys, as whole prompts are (prompt_f32.cu): bound by the multiply-adds
//   single tokens                    up to 4 query heads of a KV head; a warp (D = 64: half of one) reads a key's
//                                    row at a time, 4 of them on their way while 4 are worked on, and the
//                                    warps join at the end of the unit: bound by the K/V bytes
// 1500 rows of a prompt, 8 heads of 64: 87 us (whole prompts: 77); 8 single tokens of 2000 rows, 40 heads of 128:
// 148 us (4.4 TB/s); 24 of 4000 rows, 32/8 heads: 222 us (3.5 TB/s: four rows' sums over 32 lanes).
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "chunk.cuh"
#include "common.cuh"
#include "f32_tiles.cuh"

namespace medusa {
namespace {

using namespace f32;

constexpr int kSms = 152;
// What a unit counts for beside its key tiles.
constexpr int kTileExtra = 1, kTokenExtra = 2;

struct Work {
  int kind;            // 0: none is left, 1: 64 rows, 2: a single token
  int pos0, left;      // first packed row, positions from it on
  int h0, kvh, b;
  int s, end, p0;      // the sequence's logical rows [s, end); logical row of the first position
  int off, m, skip;    // key tiles [off, off + m) of the unit, what they skip behind the first rows
  int part;            // first row of the partial result, or -1
};

// What the kernel keeps: where page b, key lies.
struct Cache {
  const ChunkArgs& a;
  const float *K, *V;
  int D;
  // offset of the rows that a tile's keys from key0 on have, or -1 (a page outside the pool: zeros)
  __device__ __forceinline__ int64_t at(const Work& w, int page, int key0) const {
    return page >= 0 && page < a.num_pages ? (((int64_t)page * a.Hkv + w.kvh) * a.page_rows + key0 % a.page_rows) * D : -1;
  }
  __device__ __forceinline__ int page(const Work& w, int key0) const { return a.table[(size_t)w.b * a.max_pages + key0 / a.page_rows]; }
};

// 64 rows.
template <int D>
__device__ __forceinline__ void tile_unit(float* smem, const float* __restrict__ Q, const Cache& c, const ChunkTiles<6>& tiles,
                                          const ChunkSpace& sp, const Work& w, float* __restrict__ O, float* __restrict__ o_part,
                                          float* __restrict__ ml_part) {
  using S = Smem<D>;
  constexpr int CH = D / 4;
  const ChunkArgs& a = c.a;
  Rows<D> t;
  t.begin(smem);
  const int log_npos = 31 - __clz(sp.npos);
  auto head_of = [&](int r) { return r >> log_npos; };
  auto pos_of = [&](int r) { return r & (sp.npos - 1); };
  for (int e = threadIdx.x; e < kTileRows * CH; e += S::threads) {
    const int r = e / CH, x = e % CH;
    const bool ok = pos_of(r) < w.left;
    cp16(t.sq + r * S::ld + 4 * x, Q + (w.pos0 + (int64_t)(ok ? pos_of(r) : 0)) * a.q_stride + (int64_t)(w.h0 + head_of(r)) * D + 4 * x, ok);
  }
  // a tile of 64 rows of the cache; those that no row of the sequence sees become zeros
  auto load = [&](float* dst, int ld, const float* pool, int j) {
    const int key0 = tiles.tile(w.off + j, w.skip) * kTileKeys, page = c.page(w, key0);
    const int64_t at = c.at(w, page, key0);
    MEDUSA_CHECK(t.tid != 0 || at >= 0, MEDUSA_CHECK_PAGE);
    for (int e = t.tid; e < kTileKeys * CH; e += kGroup) {
      const int r = e / CH, x = e % CH, key = key0 + r;
      const bool ok = at >= 0 && key < w.end && (key > w.s - a.window || key < a.sinks);
      cp16(dst + r * ld + 4 * x, pool + (ok ? at + r * D : 0) + 4 * x, ok);
    }
  };
  if (t.group < w.m) load(t.sk, S::ld, c.K, t.group);
  cp_commit();
  cp_wait<0>();
  __syncthreads();       // Q
  for (int j = t.group; j < w.m; j += S::groups) {
    cp_wait<0>();        // K_j
    t.sync_group();      // ... of every thread; V and P of the tile before are no longer read
    load(t.sv, D, c.V, j);
    cp_commit();
    float2 s[4][8];
    t.scores(s);
    t.sync_group();      // K_j is no longer read
    if (j + S::groups < w.m) load(t.sk, S::ld, c.K, j + S::groups);
    cp_commit();
    const int key0 = tiles.tile(w.off + j, w.skip) * kTileKeys;
    t.weights(s, a.scale_log2, [&](int i) {
      const int p = w.p0 + pos_of(t.rg + 4 * i), high = p - key0, low = max(0, p - a.window + 1) - key0, first = a.sinks - key0;
      return [=](int key) { return key <= high && (key >= low || key < first); };
    });
    cp_wait<1>();        // V_j
    t.sync_group();      // ... and P_j
    t.values();
  }
  if (!t.join(smem)) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = t.rg + 4 * i;
    if (pos_of(r) >= w.left) continue;
    const float inv = w.part < 0 ? 1.f / t.l[i] : 1.f;
    float* op = w.part < 0 ? O + ((size_t)(w.pos0 + pos_of(r)) * a.Hq + w.h0 + head_of(r)) * D : o_part + (size_t)(w.part + r) * D;
#pragma unroll
    for (int n = 0; n < Rows<D>::NC; ++n)
      *reinterpret_cast<float4*>(op + 4 * t.cg + 32 * n) = make_float4(t.o[i][n].x * inv, t.o[i][n].y * inv, t.o[i][n].z * inv, t.o[i][n].w * inv);
    if (w.part >= 0 && t.cg == 0) *reinterpret_cast<float2*>(ml_part + 2 * (size_t)(w.part + r)) = make_float2(t.m[i], t.l[i]);
  }
}

// A single token's R query heads of a KV head.
template <int D, int R>
__device__ __forceinline__ void token_unit(float* smem, const float* __restrict__ Q, const Cache& c, const ChunkTiles<6>& tiles,
                                           const Work& w, float* __restrict__ O, float* __restrict__ o_part, float* __restrict__ ml_part) {
  constexpr int kLanes = D / 4, kWide = 32 / kLanes, X = 4, kStep = X * kWide;   // lanes of a key, keys a warp reads at once, its step
  constexpr int kWarps = Smem<D>::threads / 32, kStreams = kWarps * kWide, kPer = kTileKeys / kStep;
  const ChunkArgs& a = c.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane % kLanes, stream = warp * kWide + lane / kLanes;
  const int p = w.p0, low = max(0, p - a.window + 1), steps = w.m * kPer;
  auto key_of = [&](int q) { return tiles.tile(w.off + q / kPer, w.skip) * kTileKeys + q % kPer * kStep; };   // of a step
  float4 q[R], o[R], k[X], v[X];
  float m[R], l[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    q[r] = *reinterpret_cast<const float4*>(Q + w.pos0 * a.q_stride + (int64_t)(w.h0 + r) * D + 4 * sub);
    q[r] = make_float4(q[r].x * a.scale_log2, q[r].y * a.scale_log2, q[r].z * a.scale_log2, q[r].w * a.scale_log2);
    o[r] = make_float4(0.f, 0.f, 0.f, 0.f);
    m[r] = -INFINITY;
    l[r] = 0.f;
  }
  auto seen = [&](int key) { return key <= p && (key >= low || key < a.sinks); };
  auto fetch = [&](int at_step, int page) {
    const int key0 = key_of(at_step);
    const int64_t at = c.at(w, page, key0);
    MEDUSA_CHECK(lane != 0 || at >= 0, MEDUSA_CHECK_PAGE);
#pragma unroll
    for (int x = 0; x < X; ++x) {
      const int i = lane / kLanes * X + x;
      const bool ok = at >= 0 && seen(key0 + i);
      k[x] = ok ? __ldg(reinterpret_cast<const float4*>(c.K + at + i * D + 4 * sub)) : make_float4(0.f, 0.f, 0.f, 0.f);
      v[x] = ok ? __ldg(reinterpret_cast<const float4*>(c.V + at + i * D + 4 * sub)) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  };
  // (every lane of a warp takes every step: the sums are collective)
  int page = warp < steps ? c.page(w, key_of(warp)) : -1;
  if (warp < steps) fetch(warp, page);
  page = warp + kWarps < steps ? c.page(w, key_of(warp + kWarps)) : -1;
  for (int at = warp; at < steps; at += kWarps) {
    float4 kk[X], vv[X];
#pragma unroll
    for (int x = 0; x < X; ++x) {
      kk[x] = k[x];
      vv[x] = v[x];
    }
    const int key0 = key_of(at) + lane / kLanes * X;
    if (at + kWarps < steps) fetch(at + kWarps, page);
    if (at + 2 * kWarps < steps) page = c.page(w, key_of(at + 2 * kWarps));
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float s[X], mn = m[r];
#pragma unroll
      for (int x = 0; x < X; ++x) {
        s[x] = q[r].x * kk[x].x;
        s[x] = fmaf(q[r].y, kk[x].y, s[x]);
        s[x] = fmaf(q[r].z, kk[x].z, s[x]);
        s[x] = fmaf(q[r].w, kk[x].w, s[x]);
      }
#pragma unroll
      for (int d = kLanes / 2; d > 0; d >>= 1)
#pragma unroll
        for (int x = 0; x < X; ++x) s[x] += __shfl_xor_sync(0xffffffffu, s[x], d);
#pragma unroll
      for (int x = 0; x < X; ++x) {
        if (!seen(key0 + x)) s[x] = -INFINITY;
        mn = fmaxf(mn, s[x]);
      }
      const float mu = mn == -INFINITY ? 0.f : mn, corr = exp2f(m[r] - mu);
      m[r] = mn;
      l[r] *= corr;
      o[r] = make_float4(o[r].x * corr, o[r].y * corr, o[r].z * corr, o[r].w * corr);
#pragma unroll
      for (int x = 0; x < X; ++x) {
        const float e = exp2f(s[x] - mu);
        l[r] += e;
        o[r] = make_float4(fmaf(e, vv[x].x, o[r].x), fmaf(e, vv[x].y, o[r].y), fmaf(e, vv[x].z, o[r].z), fmaf(e, vv[x].w, o[r].w));
      }
    }
  }
  // [stream][R] results, then their maxima and sums; a warp joins a row
  float* sml = smem + kStreams * R * D;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    *reinterpret_cast<float4*>(smem + (stream * R + r) * D + 4 * sub) = o[r];
    if (sub == 0) *reinterpret_cast<float2*>(sml + 2 * (stream * R + r)) = make_float2(m[r], l[r]);
  }
  __syncthreads();
  if (warp >= R) return;
  constexpr int N = D / 32;
  using V = std::conditional_t<N == 4, float4, float2>;
  float M = -INFINITY, sum = 0.f, acc[N] = {};
  for (int i = 0; i < kStreams; ++i) {
    const float2 ml = *reinterpret_cast<const float2*>(sml + 2 * (i * R + warp));
    if (ml.x == -INFINITY && ml.y == 0.f) continue;
    const V part = *reinterpret_cast<const V*>(smem + (i * R + warp) * D + N * lane);
    const float mn = fmaxf(M, ml.x), mu = mn == -INFINITY ? 0.f : mn, w0 = exp2f(M - mu), w1 = exp2f(ml.x - mu);
    M = mn;
    sum = sum * w0 + ml.y * w1;
#pragma unroll
    for (int x = 0; x < N; ++x) acc[x] = acc[x] * w0 + reinterpret_cast<const float*>(&part)[x] * w1;
  }
  const float inv = w.part < 0 ? 1.f / sum : 1.f;   // (0 where every visible score is -inf: no number)
  V out;
#pragma unroll
  for (int x = 0; x < N; ++x) reinterpret_cast<float*>(&out)[x] = acc[x] * inv;
  float* op = w.part < 0 ? O + ((size_t)w.pos0 * a.Hq + w.h0 + warp) * D : o_part + (size_t)(w.part + warp) * D;
  *reinterpret_cast<V*>(op + N * lane) = out;
  if (w.part >= 0 && lane == 0) *reinterpret_cast<float2*>(ml_part + 2 * (size_t)(w.part + warp)) = make_float2(M, sum);
}

// Warp 0 finds the next unit: `work` becomes it. kind: what was worked on last (0: nothing yet, 1: 64 rows, 2: single
// tokens). A function of its own, as what it keeps in registers is not for the others to go without (in line: 24 single
// tokens of 2000 rows, 8/4 heads of 64, 43 us, so 38; 8 of 2000 rows, 40 heads of 128, 167 and 148).
template <int R>
__device__ __noinline__ void find_work(const ChunkArgs& a, const ChunkSpace& sp, ChunkWalk<6>& place, Work& work, ChunkCut* cuts, int kind) {
  const int lane = threadIdx.x & 31;
  ChunkWalk<6> walk;
  bool open = kind == 0;
  if (open) {
    walk.begin(a, 0);
    kind = sp.pair_streams ? 0 : 1;
  } else {
    walk = place;
  }
  ChunkPart part;
  part.m = 0;
  while (kind < 3) {
    bool more;
    if (open) {
      ++kind;
      if (kind == 3) break;
      if (lane == 0) cuts[(kind == 1 ? 0 : sp.pair_streams) + blockIdx.x] = ChunkCut{0, 0, 0, 0};
      if (walk.B <= 32) walk.load(0);
      walk.HG = kind == 1 ? a.Hq >> sp.gp_shift : a.Hq / R;
      more = walk.open(kind == 1 ? 31 - __clz(sp.npos) : 0, kind == 1 ? 2 : 1, kind == 1 ? INT32_MAX : 1,
                       kind == 1 ? kTileExtra : kTokenExtra, (int)blockIdx.x, kSms);
    } else {   // behind the unit that has just been worked on
      if (walk.hg + 1 >= walk.HG && walk.t + 1 >= walk.units) walk.load(walk.group);   // (what the lanes hold is not kept)
      more = walk.next(work.m);
    }
    open = !(more && walk.part(part));
    if (!open) break;
  }
  __syncwarp();
  if (lane != 0) return;
  place = walk;
  work.kind = kind == 3 ? 0 : kind;
  if (kind == 3) return;
  const int at = (int)blockIdx.x, second = part.off == 0;
  work.pos0 = part.c0 + part.row;
  work.left = part.n - part.row;
  work.h0 = kind == 1 ? part.hg << sp.gp_shift : part.hg * R;
  work.kvh = work.h0 / (a.Hq / a.Hkv);
  work.b = part.b;
  work.s = part.s;
  work.end = part.s + part.n;
  work.p0 = part.s + part.row;
  work.off = part.off;
  work.m = part.m;
  work.skip = walk.tiles.skip(work.p0);
  work.part = !part.cut() ? -1 : (int)(kind == 1 ? sp.pair_part(at, second) : sp.single_part(at, second));
  if (part.cut() && second)
    cuts[(kind == 1 ? 0 : sp.pair_streams) + at] = ChunkCut{work.pos0, work.left, work.h0, (part.x + part.all - 1) / walk.range - at};
}

template <int D, int R>
__global__ void __launch_bounds__(Smem<D>::threads, 1)
chunk_f32_kernel(const float* __restrict__ Q, const float* __restrict__ Kp, const float* __restrict__ Vp, float* __restrict__ O,
                 const __grid_constant__ ChunkArgs a, const __grid_constant__ ChunkSpace sp, float* __restrict__ o_part,
                 float* __restrict__ ml_part, ChunkCut* cuts) {
  extern __shared__ __align__(16) float smem[];
  __shared__ Work work;
  __shared__ ChunkWalk<6> place;
  pdl_trigger();   // (one CTA per SM, as many as there are, leaves nothing to crowd)
  pdl_wait();
  ChunkTiles<6> tiles;
  tiles.begin(a.window, a.sinks);
  const Cache cache{a, Kp, Vp, D};
  for (int kind = 0;;) {
    if (threadIdx.x < 32) find_work<R>(a, sp, place, work, cuts, kind);
    __syncthreads();
    kind = work.kind;
    if (kind == 0) return;
    if (kind == 1) tile_unit<D>(smem, Q, cache, tiles, sp, work, O, o_part, ml_part);
    else token_unit<D, R>(smem, Q, cache, tiles, work, O, o_part, ml_part);
    __syncthreads();   // the next unit goes where this one was
  }
}

template <int D, int R>
cudaError_t run(const float* Q, const float* Kp, const float* Vp, float* O, const ChunkArgs& a, const ChunkSpace& sp, char* ws, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(chunk_f32_kernel<D, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::bytes);
  if (e != cudaSuccess) return e;
  e = launch_pdl(chunk_f32_kernel<D, R>, kSms, Smem<D>::threads, Smem<D>::bytes, st, Q, Kp, Vp, O, a, sp,
                 reinterpret_cast<float*>(ws), reinterpret_cast<float*>(ws + sp.ml), reinterpret_cast<ChunkCut*>(ws + sp.cuts));
  note_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

MEDUSA_CHECK_TAKE(chunk_take_checks)

cudaError_t launch_chunk_f32(const medusa_cfg& c, const void* Q, const void* Kp, const void* Vp, void* O, const ChunkArgs& a,
                             const ChunkSpace& sp, void* ws, cudaStream_t st) {
  static_assert(kSms == kChunkStreams, "a stream per CTA");
  const auto kernel = c.D == 64 ? (sp.single_rows == 1 ? run<64, 1> : sp.single_rows == 2 ? run<64, 2> : run<64, 4>)
                                : (sp.single_rows == 1 ? run<128, 1> : sp.single_rows == 2 ? run<128, 2> : run<128, 4>);
  return kernel(static_cast<const float*>(Q), static_cast<const float*>(Kp), static_cast<const float*>(Vp), static_cast<float*>(O), a, sp,
                static_cast<char*>(ws), st);
}

}  // namespace medusa
