// Attention of new tokens over the pages of a cache: a warp per query row, one pass over the keys
// that the row sees, with the running maximum and sum of "최적화 2편" (beengineer500), section 3.3.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "chunk.cuh"
#include "common.cuh"

namespace medusa {
namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t* p, float v) {   // (v may be no number)
  asm("{ .reg .b16 h; cvt.rn.bf16.f32 h, %1; mov.b16 %0, h; }" : "=h"(*p) : "f"(v));
}

template <typename T, int D>
__global__ void __launch_bounds__(32 * kWarps)
chunk_rows_kernel(const T* __restrict__ Q, const T* __restrict__ Kp, const T* __restrict__ Vp, T* __restrict__ O,
                  const ChunkArgs a) {
  constexpr int X = D / 32;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  for (int b = 0; b < a.B; ++b) {
    const int c0 = a.cu[b], c1 = a.cu[b + 1];
    if (c1 < c0) return;
    const int s = a.start ? a.start[b] : 0;
    if (c0 < 0 || c1 > a.T || s < 0 || s > a.L_cap - (c1 - c0)) continue;
    const int64_t rows = (int64_t)(c1 - c0) * a.Hq;
    for (int64_t r = blockIdx.x * kWarps + (threadIdx.x >> 5); r < rows; r += (int64_t)gridDim.x * kWarps) {
      const int i = (int)(r / a.Hq), h = (int)(r % a.Hq), p = s + i, kvh = h / (a.Hq / a.Hkv);
      float q[X], o[X], m = -INFINITY, l = 0.f;
#pragma unroll
      for (int x = 0; x < X; ++x) {
        q[x] = Elt<T>::load(Q, (c0 + i) * a.q_stride + (int64_t)h * D + lane + 32 * x);
        o[x] = 0.f;
      }
      const int low = max(0, p - a.window + 1);
      for (int j = min(a.sinks, low) > 0 ? 0 : low; j <= p; ++j) {
        if (j >= a.sinks && j < low) j = low;
        const int page = a.table[(size_t)b * a.max_pages + j / a.page_rows];
        const bool in_pool = page >= 0 && page < a.num_pages;
        MEDUSA_CHECK(in_pool, MEDUSA_CHECK_PAGE);
        const size_t at = (((size_t)(in_pool ? page : 0) * a.Hkv + kvh) * a.page_rows + j % a.page_rows) * D + lane;
        float t = 0.f;
#pragma unroll
        for (int x = 0; x < X; ++x) t = fmaf(q[x], in_pool ? Elt<T>::load(Kp, at + 32 * x) : 0.f, t);
        t = warp_sum(t) * a.scale_log2;
        const float mn = fmaxf(m, t), mu = mn == -INFINITY ? 0.f : mn, corr = exp2f(m - mu), w = exp2f(t - mu);
        m = mn;
        l = l * corr + w;
#pragma unroll
        for (int x = 0; x < X; ++x) o[x] = fmaf(w, in_pool ? Elt<T>::load(Vp, at + 32 * x) : 0.f, o[x] * corr);
      }
#pragma unroll
      for (int x = 0; x < X; ++x) put(O + ((size_t)(c0 + i) * a.Hq + h) * D + lane + 32 * x, o[x] / l);
    }
  }
}

template <typename T, int D>
cudaError_t run(const void* Q, const void* Kp, const void* Vp, void* O, const ChunkArgs& a, cudaStream_t st) {
  const cudaError_t e = launch_pdl(chunk_rows_kernel<T, D>, 152 * 8, 32 * kWarps, 0, st, static_cast<const T*>(Q),
                                   static_cast<const T*>(Kp), static_cast<const T*>(Vp), static_cast<T*>(O), a);
  note_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// Joins the partial results of the units that were cut: O = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s, a warp
// per row, several parts on their way at a time. Bound by the partial results' bytes, which lie in L2.
constexpr int kMergeThreads = 256, kMergeRows = kMergeThreads / 32, kMergeParts = 4;

template <int X>
struct Vec;
template <>
struct Vec<2> { using type = float2; };
template <>
struct Vec<4> { using type = float4; };

template <typename T, int D>
__global__ void __launch_bounds__(kMergeThreads)
chunk_merge_kernel(const float* __restrict__ o_part, const float* __restrict__ ml_part, const ChunkCut* __restrict__ cuts,
                   const ChunkSpace sp, int Hq, T* __restrict__ O) {
  constexpr int X = D / 32;
  using V = typename Vec<X>::type;
  pdl_wait();
  pdl_trigger();
  // blocks: kMergeRows rows of each stream of pairs, then of single tiles
  const int per_pair = sp.pair_rows / kMergeRows, per_single = (sp.single_rows + kMergeRows - 1) / kMergeRows;
  const bool pair = (int)blockIdx.x < sp.pair_streams * per_pair;
  const int y = pair ? (int)blockIdx.x : (int)blockIdx.x - sp.pair_streams * per_pair;
  const int stream = y / (pair ? per_pair : per_single), lane = threadIdx.x & 31;
  const int r = (y - stream * (pair ? per_pair : per_single)) * kMergeRows + (threadIdx.x >> 5);
  const ChunkCut cut = cuts[(pair ? 0 : sp.pair_streams) + stream];
  if (cut.parts == 0 || r >= (pair ? sp.pair_rows : sp.single_rows)) return;
  const int along = pair ? sp.npos : sp.single_npos, tile_rows = along << sp.gp_shift;   // rows of a tile: [head][position]
  const int tile = r / tile_rows, head = (r - tile * tile_rows) / along, pos = r - tile * tile_rows - head * along + tile * along;
  if (pos >= cut.left) return;
  float M = -INFINITY, sum = 0.f, acc[X] = {};
  for (int s0 = 0; s0 <= cut.parts; s0 += kMergeParts) {
    float2 ml[kMergeParts];
    V v[kMergeParts];
#pragma unroll
    for (int i = 0; i < kMergeParts; ++i) {
      const int s = min(s0 + i, cut.parts);
      const int64_t at = (pair ? sp.pair_part(stream + s, s == 0) : sp.single_part(stream + s, s == 0)) + r;
      ml[i] = *reinterpret_cast<const float2*>(ml_part + 2 * at);
      v[i] = *reinterpret_cast<const V*>(o_part + at * D + X * lane);
    }
#pragma unroll
    for (int i = 0; i < kMergeParts; ++i) {
      // (where nothing was visible its O need not have been written)
      if (s0 + i > cut.parts || (ml[i].x == -INFINITY && ml[i].y == 0.f)) continue;
      const float* o = reinterpret_cast<const float*>(&v[i]);
      const float mn = fmaxf(M, ml[i].x), mu = mn == -INFINITY ? 0.f : mn, w0 = exp2f(M - mu), w1 = exp2f(ml[i].x - mu);
      M = mn;
      sum = sum * w0 + ml[i].y * w1;
#pragma unroll
      for (int x = 0; x < X; ++x) acc[x] = acc[x] * w0 + o[x] * w1;
    }
  }
  const float inv = 1.f / sum;   // (0 where every visible score is -inf: no number)
  T* op = O + ((size_t)(cut.pos0 + pos) * Hq + cut.h0 + head) * D + X * lane;
  if constexpr (sizeof(T) == 4) {
    V v;
#pragma unroll
    for (int x = 0; x < X; ++x) reinterpret_cast<float*>(&v)[x] = acc[x] * inv;
    *reinterpret_cast<V*>(op) = v;
  } else {
#pragma unroll
    for (int x = 0; x < X; x += 2) {
      uint32_t w;
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(acc[x + 1] * inv), "f"(acc[x] * inv));
      reinterpret_cast<uint32_t*>(op)[x / 2] = w;
    }
  }
}

template <typename T, int D>
cudaError_t merge(const medusa_cfg& c, void* O, const ChunkSpace& sp, void* ws, cudaStream_t st) {
  const int blocks = sp.pair_streams * (sp.pair_rows / kMergeRows) + sp.streams * ((sp.single_rows + kMergeRows - 1) / kMergeRows);
  const char* base = static_cast<const char*>(ws);
  const cudaError_t e = launch_pdl(chunk_merge_kernel<T, D>, blocks, kMergeThreads, 0, st, reinterpret_cast<const float*>(base),
                                   reinterpret_cast<const float*>(base + sp.ml), reinterpret_cast<const ChunkCut*>(base + sp.cuts), sp,
                                   c.Hq, static_cast<T*>(O));
  note_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

MEDUSA_CHECK_TAKE(chunk_take_checks)

ChunkSpace chunk_space(const medusa_cfg& c, int T) {
  constexpr int kSms = 152, kRows = 128;
  ChunkSpace sp{};
  const int G = c.Hq / c.Hkv;
  while (sp.gp_shift < 4 && G % (2 << sp.gp_shift) == 0) ++sp.gp_shift;   // the largest power of two that divides the group
  sp.npos = kRows >> sp.gp_shift;
  sp.pair_streams = T > sp.npos ? kSms : 0;   // (no sequence has more rows than there are)
  sp.pair_rows = 2 * kRows;
  sp.streams = kSms;
  sp.single_npos = T < sp.npos ? T : sp.npos;
  sp.single_rows = sp.single_npos << sp.gp_shift;
  const size_t rows = (size_t)2 * sp.pair_streams * sp.pair_rows + (size_t)2 * sp.streams * sp.single_rows;
  sp.ml = align_up(rows * c.D * 4, 256);
  sp.cuts = sp.ml + align_up(rows * 8, 256);
  sp.total = sp.cuts + align_up((sp.pair_streams + sp.streams) * sizeof(ChunkCut), 256);
  return sp;
}

bool chunk_countable(const medusa_cfg& c, int T) {
  const ChunkSpace sp = chunk_space(c, T);
  const double units = ((double)T / sp.npos + c.B) * (c.Hq >> sp.gp_shift);
  return units * (c.L_cap / 128 + 4.0) < 2147483647.0;   // (4: the tile that is begun, what a unit counts for beside)
}

size_t chunk_workspace(const medusa_cfg& c, int T) { return c.dtype == MEDUSA_F32 ? 0 : chunk_space(c, T).total; }

cudaError_t launch_chunk_attention(const medusa_cfg& c, const void* Q, const void* Kp, const void* Vp, void* O, const ChunkArgs& a,
                                   void* ws, cudaStream_t st) {
  if (c.dtype == MEDUSA_F32) return c.D == 64 ? run<float, 64>(Q, Kp, Vp, O, a, st) : run<float, 128>(Q, Kp, Vp, O, a, st);
  const ChunkSpace sp = chunk_space(c, a.T);
  const cudaError_t e = launch_chunk_tc(c, Q, Kp, Vp, O, a, sp, ws, st);
  if (e != cudaSuccess) return e;
  return c.D == 64 ? merge<uint16_t, 64>(c, O, sp, ws, st) : merge<uint16_t, 128>(c, O, sp, ws, st);
}

}  // namespace medusa
