// Attention of new tokens over the pages of a cache: the workspace, the merge of what was cut, and the call.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "chunk.cuh"
#include "common.cuh"

namespace medusa {
namespace {

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

ChunkSpace chunk_space(const medusa_cfg& c, int T) {
  const bool f32 = c.dtype == MEDUSA_F32;
  const int rows = f32 ? 64 : 128;   // of a tile
  ChunkSpace sp{};
  const int G = c.Hq / c.Hkv;
  while (sp.gp_shift < 4 && G % (2 << sp.gp_shift) == 0) ++sp.gp_shift;   // the largest power of two that divides the group
  sp.npos = rows >> sp.gp_shift;
  // (no sequence has more rows than there are)
  sp.pair_streams = T > (f32 ? 1 : sp.npos) ? kChunkStreams : 0;
  sp.pair_rows = f32 ? rows : 2 * rows;
  sp.streams = kChunkStreams;
  sp.single_npos = f32 ? 1 : T < sp.npos ? T : sp.npos;
  sp.single_rows = f32 ? 1 << (sp.gp_shift < 2 ? sp.gp_shift : 2) : sp.single_npos << sp.gp_shift;
  const size_t all = (size_t)2 * sp.pair_streams * sp.pair_rows + (size_t)2 * sp.streams * sp.single_rows;
  sp.ml = align_up(all * c.D * 4, 256);
  sp.cuts = sp.ml + align_up(all * 8, 256);
  sp.total = sp.cuts + align_up((sp.pair_streams + sp.streams) * sizeof(ChunkCut), 256);
  return sp;
}

bool chunk_countable(const medusa_cfg& c, int T) {
  const ChunkSpace sp = chunk_space(c, T);
  const bool f32 = c.dtype == MEDUSA_F32;
  const double units = ((double)T / sp.npos + c.B) * (c.Hq >> sp.gp_shift) + (f32 ? (double)c.B * c.Hq / sp.single_rows : 0.0);
  return units * (c.L_cap / (f32 ? 64 : 128) + 4.0) < 2147483647.0;   // (4: the tile that is begun, what a unit counts for beside)
}

size_t chunk_workspace(const medusa_cfg& c, int T) { return chunk_space(c, T).total; }

cudaError_t launch_chunk_attention(const medusa_cfg& c, const void* Q, const void* Kp, const void* Vp, void* O, const ChunkArgs& a,
                                   void* ws, cudaStream_t st) {
  const ChunkSpace sp = chunk_space(c, a.T);
  const bool f32 = c.dtype == MEDUSA_F32;
  const cudaError_t e = f32 ? launch_chunk_f32(c, Q, Kp, Vp, O, a, sp, ws, st) : launch_chunk_tc(c, Q, Kp, Vp, O, a, sp, ws, st);
  if (e != cudaSuccess) return e;
  if (f32) return c.D == 64 ? merge<float, 64>(c, O, sp, ws, st) : merge<float, 128>(c, O, sp, ws, st);
  return c.D == 64 ? merge<uint16_t, 64>(c, O, sp, ws, st) : merge<uint16_t, 128>(c, O, sp, ws, st);
}

}  // namespace medusa
