// Attention of new tokens over the pages of a cache: the workspace, the merge of what was cut, and the call.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "chunk.cuh"
#include "common.cuh"

namespace medusa {
namespace {

// Joins the partial results of the units that were cut: O = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s. Eight
// lanes to a row, each with its weights and D / 8 head dims, four of them next to each other in every 32. Bound by the
// partial results' bytes, which lie in L2. (A warp to a row worked out where that is, and its weights, 32 times over:
// 20 us behind 2048 rows after 14336, now 12.6.)
constexpr int kMergeThreads = 256, kMergeLanes = 8, kMergeRows = kMergeThreads / kMergeLanes;
constexpr int kMergeSplit = 4;   // groups of lanes to a row of a single tile, whose parts they divide: there are few rows, of many parts
constexpr int kMergeBlocks = 2;
// Parts on their way at a time. In bf16 most rows have two or three (two: 12.6 us behind 2048 rows after 14336, four:
// 16); in float32, where little work is cut into many, up to thirty. Whole calls in float32 with four, and with two: one token
// of 8000 rows, 8/4 heads, 17.3 and 18.0 us with D = 64, 18.9 and 19.4 with D = 128; five sequences of 0 to 700 rows 46.9 and 47.0,
// 62.1 and 61.7; 24 tokens of 4000 rows, 32/8 heads of 128, 227 both.
template <typename T> constexpr int kMergeParts = sizeof(T) == 4 ? 4 : 2;

// 2^x. In float32 as the attention kernel has it, down to 2^-149: a part 2^-130 below the row's maximum may still count.
template <typename T>
__device__ __forceinline__ float ex2(float x) {
  if constexpr (sizeof(T) == 4) {
    return exp2f(x);
  } else {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
  }
}

// Row i of a cut: its parts turn, turn + step, ... by eight lanes, or by the four groups of eight of a warp.
template <typename T, int D>
__device__ __forceinline__ void join(const float* __restrict__ o_part, const float* __restrict__ ml_part, const ChunkSpace& sp,
                                     const ChunkCut& cut, bool pair, int stream, int i, int turn, int step, int sub, int Hq,
                                     T* __restrict__ O) {
  constexpr int X = D / 32, P = kMergeParts<T>;
  // rows of a tile lie [head][position]
  const int along = pair ? sp.npos : sp.single_npos, tile_rows = along << sp.gp_shift;
  const int tile = pair && i >= tile_rows, in_tile = i - tile * tile_rows;
  const int head = in_tile / (pair ? along : cut.left), at_pos = in_tile - head * (pair ? along : cut.left), pos = at_pos + tile * along;
  const int r = pair ? i : head * along + at_pos;
  if (pos >= cut.left) return;
  const int64_t rows = pair ? sp.pair_rows : sp.single_rows;
  // part 0 is the stream's second one, the others are the first ones of those behind it
  const int64_t at0 = (pair ? sp.pair_part(stream, 1) : sp.single_part(stream, 1)) + r;
  auto place = [&](int s) { return s == 0 ? at0 : at0 + (2 * s - 1) * rows; };
  // a row's lanes, which are here together: eight of them, or a whole warp
  const int wide = kMergeLanes * step;
  const unsigned lanes = pair ? ((1u << kMergeLanes) - 1) << (threadIdx.x & 31) / kMergeLanes * kMergeLanes : 0xffffffffu;
  float M = -INFINITY;   // (they take the parts in turn)
  for (int s = turn * kMergeLanes + sub; s <= cut.parts; s += wide) M = fmaxf(M, ml_part[2 * place(s)]);
  for (int o = wide / 2; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(lanes, M, o));
  const float mu = M == -INFINITY ? 0.f : M;
  float sum = 0.f;
  float4 acc[X];
#pragma unroll
  for (int x = 0; x < X; ++x) acc[x] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = turn; s0 <= cut.parts; s0 += P * step) {
    float2 ml[P];
    float4 o[P][X];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      ml[i] = make_float2(-INFINITY, 0.f);
      if (s0 + i * step > cut.parts) continue;
      const int64_t at = place(s0 + i * step);
      ml[i] = *reinterpret_cast<const float2*>(ml_part + 2 * at);
#pragma unroll
      for (int x = 0; x < X; ++x) o[i][x] = *reinterpret_cast<const float4*>(o_part + at * D + 32 * x + 4 * sub);
    }
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if (ml[i].x == -INFINITY && ml[i].y == 0.f) continue;   // nothing was visible: its O need not have been written
      const float w = ex2<T>(ml[i].x - mu);
      sum = fmaf(ml[i].y, w, sum);
#pragma unroll
      for (int x = 0; x < X; ++x) {
        const float4 v = o[i][x];
        acc[x] = make_float4(fmaf(v.x, w, acc[x].x), fmaf(v.y, w, acc[x].y), fmaf(v.z, w, acc[x].z), fmaf(v.w, w, acc[x].w));
      }
    }
  }
  if (!pair) {
#pragma unroll
    for (int o = kMergeLanes; o < 32; o <<= 1) {
      sum += __shfl_xor_sync(lanes, sum, o);
#pragma unroll
      for (int x = 0; x < X; ++x) {
        acc[x].x += __shfl_xor_sync(lanes, acc[x].x, o);
        acc[x].y += __shfl_xor_sync(lanes, acc[x].y, o);
        acc[x].z += __shfl_xor_sync(lanes, acc[x].z, o);
        acc[x].w += __shfl_xor_sync(lanes, acc[x].w, o);
      }
    }
    if (turn) return;
  }
  const float inv = 1.f / sum;   // (0 where every visible score is -inf: no number)
  T* op = O + ((size_t)(cut.pos0 + pos) * Hq + cut.h0 + head) * D + 4 * sub;
#pragma unroll
  for (int x = 0; x < X; ++x) {
    const float4 v = make_float4(acc[x].x * inv, acc[x].y * inv, acc[x].z * inv, acc[x].w * inv);
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<float4*>(op + 32 * x) = v;
    } else {
      uint2 w;
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.x) : "f"(v.y), "f"(v.x));
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.y) : "f"(v.w), "f"(v.z));
      *reinterpret_cast<uint2*>(op + 32 * x) = w;
    }
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kMergeThreads)
chunk_merge_kernel(const float* __restrict__ o_part, const float* __restrict__ ml_part, const ChunkCut* __restrict__ cuts,
                   const ChunkSpace sp, int Hq, T* __restrict__ O) {
  static_assert(kMergeLanes * kMergeSplit == 32, "a row of a single tile is a warp's");
  pdl_wait();
  pdl_trigger();
  // blocks: kMergeRows rows of each stream of pairs; then kMergeBlocks for each stream of single tiles, which go
  // through the rows that its cut has (most have few: a block for every eight that there may be took 2 us more)
  const int per_pair = sp.pair_rows / kMergeRows;
  const bool pair = (int)blockIdx.x < sp.pair_streams * per_pair;
  const int y = pair ? (int)blockIdx.x : (int)blockIdx.x - sp.pair_streams * per_pair, per = pair ? per_pair : kMergeBlocks;
  const int stream = y / per, sub = threadIdx.x % kMergeLanes, step = pair ? 1 : kMergeSplit;
  const int slot = (y - stream * per) * kMergeRows + threadIdx.x / kMergeLanes;
  const int turn = pair ? 0 : slot % kMergeSplit;   // the row's parts turn, turn + step, ... are this group's
  const ChunkCut cut = cuts[(pair ? 0 : sp.pair_streams) + stream];
  if (cut.parts == 0) return;
  const int count = pair ? sp.pair_rows : cut.left << sp.single_shift;
  for (int i = pair ? slot : slot / kMergeSplit; i < count; i += pair ? count : kMergeBlocks * kMergeRows / kMergeSplit)
    join<T, D>(o_part, ml_part, sp, cut, pair, stream, i, turn, step, sub, Hq, O);
}

template <typename T, int D>
cudaError_t merge(const medusa_cfg& c, void* O, const ChunkSpace& sp, void* ws, cudaStream_t st) {
  const int blocks = sp.pair_streams * (sp.pair_rows / kMergeRows) + sp.streams * kMergeBlocks;
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
  sp.single_shift = f32 && sp.gp_shift > 2 ? 2 : sp.gp_shift;
  sp.single_rows = sp.single_npos << sp.single_shift;
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
