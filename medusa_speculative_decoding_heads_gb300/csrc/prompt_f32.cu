// Causal attention over packed prompts in float32 on the CUDA cores.
//
// O = softmax(q.k / sqrt(D)) v, 64 rows of one head against tiles of 64 keys, with the
// running maximum and sum of "최적화 2편" (beengineer500), section 3.3; everything float32.
// Bound by the float32 multiply-adds (128 per SM and clock): 4 rows keys D operations. Measured
// alone from registers they reach 68 TFLOP/s one by one and 57-61 in pairs (the registers'
// bandwidth), but one by one they leave no issue slots for the rest, so pairs it is (prompts of
// 700, 1, 129 and 1500 tokens, 8 heads of 64: 89 us one by one, 80 in pairs, now 76). A thread owns 4 rows x 8 keys of the scores and 4 rows x D / 8 head dims of O:
// four head dims (or keys) cost it 12 shared-memory words of 16 bytes for 128 multiply-adds. A
// half-warp's words come in one wavefront if neighbouring lanes (or every second pair) want
// the same one, so lane bit 0 is a row's and bit 1 a key's: 24 wavefronts per warp, 40 with
// rows in bits 3 and 4 (86 us). Rows of Q, K and P are padded, and a thread's rows and keys
// lie apart, so that no two words meet in a bank.
// K_{j+1} arrives while tile j's weights and values are worked on, V_j while its scores are.
// Groups of 128 threads (3 with D = 64, 2 with D = 128: as many as registers and shared memory
// hold tiles for) take the unit's key tiles in turn, each with its own maximum, sum and O, and
// merge at the end: a causal prompt's last rows are its longest chain. One CTA per SM at a time and,
// up to 64 prompts, per unit; those with the most keys first. 8192 tokens, 8 heads of 64: 1375 us, 50
// TFLOP/s; of 128: 2665 us, 51.6; 1500 tokens 77 and 147 us (fewer than two waves of units).
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "common.cuh"
#include "f32_tiles.cuh"
#include "prompt_walk.cuh"

namespace medusa {
namespace {

// Batches of more prompts than this look for each unit's sequence from where the CTA's last one was
// (4 CTAs per SM, one at a time): 512 of 1 to 60 rows 227 us with a CTA per unit, 189 so, 4096 of
// them 3865 and 1541 (two CTAs per SM 185 and 1493); 128 of them and one of 4000 rows 403 and 399
// (409), but 64 with one of 4000 373 and 385.
constexpr int kManyPrompts = 64, kManyGrid = 4 * 152;
using namespace f32;

// 64 rows of `stride` floats from src into rows of ld floats, by thread `tid` of `threads`; rows
// past `live` become zeros.
template <int D>
__device__ __forceinline__ void load_tile(float* dst, int ld, const float* src, int64_t stride, int live, int tid, int threads) {
  constexpr int CH = D / 4;
  for (int e = tid; e < 64 * CH; e += threads) {
    const int r = e / CH, c = e % CH;
    const bool ok = r < live;
    cp16(dst + r * ld + 4 * c, src + (ok ? r : 0) * stride + 4 * c, ok);
  }
}

// Rows r0 to r0 + 63 of sequence b in head h, by the whole CTA.
template <int D>
__device__ __forceinline__ void prompt_unit(float* smem, const float* __restrict__ Q, const float* __restrict__ K,
                                            const float* __restrict__ V, int64_t qs, int64_t ks, int64_t vs,
                                            const int32_t* __restrict__ cu, int Hq, int Hkv, float scale_log2,
                                            float* __restrict__ O, int b, int r0, int h) {
  using S = Smem<D>;
  Rows<D> t;
  t.begin(smem);
  const int group = t.group, tid = t.tid;
  const int kvh = h / (Hq / Hkv);
  const int64_t c0 = cu[b];
  const int len = cu[b + 1] - (int)c0, rows = min(kTileRows, len - r0), keys = r0 + rows;
  const int nt = (keys + kTileKeys - 1) / kTileKeys;
  const float* kp = K + c0 * ks + (size_t)kvh * D;
  const float* vp = V + c0 * vs + (size_t)kvh * D;
  load_tile<D>(t.sq, S::ld, Q + (c0 + r0) * qs + (size_t)h * D, qs, rows, threadIdx.x, S::threads);
  if (group < nt) load_tile<D>(t.sk, S::ld, kp + (int64_t)group * kTileKeys * ks, ks, keys - group * kTileKeys, tid, kGroup);
  cp_commit();
  cp_wait<0>();
  __syncthreads();       // Q
  for (int j = group; j < nt; j += S::groups) {
    const int k0 = j * kTileKeys;
    cp_wait<0>();        // K_j
    t.sync_group();      // ... of every thread; V and P of the tile before are no longer read
    load_tile<D>(t.sv, D, vp + k0 * vs, vs, keys - k0, tid, kGroup);
    cp_commit();
    float2 s[4][8];
    t.scores(s);
    t.sync_group();      // K_j is no longer read
    constexpr int ahead = S::groups * kTileKeys;
    if (j + S::groups < nt) load_tile<D>(t.sk, S::ld, kp + (int64_t)(k0 + ahead) * ks, ks, keys - k0 - ahead, tid, kGroup);
    cp_commit();
    t.weights(s, scale_log2, [&](int i) {
      const int see = r0 + t.rg + 4 * i - k0;   // keys 0..see of the tile are visible to the row
      return [see](int key) { return key <= see; };
    });
    cp_wait<1>();        // V_j
    t.sync_group();      // ... and P_j
    t.values();
  }
  if (!t.join(smem, rows)) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = t.rg + 4 * i;
    if (r >= rows) continue;
    const float inv = 1.f / t.l[i];
    float* op = O + ((size_t)(c0 + r0 + r) * Hq + h) * D + 4 * t.cg;
#pragma unroll
    for (int n = 0; n < Rows<D>::NC; ++n)
      *reinterpret_cast<float4*>(op + 32 * n) = make_float4(t.o[i][n].x * inv, t.o[i][n].y * inv, t.o[i][n].z * inv, t.o[i][n].w * inv);
  }
}

// A CTA per unit; kMany: it takes unit blockIdx.x and every gridDim.x-th behind it, and keeps its
// place among them.
template <int D, bool kMany>
__global__ void __launch_bounds__(Smem<D>::threads, 1)
prompt_f32_kernel(const float* __restrict__ Q, const float* __restrict__ K, const float* __restrict__ V, int T, int64_t qs,
                  int64_t ks, int64_t vs, const int32_t* __restrict__ cu, int B, int Hq, int Hkv, float scale_log2,
                  unsigned units, float* __restrict__ O) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ __align__(16) float smem[];
  __shared__ int unit_b, unit_t;
  __shared__ PromptWalk place;
  for (unsigned u = blockIdx.x;; u += gridDim.x) {
    if (threadIdx.x < 32) {
      PromptWalk walk;
      if (!kMany || u == blockIdx.x) walk.begin(cu, B, T, kTileShift);
      else walk = place;
      const int b = walk.find((int)(u / Hq));
      __syncwarp();
      if (threadIdx.x == 0) {
        unit_b = b;
        unit_t = walk.t;
        if (kMany) place = walk;
      }
    }
    __syncthreads();
    if (unit_b < 0) return;   // (there may be fewer units than blocks)
    prompt_unit<D>(smem, Q, K, V, qs, ks, vs, cu, Hq, Hkv, scale_log2, O, unit_b, unit_t * kTileRows, (int)(u % Hq));
    if (!kMany || units - u <= gridDim.x) return;
    __syncthreads();   // the next unit's tiles and place go where this one's were
  }
}

template <int D>
cudaError_t run(const medusa_cfg& c, const void* Q, const void* K, const void* V, int T, int64_t qs, int64_t ks, int64_t vs,
                const int32_t* cu, void* O, cudaStream_t st) {
  const float scale_log2 = (float)(1.4426950408889634 / sqrt((double)D));
  const int units = (int)(((int64_t)T / kTileRows + c.B) * c.Hq);   // at least as many as there are
  const bool many = c.B > kManyPrompts && units > kManyGrid;
  const auto kernel = many ? prompt_f32_kernel<D, true> : prompt_f32_kernel<D, false>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::bytes);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kernel, (unsigned)(many ? kManyGrid : units), Smem<D>::threads, Smem<D>::bytes, st, static_cast<const float*>(Q),
                 static_cast<const float*>(K), static_cast<const float*>(V), T, qs, ks, vs, cu, c.B, c.Hq, c.Hkv, scale_log2,
                 (unsigned)units, static_cast<float*>(O));
  note_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_prompt_f32(const medusa_cfg& c, const void* Q, const void* K, const void* V, int T, int64_t q_stride,
                              int64_t k_stride, int64_t v_stride, const int32_t* cu, void* O, cudaStream_t st) {
  return c.D == 64 ? run<64>(c, Q, K, V, T, q_stride, k_stride, v_stride, cu, O, st)
                   : run<128>(c, Q, K, V, T, q_stride, k_stride, v_stride, cu, O, st);
}

}  // namespace medusa
