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

}  // namespace

MEDUSA_CHECK_TAKE(chunk_take_checks)

size_t chunk_workspace(const medusa_cfg&, int) { return 0; }

cudaError_t launch_chunk_attention(const medusa_cfg& c, const void* Q, const void* Kp, const void* Vp, void* O, const ChunkArgs& a,
                                   void*, cudaStream_t st) {
  if (c.dtype == MEDUSA_F32) return c.D == 64 ? run<float, 64>(Q, Kp, Vp, O, a, st) : run<float, 128>(Q, Kp, Vp, O, a, st);
  return c.D == 64 ? run<uint16_t, 64>(Q, Kp, Vp, O, a, st) : run<uint16_t, 128>(Q, Kp, Vp, O, a, st);
}

}  // namespace medusa
