// Causal attention over packed prompts: one warp per query row and head (float32, and bf16
// with D = 64; bf16 with D = 128 takes the tcgen05 kernel of rows_tc.cu).
//
// O = softmax(q.k / sqrt(D)) v over the visible keys, 32 keys at a time: lane = key for
// the scores, lane = head dim for the weighted sum of values, with the running maximum and
// sum of "최적화 2편" (beengineer500), section 3.3. Scores, statistics and sums are float32.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "common.cuh"

namespace medusa {
namespace {

constexpr int kRowWarps = 8;

// Online softmax over blocks of 32 keys of one query row held by a warp.
template <typename T, int D>
struct WarpRow {
  float q[D];   // every lane holds the whole (scaled) query row
  float m = -INFINITY, l = 0.f, o[D / 32];

  __device__ __forceinline__ void begin(const T* qp, float scale_log2) {
#pragma unroll
    for (int d = 0; d < D; ++d) q[d] = Elt<T>::load(qp, d) * scale_log2;
#pragma unroll
    for (int j = 0; j < D / 32; ++j) o[j] = 0.f;
  }
  // kp, vp: this lane's key and value row (nullptr: not visible)
  __device__ __forceinline__ void block(const T* kp, const T* vp) {
    float s = -INFINITY;
    if (kp) {
      s = 0.f;
#pragma unroll
      for (int d = 0; d < D; ++d) s = fmaf(q[d], Elt<T>::load(kp, d), s);
    }
    const float mt = warp_max(s);
    const float mn = fmaxf(m, mt);
    if (mn == -INFINITY) return;
    const float corr = exp2f(m - mn), p = kp ? exp2f(s - mn) : 0.f;
    l = l * corr + warp_sum(p);
#pragma unroll
    for (int j = 0; j < D / 32; ++j) o[j] *= corr;
    m = mn;
    const int lane = threadIdx.x & 31;
    for (unsigned live = __ballot_sync(0xffffffffu, kp != nullptr); live; live &= live - 1) {
      const int j = __ffs(live) - 1;
      const float pj = __shfl_sync(0xffffffffu, p, j);
      const T* v = reinterpret_cast<const T*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(vp), j));
#pragma unroll
      for (int x = 0; x < D / 32; ++x) o[x] = fmaf(pj, Elt<T>::load(v, lane + 32 * x), o[x]);
    }
  }
  __device__ __forceinline__ void store(T* op) {
    const int lane = threadIdx.x & 31;
    const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
    for (int x = 0; x < D / 32; ++x) Elt<T>::store(op, lane + 32 * x, o[x] * inv);
  }
};

template <typename T, int D>
__global__ void __launch_bounds__(kRowWarps * 32)
prompt_rows_kernel(const T* __restrict__ Q, const T* __restrict__ K, const T* __restrict__ V, int T_rows, int64_t qs,
                   int64_t ks, int64_t vs, const int32_t* __restrict__ cu, int B, int Hq, int Hkv, float scale_log2,
                   T* __restrict__ O) {
  pdl_wait();
  pdl_trigger();
  const int64_t w = (int64_t)blockIdx.x * kRowWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int t = (int)(w / Hq), h = (int)(w % Hq);
  if (t >= T_rows) return;
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= t) lo = mid;
    else hi = mid;
  }
  const int c0 = cu[lo], c1 = cu[lo + 1];
  if (!(c0 >= 0 && c1 <= T_rows && t >= c0 && t < c1)) return;
  const int kvh = h / (Hq / Hkv);
  WarpRow<T, D> r;
  r.begin(Q + t * qs + (size_t)h * D, scale_log2);
  for (int k0 = c0; k0 <= t; k0 += 32) {
    const int64_t key = k0 + lane;
    const bool see = key <= t;
    r.block(see ? K + key * ks + (size_t)kvh * D : nullptr, see ? V + key * vs + (size_t)kvh * D : nullptr);
  }
  r.store(O + ((size_t)t * Hq + h) * D);
}

template <typename T, int D>
cudaError_t run_prompt(const medusa_cfg& c, const void* Q, const void* K, const void* V, int T_rows, int64_t qs, int64_t ks,
                       int64_t vs, const int32_t* cu, void* O, cudaStream_t st) {
  const float scale_log2 = (float)(1.4426950408889634 / sqrt((double)D));
  const int64_t warps = (int64_t)T_rows * c.Hq;
  return launch_pdl(prompt_rows_kernel<T, D>, (unsigned)((warps + kRowWarps - 1) / kRowWarps), kRowWarps * 32, 0, st,
                    static_cast<const T*>(Q), static_cast<const T*>(K), static_cast<const T*>(V), T_rows, qs, ks, vs, cu,
                    c.B, c.Hq, c.Hkv, scale_log2, static_cast<T*>(O));
}

}  // namespace

cudaError_t launch_prompt_attention(const medusa_cfg& c, const void* Q, const void* K, const void* V, int T_rows, int64_t qs,
                                    int64_t ks, int64_t vs, const int32_t* cu, void* O, cudaStream_t st) {
  if (c.dtype == MEDUSA_BF16 && c.D == 128) return launch_prompt_tc(c, Q, K, V, T_rows, qs, ks, vs, cu, O, st);
  cudaError_t e;
  if (c.dtype == MEDUSA_F32)
    e = c.D == 64 ? run_prompt<float, 64>(c, Q, K, V, T_rows, qs, ks, vs, cu, O, st)
                  : run_prompt<float, 128>(c, Q, K, V, T_rows, qs, ks, vs, cu, O, st);
  else
    e = run_prompt<uint16_t, 64>(c, Q, K, V, T_rows, qs, ks, vs, cu, O, st);
  note_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace medusa
