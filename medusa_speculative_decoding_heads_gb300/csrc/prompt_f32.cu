// Causal attention over packed prompts in float32 on the CUDA cores.
//
// O = softmax(q.k / sqrt(D)) v, 64 rows of one head against tiles of 64 keys, with the
// running maximum and sum of "최적화 2편" (beengineer500), section 3.3; everything float32.
// Bound by the float32 multiply-adds (128 per SM and clock): 4 rows keys D operations. A
// thread owns 4 rows x 4 keys of the scores and 4 rows x D / 16 head dims of O, so that four
// head dims (or keys) cost 8 shared-memory words of 16 bytes for 64 multiply-adds, 12
// bank-conflict-free wavefronts per warp; rows of Q, K and P are padded by 16 bytes for that.
// K_{j+1} arrives while tile j's weights and values are worked on, V_j while its scores are.
// Two groups of 256 threads take the unit's even and odd key tiles, each with its own
// maximum, sum and O, and merge at the end: a causal prompt's last rows are its longest
// chain, and this halves it.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "common.cuh"
#include "prompt_walk.cuh"

namespace medusa {
namespace {

constexpr int kTileRows = 64, kTileKeys = 64;
constexpr int kGroup = 256, kGroups = 2;
constexpr int kThreadsF32 = kGroup * kGroups;

template <int D>
struct Smem {
  static constexpr int kLd = D + 4;            // padded row of Q and K (floats)
  static constexpr int kLdP = kTileKeys + 4;   // padded row of P
  static constexpr int q = 0;
  static constexpr int k = q + kTileRows * kLd;
  static constexpr int v = k + kTileKeys * kLd;
  static constexpr int p = v + kTileKeys * D;
  static constexpr int per_group = p + kTileRows * kLdP - k;   // K, V and P, once per group
  static constexpr int bytes = (k + kGroups * per_group) * 4;
  static_assert(kTileRows * (D + 2) <= per_group, "the second group's result must fit its tiles");
};

__device__ __forceinline__ void cp16(float* dst, const float* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
               "r"(valid ? 16 : 0));
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;\n" ::); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;\n" ::"n"(N)); }

// 64 rows of `stride` floats from src into rows of ld floats, by thread `tid` of a group;
// rows past `live` become zeros.
template <int D>
__device__ __forceinline__ void load_tile(float* dst, int ld, const float* src, int64_t stride, int live, int tid) {
  constexpr int CH = D / 4;
#pragma unroll
  for (int e = tid; e < 64 * CH; e += kGroup) {
    const int r = e / CH, c = e % CH;
    const bool ok = r < live;
    cp16(dst + r * ld + 4 * c, src + (ok ? r : 0) * stride + 4 * c, ok);
  }
}

template <int D>
__global__ void __launch_bounds__(kThreadsF32, 1)
prompt_f32_kernel(const float* __restrict__ Q, const float* __restrict__ K, const float* __restrict__ V, int T, int64_t qs,
                  int64_t ks, int64_t vs, const int32_t* __restrict__ cu, int B, int Hq, int Hkv, float scale_log2,
                  float* __restrict__ O) {
  using S = Smem<D>;
  constexpr int NC = D / 64;   // 4-column groups of O per thread, 64 columns apart
  pdl_wait();
  pdl_trigger();
  extern __shared__ __align__(16) float smem[];
  __shared__ int unit_b, unit_t;
  const int group = threadIdx.x / kGroup, tid = threadIdx.x % kGroup;
  float *sq = smem + S::q, *sk = smem + S::k + group * S::per_group, *sv = sk + S::v - S::k, *sp = sk + S::p - S::k;
  const int rg = tid >> 4, cg = tid & 15;   // rows 4 rg .., keys cg + 16 i, head dims 4 cg + 64 n ..
  auto sync_group = [&] { asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(kGroup) : "memory"); };
  PromptWalk walk;
  if (threadIdx.x < 32) walk.begin(cu, B, T, kTileRows);

  for (int64_t u = blockIdx.x;; u += gridDim.x) {
    if (threadIdx.x < 32) {
      const int b = walk.find((int)(u / Hq));
      if (threadIdx.x == 0) {
        unit_b = b;
        unit_t = walk.t;
      }
    }
    __syncthreads();
    const int b = unit_b, r0 = unit_t * kTileRows;
    if (b < 0) break;
    const int h = (int)(u % Hq), kvh = h / (Hq / Hkv);
    const int64_t c0 = cu[b];
    const int len = cu[b + 1] - (int)c0, rows = min(kTileRows, len - r0), keys = r0 + rows;
    const int nt = (keys + kTileKeys - 1) / kTileKeys;
    const float* kp = K + c0 * ks + (size_t)kvh * D;
    const float* vp = V + c0 * vs + (size_t)kvh * D;
    if (group == 0) load_tile<D>(sq, S::kLd, Q + (c0 + r0) * qs + (size_t)h * D, qs, rows, tid);
    if (group < nt) load_tile<D>(sk, S::kLd, kp + (int64_t)group * kTileKeys * ks, ks, keys - group * kTileKeys, tid);
    cp_commit();

    float4 o[4][NC];
    float m[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int n = 0; n < NC; ++n) o[i][n] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    cp_wait<0>();
    __syncthreads();       // Q of group 0
    for (int j = group; j < nt; j += kGroups) {
      const int k0 = j * kTileKeys;
      cp_wait<0>();        // K_j
      sync_group();        // ... of every thread; V and P of the tile before are no longer read
      load_tile<D>(sv, D, vp + k0 * vs, vs, keys - k0, tid);
      cp_commit();
      float2 s[4][4];   // (even, odd) head dims
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) s[i][c] = make_float2(0.f, 0.f);
#pragma unroll 4
      for (int d = 0; d < D; d += 4) {
        float4 a[4], w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4*>(sq + (4 * rg + i) * S::kLd + d);
#pragma unroll
        for (int c = 0; c < 4; ++c) w[c] = *reinterpret_cast<const float4*>(sk + (cg + 16 * c) * S::kLd + d);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            s[i][c] = __ffma2_rn(make_float2(a[i].x, a[i].y), make_float2(w[c].x, w[c].y), s[i][c]);
            s[i][c] = __ffma2_rn(make_float2(a[i].z, a[i].w), make_float2(w[c].z, w[c].w), s[i][c]);
          }
      }
      sync_group();        // K_j is no longer read
      constexpr int ahead = kGroups * kTileKeys;
      if (j + kGroups < nt) load_tile<D>(sk, S::kLd, kp + (int64_t)(k0 + ahead) * ks, ks, keys - k0 - ahead, tid);
      cp_commit();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int see = r0 + 4 * rg + i - k0;   // keys 0..see of the tile are visible to the row
        float x[4], mt = -INFINITY;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          x[c] = cg + 16 * c <= see ? (s[i][c].x + s[i][c].y) * scale_log2 : -INFINITY;
          mt = fmaxf(mt, x[c]);
        }
#pragma unroll
        for (int w = 8; w > 0; w >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, w));   // the row's 16 threads
        const float mn = fmaxf(m[i], mt), mu = mn == -INFINITY ? 0.f : mn;
        const float corr = exp2f(m[i] - mu);
        m[i] = mn;
        float ps = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float p = exp2f(x[c] - mu);
          ps += p;
          sp[(4 * rg + i) * S::kLdP + cg + 16 * c] = p;
        }
        l[i] = l[i] * corr + ps;
#pragma unroll
        for (int n = 0; n < NC; ++n) {
          o[i][n].x *= corr;
          o[i][n].y *= corr;
          o[i][n].z *= corr;
          o[i][n].w *= corr;
        }
      }
      cp_wait<1>();        // V_j
      sync_group();        // ... and P_j
#pragma unroll 4
      for (int k = 0; k < kTileKeys; k += 4) {
        float4 p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const float4*>(sp + (4 * rg + i) * S::kLdP + k);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          float4 w[NC];
#pragma unroll
          for (int n = 0; n < NC; ++n) w[n] = *reinterpret_cast<const float4*>(sv + (k + x) * D + 64 * n + 4 * cg);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float pv = x == 0 ? p[i].x : x == 1 ? p[i].y : x == 2 ? p[i].z : p[i].w;
            const float2 pp = make_float2(pv, pv);
#pragma unroll
            for (int n = 0; n < NC; ++n) {
              const float2 lo = __ffma2_rn(pp, make_float2(w[n].x, w[n].y), make_float2(o[i][n].x, o[i][n].y));
              const float2 hi = __ffma2_rn(pp, make_float2(w[n].z, w[n].w), make_float2(o[i][n].z, o[i][n].w));
              o[i][n] = make_float4(lo.x, lo.y, hi.x, hi.y);
            }
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int w = 8; w > 0; w >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], w);
    // group 1 leaves its maximum, sum and O where its tiles were; group 0 merges and stores
    float* so = smem + S::k + S::per_group;
    float* sml = so + kTileRows * D;
    if (group == 1) {
      sync_group();        // its last tile is no longer read
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (cg == 0) {
          sml[2 * (4 * rg + i)] = m[i];
          sml[2 * (4 * rg + i) + 1] = l[i];
        }
#pragma unroll
        for (int n = 0; n < NC; ++n) *reinterpret_cast<float4*>(so + (4 * rg + i) * D + 64 * n + 4 * cg) = o[i][n];
      }
    }
    cp_wait<0>();
    __syncthreads();
    if (group == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float m1 = sml[2 * (4 * rg + i)], l1 = sml[2 * (4 * rg + i) + 1], M = fmaxf(m[i], m1);
        if (4 * rg + i < rows) {   // such a row saw its own key at least, so M is no -inf (unless it is no number)
          const float w0 = m[i] == M ? 1.f : exp2f(m[i] - M), w1 = m1 == M ? 1.f : exp2f(m1 - M);
          const float inv = 1.f / (l[i] * w0 + l1 * w1);
          float* op = O + ((size_t)(c0 + r0 + 4 * rg + i) * Hq + h) * D + 4 * cg;
#pragma unroll
          for (int n = 0; n < NC; ++n) {
            const float4 x = *reinterpret_cast<const float4*>(so + (4 * rg + i) * D + 64 * n + 4 * cg);
            *reinterpret_cast<float4*>(op + 64 * n) =
                make_float4((o[i][n].x * w0 + x.x * w1) * inv, (o[i][n].y * w0 + x.y * w1) * inv,
                            (o[i][n].z * w0 + x.z * w1) * inv, (o[i][n].w * w0 + x.w * w1) * inv);
          }
        }
      }
    }
    __syncthreads();   // the unit, Q and the tiles may be overwritten
  }
}

template <int D>
cudaError_t run(const medusa_cfg& c, const void* Q, const void* K, const void* V, int T, int64_t qs, int64_t ks, int64_t vs,
                const int32_t* cu, void* O, cudaStream_t st) {
  const float scale_log2 = (float)(1.4426950408889634 / sqrt((double)D));
  cudaError_t e = cudaFuncSetAttribute(prompt_f32_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::bytes);
  if (e != cudaSuccess) return e;
  const int64_t units = ((int64_t)T / kTileRows + c.B) * c.Hq;   // at least as many as there are
  const int64_t resident = 152;   // one CTA per SM
  e = launch_pdl(prompt_f32_kernel<D>, (unsigned)(units < resident ? units : resident), kThreadsF32, Smem<D>::bytes, st,
                 static_cast<const float*>(Q), static_cast<const float*>(K), static_cast<const float*>(V), T, qs, ks, vs, cu,
                 c.B, c.Hq, c.Hkv, scale_log2, static_cast<float*>(O));
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
