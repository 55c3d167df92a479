// Causal attention over packed prompts in float32 on the CUDA cores.
//
// O = softmax(q.k / sqrt(D)) v, 64 rows of one head against tiles of 64 keys, with the
// running maximum and sum of "최적화 2편" (beengineer500), section 3.3; everything float32.
// Bound by the float32 multiply-adds (128 per SM and clock): 4 rows keys D operations. A
// thread owns 8 rows x 4 keys of the scores and 8 rows x D / 16 head dims of O, so that four
// head dims (or keys) cost it 12 shared-memory words of 16 bytes, 16 wavefronts of its warp,
// for 128 multiply-adds, issued in pairs (prompts of 700, 1, 129 and 1500 tokens, 8 heads of
// 64: 155 us with 4 x 4 per thread, bound by shared memory; 101 us with single multiply-adds,
// by their issue; 85 us so, 39 TFLOP/s on longer ones). Rows of Q, K and P are padded by 16
// bytes, and a thread's rows lie 8 apart, so that no two of a warp's words meet in a bank.
// K_{j+1} arrives while tile j's weights and values are worked on, V_j while its scores are.
// Groups of 128 threads (3 with D = 64, 2 with D = 128: as many as registers and shared memory
// hold tiles for) take the unit's key tiles in turn, each with its own maximum, sum and O, and
// merge at the end: a causal prompt's last rows are its longest chain. One CTA per unit and SM,
// those with the most keys first.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "common.cuh"
#include "prompt_walk.cuh"

namespace medusa {
namespace {

constexpr int kTileRows = 64, kTileKeys = 64, kGroup = 128;

template <int D>
struct Smem {
  static constexpr int groups = D == 64 ? 3 : 2;
  static constexpr int threads = groups * kGroup;
  static constexpr int ld = D + 4;            // padded row of Q and K (floats)
  static constexpr int ldp = kTileKeys + 4;   // padded row of P
  static constexpr int k = kTileRows * ld;    // behind Q: K, V and P of each group
  static constexpr int v = k + kTileKeys * ld;
  static constexpr int p = v + kTileKeys * D;
  static constexpr int per_group = p + kTileRows * ldp - k;
  static constexpr int bytes = (k + groups * per_group) * 4;
  static_assert(kTileRows * (D + 2) <= per_group, "a group's result must fit its tiles");
  static_assert(bytes <= 227 * 1024, "shared memory of one CTA");
};

__device__ __forceinline__ void cp16(float* dst, const float* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
               "r"(valid ? 16 : 0));
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;\n" ::); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;\n" ::"n"(N)); }

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

template <int D>
__global__ void __launch_bounds__(Smem<D>::threads, 1)
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
  float *sq = smem, *sk = smem + S::k + group * S::per_group, *sv = sk + S::v - S::k, *sp = sk + S::p - S::k;
  const int rg = tid >> 4, cg = tid & 15;   // rows rg + 8 i, keys cg + 16 c, head dims 4 cg + 64 n ..
  auto sync_group = [&] { asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(kGroup) : "memory"); };

  if (threadIdx.x < 32) {
    PromptWalk walk;
    walk.begin(cu, B, T, kTileRows);
    const int b = walk.find((int)(blockIdx.x / Hq));
    if (threadIdx.x == 0) {
      unit_b = b;
      unit_t = walk.t;
    }
  }
  __syncthreads();
  const int b = unit_b, r0 = unit_t * kTileRows;
  if (b < 0) return;   // (the grid may hold more blocks than there are units)
  const int h = (int)(blockIdx.x % Hq), kvh = h / (Hq / Hkv);
  const int64_t c0 = cu[b];
  const int len = cu[b + 1] - (int)c0, rows = min(kTileRows, len - r0), keys = r0 + rows;
  const int nt = (keys + kTileKeys - 1) / kTileKeys;
  const float* kp = K + c0 * ks + (size_t)kvh * D;
  const float* vp = V + c0 * vs + (size_t)kvh * D;
  load_tile<D>(sq, S::ld, Q + (c0 + r0) * qs + (size_t)h * D, qs, rows, threadIdx.x, S::threads);
  if (group < nt) load_tile<D>(sk, S::ld, kp + (int64_t)group * kTileKeys * ks, ks, keys - group * kTileKeys, tid, kGroup);
  cp_commit();

  float4 o[8][NC];
  float m[8], l[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int n = 0; n < NC; ++n) o[i][n] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  cp_wait<0>();
  __syncthreads();       // Q
  for (int j = group; j < nt; j += S::groups) {
    const int k0 = j * kTileKeys;
    cp_wait<0>();        // K_j
    sync_group();        // ... of every thread; V and P of the tile before are no longer read
    load_tile<D>(sv, D, vp + k0 * vs, vs, keys - k0, tid, kGroup);
    cp_commit();
    float2 s[8][4];   // (even, odd) head dims
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) s[i][c] = make_float2(0.f, 0.f);
#pragma unroll 2
    for (int d = 0; d < D; d += 4) {
      float4 w[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) w[c] = *reinterpret_cast<const float4*>(sk + (cg + 16 * c) * S::ld + d);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 a = *reinterpret_cast<const float4*>(sq + (rg + 8 * i) * S::ld + d);
#pragma unroll
        for (int c = 0; c < 4; ++c) s[i][c] = __ffma2_rn(make_float2(a.x, a.y), make_float2(w[c].x, w[c].y), s[i][c]);
#pragma unroll
        for (int c = 0; c < 4; ++c) s[i][c] = __ffma2_rn(make_float2(a.z, a.w), make_float2(w[c].z, w[c].w), s[i][c]);
      }
    }
    sync_group();        // K_j is no longer read
    constexpr int ahead = S::groups * kTileKeys;
    if (j + S::groups < nt) load_tile<D>(sk, S::ld, kp + (int64_t)(k0 + ahead) * ks, ks, keys - k0 - ahead, tid, kGroup);
    cp_commit();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int see = r0 + rg + 8 * i - k0;   // keys 0..see of the tile are visible to the row
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
        sp[(rg + 8 * i) * S::ldp + cg + 16 * c] = p;
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
#pragma unroll 2
    for (int k = 0; k < kTileKeys; k += 4) {
      float4 w[4][NC];
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int n = 0; n < NC; ++n) w[x][n] = *reinterpret_cast<const float4*>(sv + (k + x) * D + 64 * n + 4 * cg);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 p = *reinterpret_cast<const float4*>(sp + (rg + 8 * i) * S::ldp + k);
#pragma unroll
        for (int n = 0; n < NC; ++n) {
          float2 lo = make_float2(o[i][n].x, o[i][n].y), hi = make_float2(o[i][n].z, o[i][n].w);
          const float pk[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float2 pp = make_float2(pk[x], pk[x]);
            lo = __ffma2_rn(pp, make_float2(w[x][n].x, w[x][n].y), lo);
            hi = __ffma2_rn(pp, make_float2(w[x][n].z, w[x][n].w), hi);
          }
          o[i][n] = make_float4(lo.x, lo.y, hi.x, hi.y);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int w = 8; w > 0; w >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], w);
  // The other groups leave their maximum, sum and O where their tiles were; group 0 merges and stores.
  if (group > 0) {
    sync_group();        // the group's last tile is no longer read
    float *so = sk, *sml = so + kTileRows * D;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = rg + 8 * i;
      if (cg == 0) {
        sml[2 * r] = m[i];
        sml[2 * r + 1] = l[i];
      }
#pragma unroll
      for (int n = 0; n < NC; ++n) *reinterpret_cast<float4*>(so + r * D + 64 * n + 4 * cg) = o[i][n];
    }
  }
  cp_wait<0>();
  __syncthreads();
  if (group > 0) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = rg + 8 * i;
    if (r >= rows) continue;
    // A row saw its own key at least, so its largest maximum is no -inf (unless it is no number).
    float M = m[i];
    for (int g = 1; g < S::groups; ++g) M = fmaxf(M, smem[S::k + g * S::per_group + kTileRows * D + 2 * r]);
    float w = m[i] == M ? 1.f : exp2f(m[i] - M), sum = l[i] * w;
#pragma unroll
    for (int n = 0; n < NC; ++n) o[i][n] = make_float4(o[i][n].x * w, o[i][n].y * w, o[i][n].z * w, o[i][n].w * w);
    for (int g = 1; g < S::groups; ++g) {
      const float* so = smem + S::k + g * S::per_group;
      const float mg = so[kTileRows * D + 2 * r];
      w = mg == M ? 1.f : exp2f(mg - M);
      sum += so[kTileRows * D + 2 * r + 1] * w;
#pragma unroll
      for (int n = 0; n < NC; ++n) {
        const float4 x = *reinterpret_cast<const float4*>(so + r * D + 64 * n + 4 * cg);
        o[i][n] = make_float4(o[i][n].x + x.x * w, o[i][n].y + x.y * w, o[i][n].z + x.z * w, o[i][n].w + x.w * w);
      }
    }
    const float inv = 1.f / sum;
    float* op = O + ((size_t)(c0 + r0 + r) * Hq + h) * D + 4 * cg;
#pragma unroll
    for (int n = 0; n < NC; ++n)
      *reinterpret_cast<float4*>(op + 64 * n) = make_float4(o[i][n].x * inv, o[i][n].y * inv, o[i][n].z * inv, o[i][n].w * inv);
  }
}

template <int D>
cudaError_t run(const medusa_cfg& c, const void* Q, const void* K, const void* V, int T, int64_t qs, int64_t ks, int64_t vs,
                const int32_t* cu, void* O, cudaStream_t st) {
  const float scale_log2 = (float)(1.4426950408889634 / sqrt((double)D));
  cudaError_t e = cudaFuncSetAttribute(prompt_f32_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::bytes);
  if (e != cudaSuccess) return e;
  const int64_t units = ((int64_t)T / kTileRows + c.B) * c.Hq;   // at least as many as there are
  e = launch_pdl(prompt_f32_kernel<D>, (unsigned)units, Smem<D>::threads, Smem<D>::bytes, st, static_cast<const float*>(Q),
                 static_cast<const float*>(K), static_cast<const float*>(V), T, qs, ks, vs, cu, c.B, c.Hq, c.Hkv, scale_log2,
                 static_cast<float*>(O));
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
