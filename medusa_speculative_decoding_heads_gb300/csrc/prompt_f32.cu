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
#include "prompt_walk.cuh"

namespace medusa {
namespace {

// Batches of more prompts than this look for each unit's sequence from where the CTA's last one was
// (4 CTAs per SM, one at a time): 512 of 1 to 60 rows 227 us with a CTA per unit, 189 so, 4096 of
// them 3865 and 1541 (two CTAs per SM 185 and 1493); 128 of them and one of 4000 rows 403 and 399
// (409), but 64 with one of 4000 373 and 385.
constexpr int kManyPrompts = 64, kManyGrid = 4 * 152;
constexpr int kTileShift = 6, kTileRows = 1 << kTileShift, kTileKeys = 64, kGroup = 128;

template <int D>
struct Smem {
  static constexpr int groups = D == 64 ? 3 : 2;
  static constexpr int threads = groups * kGroup;
  static constexpr int ld = D + 4;            // padded row of Q and K (floats)
  static constexpr int ldp = kTileKeys + 8;   // padded row of P
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

// Rows r0 to r0 + 63 of sequence b in head h, by the whole CTA.
template <int D>
__device__ __forceinline__ void prompt_unit(float* smem, const float* __restrict__ Q, const float* __restrict__ K,
                                            const float* __restrict__ V, int64_t qs, int64_t ks, int64_t vs,
                                            const int32_t* __restrict__ cu, int Hq, int Hkv, float scale_log2,
                                            float* __restrict__ O, int b, int r0, int h) {
  using S = Smem<D>;
  constexpr int NC = D / 32;   // 4-column groups of O per thread, 32 columns apart
  const int group = threadIdx.x / kGroup, tid = threadIdx.x % kGroup;
  float *sq = smem, *sk = smem + S::k + group * S::per_group, *sv = sk + S::v - S::k, *sp = sk + S::p - S::k;
  const int rg = (tid >> 5) * 16 + ((tid & 1) | ((tid >> 3) & 2)), cg = (tid >> 1) & 7;   // rows rg + 4 i, keys cg + 8 c, head dims 4 cg + 32 n ..
  auto sync_group = [&] { asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(kGroup) : "memory"); };
  const int kvh = h / (Hq / Hkv);
  const int64_t c0 = cu[b];
  const int len = cu[b + 1] - (int)c0, rows = min(kTileRows, len - r0), keys = r0 + rows;
  const int nt = (keys + kTileKeys - 1) / kTileKeys;
  const float* kp = K + c0 * ks + (size_t)kvh * D;
  const float* vp = V + c0 * vs + (size_t)kvh * D;
  load_tile<D>(sq, S::ld, Q + (c0 + r0) * qs + (size_t)h * D, qs, rows, threadIdx.x, S::threads);
  if (group < nt) load_tile<D>(sk, S::ld, kp + (int64_t)group * kTileKeys * ks, ks, keys - group * kTileKeys, tid, kGroup);
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
  __syncthreads();       // Q
  for (int j = group; j < nt; j += S::groups) {
    const int k0 = j * kTileKeys;
    cp_wait<0>();        // K_j
    sync_group();        // ... of every thread; V and P of the tile before are no longer read
    load_tile<D>(sv, D, vp + k0 * vs, vs, keys - k0, tid, kGroup);
    cp_commit();
    float2 s[4][8];   // (even, odd) head dims
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int c = 0; c < 8; ++c) s[i][c] = make_float2(0.f, 0.f);
#pragma unroll 1
    for (int d = 0; d < D; d += 4) {
      float4 a[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4*>(sq + (rg + 4 * i) * S::ld + d);
#pragma unroll
      for (int half = 0; half < 8; half += 4) {
        float4 w[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) w[c] = *reinterpret_cast<const float4*>(sk + (cg + 8 * (half + c)) * S::ld + d);
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[i][half + c] = __ffma2_rn(make_float2(a[i].x, a[i].y), make_float2(w[c].x, w[c].y), s[i][half + c]);
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[i][half + c] = __ffma2_rn(make_float2(a[i].z, a[i].w), make_float2(w[c].z, w[c].w), s[i][half + c]);
      }
    }
    sync_group();        // K_j is no longer read
    constexpr int ahead = S::groups * kTileKeys;
    if (j + S::groups < nt) load_tile<D>(sk, S::ld, kp + (int64_t)(k0 + ahead) * ks, ks, keys - k0 - ahead, tid, kGroup);
    cp_commit();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int see = r0 + rg + 4 * i - k0;   // keys 0..see of the tile are visible to the row
      float x[8], mt = -INFINITY;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        x[c] = cg + 8 * c <= see ? (s[i][c].x + s[i][c].y) * scale_log2 : -INFINITY;
        mt = fmaxf(mt, x[c]);
      }
#pragma unroll
      for (int w = 8; w > 1; w >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, w));   // the row's 8 threads
      const float mn = fmaxf(m[i], mt), mu = mn == -INFINITY ? 0.f : mn;
      const float corr = exp2f(m[i] - mu);
      m[i] = mn;
      float ps = 0.f;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const float p = exp2f(x[c] - mu);
        ps += p;
        sp[(rg + 4 * i) * S::ldp + cg + 8 * c] = p;
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
      float p[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 x = *reinterpret_cast<const float4*>(sp + (rg + 4 * i) * S::ldp + k);
        p[i][0] = x.x;
        p[i][1] = x.y;
        p[i][2] = x.z;
        p[i][3] = x.w;
      }
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int n = 0; n < NC; ++n) {
          const float4 w = *reinterpret_cast<const float4*>(sv + (k + x) * D + 32 * n + 4 * cg);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 pp = make_float2(p[i][x], p[i][x]);
            const float2 lo = __ffma2_rn(pp, make_float2(w.x, w.y), make_float2(o[i][n].x, o[i][n].y));
            const float2 hi = __ffma2_rn(pp, make_float2(w.z, w.w), make_float2(o[i][n].z, o[i][n].w));
            o[i][n] = make_float4(lo.x, lo.y, hi.x, hi.y);
          }
        }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int w = 8; w > 1; w >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], w);
  // The other groups leave their maximum, sum and O where their tiles were; group 0 merges and stores.
  if (group > 0) {
    sync_group();        // the group's last tile is no longer read
    float *so = sk, *sml = so + kTileRows * D;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = rg + 4 * i;
      if (cg == 0) {
        sml[2 * r] = m[i];
        sml[2 * r + 1] = l[i];
      }
#pragma unroll
      for (int n = 0; n < NC; ++n) *reinterpret_cast<float4*>(so + r * D + 32 * n + 4 * cg) = o[i][n];
    }
  }
  cp_wait<0>();
  __syncthreads();
  if (group > 0) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = rg + 4 * i;
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
        const float4 x = *reinterpret_cast<const float4*>(so + r * D + 32 * n + 4 * cg);
        o[i][n] = make_float4(o[i][n].x + x.x * w, o[i][n].y + x.y * w, o[i][n].z + x.z * w, o[i][n].w + x.w * w);
      }
    }
    const float inv = 1.f / sum;
    float* op = O + ((size_t)(c0 + r0 + r) * Hq + h) * D + 4 * cg;
#pragma unroll
    for (int n = 0; n < NC; ++n)
      *reinterpret_cast<float4*>(op + 32 * n) = make_float4(o[i][n].x * inv, o[i][n].y * inv, o[i][n].z * inv, o[i][n].w * inv);
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
