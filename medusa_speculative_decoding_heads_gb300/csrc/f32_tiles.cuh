// Attention of 64 query rows against tiles of 64 keys in float32 on the CUDA cores, for new tokens over a paged cache.
// The layout is that of whole prompts (prompt_f32.cu, which has its reasons and figures, and keeps code of
// its own: on these functions 8192 tokens, 8 heads of 64, took 1409 us instead of 1374).
#pragma once

#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

namespace medusa {
namespace f32 {

constexpr int kTileRows = 64, kTileKeys = 64, kGroup = 128;

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

// A thread's place: rows rg + 4 i, keys cg + 8 c, head dims 4 cg + 32 n .. of its group's tile, and what it
// holds of its rows.
template <int D>
struct Rows {
  static constexpr int NC = D / 32;   // 4-column groups of O per thread, 32 columns apart
  int group, tid, rg, cg;
  float *sq, *sk, *sv, *sp;
  float4 o[4][NC];
  float m[4], l[4];
  __device__ __forceinline__ void begin(float* smem) {
    using S = Smem<D>;
    group = threadIdx.x / kGroup;
    tid = threadIdx.x % kGroup;
    sq = smem;
    sk = smem + S::k + group * S::per_group;
    sv = sk + S::v - S::k;
    sp = sk + S::p - S::k;
    rg = (tid >> 5) * 16 + ((tid & 1) | ((tid >> 3) & 2));
    cg = (tid >> 1) & 7;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int n = 0; n < NC; ++n) o[i][n] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  __device__ __forceinline__ void sync_group() const { asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(kGroup) : "memory"); }

  // Scores of the K tile, (even, odd) head dims.
  __device__ __forceinline__ void scores(float2 (&s)[4][8]) const {
    using S = Smem<D>;
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
  }
  // The running maximum and sum, and the weights into P; see(i, key of the tile) says what is visible.
  template <typename See>
  __device__ __forceinline__ void weights(const float2 (&s)[4][8], float scale_log2, See see) {
    using S = Smem<D>;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const auto row = see(i);
      float x[8], mt = -INFINITY;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        x[c] = row(cg + 8 * c) ? (s[i][c].x + s[i][c].y) * scale_log2 : -INFINITY;
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
  }
  // O += P V.
  __device__ __forceinline__ void values() {
    using S = Smem<D>;
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
  // The groups' results joined in group 0 (whose threads get true): m, l and o of the tile's rows.
  __device__ __forceinline__ bool join(float* smem) {
    using S = Smem<D>;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int w = 8; w > 1; w >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], w);
    // The other groups leave their maximum, sum and O where their tiles were.
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
    if (group > 0) return false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = rg + 4 * i;
      float M = m[i];
      for (int g = 1; g < S::groups; ++g) M = fmaxf(M, smem[S::k + g * S::per_group + kTileRows * D + 2 * r]);
      // (a row's largest maximum is -inf only where it has seen nothing but -inf)
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
      m[i] = M;
      l[i] = sum;
    }
    return true;
  }
};

}  // namespace f32
}  // namespace medusa
