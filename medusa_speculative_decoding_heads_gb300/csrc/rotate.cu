// Norms of queries and keys, each head by itself, and their rotation by position, in one pass.
//
// y = x w / sqrt(mean(x^2) + eps); then pairs (y_u, y_v) of the first R head dims turn by the angle
// a = pos f_i: (y_u cos a - y_v sin a, y_v cos a + y_u sin a). Bound by the bytes of Q and K, read
// once and written once: 8191 tokens of 40/40 heads in bf16 59.4 to 60.1 us (5.6 TB/s, 0.83 of the measured copy).
//
// D / 8 lanes hold a head, 8 head dims each, in two pieces of 4 that lie so that both dims of a pair
// are in the same lane: R / 2 apart where halves turn against each other, next to each other where
// neighbours do. A group of such lanes takes up to H heads of one token: all of them are on their way
// while the lane works out its 4 angles, which the heads share. At most 32 blocks per SM go through the
// groups, so that what depends on a lane's frequencies alone is worked out once for several of them. (Five blocks
// are there at a time, at 88 to 91 registers. 8191 tokens of 40/40 heads in bf16 59.8 us; without a limit 63.6; with five
// 56.5, but without norms 57.5 instead of 50.9, and 57.4 instead of 50.4 in float32 with 32/8 heads.)
//
// Angles. pos f in float32 is off by 2^-25 pos f, 0.03 at a position of a million; here f / 2 pi
// becomes a 64-bit fraction of a turn, in whole numbers (off by 2^-64 of itself, and of a turn), so that
// pos times it modulo 2^64 is the remainder. Its nearest quarter turn is taken off, and the rest, |a| <=
// pi / 4, goes into the Taylor series of sine and cosine (to a^9 and a^10: off by 2e-9 and 2e-10). (The
// fraction from a product in float64, for each group: 8191 tokens of 40/40 heads 121 us.)
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "common.cuh"

namespace medusa {
namespace {

constexpr int kThreads = 128, kBlocks = 152 * 32, kFew = 152 * 64;   // kBlocks: of a grid at most; kFew: heads of a call

struct RotateArgs {
  const void *Q, *K, *qw, *kw;
  void *Qo, *Ko;
  int64_t qs, ks, qos, kos;   // elements from row to row; kos 0: the trees' staged layout
  const float* freq;
  const int32_t* pos;
  int64_t groups;             // T * (groups of a token)
  int per_token, q_groups;    // groups of a token, and how many of them are the queries'
  int Hq, Hkv, N, R, pairs;
  float eps;
};

// 4 values as they come, and unpacked.
__device__ __forceinline__ float4 get4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ uint2 get4(const uint16_t* p) { return *reinterpret_cast<const uint2*>(p); }
__device__ __forceinline__ float4 values(const float4& w) { return w; }
__device__ __forceinline__ float4 values(const uint2& w) { return make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y)); }
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void put4(float* p, const float4& v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void put4(uint16_t* p, const float4& v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack2(v.x, v.y), pack2(v.z, v.w));
}

// freq / 2 pi in 2^-64 turns, modulo a turn: freq is m 2^e, and m times 2^66 / 2 pi has 88 bits.
__device__ __forceinline__ uint64_t turns_of(float freq) {
  const uint32_t bits = __float_as_uint(freq), field = (bits >> 23) & 255u;
  const uint64_t m = (bits & 0x7fffffu) | (field ? 0x800000u : 0u), c = 0xa2f9836e4e44152aull;   // 2^66 / 2 pi
  const uint64_t lo = m * c, hi = __umul64hi(m, c);
  const int s = 152 - (int)(field ? field : 1u);   // to the right by 2 - e
  uint64_t f;
  if (s <= 0) f = s > -64 ? lo << -s : 0;
  else if (s < 64) f = lo >> s | hi << (64 - s);
  else f = s < 128 ? hi >> (s - 64) : 0;
  return bits >> 31 ? 0 - f : f;
}
// (cos, sin) of the angle of `turns` 2^-64 turns.
__device__ __forceinline__ float2 turn(uint64_t turns) {
  const int h = (int)(turns >> 32), quarter = (int)((uint32_t)h + (1u << 29)) >> 30;
  const int rest = (int)((uint32_t)h - ((uint32_t)quarter << 30));
  const float a = (float)rest * 1.4629180792671596e-9f;   // pi 2^-31
  const float s2 = a * a;
  float s = fmaf(s2, 2.7557319e-6f, -1.9841270e-4f);
  s = fmaf(s2, s, 8.3333333e-3f);
  s = fmaf(s2, s, -1.6666667e-1f);
  s = fmaf(a * s2, s, a);
  float c = fmaf(s2, -2.7557319e-7f, 2.4801587e-5f);
  c = fmaf(s2, c, -1.3888889e-3f);
  c = fmaf(s2, c, 4.1666667e-2f);
  c = fmaf(s2, c, -0.5f);
  c = fmaf(s2, c, 1.f);
  const float x = quarter & 1 ? s : c, y = quarter & 1 ? c : s;   // a quarter turn on: (c, s) -> (-s, c)
  return make_float2(((quarter + 1) & 2) ? -x : x, (quarter & 2) ? -y : y);
}

template <typename T, int D, int H>
__global__ void __launch_bounds__(kThreads)
qk_norm_rotate_kernel(const RotateArgs a) {
  constexpr int kLanes = D / 8;   // 8 or 16
  const int l = threadIdx.x % kLanes;
  pdl_wait();
  pdl_trigger();
  const unsigned mask = ((1u << kLanes) - 1u) << ((threadIdx.x & 31) / kLanes * kLanes);
  // the lane's two pieces and its frequencies
  const bool turns = 8 * l < a.R;
  const int c0 = a.pairs ? 8 * l : turns ? 4 * l : 8 * l, c1 = a.pairs || !turns ? c0 + 4 : (a.R >> 1) + 4 * l;
  uint64_t f[4];
  bool number[4] = {true, true, true, true};
  if (turns) {
    const float4 w = *reinterpret_cast<const float4*>(a.freq + 4 * l);
    const float x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = turns_of(x[i]);
      number[i] = isfinite(x[i]);
    }
  }
  // (whole groups leave the loop: the shuffles name a group's lanes only)
  for (int64_t g = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / kLanes; g < a.groups; g += (int64_t)gridDim.x * (kThreads / kLanes)) {
    const int t = (int)((uint32_t)g / (uint32_t)a.per_token), of = (int)g - t * a.per_token;   // (groups are counted in 31 bits)
    const bool isq = of < a.q_groups;
    const int h0 = (isq ? of : of - a.q_groups) * H, heads = min(H, (isq ? a.Hq : a.Hkv) - h0);
    const T* src = static_cast<const T*>(isq ? a.Q : a.K) + t * (isq ? a.qs : a.ks) + (int64_t)h0 * D;
    decltype(get4(src)) x0[H], x1[H];
#pragma unroll
    for (int i = 0; i < H; ++i)
      if (i < heads) {
        x0[i] = get4(src + i * D + c0);
        x1[i] = get4(src + i * D + c1);
      }
    const T* w = static_cast<const T*>(isq ? a.qw : a.kw);
    float4 w0, w1;
    if (w) {
      w0 = values(get4(w + c0));
      w1 = values(get4(w + c1));
    }
    float2 cs[4];
    if (turns) {
      const uint64_t pos = (uint64_t)(int64_t)a.pos[t];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        cs[i] = turn(f[i] * pos);
        if (!number[i]) cs[i] = make_float2(NAN, NAN);
      }
    }
    T* dst;
    int64_t step = D;
    if (isq) {
      dst = static_cast<T*>(a.Qo) + t * a.qos + (int64_t)h0 * D;
    } else if (a.kos) {
      dst = static_cast<T*>(a.Ko) + t * a.kos + (int64_t)h0 * D;
    } else {
      const int64_t b = t / a.N;
      dst = static_cast<T*>(a.Ko) + ((b * a.Hkv + h0) * a.N + (t - b * a.N)) * D;
      step = (int64_t)a.N * D;
    }
#pragma unroll
    for (int i = 0; i < H; ++i) {
      if (i >= heads) break;
      float4 u = values(x0[i]), v = values(x1[i]);
      if (w) {
        float s = u.x * u.x;
        s = fmaf(u.y, u.y, s);
        s = fmaf(u.z, u.z, s);
        s = fmaf(u.w, u.w, s);
        s = fmaf(v.x, v.x, s);
        s = fmaf(v.y, v.y, s);
        s = fmaf(v.z, v.z, s);
        s = fmaf(v.w, v.w, s);
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) s += __shfl_xor_sync(mask, s, o);
        const float r = rsqrtf(fmaf(s, 1.f / D, a.eps));
        u = make_float4(u.x * r * w0.x, u.y * r * w0.y, u.z * r * w0.z, u.w * r * w0.w);
        v = make_float4(v.x * r * w1.x, v.y * r * w1.y, v.z * r * w1.z, v.w * r * w1.w);
      }
      if (turns) {
        auto both = [](float& p, float& q, const float2& c) {
          const float x = p * c.x - q * c.y;
          q = q * c.x + p * c.y;
          p = x;
        };
        if (a.pairs) {
          both(u.x, u.y, cs[0]);
          both(u.z, u.w, cs[1]);
          both(v.x, v.y, cs[2]);
          both(v.z, v.w, cs[3]);
        } else {
          both(u.x, v.x, cs[0]);
          both(u.y, v.y, cs[1]);
          both(u.z, v.z, cs[2]);
          both(u.w, v.w, cs[3]);
        }
      }
      put4(dst + i * step + c0, u);
      put4(dst + i * step + c1, v);
    }
  }
}

template <typename T, int D, int H>
cudaError_t run(const medusa_cfg& c, RotateArgs a, int T_, cudaStream_t st) {
  a.q_groups = (c.Hq + H - 1) / H;
  a.per_token = a.q_groups + (c.Hkv + H - 1) / H;
  a.groups = (int64_t)T_ * a.per_token;
  constexpr int per_block = kThreads * 8 / D;
  const int64_t blocks = (a.groups + per_block - 1) / per_block;
  const cudaError_t e = launch_pdl(qk_norm_rotate_kernel<T, D, H>, (unsigned)(blocks < kBlocks ? blocks : kBlocks), kThreads, 0, st, a);
  note_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}
template <typename T, int H>
cudaError_t run(const medusa_cfg& c, const RotateArgs& a, int T_, cudaStream_t st) {
  return c.D == 64 ? run<T, 64, H>(c, a, T_, st) : run<T, 128, H>(c, a, T_, st);
}

}  // namespace

cudaError_t launch_qk_norm_rotate(const medusa_cfg& c, const void* Q, const void* K, int T, int64_t q_stride, int64_t k_stride,
                                  const void* q_weight, const void* k_weight, float eps, const float* inv_freq, int rot_dim,
                                  int pairing, const int32_t* pos, void* Qo, void* Ko, int64_t qo_stride, int64_t ko_stride,
                                  cudaStream_t st) {
  RotateArgs a{};
  a.Q = Q;
  a.K = K;
  a.qw = q_weight;
  a.kw = k_weight;
  a.Qo = Qo;
  a.Ko = Ko;
  a.qs = q_stride;
  a.ks = k_stride;
  a.qos = qo_stride;
  a.kos = ko_stride;
  a.freq = inv_freq;
  a.pos = pos;
  a.Hq = c.Hq;
  a.Hkv = c.Hkv;
  a.N = tree_shape(c).N;
  a.R = rot_dim;
  a.pairs = pairing == MEDUSA_ROTATE_PAIRS;
  a.eps = eps;
  // Two heads to a group while the SMs hold all such groups at once (a shorter chain in each), more beyond, which
  // share their angles: one token of 32/8 heads 2.3 us so and 3.4 with eight, 64 tokens of 40/40 2.8 and 3.7;
  // 700 tokens 9.0 and 7.7, 8191 74 and 59.4 (four: 59.7).
  const bool few = (int64_t)T * (c.Hq + c.Hkv) <= kFew;
  if (c.dtype == MEDUSA_F32) return few ? run<float, 2>(c, a, T, st) : run<float, 4>(c, a, T, st);
  return few ? run<uint16_t, 2>(c, a, T, st) : run<uint16_t, 8>(c, a, T, st);
}

}  // namespace medusa
