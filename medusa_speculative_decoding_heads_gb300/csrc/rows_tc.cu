// Attention of packed query rows on 5th-generation tensor cores (tcgen05, TMEM
// accumulators, TMA), bf16 with D = 128: whole prompts (causal), and tree attention
// behind a prefix that the batch shares.
//
// O = softmax(Q K^T / sqrt(D)) V in one pass over the keys, with the running maximum and
// sum of "최적화 2편" (beengineer500), section 3.3. 4 rows keys D operations against
// 2 keys D elements of K and V per 256 rows: bound by the tensor cores and, beside them,
// by the exponentials, as long as there are rows; by the K/V bytes for a few single tokens.
//
// A unit of work is 256 query rows of one KV head (two tiles of 128) against a range of
// keys. A tile's rows are Gp query heads of the KV head's group times 128 / Gp positions
// (Gp: the largest power of two that divides the group, at most 16), so that one TMA box
// loads it and the heads share every K/V tile. 12 warps, one CTA per SM, which walks
// units u = blockIdx.x, + gridDim.x, ...:
//   warps 0-3, 4-7  softmax of tile 0 and of tile 1: thread = row = TMEM lane; S (f32) to
//                   registers, mask, maximum, 2^(s - m) rounded to bf16 back over S, sums
//                   in f32. O is rescaled only when the maximum rises by more than 2^8.
//   warp 8          issues every MMA: S_t(j) = Q_t K_j^T (both operands in shared memory)
//                   and O_t += P_t(j) V_j (P from TMEM), so that one tile's products run
//                   while the other tile's softmax does. MMAs of one issuing thread run in
//                   order: S_t(j + 1), which overwrites P_t(j), follows O_t += P_t(j) V_j.
//   warp 9          TMA: Q tiles, then K and V tiles of 128 keys alternating through one
//                   5-stage ring. V rows past the last key that may be read are zeroed in
//                   shared memory (0 x NaN must not reach a result).
//   warp 10         the schedule: decodes the next unit while the others work on this one.
// TMEM: S_0, S_1, O_0, O_1 (128 columns each). Every mbarrier wait is bounded.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <mutex>

#include "common.cuh"
#include "tc_common.cuh"

namespace medusa {

__device__ uint32_t g_rows_tc_error = 0;

namespace {

constexpr int kD = 128, kRows = 128, kKeys = 128;
constexpr int kHalf = 128 * 128;            // 128 rows x 64 bf16, 128-byte swizzle: half a tile (16 KB)
constexpr int kTile = 2 * kHalf;            // 128 x 128 bf16 (32 KB)
constexpr int kStages = 5;                  // K/V ring
constexpr int kOffRing = 2 * kTile;         // behind the two Q tiles
constexpr int kSmem = kOffRing + kStages * kTile + 1024;   // + alignment slack
constexpr int kMmaWarp = 8, kLoadWarp = 9, kPlanWarp = 10;
constexpr int kThreads = 384;
constexpr uint32_t kTmemCols = 512;
constexpr int kSms = 152;
// The running maximum moves (and O is rescaled) only when a tile's maximum exceeds it by more
// than this many binary orders of magnitude: weights stay below 2^8, far inside bf16 and f32.
constexpr float kLazy = 8.f;

__host__ __device__ constexpr uint32_t col_S(int t) { return 128u * t; }
__host__ __device__ constexpr uint32_t col_O(int t) { return 256u + 128u * t; }

struct RowsArgs {
  const int32_t* cu;       // prompts: [B + 1]
  const int32_t* L;        // prefix: [B]
  const uint64_t* bits;    // prefix: [N][2]
  const int32_t* prefix;   // prefix: pages of the shared rows
  const int32_t* table;    // prefix: [B][max_pages]
  int B, N, T;             // T: rows of Q (prefix: B * N)
  int Hq, Hkv, gp_shift;   // log2 of Gp
  int L_cap, page_rows, max_pages, num_pages, shared;
  int splits_s, chunk_s, splits_u, chunk_u;   // key splits of the shared and of the own rows
  float scale_log2;
  uint16_t* O;             // prompts
  float* o_part;           // prefix: [split][row][D], row = position * Hq + head
  float* ml_part;          // prefix: [split][row][2]
};

enum UnitKind : int { kEnd = 0, kPrompt = 1, kShared = 2, kOwn = 3 };

// What the scheduling warp hands to the others.
struct Unit {
  int kind;
  int pos0;      // Q row (position) of tile 0's first row; tile 1 begins 128 / Gp later
  int left;      // positions from pos0 on that exist
  int h0, kvh;   // first query head, KV head
  int n0, n1;    // key tiles of tile 0 and tile 1 (the tree tile included)
  int k0, kend;  // key range
  int base;      // prompts: packed row of the sequence's row 0; prefix: the sequence
  int tree;      // number of the tree tile, or -1
  int part;      // prefix: split the partial result belongs to
};

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          tc::saddr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(tc::saddr(bar))
      : "memory");
}

// Walks the prompts' units, those with the most keys first: by tile number from the last one
// down, then by sequence. A whole warp calls it; units must be asked for in ascending order.
struct PromptWalk {
  int t = -1, before = 0, count = 0;   // units of tile number t follow `before` earlier ones

  static __device__ __forceinline__ int tiles(const RowsArgs& a, int b, int per) {
    if (b >= a.B) return 0;
    const int c0 = a.cu[b], c1 = a.cu[b + 1];
    return (c0 >= 0 && c1 >= c0 && c1 <= a.T) ? (int)(((int64_t)(c1 - c0) + per - 1) / per) : 0;
  }
  __device__ int above(const RowsArgs& a, int per) const {   // sequences with more than t tiles
    int c = 0;
    for (int b = threadIdx.x & 31; b < a.B; b += 32) c += tiles(a, b, per) > t;
    return __reduce_add_sync(0xffffffffu, c);
  }
  __device__ void begin(const RowsArgs& a, int per) {
    int most = 0;
    for (int b = threadIdx.x & 31; b < a.B; b += 32) most = max(most, tiles(a, b, per));
    t = __reduce_max_sync(0xffffffffu, most) - 1;
    count = t >= 0 ? above(a, per) : 0;
  }
  // Sequence of unit u's rows (and t: its tile number), or -1 past the last unit.
  __device__ int find(const RowsArgs& a, int per, int u) {
    while (t >= 0 && u >= before + count) {
      before += count;
      --t;
      count = t >= 0 ? above(a, per) : 0;
    }
    if (t < 0) return -1;
    int rank = u - before;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      const unsigned votes = __ballot_sync(0xffffffffu, tiles(a, b0 + (threadIdx.x & 31), per) > t);
      const int c = __popc(votes);
      if (rank < c) return b0 + (int)__fns(votes, 0, rank + 1);
      rank -= c;
    }
    return -1;
  }
};

template <bool kPrefix>
__device__ Unit decode(const RowsArgs& a, PromptWalk& walk, int u) {
  Unit w;
  const int npos = kRows >> a.gp_shift, per = 2 * npos;   // positions of a tile, of a unit
  const int G = a.Hq / a.Hkv, HG = a.Hq >> a.gp_shift;
  w.kind = kEnd;
  w.tree = -1;
  w.part = 0;
  if (!kPrefix) {
    const int b = walk.find(a, per, u / HG);
    if (b < 0) return w;
    const int c0 = a.cu[b], len = a.cu[b + 1] - c0, i0 = walk.t * per;
    w.kind = kPrompt;
    w.pos0 = c0 + i0;
    w.left = len - i0;
    w.h0 = (u % HG) << a.gp_shift;
    w.k0 = 0;
    w.kend = len;
    w.base = c0;
    w.n0 = (min(len, i0 + npos) + kKeys - 1) / kKeys;
    w.n1 = w.left > npos ? (min(len, i0 + per) + kKeys - 1) / kKeys : 0;
  } else {
    const int rows = a.T, ru = (rows + per - 1) / per, us = a.splits_s * HG * ru;
    const int nu = (a.N + per - 1) / per;
    if (u < us) {   // shared rows: all positions of the batch
      const int r = u / ru, split = r / HG;
      w.kind = kShared;
      w.pos0 = (u % ru) * per;
      w.left = rows - w.pos0;
      w.h0 = (r % HG) << a.gp_shift;
      w.k0 = split * a.chunk_s;
      w.kend = min(a.shared, w.k0 + a.chunk_s);
      w.base = 0;
      w.part = split;
      w.n0 = (w.kend - w.k0) / kKeys;
    } else {        // a sequence's own rows and tree
      const int v = u - us, r = v / nu, hb = r / HG, b = hb % a.B, split = hb / a.B;
      if (split >= a.splits_u) return w;
      const int Lb = a.L[b];
      const bool ok = Lb >= 0 && Lb <= a.L_cap - a.N;
      const int node0 = (v % nu) * per;
      w.kind = kOwn;
      w.pos0 = b * a.N + node0;
      w.left = a.N - node0;
      w.h0 = (r % HG) << a.gp_shift;
      w.k0 = a.shared + split * a.chunk_u;
      w.kend = ok ? min(Lb, w.k0 + a.chunk_u) : 0;
      w.base = b;
      w.part = a.splits_s + split;
      w.n0 = w.kend > w.k0 ? (w.kend - w.k0 + kKeys - 1) / kKeys : 0;
      if (ok && split == a.splits_u - 1) w.tree = w.n0++;
    }
    w.n1 = w.left > npos ? w.n0 : 0;
  }
  w.kvh = w.h0 / G;
  return w;
}

template <bool kPrefix>
__global__ void __launch_bounds__(kThreads, 1)
rows_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
               const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmKt,
               const __grid_constant__ CUtensorMap tmVt, const __grid_constant__ RowsArgs a) {
  pdl_trigger();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = sm + kOffRing;
  __shared__ __align__(8) uint64_t kv_full[kStages], kv_empty[kStages];
  __shared__ __align__(8) uint64_t q_full[2], q_empty[2], s_full[2], p_full[2], o_done[2];
  __shared__ __align__(8) uint64_t unit_full[2], unit_empty[2], tail;
  __shared__ Unit units[2];
  __shared__ uint32_t tmem_slot;
  uint32_t* err = &g_rows_tc_error;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      tc::mbar_init(&kv_full[i], 1);
      tc::mbar_init(&kv_empty[i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      tc::mbar_init(&q_full[t], 1);
      tc::mbar_init(&q_empty[t], 1);
      tc::mbar_init(&s_full[t], 1);
      tc::mbar_init(&p_full[t], kRows);
      tc::mbar_init(&o_done[t], 1);
      tc::mbar_init(&unit_full[t], 1);
      tc::mbar_init(&unit_empty[t], 10);   // 8 softmax warps, the MMA warp, the load warp
    }
    tc::mbar_init(&tail, 1);
    tc::mbar_fence_init();
  }
  if (warp == kMmaWarp) tc::tmem_alloc(&tmem_slot, kTmemCols);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  pdl_wait();   // lengths, tables and the rows themselves are visible from here on
  const uint32_t tmem = tmem_slot;
  const int npos = kRows >> a.gp_shift;

  // The next unit from the schedule: false when a wait ran out. The warp's lane 0 gives the
  // slot back once every lane has its copy.
  auto next_unit = [&](int i, Unit& w) {
    if (!__all_sync(0xffffffffu, tc::mbar_wait(&unit_full[i & 1], (i >> 1) & 1, err, 1))) return false;
    w = units[i & 1];
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&unit_empty[i & 1]);
    return w.kind != kEnd;
  };

  if (warp == kPlanWarp) {
    // ------------------------------------------------------------------ schedule
    PromptWalk walk;
    if (!kPrefix) walk.begin(a, 2 * npos);
    for (int i = 0;; ++i) {
      const Unit w = decode<kPrefix>(a, walk, (int)blockIdx.x + i * (int)gridDim.x);
      if (i >= 2 && !__all_sync(0xffffffffu, tc::mbar_wait(&unit_empty[i & 1], ((i >> 1) - 1) & 1, err, 2))) break;
      if (lane == 0) {
        units[i & 1] = w;
        tc::mbar_arrive(&unit_full[i & 1]);
      }
      __syncwarp();
      if (w.kind == kEnd) break;
    }
  } else if (warp == kLoadWarp) {
    // ------------------------------------------------------------------ TMA loads
    Unit w;
    int it = 0, nq[2] = {0, 0}, fixes = 0;   // ring position, Q tiles loaded, tails zeroed
    bool ok = true;
    for (int i = 0; ok && next_unit(i, w); ++i) {
      const int nt = max(w.n0, w.n1);
      int page_reg = 0;
      for (int s = 0; ok && s < 2 * nt; ++s) {   // K_0, V_0, K_1, V_1, ...
        const int j = s >> 1;
        const bool isv = s & 1;
        if (s < 2 && (s == 0 ? w.n0 : w.n1) > 0) {   // Q tile s, ahead of its first use
          if (nq[s] > 0) ok = __all_sync(0xffffffffu, tc::mbar_wait(&q_empty[s], (nq[s] - 1) & 1, err, 4));
          if (!ok) break;
          if (lane == 0) {
            uint8_t* dst = sm + s * kTile;
            tc::mbar_arrive_expect(&q_full[s], kTile);
            tma_load_3d(dst, &tmQ, 0, w.pos0 + s * npos, w.h0, &q_full[s]);
            tma_load_3d(dst + kHalf, &tmQ, 64, w.pos0 + s * npos, w.h0, &q_full[s]);
          }
          ++nq[s];
        }
        const int st = it % kStages;
        if (it >= kStages) ok = __all_sync(0xffffffffu, tc::mbar_wait<true>(&kv_empty[st], (it / kStages - 1) & 1, err, 8));
        if (!ok) break;
        const bool tree = kPrefix && j == w.tree;
        const int key0 = w.k0 + j * kKeys;
        int y, z;
        if (!kPrefix) {
          y = w.base + key0;
          z = w.kvh;
        } else if (tree) {
          y = 0;
          z = w.base * a.Hkv + w.kvh;
        } else {
          if (!isv && (j & 31) == 0) {   // 32 tiles' pages at a time, one per lane
            const int key = w.k0 + (j + lane) * kKeys;
            page_reg = -1;
            if (key < w.kend)
              page_reg = w.kind == kShared ? a.prefix[key / a.page_rows]
                                           : a.table[(size_t)w.base * a.max_pages + key / a.page_rows];
          }
          const int page = __shfl_sync(0xffffffffu, page_reg, j & 31);
          const bool in_pool = page >= 0 && page < a.num_pages;
          MEDUSA_CHECK(isv || lane != 0 || in_pool, MEDUSA_CHECK_PAGE);
          y = key0 % a.page_rows;
          z = (in_pool ? page : a.num_pages) * a.Hkv + w.kvh;   // outside the pool: TMA fills zeros
        }
        const CUtensorMap* m = tree ? (isv ? &tmVt : &tmKt) : (isv ? &tmV : &tmK);
        uint8_t* dst = ring + st * kTile;
        const int live = tree ? kKeys : min(kKeys, w.kend - key0);   // (rows past the tree's nodes arrive as zeros)
        const bool fix = isv && live < kKeys;
        uint64_t* bar = fix ? &tail : &kv_full[st];
        if (lane == 0) {
          tc::mbar_arrive_expect(bar, kTile);
          tma_load_3d(dst, m, 0, y, z, bar);
          tma_load_3d(dst + kHalf, m, 64, y, z, bar);
        }
        __syncwarp();
        if (fix) {   // rows [live, 128) of both halves become zero before the MMA warp may see the tile
          ok = __all_sync(0xffffffffu, tc::mbar_wait<true>(&tail, fixes & 1, err, 16));
          ++fixes;
          if (!ok) break;
          for (int c = live * 8 + lane; c < kKeys * 8; c += 32) {
            reinterpret_cast<uint4*>(dst)[c] = make_uint4(0, 0, 0, 0);
            reinterpret_cast<uint4*>(dst + kHalf)[c] = make_uint4(0, 0, 0, 0);
          }
          tc::fence_proxy_async();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&kv_full[st]);
        }
        ++it;
      }
    }
    // never leave with copies still landing in shared memory
    for (int x = it > kStages ? it - kStages : 0; x < it; ++x) tc::mbar_wait(&kv_full[x % kStages], (x / kStages) & 1, err, 32);
    for (int t = 0; t < 2; ++t)
      if (nq[t] > 0) tc::mbar_wait(&q_full[t], (nq[t] - 1) & 1, err, 64);
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------------ MMA issue
    // The whole warp walks the schedule; one elected lane issues.
    constexpr uint32_t idS = tc::idesc_bf16_f32(kRows, kKeys, 0, 0);
    constexpr uint32_t idPV = tc::idesc_bf16_f32(kRows, kD, 0, 1);
    const uint64_t dQ = tc::sw128_desc(tc::saddr(sm), 16, 1024);
    const uint64_t dK = tc::sw128_desc(tc::saddr(ring), 16, 1024);
    const uint64_t dV = tc::sw128_desc(tc::saddr(ring), kHalf, 1024);   // MN-major: LBO = the 64-column half
    Unit w;
    int it = 0, nq[2] = {0, 0}, np[2] = {0, 0};   // ring position, Q tiles used, P tiles used
    bool ok = true;
    auto wait_kv = [&](int x) {
      return __all_sync(0xffffffffu, tc::mbar_wait<true>(&kv_full[x % kStages], (x / kStages) & 1, err, 128));
    };
    // S_t = Q_t K^T with the K tile at ring position x; `last`: Q_t is not needed any more
    auto issue_S = [&](int t, int x, bool last) {
      tc::fence_after();
      if (tc::elect_one()) {
        const uint64_t q0 = dQ + (uint64_t)((t * kTile) >> 4), b0 = dK + (uint64_t)(((x % kStages) * kTile) >> 4);
#pragma unroll
        for (int kk = 0; kk < kD / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
          tc::mma_bf16(tmem + col_S(t), q0 + off, b0 + off, idS, kk > 0);
        }
        tc::commit(&s_full[t]);
        if (last) tc::commit(&q_empty[t]);
      }
      __syncwarp();
    };
    // O_t (+)= P_t V with the V tile at ring position x
    auto issue_PV = [&](int t, int x, bool first) {
      tc::fence_after();
      if (tc::elect_one()) {
        const uint64_t b0 = dV + (uint64_t)(((x % kStages) * kTile) >> 4);
#pragma unroll
        for (int kk = 0; kk < kKeys / 16; ++kk)   // keys [16 kk, 16 kk + 16): P columns 32 (kk / 2) + 8 (kk % 2)
          tc::mma_bf16_tmem_a(tmem + col_O(t), tmem + col_S(t) + 32 * (kk >> 1) + 8 * (kk & 1),
                              b0 + (uint64_t)((kk * 2048) >> 4), idPV, (!first || kk > 0) ? 1 : 0);
        tc::commit(&o_done[t]);
      }
      __syncwarp();
    };
    auto release = [&](int x) {   // the stage is free once everything issued so far has read it
      if (tc::elect_one()) tc::commit(&kv_empty[x % kStages]);
      __syncwarp();
    };
    for (int i = 0; ok && next_unit(i, w); ++i) {
      const int n[2] = {w.n0, w.n1}, nt = max(w.n0, w.n1);
      if (nt == 0) continue;
      ok = wait_kv(it);
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (ok && n[t] > 0) {
          ok = __all_sync(0xffffffffu, tc::mbar_wait<true>(&q_full[t], nq[t] & 1, err, 256));
          ++nq[t];
          if (ok) issue_S(t, it, n[t] == 1);
        }
      }
      if (!ok) break;
      release(it);
      for (int j = 0; ok && j < nt; ++j) {
        const int xv = it + 2 * j + 1, xk = xv + 1;
        ok = wait_kv(xv);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (ok && j < n[t]) {
            ok = __all_sync(0xffffffffu, tc::mbar_wait<true>(&p_full[t], np[t] & 1, err, 512));
            ++np[t];
            if (ok) issue_PV(t, xv, j == 0);
            if (ok && j + 1 < n[t]) {
              ok = wait_kv(xk);
              if (ok) issue_S(t, xk, j + 2 == n[t]);
            }
          }
        }
        if (!ok) break;
        release(xv);
        if (j + 1 < nt) release(xk);
      }
      it += 2 * nt;
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------------ softmax
    const int t = warp >> 2, row = 32 * (warp & 3) + lane;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t tS = tmem + col_S(t) + lanes, tO = tmem + col_O(t) + lanes;
    const int rpos = t * npos + (row & (npos - 1)), rhead = row >> (7 - a.gp_shift);
    Unit w;
    int ns = 0;   // S tiles taken
    bool ok = true;
    for (int i = 0; ok && next_unit(i, w); ++i) {
      const int n = t ? w.n1 : w.n0;
      const bool row_ok = rpos < w.left;
      const int pos = w.pos0 + rpos, head = w.h0 + rhead;
      // keys below `limit` are visible to this row
      int limit = w.kend;
      uint64_t word0 = 0, word1 = 0;
      if (!kPrefix) {
        limit = pos - w.base + 1;
      } else if (row_ok) {
        const int b = pos / a.N;
        if (w.kind == kShared) {
          const int Lb = a.L[b];
          limit = (Lb >= 0 && Lb <= a.L_cap - a.N) ? min(Lb, w.kend) : 0;
        } else if (w.tree >= 0) {
          word0 = a.bits[2 * (pos - b * a.N)];
          word1 = a.bits[2 * (pos - b * a.N) + 1];
        }
      }
      const bool busy = __any_sync(0xffffffffu, row_ok);   // a warp without rows only keeps the pace
      float m_run = -INFINITY, l_run = 0.f;
      for (int j = 0; j < n; ++j, ++ns) {
        ok = __all_sync(0xffffffffu, tc::mbar_wait(&s_full[t], ns & 1, err, 1024));
        if (!ok) break;
        if (busy) {
          tc::fence_after();
          uint32_t v[128];
#pragma unroll
          for (int c = 0; c < 4; ++c) tc::tmem_ld32(tS + 32 * c, v + 32 * c);
          tc::tmem_wait_ld();
          if (kPrefix && j == w.tree) {
#pragma unroll
            for (int c = 0; c < 128; ++c)
              if (!(((c < 64 ? word0 : word1) >> (c & 63)) & 1ull)) v[c] = __float_as_uint(-INFINITY);
          } else {
            const int vis = limit - (w.k0 + j * kKeys);
            if (__any_sync(0xffffffffu, vis < kKeys)) {
#pragma unroll
              for (int c = 0; c < 128; ++c)
                if (c >= vis) v[c] = __float_as_uint(-INFINITY);
            }
          }
          float m4[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float m = __uint_as_float(v[32 * c]);
#pragma unroll
            for (int x = 1; x < 31; x += 2) m = max3(m, __uint_as_float(v[32 * c + x]), __uint_as_float(v[32 * c + x + 1]));
            m4[c] = fmaxf(m, __uint_as_float(v[32 * c + 31]));
          }
          const float m_tile = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * a.scale_log2;
          float corr = 1.f;
          if (m_tile > m_run + kLazy) {   // also on the first visible tile (m_run = -inf): corr = 0
            corr = tc::ex2(m_run - m_tile);
            m_run = m_tile;
          }
          const float neg_m = m_run == -INFINITY ? 0.f : -m_run;
          const float2 sc = make_float2(a.scale_log2, a.scale_log2), nm = make_float2(neg_m, neg_m);
          float2 acc0 = make_float2(0.f, 0.f), acc1 = make_float2(0.f, 0.f);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t pk[16];
#pragma unroll
            for (int x = 0; x < 16; ++x) {
              const float2 e = __ffma2_rn(make_float2(__uint_as_float(v[32 * c + 2 * x]), __uint_as_float(v[32 * c + 2 * x + 1])),
                                          sc, nm);
              float2 p;
              p.x = tc::ex2(e.x);
              p.y = tc::ex2(e.y);
              if (x & 1)
                acc1 = __fadd2_rn(acc1, p);
              else
                acc0 = __fadd2_rn(acc0, p);
              pk[x] = pack_bf16x2(p.x, p.y);
            }
            tc::tmem_st16(tS + 32 * c, pk);   // P of keys [32 c, 32 c + 32) over the first half of their scores
          }
          const float2 s2 = __fadd2_rn(acc0, acc1);
          l_run = l_run * corr + (s2.x + s2.y);
          if (j > 0 && __any_sync(0xffffffffu, corr != 1.f)) {
            // O += P_{j-1} V_{j-1} was issued before S_j and has landed with it
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t o[32];
              tc::tmem_ld32(tO + 32 * c, o);
              tc::tmem_wait_ld();
#pragma unroll
              for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * corr);
              tc::tmem_st32(tO + 32 * c, o);
            }
          }
          tc::tmem_wait_st();
          tc::fence_before();
        }
        tc::mbar_arrive(&p_full[t]);
      }
      if (!ok) break;
      if (n > 0) {
        ok = __all_sync(0xffffffffu, tc::mbar_wait(&o_done[t], (ns - 1) & 1, err, 2048));
        if (!ok) break;
        tc::fence_after();
      }
      if (!busy) continue;
      const size_t orow = (size_t)pos * a.Hq + head;
      if (!kPrefix) {
        const float inv = l_run > 0.f ? 1.f / l_run : l_run;   // (a NaN sum stays NaN)
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t o[32];
          tc::tmem_ld32(tO + 32 * c, o);
          tc::tmem_wait_ld();
          if (row_ok) {
            uint4* op = reinterpret_cast<uint4*>(a.O + orow * kD + 32 * c);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              uint32_t pk[4];
#pragma unroll
              for (int y = 0; y < 4; ++y)
                pk[y] = pack_bf16x2(__uint_as_float(o[8 * x + 2 * y]) * inv, __uint_as_float(o[8 * x + 2 * y + 1]) * inv);
              op[x] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
            }
          }
        }
      } else {
        const size_t prow = (size_t)w.part * a.T * a.Hq + orow;
        if (n > 0) {
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t o[32];
            tc::tmem_ld32(tO + 32 * c, o);
            tc::tmem_wait_ld();
            if (row_ok) {
              uint4* op = reinterpret_cast<uint4*>(a.o_part + prow * kD + 32 * c);
#pragma unroll
              for (int x = 0; x < 8; ++x) op[x] = make_uint4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
            }
          }
        }
        if (row_ok) {
          a.ml_part[2 * prow] = m_run;
          a.ml_part[2 * prow + 1] = l_run;
        }
      }
      tc::fence_before();   // O has been read before the next unit's first P is announced
    }
  }

  tc::fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::fence_after();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

// O = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s over the splits; one warp per output row.
__global__ void __launch_bounds__(256)
rows_merge_kernel(const float* __restrict__ o_part, const float* __restrict__ ml_part, int64_t rows, int splits,
                  uint16_t* __restrict__ O) {
  pdl_wait();
  pdl_trigger();
  const int64_t row = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (row >= rows) return;
  float M = -INFINITY;
  for (int s = 0; s < splits; ++s) M = fmaxf(M, ml_part[2 * (s * rows + row)]);
  float l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s = 0; s < splits; ++s) {
    const float m = ml_part[2 * (s * rows + row)], ls = ml_part[2 * (s * rows + row) + 1];
    if (m == -INFINITY && ls == 0.f) continue;   // nothing was visible: its O need not have been written
    const float wgt = exp2f(m - M);
    const float4 o = *reinterpret_cast<const float4*>(o_part + (s * rows + row) * kD + 4 * lane);
    l += wgt * ls;
    acc.x += wgt * o.x;
    acc.y += wgt * o.y;
    acc.z += wgt * o.z;
    acc.w += wgt * o.w;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  *reinterpret_cast<uint2*>(O + row * kD + 4 * lane) =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
}

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

// [planes][rows][128] bf16, boxes of 64 columns, `box_rows` rows and `box_planes` planes.
bool encode_3d(CUtensorMap* map, const void* base, uint64_t rows, uint64_t planes, uint64_t row_bytes, uint64_t plane_bytes,
               uint32_t box_rows, uint32_t box_planes) {
  std::call_once(g_encode_once, [] {
    cudaDriverEntryPointQueryResult q;
    void* fn = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  if (!g_encode) return false;
  cuuint64_t dims[3] = {(cuuint64_t)kD, rows, planes};
  cuuint64_t strides[2] = {row_bytes, plane_bytes};
  cuuint32_t box[3] = {64, box_rows, box_planes};
  cuuint32_t estr[3] = {1, 1, 1};
  return g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// log2 of the query heads that share a tile: the largest power of two dividing the group, at most 16
// (8 positions: whole 8-row groups of the swizzled layout).
int gp_shift_of(int G) {
  int s = 0;
  while (s < 4 && G % (2 << s) == 0) ++s;
  return s;
}

// How the key ranges are split: while all units fit one wave, one CTA per SM.
struct PrefixPlan {
  int gp_shift, splits_s, chunk_s, splits_u, chunk_u;
  size_t o_part, ml_part, total;
};
PrefixPlan plan_prefix(const medusa_cfg& c, int shared) {
  PrefixPlan p{};
  const TreeShape ts = tree_shape(c);
  p.gp_shift = gp_shift_of(c.Hq / c.Hkv);
  const int per = 2 * (kRows >> p.gp_shift), HG = c.Hq >> p.gp_shift;
  const int64_t us = (((int64_t)c.B * ts.N + per - 1) / per) * HG, uo = (int64_t)c.B * HG * ((ts.N + per - 1) / per);
  auto split = [](int64_t units, int64_t keys, int* splits, int* chunk) {
    int64_t want = kSms / units, most = (keys + 255) / 256;   // at least two tiles each
    if (want > most) want = most;
    if (want > 32) want = 32;
    if (want < 1) want = 1;
    *chunk = (int)(keys > 0 ? ((keys + want - 1) / want + kKeys - 1) / kKeys * kKeys : kKeys);
    *splits = (int)(keys > 0 ? (keys + *chunk - 1) / *chunk : 1);
  };
  split(us, shared, &p.splits_s, &p.chunk_s);
  if (shared == 0) p.splits_s = 0;
  const int own = c.L_cap - ts.N - shared;
  split(uo, own > 0 ? own : 0, &p.splits_u, &p.chunk_u);
  const size_t rows = (size_t)c.B * ts.N * c.Hq, parts = p.splits_s + p.splits_u;
  p.ml_part = align_up(parts * rows * kD * 4, 256);
  p.total = p.ml_part + align_up(parts * rows * 8, 256);
  return p;
}

template <bool kPrefix>
cudaError_t launch_rows(const CUtensorMap* m, const RowsArgs& a, int64_t units, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(rows_tc_kernel<kPrefix>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(rows_tc_kernel<kPrefix>, (unsigned)(units < kSms ? units : kSms), kThreads, kSmem, st, m[0], m[1], m[2], m[3],
                 m[4], a);
  note_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

MEDUSA_CHECK_TAKE(rows_tc_take_checks)

cudaError_t rows_tc_take_error(uint32_t* out, cudaStream_t st) {
  static const uint32_t zero = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(out, g_rows_tc_error, sizeof(uint32_t), 0, cudaMemcpyDeviceToHost, st);
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbolAsync(g_rows_tc_error, &zero, sizeof(uint32_t), 0, cudaMemcpyHostToDevice, st);
}

cudaError_t launch_prompt_tc(const medusa_cfg& c, const void* Q, const void* K, const void* V, int T, int64_t q_stride,
                             int64_t k_stride, int64_t v_stride, const int32_t* cu, void* O, cudaStream_t st) {
  RowsArgs a{};
  a.cu = cu;
  a.B = c.B;
  a.T = T;
  a.Hq = c.Hq;
  a.Hkv = c.Hkv;
  a.gp_shift = gp_shift_of(c.Hq / c.Hkv);
  a.scale_log2 = (float)(1.4426950408889634 / sqrt((double)kD));
  a.O = static_cast<uint16_t*>(O);
  const int npos = kRows >> a.gp_shift;
  CUtensorMap m[5];
  if (!encode_3d(&m[0], Q, T, c.Hq, q_stride * 2, kD * 2, npos, 1u << a.gp_shift) ||
      !encode_3d(&m[1], K, T, c.Hkv, k_stride * 2, kD * 2, kKeys, 1) ||
      !encode_3d(&m[2], V, T, c.Hkv, v_stride * 2, kD * 2, kKeys, 1))
    return cudaErrorInvalidValue;
  m[3] = m[1];
  m[4] = m[2];
  const int64_t units = ((int64_t)T / (2 * npos) + c.B) * (c.Hq >> a.gp_shift);   // at least as many as there are
  return launch_rows<false>(m, a, units, st);
}

size_t prefix_workspace(const medusa_cfg& c, int shared) { return plan_prefix(c, shared).total; }

cudaError_t launch_prefix_attention(const medusa_cfg& c, const void* Q, const void* Kp, const void* Vp, int num_pages,
                                    int page_rows, const int32_t* prefix, int shared, const int32_t* table, const void* Kt,
                                    const void* Vt, const int32_t* L, const uint64_t* bits, void* O, void* ws,
                                    cudaStream_t st) {
  const TreeShape ts = tree_shape(c);
  const PrefixPlan p = plan_prefix(c, shared);
  RowsArgs a{};
  a.L = L;
  a.bits = bits;
  a.prefix = prefix;
  a.table = table;
  a.B = c.B;
  a.N = ts.N;
  a.T = c.B * ts.N;
  a.Hq = c.Hq;
  a.Hkv = c.Hkv;
  a.gp_shift = p.gp_shift;
  a.L_cap = c.L_cap;
  a.page_rows = page_rows;
  a.max_pages = c.L_cap / page_rows;
  a.num_pages = num_pages;
  a.shared = shared;
  a.splits_s = p.splits_s;
  a.chunk_s = p.chunk_s;
  a.splits_u = p.splits_u;
  a.chunk_u = p.chunk_u;
  a.scale_log2 = (float)(1.4426950408889634 / sqrt((double)kD));
  a.o_part = static_cast<float*>(ws);
  a.ml_part = reinterpret_cast<float*>(static_cast<char*>(ws) + p.ml_part);
  const int npos = kRows >> a.gp_shift, per = 2 * npos, HG = c.Hq >> a.gp_shift;
  const uint64_t planes = (uint64_t)num_pages * c.Hkv, tplanes = (uint64_t)c.B * c.Hkv;
  CUtensorMap m[5];
  if (!encode_3d(&m[0], Q, a.T, c.Hq, (uint64_t)c.Hq * kD * 2, kD * 2, npos, 1u << a.gp_shift) ||
      !encode_3d(&m[1], Kp, page_rows, planes, kD * 2, (uint64_t)page_rows * kD * 2, kKeys, 1) ||
      !encode_3d(&m[2], Vp, page_rows, planes, kD * 2, (uint64_t)page_rows * kD * 2, kKeys, 1) ||
      !encode_3d(&m[3], Kt, ts.N, tplanes, kD * 2, (uint64_t)ts.N * kD * 2, kKeys, 1) ||
      !encode_3d(&m[4], Vt, ts.N, tplanes, kD * 2, (uint64_t)ts.N * kD * 2, kKeys, 1))
    return cudaErrorInvalidValue;
  const int64_t units = (int64_t)p.splits_s * HG * ((a.T + per - 1) / per) +
                        (int64_t)p.splits_u * c.B * HG * ((ts.N + per - 1) / per);
  cudaError_t e = launch_rows<true>(m, a, units, st);
  if (e != cudaSuccess) return e;
  const int64_t rows = (int64_t)a.T * c.Hq;
  e = launch_pdl(rows_merge_kernel, (unsigned)((rows * 32 + 255) / 256), 256, 0, st, static_cast<const float*>(a.o_part),
                 static_cast<const float*>(a.ml_part), rows, p.splits_s + p.splits_u, static_cast<uint16_t*>(O));
  note_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace medusa
