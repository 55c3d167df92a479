// Attention of packed query rows on 5th-generation tensor cores (tcgen05, TMEM
// accumulators, TMA), bf16: whole prompts (causal; D = 64 or 128), and tree attention
// behind a prefix that the batch shares (D = 128).
//
// O = softmax(Q K^T / sqrt(D)) V in one pass over the keys, with the running maximum and
// sum of "최적화 2편" (beengineer500), section 3.3. 4 rows keys D operations against
// 2 keys D elements of K and V per 256 rows: bound by the tensor cores and, beside them,
// by the exponentials, as long as there are rows; by the K/V bytes for a few single tokens.
//
// A unit of work is 256 query rows of one KV head (two tiles of 128) against a range of
// keys. A tile's rows are Gp query heads of the KV head's group times 128 / Gp positions
// (Gp: the largest power of two that divides the group, at most 16), so that one TMA box
// loads it and the heads share every K/V tile. 12 warps, one CTA per SM, which takes
// units from the grid until none is left (warp 10):
//   warps 0-3, 4-7  softmax of tile 0 and of tile 1: thread = row = TMEM lane; S (f32) to
//                   registers, mask, maximum, 2^(s - m) rounded to bf16 back over S, sums
//                   in f32. O is rescaled only when the maximum rises by more than 2^8.
//                   The product with V begins once half of the weights are there. (bf16 is what
//                   the matrix instruction takes beside a bf16 V: each weight is off by 2^-8 of itself at
//                   most, an output by 2^-8 of its weights times |v|. Against 64 bits, relative: 0.0020 to
//                   0.0023 on the cases measured, and 0.0016 for float32 rounded once at the end.)
//   warp 8          issues every MMA: S_t(j) = Q_t K_j^T (both operands in shared memory)
//                   and O_t += P_t(j) V_j (P from TMEM), so that one tile's products run
//                   while the other tile's softmax does. MMAs of one issuing thread run in
//                   order: S_t(j + 1), which overwrites P_t(j), follows O_t += P_t(j) V_j.
//   warp 9          TMA: Q tiles, then K and V tiles of 128 keys alternating through one
//                   ring of 160 KB. V rows past the last key that any row sees are zeroed in
//                   shared memory (0 x NaN must not reach a result).
//   warp 10         the schedule: a unit per block of the grid, longest first; this warp takes over
//                   blocks that have not started (cluster launch control) and decodes the next
//                   unit while the others work on this one.
// TMEM: S_0, S_1, O_0, O_1 (128 columns each; O uses D of them). Every mbarrier wait is bounded.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <mutex>
#include <type_traits>

#include "common.cuh"
#include "prompt_walk.cuh"
#include "tc_common.cuh"

namespace medusa {

__device__ uint32_t g_rows_tc_error = 0;

namespace {

constexpr int kRows = 128, kKeys = 128;
constexpr int kHalf = 128 * 128;            // 128 rows x 64 bf16, 128-byte swizzle (16 KB): a tile of D = 64
template <int D>
struct Layout {
  static constexpr int halves = D / 64;
  static constexpr int tile = halves * kHalf;        // 128 x D bf16
  static constexpr int stages = 160 * 1024 / tile;   // K/V ring
  static constexpr int ring = 2 * tile;              // behind the two Q tiles
  static constexpr int smem = ring + stages * tile + 1024;   // + alignment slack
};
constexpr int kMmaWarp = 8, kLoadWarp = 9, kPlanWarp = 10;
constexpr int kThreads = 384;
constexpr uint32_t kTmemCols = 512;
constexpr int kSms = 152;
constexpr int kLeastKeys = 256;   // of a key range that is one of several: two tiles
constexpr int kAhead = 8;   // steps (K and V tiles) of a unit still to be loaded when the next unit is fetched
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
  int units_s, splits_s, chunk_s, dual_s;   // units, key ranges and their length of the shared rows; 1: dual units
  int units_u, splits_u, dual_u;            // the same of the sequences' own rows (a length for each sequence)
  float scale_log2;
  uint16_t* O;             // prompts
  float* o_part;           // prefix: [split][row][D], row = position * Hq + head
  float* ml_part;          // prefix: [split][row][2]
};

enum UnitKind : int { kEnd = 0, kPrompt = 1, kShared = 2, kOwn = 3 };

// What the scheduling warp hands to the others. Where the rows of a key range fill one tile only
// (prefix), the two tiles are two such pieces of work, so that there is still one tile's softmax
// to hide behind the other's products; they then share no K/V tile (`dual`).
struct Unit {
  int kind, dual;
  int pos0[2], left[2];   // a tile's first Q row (position), and how many positions there are from it on
  int h0[2], kvh[2];      // first query head, KV head
  int base[2];            // prompts: packed row of the sequence's row 0; prefix: the sequence
  int k0[2], kend[2];     // key range
  int n[2], tree[2];      // key tiles (the tree tile included); number of the tree tile, or -1
  int part[2];            // prefix: which partial result the tile writes
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
// Cluster launch control: asks for a block of this grid that has not started yet; its index
// arrives as 16 bytes at `slot` (16-byte aligned), completing on `bar`.
__device__ __forceinline__ void steal_ask(void* slot, uint64_t* bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   tc::saddr(slot)),
               "r"(tc::saddr(bar))
               : "memory");
}
// The block index that was taken over, or -1: every block has started.
__device__ __forceinline__ int steal_answer(const void* slot) {
  uint32_t x, got;
  asm volatile(
      "{ .reg .pred p; .reg .b128 r; ld.shared.b128 r, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "selp.u32 %1, 1, 0, p;\n\t"
      "mov.u32 %0, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%0, _, _, _}, r; }"
      : "=r"(x), "=r"(got)
      : "r"(tc::saddr(slot))
      : "memory");
  return got ? (int)x : -1;
}
// mbarrier.test_wait: asks without being suspended.
__device__ __forceinline__ bool mbar_test(uint64_t* b, uint32_t parity) {
  uint32_t ok;
  asm volatile("{ .reg .pred p; mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
               : "=r"(ok)
               : "r"(tc::saddr(b)), "r"(parity)
               : "memory");
  return ok != 0;
}
// Bounded wait of the issuing thread: it polls, since being suspended and woken costs more than
// the gaps that it has to fill.
__device__ __forceinline__ bool mbar_poll(uint64_t* b, uint32_t parity, uint32_t* err, uint32_t code) {
  if (mbar_test(b, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_test(b, parity)) {
    if (clock64() - t0 > 4000000000LL) {
      atomicOr(err, code);
      return false;
    }
  }
  return true;
}
// 32 columns of this warp's TMEM lanes, and the wait that makes them readable: the registers
// pass through it, so that no use of them can be moved ahead of it.
__device__ __forceinline__ void tmem_landed32(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                 "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                 "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}
__device__ __forceinline__ float max32(const uint32_t* v) {
  float m = __uint_as_float(v[0]);
#pragma unroll
  for (int x = 1; x < 31; x += 2) m = max3(m, __uint_as_float(v[x]), __uint_as_float(v[x + 1]));
  return fmaxf(m, __uint_as_float(v[31]));
}
// p = 2^(s scale - m) of 32 scores as 16 bf16 pairs; their float32 values are added to acc.
__device__ __forceinline__ void exp32(const uint32_t* v, float scale_log2, float neg_m, uint32_t* pk, float2* acc) {
  const float2 sc = make_float2(scale_log2, scale_log2), nm = make_float2(neg_m, neg_m);
#pragma unroll
  for (int x = 0; x < 16; ++x) {
    const float2 e = __ffma2_rn(make_float2(__uint_as_float(v[2 * x]), __uint_as_float(v[2 * x + 1])), sc, nm);
    float2 p;
    p.x = tc::ex2(e.x);
    p.y = tc::ex2(e.y);
    acc[x & 1] = __fadd2_rn(acc[x & 1], p);
    pk[x] = pack_bf16x2(p.x, p.y);
  }
}
// Four lanes hold four 16-byte pieces of a row each (r[4 i ..]: piece i); afterwards lane l of
// the four holds piece l of rows 0..3 (r[4 k ..]: row k).
__device__ __forceinline__ void transpose4(uint32_t* r) {
  const int lane = threadIdx.x;
#pragma unroll
  for (int s = 1; s <= 2; s <<= 1) {
    const bool up = lane & s;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i & s) continue;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        uint32_t &lo = r[4 * i + x], &hi = r[4 * (i | s) + x];
        const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? lo : hi, s);
        if (up) lo = got;
        else hi = got;
      }
    }
  }
}
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          tc::saddr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(tc::saddr(bar))
      : "memory");
}

// One tile's part of a unit, as decoded by lanes t, t + 2, ... of the scheduling warp. (What runs
// once per unit is kept short: between two units its instructions come from beyond the
// instruction caches, which the softmax fills.)
struct Piece {
  int kind, dual, pos0, left, h0, kvh, base, k0, kend, n, tree, part;
};

// Unit u of the prompts: 256 rows, both tiles over the same keys.
__device__ __forceinline__ Piece decode_prompt(const RowsArgs& a, PromptWalk& walk, int u, int t) {
  Piece w = {};
  const int npos = kRows >> a.gp_shift, HG = a.Hq >> a.gp_shift;
  const int x = u / HG, b = walk.find(x);
  if (b < 0) return w;
  const int c0 = a.cu[b], len = a.cu[b + 1] - c0, i = (2 * walk.t + t) * npos;
  w.kind = kPrompt;
  w.pos0 = c0 + i;
  w.left = len - i;
  w.h0 = (u - x * HG) << a.gp_shift;
  w.kvh = w.h0 / (a.Hq / a.Hkv);
  w.base = c0;
  w.kend = len;
  w.n = i < len ? (min(len, i + npos) + kKeys - 1) / kKeys : 0;
  w.tree = -1;
  return w;
}

// Unit u of tree attention behind a prefix: the shared rows come first, for all positions of the
// batch (a.units_s units), then the sequences' own rows and trees (a.units_u).
__device__ __forceinline__ Piece decode_prefix(const RowsArgs& a, int u, int t) {
  Piece w = {};
  const int npos = kRows >> a.gp_shift, HG = a.Hq >> a.gp_shift;
  if (u >= a.units_s + a.units_u) return w;
  const bool shared = u < a.units_s;
  w.kind = shared ? kShared : kOwn;
  w.dual = shared ? a.dual_s : a.dual_u;
  w.tree = -1;
  const int v = shared ? u : u - a.units_s;
  const int positions = shared ? a.T : a.N;   // that meet the same keys
  // piece x: (split, [sequence,] head group), for the two tiles together or for one
  const int per = w.dual ? npos : 2 * npos, ru = (positions + per - 1) / per;
  const int vt = w.dual ? 2 * v + t : v, x = vt / ru, row0 = (vt - x * ru) * per + (w.dual ? 0 : t * npos);
  const int y = x / HG, split = shared ? y : y / a.B, b = shared ? 0 : y - split * a.B;
  w.left = positions - row0;
  if (split >= (shared ? a.splits_s : a.splits_u)) w.left = 0;   // the last unit of an odd number of pieces
  if (w.left <= 0) return w;
  w.pos0 = b * a.N + row0;
  w.h0 = (x - y * HG) << a.gp_shift;
  w.kvh = w.h0 / (a.Hq / a.Hkv);
  w.base = b;
  w.part = shared ? split : a.splits_s + split;
  bool tree = false;
  if (shared) {
    w.k0 = split * a.chunk_s;
    w.kend = min(a.shared, w.k0 + a.chunk_s);
  } else {
    const int Lb = a.L[b];
    const bool ok = Lb >= 0 && Lb <= a.L_cap - a.N;
    // The ranges divide the rows that the sequence has, not those that it may come to have: four
    // tokens of 32 heads with 300 to 2800 own rows in a cache of 32768: 63 us by capacity, 30 so.
    const int own = ok ? max(0, Lb - a.shared) : 0;
    const int chunk = max(kLeastKeys, ((own + a.splits_u - 1) / a.splits_u + kKeys - 1) & ~(kKeys - 1));
    w.k0 = a.shared + split * chunk;
    w.kend = ok ? min(Lb, w.k0 + chunk) : 0;
    tree = ok && split == a.splits_u - 1;
  }
  w.n = w.kend > w.k0 ? (w.kend - w.k0 + kKeys - 1) / kKeys : 0;
  if (tree) w.tree = w.n++;
  return w;
}

template <int kD, bool kPrefix>
__global__ void __launch_bounds__(kThreads, 1)
rows_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
               const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmKt,
               const __grid_constant__ CUtensorMap tmVt, const __grid_constant__ RowsArgs a) {
  using Lay = Layout<kD>;
  constexpr int kStages = Lay::stages, kTile = Lay::tile, kHalves = Lay::halves;
  // (Behind a prefix the next kernel's blocks, started early, would crowd the SMs that are done first.)
  if (!kPrefix) pdl_trigger();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = sm + Lay::ring;
  __shared__ __align__(8) uint64_t kv_full[kStages], kv_empty[kStages];
  __shared__ __align__(8) uint64_t q_full[2], q_empty[2], s_full[2], p_half[2], p_full[2], o_done[2];
  __shared__ __align__(8) uint64_t unit_full[2], unit_empty[2], tail, stolen, want;
  __shared__ __align__(16) uint4 steal_slot[1];
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
      tc::mbar_init(&p_half[t], kRows);
      tc::mbar_init(&p_full[t], kRows);
      tc::mbar_init(&o_done[t], 1);
      tc::mbar_init(&unit_full[t], 1);
      tc::mbar_init(&unit_empty[t], 10);   // 8 softmax warps, the MMA warp, the load warp
    }
    tc::mbar_init(&tail, 1);
    tc::mbar_init(&stolen, 1);
    tc::mbar_init(&want, 1);
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
    // Block indices are units in order. The CTA begins with its own and then takes over blocks
    // that have not started, so that the SMs run out of work together.
    PromptWalk walk;
    if (!kPrefix) walk.begin(a.cu, a.B, a.T, 8 - a.gp_shift);
    int u = (int)blockIdx.x, asked = 0, i = 0;   // i: units handed out
    bool ok = true;
    while (ok && u >= 0) {
      const int t = lane & 1;
      const Piece w = kPrefix ? decode_prefix(a, u, t) : decode_prompt(a, walk, u, t);
      if (w.kind != kEnd) {   // (the grid may hold more blocks than there are units)
        if (i >= 2) ok = __all_sync(0xffffffffu, tc::mbar_wait(&unit_empty[i & 1], ((i >> 1) - 1) & 1, err, 2));
        if (!ok) break;
        Unit& d = units[i & 1];
        if (lane < 2) {
          d.kind = w.kind;
          d.dual = w.dual;
          d.pos0[t] = w.pos0;
          d.left[t] = w.left;
          d.h0[t] = w.h0;
          d.kvh[t] = w.kvh;
          d.base[t] = w.base;
          d.k0[t] = w.k0;
          d.kend[t] = w.kend;
          d.n[t] = w.n;
          d.tree[t] = w.tree;
          d.part[t] = w.part;
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&unit_full[i & 1]);
        __syncwarp();
        // not before the loads of this unit near their end: what is taken too early is missing elsewhere
        ok = __all_sync(0xffffffffu, tc::mbar_wait(&want, i & 1, err, 16384));
        ++i;
        if (!ok) break;
      }
      if (lane == 0) {
        tc::mbar_arrive_expect(&stolen, 16);
        steal_ask(steal_slot, &stolen);
      }
      __syncwarp();
      ok = __all_sync(0xffffffffu, tc::mbar_wait(&stolen, asked & 1, err, 8192));
      ++asked;
      if (!ok) break;
      u = steal_answer(steal_slot);
      tc::fence_proxy_async();   // the slot has been read before the next answer may land in it
      __syncwarp();
    }
    if (i >= 2) tc::mbar_wait(&unit_empty[i & 1], ((i >> 1) - 1) & 1, err, 2);
    if (lane == 0) {
      units[i & 1].kind = kEnd;
      tc::mbar_arrive(&unit_full[i & 1]);
    }
    __syncwarp();
  } else if (warp == kLoadWarp) {
    // ------------------------------------------------------------------ TMA loads
    // Tiles come in the order in which the MMA warp uses them: K_0, V_0, K_1, V_1, ...; for two
    // tiles with keys of their own K_0 K'_0, V_0 K_1 V'_0 K'_1, ...
    Unit w;
    int it = 0, nq[2] = {0, 0}, fixes = 0;   // ring position, Q tiles loaded, tails zeroed
    int page_reg[2] = {-1, -1};
    int seen = -1;   // prefix: shared rows that any sequence sees (once it is known: rows past it may hold anything)
    bool ok = true;
    for (int i = 0; ok && next_unit(i, w); ++i) {
      const int nt = max(w.n[0], w.n[1]), tiles = w.dual ? 2 : 1;
      if (nt <= kAhead && lane == 0) tc::mbar_arrive(&want);   // time to fetch the next unit
#pragma unroll 1
      for (int j = nt > 0 ? -1 : 0; ok && j < nt; ++j) {   // step j: V_j and K_{j+1}
        if (j > 0 && nt - j == kAhead && lane == 0) tc::mbar_arrive(&want);
#pragma unroll 1
        for (int x = 0; ok && x < 2 * tiles; ++x) {
          const int t = x >> 1, n = w.dual ? (t ? w.n[1] : w.n[0]) : nt, jt = j + (x & 1);
          const bool isv = !(x & 1);
          if (jt < 0 || jt >= n) continue;
          // a tile's rows go ahead of its first K tile; tile 1's, where both share the keys, behind it
          const int r = j < 0 ? t : (j == 0 && x == 0 && !w.dual && w.n[1] > 0) ? 1 : -1;
          if (r >= 0) {
            const int used = r ? nq[1] : nq[0];
            if (used > 0) ok = __all_sync(0xffffffffu, tc::mbar_wait(&q_empty[r], (used - 1) & 1, err, 4));
            if (!ok) break;
            if (lane == 0) {
              uint8_t* dst = sm + r * kTile;
              tc::mbar_arrive_expect(&q_full[r], kTile);
#pragma unroll
              for (int h = 0; h < kHalves; ++h)
                tma_load_3d(dst + h * kHalf, &tmQ, 64 * h, r ? w.pos0[1] : w.pos0[0], r ? w.h0[1] : w.h0[0], &q_full[r]);
            }
            if (r) ++nq[1];
            else ++nq[0];
          }
          const int k0 = t ? w.k0[1] : w.k0[0], kend = t ? w.kend[1] : w.kend[0], base = t ? w.base[1] : w.base[0];
          const int kvh = t ? w.kvh[1] : w.kvh[0];
          const int st = it % kStages;
          if (it >= kStages) ok = __all_sync(0xffffffffu, tc::mbar_wait<true>(&kv_empty[st], (it / kStages - 1) & 1, err, 8));
          if (!ok) break;
          const bool tree = kPrefix && jt == (t ? w.tree[1] : w.tree[0]);
          const int key0 = k0 + jt * kKeys;
          int y, z;
          if (!kPrefix) {
            y = base + key0;
            z = kvh;
          } else if (tree) {
            y = 0;
            z = base * a.Hkv + kvh;
          } else {
            int pages = t ? page_reg[1] : page_reg[0];
            if (!isv && (jt & 31) == 0) {   // 32 tiles' pages at a time, one per lane
              const int key = key0 + lane * kKeys;
              pages = -1;
              if (key < kend)
                pages = w.kind == kShared ? a.prefix[key / a.page_rows] : a.table[(size_t)base * a.max_pages + key / a.page_rows];
              if (t) page_reg[1] = pages;
              else page_reg[0] = pages;
            }
            const int page = __shfl_sync(0xffffffffu, pages, jt & 31);
            const bool in_pool = page >= 0 && page < a.num_pages;
            MEDUSA_CHECK(isv || lane != 0 || in_pool, MEDUSA_CHECK_PAGE);
            y = key0 % a.page_rows;
            z = (in_pool ? page : a.num_pages) * a.Hkv + kvh;   // outside the pool: TMA fills zeros
          }
          const CUtensorMap* m = tree ? (isv ? &tmVt : &tmKt) : (isv ? &tmV : &tmK);
          uint8_t* dst = ring + st * kTile;
          if (kPrefix && isv && seen < 0 && w.kind == kShared) {   // (K and Q are on their way)
            seen = 0;
            for (int b = lane; b < a.B; b += 32) {
              const int Lb = a.L[b];
              if (Lb <= a.L_cap - a.N) seen = max(seen, Lb);
            }
            seen = __reduce_max_sync(0xffffffffu, seen);
          }
          const int last = kPrefix && w.kind == kShared ? min(kend, seen) : kend;
          const int live = tree ? kKeys : max(0, min(kKeys, last - key0));   // (rows past the tree's nodes arrive as zeros)
          const bool fix = isv && live < kKeys;
          uint64_t* bar = fix ? &tail : &kv_full[st];
          if (lane == 0) {
            tc::mbar_arrive_expect(bar, kTile);
#pragma unroll
            for (int h = 0; h < kHalves; ++h) tma_load_3d(dst + h * kHalf, m, 64 * h, y, z, bar);
          }
          __syncwarp();
          if (fix) {   // rows [live, 128) of each half become zero before the MMA warp may see the tile
            ok = __all_sync(0xffffffffu, tc::mbar_wait<true>(&tail, fixes & 1, err, 16));
            ++fixes;
            if (!ok) break;
#pragma unroll 1
            for (int c = live * 8 + lane; c < kKeys * 8; c += 32) {
#pragma unroll
              for (int h = 0; h < kHalves; ++h) reinterpret_cast<uint4*>(dst + h * kHalf)[c] = make_uint4(0, 0, 0, 0);
            }
            tc::fence_proxy_async();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&kv_full[st]);
          }
          ++it;
        }
      }
    }
    // never leave with copies still landing in shared memory
    for (int x = it > kStages ? it - kStages : 0; x < it; ++x) tc::mbar_wait(&kv_full[x % kStages], (x / kStages) & 1, err, 32);
    for (int t = 0; t < 2; ++t)
      if (nq[t] > 0) tc::mbar_wait(&q_full[t], (nq[t] - 1) & 1, err, 64);
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------------ MMA issue
    // One elected lane walks the schedule and issues; little but waits stands between two
    // batches of products, since whatever does is time without a product in flight (as a loop of
    // the whole warp with a vote after each wait: 1520 us for a 16384-token prompt, so: 1370).
    // What is left: a pair of tiles takes 2650 clocks for 2048 of products. Both operands of S
    // come from shared memory, 8 KB per 64 clocks; with V and the arriving tiles the products
    // ask for 2048 clocks of its bandwidth as well (TMEM has no room for Q beside S and O).
    constexpr uint32_t idS = tc::idesc_bf16_f32(kRows, kKeys, 0, 0);
    constexpr uint32_t idPV = tc::idesc_bf16_f32(kRows, kD, 0, 1);
    if (tc::elect_one()) {
      const uint64_t dQ = tc::sw128_desc(tc::saddr(sm), 16, 1024);
      const uint64_t dK = tc::sw128_desc(tc::saddr(ring), 16, 1024);
      const uint64_t dV = tc::sw128_desc(tc::saddr(ring), kHalf, 1024);   // MN-major: LBO = the 64-column half
      int st = 0, ph = 0;                     // ring stage of the next tile and its phase
      int nq[2] = {0, 0}, np[2] = {0, 0};     // Q tiles used, P tiles used
      bool ok = true, ahead = false;          // ahead: S_0(0) of the coming unit has been issued
      auto advance = [&](int& stage, int& phase) {
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1;
        }
      };
      // S_t = Q_t K^T with the K tile in `stage`
      auto issue_S = [&](int t, int stage) {
        const uint64_t q0 = dQ + (uint64_t)((t * kTile) >> 4), b0 = dK + (uint64_t)((stage * kTile) >> 4);
#pragma unroll
        for (int kk = 0; kk < kD / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
          tc::mma_bf16(tmem + col_S(t), q0 + off, b0 + off, idS, kk > 0);
        }
        tc::commit(&s_full[t]);
      };
      // O_t (+)= P_t V with keys [64 half, 64 half + 64) of the V tile in `stage`
      auto issue_PV = [&](int t, int stage, int half, bool first) {
        tc::fence_after();
        const uint64_t b0 = dV + (uint64_t)((stage * kTile) >> 4);
#pragma unroll
        for (int k4 = 0; k4 < kKeys / 32; ++k4) {   // keys [16 kk, 16 kk + 16): P columns 32 (kk / 2) + 8 (kk % 2)
          const int kk = (kKeys / 32) * half + k4;
          tc::mma_bf16_tmem_a(tmem + col_O(t), tmem + col_S(t) + 32 * (kk >> 1) + 8 * (kk & 1),
                              b0 + (uint64_t)((kk * 2048) >> 4), idPV, (!first || k4 > 0) ? 1 : 0);
        }
      };
      // One unit, number i of this CTA. (A template of `dual`: a test between two batches of products
      // shows, 228 -> 270 us for 32 trees behind 8192 rows.)
      auto issue_unit = [&](auto dual_c, int i, const int* n) {
        constexpr bool dual = decltype(dual_c)::value;
        const int nt = max(n[0], n[1]);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (!ok || n[t] == 0) continue;
          if (!(t == 0 && ahead)) {
            ok = mbar_poll(&kv_full[st], ph, err, 128) && mbar_poll(&q_full[t], nq[t] & 1, err, 256);
            if (!ok) break;
            ++nq[t];
            issue_S(t, st);
            if (n[t] == 1) tc::commit(&q_empty[t]);
          }
          if (dual) {   // a stage is free once everything issued so far has read it
            tc::commit(&kv_empty[st]);
            advance(st, ph);
          }
        }
        ahead = false;
        if (!dual) {
          tc::commit(&kv_empty[st]);
          advance(st, ph);
        }
        for (int j = 0; ok && j < nt; ++j) {
          int sv = 0, sk = 0;   // stages of V_j and K_{j+1}
          auto take = [&](int& stage) {
            stage = st;
            ok = ok && mbar_poll(&kv_full[st], ph, err, 128);
            advance(st, ph);
          };
          if (!dual) {
            take(sv);
            if (j + 1 < nt) take(sk);
          }
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (ok && j < n[t]) {
              if (dual) take(sv);
              ok = ok && mbar_poll(&p_half[t], np[t] & 1, err, 4096);
              if (!ok) break;
              issue_PV(t, sv, 0, j == 0);
              ok = mbar_poll(&p_full[t], np[t] & 1, err, 512);
              if (!ok) break;
              issue_PV(t, sv, 1, false);
              ++np[t];
              if (j + 1 < n[t]) {
                if (dual) {
                  tc::commit(&kv_empty[sv]);
                  take(sk);
                  if (!ok) break;
                }
                issue_S(t, sk);
                if (j + 2 == n[t]) tc::commit(&q_empty[t]);   // Q_t is not needed any more
                if (dual) tc::commit(&kv_empty[sk]);
              } else {
                tc::commit(&o_done[t]);
                if (dual) tc::commit(&kv_empty[sv]);
              }
            }
            // Tile 0 is through with the unit: its first product of the next one goes ahead of tile
            // 1's last, if everything for it is there.
            if (ok && t == 0 && !dual && j + 1 == nt && mbar_test(&unit_full[(i + 1) & 1], ((i + 1) >> 1) & 1)) {
              const int n0 = units[(i + 1) & 1].n[0];
              if (units[(i + 1) & 1].kind != kEnd && n0 > 0 && mbar_test(&kv_full[st], ph) && mbar_test(&q_full[0], nq[0] & 1)) {
                tc::fence_after();
                ++nq[0];
                issue_S(0, st);
                if (n0 == 1) tc::commit(&q_empty[0]);
                ahead = true;
              }
            }
          }
          if (!dual) {
            tc::commit(&kv_empty[sv]);
            if (j + 1 < nt) tc::commit(&kv_empty[sk]);
          }
        }
      };
      for (int i = 0; ok; ++i) {
        ok = tc::mbar_wait(&unit_full[i & 1], (i >> 1) & 1, err, 1);
        if (!ok) break;
        const bool end = units[i & 1].kind == kEnd, two = units[i & 1].dual;
        const int n[2] = {units[i & 1].n[0], units[i & 1].n[1]};
        tc::mbar_arrive(&unit_empty[i & 1]);
        if (end) break;
        if (max(n[0], n[1]) == 0) continue;
        if (kPrefix && two) issue_unit(std::true_type{}, i, n);
        else issue_unit(std::false_type{}, i, n);
      }
    }
    __syncwarp();
  } else if (warp < 8) {
    // ------------------------------------------------------------------ softmax
    const int t = warp >> 2, row = 32 * (warp & 3) + lane;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t tS = tmem + col_S(t) + lanes, tO = tmem + col_O(t) + lanes;
    const int rhead = row >> (7 - a.gp_shift), rpos = row & (npos - 1);
    int ns = 0, nu = 0;   // S tiles and units taken
    bool ok = true;
    for (int i = 0; ok; ++i) {
      ok = __all_sync(0xffffffffu, tc::mbar_wait(&unit_full[i & 1], (i >> 1) & 1, err, 1));
      if (!ok) break;
      const Unit& w = units[i & 1];
      const int kind = w.kind, n = w.n[t], k0 = w.k0[t], kend = w.kend[t], tree_tile = w.tree[t], left = w.left[t];
      const int pos = w.pos0[t] + rpos, head = w.h0[t] + rhead, base = w.base[t], part_no = w.part[t];
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&unit_empty[i & 1]);
      if (kind == kEnd) break;
      const bool row_ok = rpos < left;
      // keys below `limit` are visible to this row
      int limit = kend;
      uint64_t word0 = 0, word1 = 0;
      if (!kPrefix) {
        limit = pos - base + 1;
      } else if (row_ok) {
        const int b = pos / a.N;
        if (kind == kShared) {
          const int Lb = a.L[b];
          limit = (Lb >= 0 && Lb <= a.L_cap - a.N) ? min(Lb, kend) : 0;
        } else if (tree_tile >= 0) {
          // (bits past the last node name no key)
          word0 = a.bits[2 * (pos - b * a.N)] & (~0ull >> (a.N < 64 ? 64 - a.N : 0));
          word1 = a.N > 64 ? a.bits[2 * (pos - b * a.N) + 1] & (~0ull >> (128 - a.N)) : 0;
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
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_landed32(v + 32 * c);
          const int vis = limit - (k0 + j * kKeys);
          const bool tree = kPrefix && j == tree_tile, masked = tree || __any_sync(0xffffffffu, vis < kKeys);
          if (masked) {   // a bit per key, so that one piece of code masks the tree's tiles and the others
            uint32_t see[4] = {(uint32_t)word0, (uint32_t)(word0 >> 32), (uint32_t)word1, (uint32_t)(word1 >> 32)};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int here = vis - 32 * c;
              if (!tree) see[c] = here >= 32 ? 0xffffffffu : here <= 0 ? 0u : (1u << here) - 1u;
#pragma unroll
              for (int x = 0; x < 32; ++x)
                v[32 * c + x] = (see[c] >> x) & 1u ? v[32 * c + x] : __float_as_uint(-INFINITY);
            }
          }
          float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          float corr = 1.f;
          uint32_t pk[16];
          const float m_tile = fmaxf(fmaxf(max32(v), max32(v + 32)), fmaxf(max32(v + 64), max32(v + 96))) * a.scale_log2;
          const bool move = m_tile > m_run + kLazy;   // also on the first visible tile (m_run = -inf): corr = 0
          if (__any_sync(0xffffffffu, move)) {
            if (move) {
              corr = tc::ex2(m_run - m_tile);
              m_run = m_tile;
            }
            if (j > 0) {   // O += P_{j-1} V_{j-1} was issued before S_j and has landed with it
#pragma unroll 1
              for (int c = 0; c < kD / 8; ++c) {
                uint32_t o[8];
                tc::tmem_ld8(tO + 8 * c, o);
                tc::tmem_wait_ld();
#pragma unroll
                for (int x = 0; x < 8; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * corr);
                tc::tmem_st8(tO + 8 * c, o);
              }
            }
          }
          {
            const float neg_m = m_run == -INFINITY ? 0.f : -m_run;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              exp32(v + 32 * c, a.scale_log2, neg_m, pk, acc);
              tc::tmem_st16(tS + 32 * c, pk);
            }
          }
          tc::tmem_wait_st();
          tc::fence_before();
          tc::mbar_arrive(&p_half[t]);   // the product with V begins on these 64 keys
          const float neg_m = m_run == -INFINITY ? 0.f : -m_run;
#pragma unroll
          for (int c = 2; c < 4; ++c) {
            exp32(v + 32 * c, a.scale_log2, neg_m, pk, acc);
            tc::tmem_st16(tS + 32 * c, pk);
          }
          const float2 s2 = __fadd2_rn(acc[0], acc[1]);
          l_run = l_run * corr + (s2.x + s2.y);
          tc::tmem_wait_st();
          tc::fence_before();
        } else {
          tc::mbar_arrive(&p_half[t]);
        }
        tc::mbar_arrive(&p_full[t]);
      }
      if (!ok) break;
      if (n > 0) {
        ok = __all_sync(0xffffffffu, tc::mbar_wait(&o_done[t], nu & 1, err, 2048));
        ++nu;
        if (!ok) break;
        tc::fence_after();
      }
      if (!busy) continue;
      // Four lanes hold four consecutive positions of one head. They trade 16-byte pieces, so that
      // a store instruction writes 64 bytes of each row, not 16 (a quarter of the memory lines).
      const int quad = lane & 3;
      const size_t orow = (size_t)pos * a.Hq + head, orow0 = (size_t)(pos - quad) * a.Hq + head;
      const int rows_here = left - (rpos - quad);   // rows of the four that exist, if positive
      if (!kPrefix) {
        const float inv = 1.f / l_run;   // (0 where every visible score is -inf: 0 times inf, no number, as in float32)
#pragma unroll 1
        for (int c = 0; c < kD / 32; ++c) {
          uint32_t o[32], pk[16];
          tc::tmem_ld32(tO + 32 * c, o);
          tmem_landed32(o);
#pragma unroll
          for (int x = 0; x < 16; ++x)
            pk[x] = pack_bf16x2(__uint_as_float(o[2 * x]) * inv, __uint_as_float(o[2 * x + 1]) * inv);
          transpose4(pk);
          uint16_t* op = a.O + orow0 * kD + 32 * c + 8 * quad;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (k < rows_here)
              *reinterpret_cast<uint4*>(op + (size_t)k * a.Hq * kD) = make_uint4(pk[4 * k], pk[4 * k + 1], pk[4 * k + 2], pk[4 * k + 3]);
        }
      } else {
        const size_t part = (size_t)part_no * a.T * a.Hq;
        if (n > 0) {
#pragma unroll 1
          for (int c = 0; c < kD / 32; ++c) {
            uint32_t o[32];
            tc::tmem_ld32(tO + 32 * c, o);
            tmem_landed32(o);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              transpose4(o + 16 * x);
              float* op = a.o_part + (part + orow0) * kD + 32 * c + 16 * x + 4 * quad;
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (k < rows_here)
                  *reinterpret_cast<uint4*>(op + (size_t)k * a.Hq * kD) =
                      make_uint4(o[16 * x + 4 * k], o[16 * x + 4 * k + 1], o[16 * x + 4 * k + 2], o[16 * x + 4 * k + 3]);
            }
          }
        }
        if (row_ok) {
          a.ml_part[2 * (part + orow)] = m_run;
          a.ml_part[2 * (part + orow) + 1] = l_run;
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

constexpr int kPrefixD = 128;

// The merge of partial results of one row, 4 head dims per lane: O = sum_s 2^(m_s - M) o_s /
// sum_s 2^(m_s - M) l_s.
struct Merge {
  float M = -INFINITY, sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  __device__ __forceinline__ void add(float m, float l, const float4& o) {
    if (m == -INFINITY && l == 0.f) return;   // nothing was visible: its O need not have been written
    const float mn = fmaxf(M, m), mu = mn == -INFINITY ? 0.f : mn, w0 = exp2f(M - mu), w1 = exp2f(m - mu);
    M = mn;
    sum = sum * w0 + l * w1;
    acc = make_float4(acc.x * w0 + o.x * w1, acc.y * w0 + o.y * w1, acc.z * w0 + o.z * w1, acc.w * w0 + o.w * w1);
  }
  // parts [0, splits) of a row, X loads at a time
  template <int X>
  __device__ __forceinline__ void parts(const float* __restrict__ o_part, const float* __restrict__ ml_part, int64_t rows,
                                        int64_t row, int splits) {
    for (int s0 = 0; s0 < splits; s0 += X) {
      float2 ml[X];
      float4 o[X];
#pragma unroll
      for (int x = 0; x < X; ++x) {
        const int64_t at = (s0 + x < splits ? s0 + x : 0) * rows + row;
        ml[x] = *reinterpret_cast<const float2*>(ml_part + 2 * at);
        o[x] = *reinterpret_cast<const float4*>(o_part + at * kPrefixD + 4 * (threadIdx.x & 31));
        if (s0 + x >= splits) ml[x] = make_float2(-INFINITY, 0.f);
      }
#pragma unroll
      for (int x = 0; x < X; ++x) add(ml[x].x, ml[x].y, o[x]);
    }
  }
  __device__ __forceinline__ void store(uint16_t* O, int64_t row) const {
    const float inv = sum == 0.f ? 0.f : 1.f / sum;   // no key at all: zeros
    *reinterpret_cast<uint2*>(O + row * kPrefixD + 4 * (threadIdx.x & 31)) =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  }
};

// One warp per output row. Bound by the partial results' bytes.
__global__ void __launch_bounds__(256)
rows_merge_kernel(const float* __restrict__ o_part, const float* __restrict__ ml_part, int64_t rows, int splits,
                  uint16_t* __restrict__ O) {
  pdl_wait();
  pdl_trigger();
  const int64_t row = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  if (row >= rows) return;
  Merge m;
  m.parts<2>(o_part, ml_part, rows, row, splits);
  m.store(O, row);
}

// One or two rows per KV head (single tokens): a sequence's own keys and tree, then the merge with the
// parts of the shared rows, one CTA of 8 half-warps per (sequence, KV head). Bound by the K/V
// bytes of the own rows: 16 lanes read a key's 256 bytes, each half-warp X keys a step with S
// steps on their way to shared memory, and keep R rows of q and O in registers (8 head dims per
// lane; R = N * G). Alone, 24 sequences of 40 heads: 8.2 us with 63 own rows each (3.8 TB/s), 22
// with 256 (5.7), 11 with 1 to 294, where the longest is a chain of steps; so a step of own rows
// that are all seen has code of its own (13.3 against 17.3 us) and copies come from L2 or HBM as
// they may (11.1; all own rows asked for L2 first, 13.3). With the next step in registers, not on
// its way to shared memory: 18 us. A tensor-core unit per (sequence, KV head) spends its time on
// barriers: behind 4096 shared rows 52 us, so 34.
constexpr int kTailThreads = 128, kTailStreams = kTailThreads / 16, kTailRows = 2;

__device__ __forceinline__ void cp16(uint4* dst, const uint16_t* src, bool valid) {   // (else zeros)
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::saddr(dst)), "l"(src), "r"(valid ? 16 : 0) : "memory");
}

template <int R, int X, int S>
__global__ void __launch_bounds__(kTailThreads, R == 1 ? 6 : 4)
prefix_tail_kernel(const uint16_t* __restrict__ Q, const uint16_t* __restrict__ Kp, const uint16_t* __restrict__ Vp,
                   const uint16_t* __restrict__ Kt, const uint16_t* __restrict__ Vt, const RowsArgs a,
                   uint16_t* __restrict__ O) {
  constexpr int D = kPrefixD;
  // the ring: every thread's pieces of the next S steps, [step][key][K, V][thread]; then the streams' O
  constexpr int kRing = S * X * 2 * kTailThreads * 16, kResult = kTailStreams * R * D * 4;
  __shared__ __align__(16) uint8_t sm[kRing > kResult ? kRing : kResult];
  __shared__ float sm_m[kTailStreams][R], sm_l[kTailStreams][R];
  uint4* ring = reinterpret_cast<uint4*>(sm) + threadIdx.x;
  float* sm_o = reinterpret_cast<float*>(sm);
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.x / a.Hkv, kvh = blockIdx.x % a.Hkv, G = a.Hq / a.Hkv;
  const int stream = threadIdx.x >> 4, sub = threadIdx.x & 15;
  const int Lb = a.L[b];
  const bool ok = Lb >= 0 && Lb <= a.L_cap - a.N;
  const int own = ok ? max(0, Lb - a.shared) : 0, keys = ok ? own + a.N : 0;
  const size_t row0 = (size_t)b * a.N * a.Hq + kvh * G;   // row r: + r / G * Hq + r % G

  auto unpack8 = [](const uint4& x, float* f) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16_lo(w[i]);
      f[2 * i + 1] = bf16_hi(w[i]);
    }
  };
  // A step is kStep keys, X per stream; as page_rows and shared are multiples of 128, a step's own
  // rows lie in one page, whose id is fetched a step before its rows are.
  constexpr int kStep = kTailStreams * X;
  static_assert(128 % kStep == 0, "a step must not cross a page");
  auto page_of = [&](int k0) { return k0 < own ? a.table[(size_t)b * a.max_pages + (a.shared + k0) / a.page_rows] : -1; };
  auto fetch = [&](int k0, int stage, int page) {
    const bool in_pool = page >= 0 && page < a.num_pages;
    MEDUSA_CHECK(k0 >= own || in_pool, MEDUSA_CHECK_PAGE);
    const size_t own_at = (((size_t)(in_pool ? page : 0) * a.Hkv + kvh) * a.page_rows + (a.shared + k0) % a.page_rows + stream * X) * D + 8 * sub;
    if (k0 + kStep <= own && in_pool) {
#pragma unroll
      for (int x = 0; x < X; ++x) {
        cp16(ring + ((stage * X + x) * 2) * kTailThreads, Kp + own_at + x * D, true);
        cp16(ring + ((stage * X + x) * 2 + 1) * kTailThreads, Vp + own_at + x * D, true);
      }
    } else if (k0 < keys) {
#pragma unroll
      for (int x = 0; x < X; ++x) {
        const int key = k0 + stream * X + x;
        const uint16_t *kp = Kp, *vp = Vp;
        bool live = false;
        if (key < own) {   // (outside the pool: zeros, as the tensor-core path reads)
          live = in_pool;
          kp += own_at + x * D;
          vp += own_at + x * D;
        } else if (key < keys) {
          const size_t at = (((size_t)b * a.Hkv + kvh) * a.N + key - own) * D + 8 * sub;
          live = true;
          kp = Kt + at;
          vp = Vt + at;
        }
        cp16(ring + ((stage * X + x) * 2) * kTailThreads, kp, live);
        cp16(ring + ((stage * X + x) * 2 + 1) * kTailThreads, vp, live);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < S; ++i) fetch(i * kStep, i, page_of(i * kStep));
  int page = page_of(S * kStep);
  float q[R][8], o[R][8], m[R], l[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
    unpack8(*reinterpret_cast<const uint4*>(Q + (row0 + (size_t)(r / G) * a.Hq + r % G) * D + 8 * sub), q[r]);
#pragma unroll
    for (int d = 0; d < 8; ++d) {
      q[r][d] *= a.scale_log2;
      o[r][d] = 0.f;
    }
  }
  // One step; full: every key is one of the sequence's own rows and seen. (Every lane of a warp takes
  // every step: the reductions are collective.)
  auto step = [&](auto full_c, int k0, int st) {
    constexpr bool full = decltype(full_c)::value;
    float s[R][X];
#pragma unroll
    for (int x = 0; x < X; ++x) {
      float k[8];
      unpack8(ring[((st * X + x) * 2) * kTailThreads], k);
      const int key = k0 + stream * X + x, node = key - own;   // node >= 0: of the tree
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float t = 0.f;
#pragma unroll
        for (int d = 0; d < 8; ++d) t = fmaf(q[r][d], k[d], t);
#pragma unroll
        for (int w = 8; w > 0; w >>= 1) t += __shfl_xor_sync(0xffffffffu, t, w);
        bool see = true;
        if (!full) {
          see = key < keys;
          if (see && node >= 0) see = (a.bits[2 * (r / G) + (node >> 6)] >> (node & 63)) & 1ull;
        }
        s[r][x] = see ? t : -INFINITY;
      }
    }
    float p[R][X];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float mn = m[r];
#pragma unroll
      for (int x = 0; x < X; ++x) mn = fmaxf(mn, s[r][x]);
      const float mu = mn == -INFINITY ? 0.f : mn, corr = tc::ex2(m[r] - mu);
      m[r] = mn;
      l[r] *= corr;
#pragma unroll
      for (int d = 0; d < 8; ++d) o[r][d] *= corr;
#pragma unroll
      for (int x = 0; x < X; ++x) {
        p[r][x] = tc::ex2(s[r][x] - mu);
        l[r] += p[r][x];
      }
    }
#pragma unroll
    for (int x = 0; x < X; ++x) {
      float v[8];
      unpack8(ring[((st * X + x) * 2 + 1) * kTailThreads], v);
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (full || s[r][x] != -INFINITY) {   // what is masked may hold anything
#pragma unroll
          for (int d = 0; d < 8; ++d) o[r][d] = fmaf(p[r][x], v[d], o[r][d]);
        }
    }
  };
  for (int k0 = 0, st = 0; k0 < keys; k0 += kStep, st = st + 1 == S ? 0 : st + 1) {
    asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");   // a thread reads back what it copied itself
    if (k0 + kStep <= own) step(std::true_type{}, k0, st);
    else step(std::false_type{}, k0, st);
    const int next = page;
    page = page_of(k0 + (S + 1) * kStep);
    fetch(k0 + S * kStep, st, next);
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();   // the ring is no longer read or written
#pragma unroll
  for (int r = 0; r < R; ++r) {
#pragma unroll
    for (int d = 0; d < 8; d += 4)
      *reinterpret_cast<float4*>(sm_o + (stream * R + r) * D + 8 * sub + d) = make_float4(o[r][d], o[r][d + 1], o[r][d + 2], o[r][d + 3]);
    if (sub == 0) {
      sm_m[stream][r] = m[r];
      sm_l[stream][r] = l[r];
    }
  }
  __syncthreads();
  // merge: a warp per row, 4 head dims per lane; the streams' results, then the shared rows' parts
  const int64_t rows = (int64_t)a.T * a.Hq;
  const int lane = threadIdx.x & 31;
  for (int r = threadIdx.x >> 5; r < R; r += kTailThreads / 32) {
    const size_t row = row0 + (size_t)(r / G) * a.Hq + r % G;
    Merge merge;
    merge.parts<4>(a.o_part, a.ml_part, rows, row, a.splits_s);
#pragma unroll
    for (int x = 0; x < kTailStreams; ++x)
      merge.add(sm_m[x][r], sm_l[x][r], *reinterpret_cast<const float4*>(sm_o + (x * R + r) * D + 4 * lane));
    merge.store(O, row);
  }
}

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

// [planes][rows][D] bf16, boxes of 64 columns, `box_rows` rows and `box_planes` planes.
bool encode_3d(CUtensorMap* map, int D, const void* base, uint64_t rows, uint64_t planes, uint64_t row_bytes, uint64_t plane_bytes,
               uint32_t box_rows, uint32_t box_planes) {
  std::call_once(g_encode_once, [] {
    cudaDriverEntryPointQueryResult q;
    void* fn = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  if (!g_encode) return false;
  cuuint64_t dims[3] = {(cuuint64_t)D, rows, planes};
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

// How the key ranges are split: while all units fit one wave, one CTA per SM. Rows that fill one
// tile go two pieces to a unit.
struct PrefixPlan {
  int gp_shift, parts, tail;
  int units_s, splits_s, chunk_s, dual_s, units_u, splits_u, dual_u;
  size_t ml_part, total;
};
PrefixPlan plan_prefix(const medusa_cfg& c, int shared) {
  PrefixPlan p{};
  const TreeShape ts = tree_shape(c);
  p.gp_shift = gp_shift_of(c.Hq / c.Hkv);
  const int npos = kRows >> p.gp_shift, HG = c.Hq >> p.gp_shift;
  auto split = [&](int64_t groups, int64_t positions, int64_t keys, int* units, int* splits, int* chunk, int* dual) {
    *dual = positions <= npos;
    const int64_t tiles = groups * ((positions + 2 * npos - 1) / (2 * npos));   // units of one key range; pieces, if dual
    int64_t want = (*dual ? 2 : 1) * kSms / tiles, most = (keys + kLeastKeys - 1) / kLeastKeys;
    if (want > most) want = most;
    if (want > 32) want = 32;
    if (want < 1) want = 1;
    *chunk = (int)(keys > 0 ? ((keys + want - 1) / want + kKeys - 1) / kKeys * kKeys : kKeys);
    *splits = (int)(keys > 0 ? (keys + *chunk - 1) / *chunk : 1);
    const int64_t all = tiles * *splits;
    *units = (int)(*dual ? (all + 1) / 2 : all);
  };
  split(HG, (int64_t)c.B * ts.N, shared, &p.units_s, &p.splits_s, &p.chunk_s, &p.dual_s);
  if (shared == 0) p.units_s = p.splits_s = 0;
  const int own = c.L_cap - ts.N - shared;
  // One or two rows per KV head, and enough (sequence, KV head) pairs to keep every SM reading: 192
  // pairs of one row with 63, 256 and 1024 own rows each behind 4096: 15.7, 19, 37 us so and 20.9,
  // 21.5, 35 on the tensor cores; of four rows 20, 27, 53 and 23, 24, 39; of eight 28 and 22, 41 and
  // 23. 64 pairs of one row 14.7, 17.6, 28 and 15.5, 14.6, 20. (From about 1000 own rows each the
  // tensor cores are as quick. Lengths are on the device; the capacity, which is known here, says
  // nothing about them.)
  p.tail = ts.N * (c.Hq / c.Hkv) <= kTailRows && (int64_t)c.B * c.Hkv >= kSms;
  int most_own;   // (a sequence's own rows are divided where its length is known)
  if (!p.tail) split((int64_t)c.B * HG, ts.N, own > 0 ? own : 0, &p.units_u, &p.splits_u, &most_own, &p.dual_u);
  p.parts = p.splits_s + p.splits_u;
  const size_t rows = (size_t)c.B * ts.N * c.Hq;
  p.ml_part = align_up(p.parts * rows * kPrefixD * 4, 256);
  p.total = p.ml_part + align_up(p.parts * rows * 8, 256);
  return p;
}

template <int D, bool kPrefix>
cudaError_t launch_rows(const CUtensorMap* m, const RowsArgs& a, int64_t units, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(rows_tc_kernel<D, kPrefix>, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<D>::smem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(rows_tc_kernel<D, kPrefix>, (unsigned)units, kThreads, Layout<D>::smem, st, m[0], m[1], m[2], m[3],
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
  a.scale_log2 = (float)(1.4426950408889634 / sqrt((double)c.D));
  a.O = static_cast<uint16_t*>(O);
  const int npos = kRows >> a.gp_shift;
  CUtensorMap m[5];
  if (!encode_3d(&m[0], c.D, Q, T, c.Hq, q_stride * 2, c.D * 2, npos, 1u << a.gp_shift) ||
      !encode_3d(&m[1], c.D, K, T, c.Hkv, k_stride * 2, c.D * 2, kKeys, 1) ||
      !encode_3d(&m[2], c.D, V, T, c.Hkv, v_stride * 2, c.D * 2, kKeys, 1))
    return cudaErrorInvalidValue;
  m[3] = m[1];
  m[4] = m[2];
  const int64_t units = ((int64_t)T / (2 * npos) + c.B) * (c.Hq >> a.gp_shift);   // at least as many as there are
  return c.D == 64 ? launch_rows<64, false>(m, a, units, st) : launch_rows<128, false>(m, a, units, st);
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
  a.units_s = p.units_s;
  a.splits_s = p.splits_s;
  a.chunk_s = p.chunk_s;
  a.dual_s = p.dual_s;
  a.units_u = p.units_u;
  a.splits_u = p.splits_u;
  a.dual_u = p.dual_u;
  a.scale_log2 = (float)(1.4426950408889634 / sqrt((double)kPrefixD));
  a.o_part = static_cast<float*>(ws);
  a.ml_part = reinterpret_cast<float*>(static_cast<char*>(ws) + p.ml_part);
  const int npos = kRows >> a.gp_shift;
  const uint64_t planes = (uint64_t)num_pages * c.Hkv, tplanes = (uint64_t)c.B * c.Hkv;
  CUtensorMap m[5];
  if (!encode_3d(&m[0], kPrefixD, Q, a.T, c.Hq, (uint64_t)c.Hq * kPrefixD * 2, kPrefixD * 2, npos, 1u << a.gp_shift) ||
      !encode_3d(&m[1], kPrefixD, Kp, page_rows, planes, kPrefixD * 2, (uint64_t)page_rows * kPrefixD * 2, kKeys, 1) ||
      !encode_3d(&m[2], kPrefixD, Vp, page_rows, planes, kPrefixD * 2, (uint64_t)page_rows * kPrefixD * 2, kKeys, 1) ||
      !encode_3d(&m[3], kPrefixD, Kt, ts.N, tplanes, kPrefixD * 2, (uint64_t)ts.N * kPrefixD * 2, kKeys, 1) ||
      !encode_3d(&m[4], kPrefixD, Vt, ts.N, tplanes, kPrefixD * 2, (uint64_t)ts.N * kPrefixD * 2, kKeys, 1))
    return cudaErrorInvalidValue;
  if (p.units_s + p.units_u > 0) {
    const cudaError_t e = launch_rows<kPrefixD, true>(m, a, p.units_s + p.units_u, st);
    if (e != cudaSuccess) return e;
  }
  cudaError_t e;
  if (p.tail) {
    const auto kernel = ts.N * (c.Hq / c.Hkv) == 1 ? prefix_tail_kernel<1, 4, 2> : prefix_tail_kernel<2, 4, 2>;
    e = launch_pdl(kernel, (unsigned)(c.B * c.Hkv), kTailThreads, 0, st, static_cast<const uint16_t*>(Q),
                   static_cast<const uint16_t*>(Kp), static_cast<const uint16_t*>(Vp), static_cast<const uint16_t*>(Kt),
                   static_cast<const uint16_t*>(Vt), a, static_cast<uint16_t*>(O));
    note_launches(1);
    return e != cudaSuccess ? e : cudaGetLastError();
  }
  const int64_t rows = (int64_t)a.T * c.Hq;
  e = launch_pdl(rows_merge_kernel, (unsigned)((rows * 32 + 255) / 256), 256, 0, st, static_cast<const float*>(a.o_part),
                 static_cast<const float*>(a.ml_part), rows, p.parts, static_cast<uint16_t*>(O));
  note_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace medusa
