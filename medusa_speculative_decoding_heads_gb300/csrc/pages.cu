// Pages of a KV cache: reserving, forking, freeing and compacting them, and storing a
// prompt's keys and values in them.
//
// "Speculative Decoding 원리와 가속 아키텍처" (blog.huny.dev), sections 5 and 6, keep a
// cache that grows and is rolled back; here several sequences may hold one page, counted
// in refs[]. A page is [Hkv][page_rows][D], contiguous in every layer's pool.
//
// The decisions (which page goes where) are integer scans over refs[] and the block
// tables, a few thousand words: one CTA makes them and leaves a list in the workspace.
// The bytes are moved by a second kernel over the whole GPU, which reads that list, so
// the host never waits for a count. Free pages are taken lowest id first, in order, so
// every result is the same from run to run.
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace medusa {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kScan = 8;                            // refs per thread and step of a scan
constexpr int kScanStep = kScan * kPlanThreads;

// Up to this many sequences and free pages the planning CTA keeps its lists in shared memory, not
// in the workspace (each step that reads back what another thread wrote is a round trip).
constexpr int kSmallB = 1024, kSmallList = 2048;

// Workspace: header | list A [num_pages] | list B [num_pages] | need [B] | copies [B] (source page, new page, rows)
struct PageWs {
  int32_t* head;   // [0]: number of moves (compaction)
  int32_t* a;
  int32_t* b;
  int32_t* need;
  int32_t* copies;
};
constexpr size_t kHeadBytes = 256;

size_t page_ws_bytes(int B, int num_pages) {
  return kHeadBytes + 2 * align_up((size_t)num_pages * 4, 256) + align_up((size_t)B * 4, 256) +
         align_up((size_t)B * 12, 256);
}

PageWs page_ws(void* ws, int B, int num_pages) {
  char* w = static_cast<char*>(ws);
  PageWs p;
  p.head = reinterpret_cast<int32_t*>(w);
  w += kHeadBytes;
  p.a = reinterpret_cast<int32_t*>(w);
  w += align_up((size_t)num_pages * 4, 256);
  p.b = reinterpret_cast<int32_t*>(w);
  w += align_up((size_t)num_pages * 4, 256);
  p.need = reinterpret_cast<int32_t*>(w);
  w += align_up((size_t)B * 4, 256);
  p.copies = reinterpret_cast<int32_t*>(w);
  return p;
}

__device__ __forceinline__ int warp_inclusive(int v) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if ((int)(threadIdx.x & 31) >= o) v += u;
  }
  return v;
}

// Calls emit(id, rank) for the ids of [0, n) that take(id) accepts, rank counting them in
// ascending order; returns their number (to every thread). A whole CTA of kPlanThreads
// calls it; sums: kScan * kPlanWarps + 1 ints of shared memory. It ends with the CTA
// synchronised. Stops early once `enough` are found (the count is then a lower bound).
template <typename Take, typename Emit>
__device__ int scan_ids(int n, int enough, int* sums, Take take, Emit emit) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int found = 0;
  for (int base = 0; base < n && found < enough; base += kScanStep) {
    unsigned votes[kScan];
#pragma unroll
    for (int i = 0; i < kScan; ++i) {
      const int id = base + i * kPlanThreads + (int)threadIdx.x;
      votes[i] = __ballot_sync(0xffffffffu, id < n && take(id));
      if (lane == 0) sums[i * kPlanWarps + warp] = __popc(votes[i]);
    }
    __syncthreads();
    if (warp == 0) {   // exclusive prefix over the kScan * 32 warp counts, in id order
      int run = 0;
#pragma unroll
      for (int i = 0; i < kScan; ++i) {
        const int c = sums[i * kPlanWarps + lane];
        const int inc = warp_inclusive(c);
        sums[i * kPlanWarps + lane] = run + inc - c;
        run += __shfl_sync(0xffffffffu, inc, 31);
      }
      if (lane == 0) sums[kScan * kPlanWarps] = run;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kScan; ++i)
      if ((votes[i] >> lane) & 1u)
        emit(base + i * kPlanThreads + (int)threadIdx.x,
             found + sums[i * kPlanWarps + warp] + __popc(votes[i] & ((1u << lane) - 1u)));
    found += sums[kScan * kPlanWarps];
    __syncthreads();
  }
  return found;
}

// need[0..n) -> its inclusive prefix sums, in place; returns the total. A whole CTA calls it.
__device__ int prefix_needs(int32_t* need, int n, int* sums) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int run = 0;
  for (int base = 0; base < n; base += kPlanThreads) {
    const int i = base + (int)threadIdx.x;
    const int inc = warp_inclusive(i < n ? need[i] : 0);
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    if (warp == 0) sums[lane] = warp_inclusive(sums[lane]);
    __syncthreads();
    if (i < n) need[i] = run + inc + (warp > 0 ? sums[warp - 1] : 0);
    run += sums[kPlanWarps - 1];
    __syncthreads();
  }
  return run;
}

// Pages for the rows each sequence needs: counts, the lowest free ids, then the entries.
__global__ void __launch_bounds__(kPlanThreads)
pages_reserve_kernel(int B, int max_pages, int num_pages, int page_rows, const int32_t* __restrict__ rows,
                     int32_t* __restrict__ table, int32_t* __restrict__ refs, uint32_t* __restrict__ flags, PageWs ws) {
  pdl_wait();
  pdl_trigger();
  __shared__ int sums[kScan * kPlanWarps + 1];
  __shared__ int32_t near_need[kSmallB], near_list[kSmallList];
  int32_t* need = B <= kSmallB ? near_need : ws.need;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // pages of sequence b's first rows, or -1 when the rows are out of range
  auto pages_of = [&](int b) {
    const int r = rows[b];
    return (r < 0 || r > max_pages * page_rows) ? -1 : (int)(((int64_t)r + page_rows - 1) / page_rows);
  };
  for (int b = warp; b < B; b += kPlanWarps) {
    const int np = pages_of(b);
    int c = 0;
    for (int i = lane; i < np; i += 32) c += table[(size_t)b * max_pages + i] < 0;
    c = __reduce_add_sync(0xffffffffu, c);
    if (lane == 0) need[b] = c;
  }
  __syncthreads();
  const int total = prefix_needs(need, B, sums);
  int32_t* list = total <= kSmallList ? near_list : ws.a;
  const int avail = scan_ids(num_pages, total, sums, [&](int id) { return refs[id] <= 0; },
                             [&](int id, int rank) {
                               if (rank < total) list[rank] = id;
                             });
  for (int b = warp; b < B; b += kPlanWarps) {
    const int np = pages_of(b), at = b > 0 ? need[b - 1] : 0, mine = need[b] - at;
    const bool ok = np >= 0 && (mine == 0 || need[b] <= avail);
    if (lane == 0) flags[b] = ok ? 0u : MEDUSA_FLAG_CAPACITY;
    if (!ok || mine == 0) continue;
    int given = at;
    for (int i0 = 0; i0 < np; i0 += 32) {
      const int i = i0 + lane;
      int32_t* e = table + (size_t)b * max_pages + i;
      const bool empty = i < np && *e < 0;
      const unsigned votes = __ballot_sync(0xffffffffu, empty);
      if (empty) {
        const int page = list[given + __popc(votes & ((1u << lane) - 1u))];
        *e = page;
        refs[page] = 1;
      }
      given += __popc(votes);
    }
  }
}

// Checks every fork, gives the ones that end inside a page a new page, and writes the
// tables, counts and the list of row copies (rows = 0: nothing to copy).
__global__ void __launch_bounds__(kPlanThreads)
pages_fork_kernel(int B, int max_pages, int num_pages, int page_rows, int n, const int32_t* __restrict__ src,
                  const int32_t* __restrict__ dst, int32_t* __restrict__ table, int32_t* __restrict__ L,
                  int32_t* __restrict__ refs, uint32_t* __restrict__ flags, PageWs ws) {
  pdl_wait();
  pdl_trigger();
  __shared__ int sums[kScan * kPlanWarps + 1];
  __shared__ int32_t near_need[kSmallB], near_list[kSmallList], near_roles[kSmallB];
  int32_t* need = n <= kSmallB ? near_need : ws.need;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // What each sequence is to the forks: 1 if some fork's source, plus 2 for each fork whose destination
  // it is. (Many sequences: in place of the copies, which are listed later. With each fork reading all
  // the others, 4000 forks took 1570 us, 307 so.)
  int32_t* roles = B <= kSmallB ? near_roles : ws.copies;
  for (int b = threadIdx.x; b < B; b += kPlanThreads) roles[b] = 0;
  __syncthreads();
  for (int f = threadIdx.x; f < n; f += kPlanThreads) {
    const int s = src[f], d = dst[f];
    if (s >= 0 && s < B) atomicOr(&roles[s], 1);
    if (d >= 0 && d < B) atomicAdd(&roles[d], 2);
  }
  __syncthreads();
  for (int f = warp; f < n; f += kPlanWarps) {
    const int s = src[f], d = dst[f];
    bool ok = s >= 0 && s < B && d >= 0 && d < B;
    int len = 0;
    if (ok) {
      len = L[s];
      ok = len >= 0 && len <= max_pages * page_rows;
    }
    bool bad = !ok || roles[d] != 2;   // a source, or another fork's destination, too
    if (ok) {
      for (int i = lane; i < max_pages; i += 32) bad |= table[(size_t)d * max_pages + i] >= 0;
      const int held = (int)(((int64_t)len + page_rows - 1) / page_rows);
      for (int i = lane; i < held; i += 32) {
        const int page = table[(size_t)s * max_pages + i];
        bad |= page < 0 || page >= num_pages;
      }
    }
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) {
      flags[f] = bad ? MEDUSA_FLAG_PAGES : 0u;
      need[f] = (!bad && len % page_rows != 0) ? 1 : 0;
    }
  }
  __syncthreads();
  const int total = prefix_needs(need, n, sums);
  int32_t* list = total <= kSmallList ? near_list : ws.a;
  const int avail = scan_ids(num_pages, total, sums, [&](int id) { return refs[id] <= 0; },
                             [&](int id, int rank) {
                               if (rank < total) list[rank] = id;
                             });
  // a source's rows are read and a destination's written: no sequence is both
  for (int f = warp; f < n; f += kPlanWarps) {
    const int rank = need[f] - 1;
    const bool wants = need[f] > (f > 0 ? need[f - 1] : 0);
    const uint32_t flag = flags[f];   // read by every lane before lane 0 may change it
    __syncwarp();
    int32_t* cp = ws.copies + 3 * f;
    const bool ok = flag == 0 && !(wants && rank >= avail);
    if (!ok) {
      if (lane == 0) {
        if (flag == 0) flags[f] = MEDUSA_FLAG_CAPACITY;
        cp[2] = 0;
      }
      continue;
    }
    const int s = src[f], d = dst[f], len = L[s], full = len / page_rows;
    for (int i = lane; i < full; i += 32) {
      const int page = table[(size_t)s * max_pages + i];
      table[(size_t)d * max_pages + i] = page;
      atomicAdd(&refs[page], 1);
    }
    if (lane == 0) {
      if (wants) {
        const int page = list[rank];
        cp[0] = table[(size_t)s * max_pages + full];
        cp[1] = page;
        table[(size_t)d * max_pages + full] = page;
        refs[page] = 1;
      }
      cp[2] = wants ? len % page_rows : 0;
      L[d] = len;
    }
  }
}

// Each entry that falls from a page to -1 is taken by exactly one thread (atomicExch), so
// a sequence named twice gives its pages back once.
__global__ void __launch_bounds__(256)
pages_free_kernel(int B, int max_pages, int num_pages, int n, const int32_t* __restrict__ seqs, int32_t* __restrict__ table,
                  int32_t* __restrict__ L, int32_t* __restrict__ refs) {
  pdl_wait();
  pdl_trigger();
  for (int f = blockIdx.x; f < n; f += gridDim.x) {
    const int s = seqs[f];
    if (s < 0 || s >= B) continue;
    for (int i = threadIdx.x; i < max_pages; i += blockDim.x) {
      const int page = atomicExch(&table[(size_t)s * max_pages + i], -1);
      MEDUSA_CHECK(page < num_pages, MEDUSA_CHECK_PAGE);
      if (page >= 0 && page < num_pages) atomicSub(&refs[page], 1);
    }
    if (threadIdx.x == 0) L[s] = 0;
  }
}

// Lists the free ids below the number of live pages (a) and the live ids from it on (b):
// equally many, paired in order. Writes the page map and moves the counts.
__global__ void __launch_bounds__(kPlanThreads)
pages_compact_plan_kernel(int num_pages, int32_t* __restrict__ refs, int32_t* __restrict__ page_map,
                          int32_t* __restrict__ n_live, PageWs ws) {
  pdl_wait();
  pdl_trigger();
  __shared__ int sums[kScan * kPlanWarps + 1];
  const int live = scan_ids(num_pages, num_pages, sums,
                            [&](int id) {
                              const bool l = refs[id] > 0;
                              page_map[id] = l ? id : -1;
                              return l;
                            },
                            [](int, int) {});
  scan_ids(live, live, sums, [&](int id) { return refs[id] <= 0; }, [&](int id, int rank) { ws.a[rank] = id; });
  const int moves = scan_ids(num_pages - live, num_pages, sums, [&](int id) { return refs[live + id] > 0; },
                             [&](int id, int rank) { ws.b[rank] = live + id; });
  for (int i = threadIdx.x; i < moves; i += kPlanThreads) {
    const int to = ws.a[i], from = ws.b[i];
    page_map[from] = to;
    refs[to] = refs[from];
    refs[from] = 0;
  }
  if (threadIdx.x == 0) {
    *n_live = live;
    ws.head[0] = moves;
  }
}

constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 4;                                    // 16-byte loads in flight per thread
constexpr int kCopyVec = kCopyThreads * kCopyUnroll;              // 16 KB per piece of a page

// `vecs` 16-byte words from s to d, by one CTA.
__device__ __forceinline__ void copy_block(const uint4* __restrict__ s, uint4* __restrict__ d, int vecs) {
  for (int i0 = threadIdx.x; i0 < vecs; i0 += kCopyVec) {
    uint4 v[kCopyUnroll];
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u)
      if (i0 + u * kCopyThreads < vecs) v[u] = s[i0 + u * kCopyThreads];
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u)
      if (i0 + u * kCopyThreads < vecs) d[i0 + u * kCopyThreads] = v[u];
  }
}

// Moves the listed pages in every layer, 16 KB pieces dealt out over the grid, and renames
// the block-table entries.
__global__ void __launch_bounds__(kCopyThreads)
pages_compact_move_kernel(uint4* __restrict__ Kp, uint4* __restrict__ Vp, size_t layer_vec, int page_vec, int n_layers,
                          int32_t* __restrict__ table, size_t entries, int num_pages,
                          const int32_t* __restrict__ page_map, PageWs ws) {
  pdl_wait();
  pdl_trigger();
  for (size_t e = blockIdx.x * (size_t)kCopyThreads + threadIdx.x; e < entries; e += (size_t)gridDim.x * kCopyThreads) {
    const int page = table[e];
    if (page >= 0 && page < num_pages) table[e] = page_map[page];
  }
  const int moves = ws.head[0];
  const int pieces = (page_vec + kCopyVec - 1) / kCopyVec;
  const size_t items = (size_t)moves * n_layers * 2 * pieces;
  for (size_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int piece = (int)(it % pieces);
    const size_t r = it / pieces;
    const int move = (int)(r / (2 * n_layers)), lk = (int)(r % (2 * n_layers));
    uint4* base = ((lk & 1) ? Vp : Kp) + (lk >> 1) * layer_vec + (size_t)piece * kCopyVec;
    const int left = page_vec - piece * kCopyVec;
    copy_block(base + (size_t)ws.b[move] * page_vec, base + (size_t)ws.a[move] * page_vec,
               left < kCopyVec ? left : kCopyVec);
  }
}

// The forks' row copies: one (fork, layer, K or V, head) run of rows per CTA and step.
__global__ void __launch_bounds__(kCopyThreads)
pages_fork_copy_kernel(uint4* __restrict__ Kp, uint4* __restrict__ Vp, size_t layer_vec, int head_vec, int row_vec, int Hkv,
                       int n_layers, int n, PageWs ws) {
  pdl_wait();
  pdl_trigger();
  const size_t items = (size_t)n * n_layers * 2 * Hkv;
  for (size_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int h = (int)(it % Hkv);
    const size_t r = it / Hkv;
    const int lk = (int)(r % (2 * n_layers));
    const int32_t* cp = ws.copies + 3 * (r / (2 * n_layers));
    const int rows = cp[2];
    if (rows == 0) continue;
    uint4* base = ((lk & 1) ? Vp : Kp) + (lk >> 1) * layer_vec + (size_t)h * head_vec;
    copy_block(base + (size_t)cp[0] * Hkv * head_vec, base + (size_t)cp[1] * Hkv * head_vec, rows * row_vec);
  }
}

// Packed prompt rows into pages: kStoreRows rows per CTA. Their places are looked up first
// (one thread per row), then the CTA copies K and V, 16 bytes per thread and step.
constexpr int kStoreRows = 8;

__global__ void __launch_bounds__(kCopyThreads)
kv_store_paged_kernel(const uint4* __restrict__ K, const uint4* __restrict__ V, int T, int64_t k_vec, int64_t v_vec,
                      const int32_t* __restrict__ cu, const int32_t* __restrict__ start, int B, uint4* __restrict__ Kp,
                      uint4* __restrict__ Vp, int num_pages, int page_rows, const int32_t* __restrict__ table, int max_pages,
                      int Hkv, int row_vec) {
  pdl_wait();
  pdl_trigger();
  __shared__ int64_t place[kStoreRows];   // first 16-byte word of the row in head 0 of its page; -1: not written
  const int row0 = blockIdx.x * kStoreRows;
  if (threadIdx.x < kStoreRows) {
    const int row = row0 + threadIdx.x;
    int64_t at = -1;
    if (row < T) {
      int lo = 0, hi = B;   // the last sequence that begins at or before the row
      while (hi - lo > 1) {
        const int mid = lo + ((hi - lo) >> 1);
        if (cu[mid] <= row) lo = mid;
        else hi = mid;
      }
      const int c0 = cu[lo], c1 = cu[lo + 1];
      if (c0 >= 0 && c1 <= T && row >= c0 && row < c1) {
        const int64_t lr = (int64_t)(start ? start[lo] : 0) + (row - c0);
        if (lr >= 0 && lr < (int64_t)max_pages * page_rows) {
          const int page = table[(size_t)lo * max_pages + (int)(lr / page_rows)];
          MEDUSA_CHECK(page >= 0 && page < num_pages, MEDUSA_CHECK_PAGE);
          if (page >= 0 && page < num_pages) at = ((int64_t)page * Hkv * page_rows + lr % page_rows) * row_vec;
        }
      }
    }
    place[threadIdx.x] = at;
  }
  __syncthreads();
  const int per_row = Hkv * row_vec, items = kStoreRows * 2 * per_row;
  const size_t head_vec = (size_t)page_rows * row_vec;
  for (int i0 = threadIdx.x; i0 < items; i0 += kCopyVec) {
    uint4 v[kCopyUnroll];
    uint4* d[kCopyUnroll];
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u) {
      const int i = i0 + u * kCopyThreads;
      const int c = i % per_row, rk = i / per_row;   // word within the row; (row, K or V)
      const int64_t at = i < items ? place[rk >> 1] : -1;
      d[u] = nullptr;
      if (at >= 0) {
        const int64_t row = row0 + (rk >> 1);
        v[u] = (rk & 1) ? V[row * v_vec + c] : K[row * k_vec + c];
        d[u] = ((rk & 1) ? Vp : Kp) + at + (c / row_vec) * head_vec + c % row_vec;
      }
    }
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u)
      if (d[u]) *d[u] = v[u];
  }
}

int max_pages_of(const medusa_cfg& c, int page_rows) { return c.L_cap / page_rows; }
int elt_of(const medusa_cfg& c) { return c.dtype == MEDUSA_F32 ? 4 : 2; }

// CTAs of a copy at most, 8 of which fit an SM at a time: with four rounds of them the SMs end
// together (compacting 48 sequences' pages 246 us with one round, 229 with four; 31 forks 81, 72).
constexpr int kCopyGrid = 152 * 32;

}  // namespace

MEDUSA_CHECK_TAKE(pages_take_checks)

size_t pages_workspace(const medusa_cfg& c, int num_pages) { return page_ws_bytes(c.B, num_pages); }

cudaError_t launch_pages_reserve(const medusa_cfg& c, int num_pages, int page_rows, const int32_t* rows, int32_t* table,
                                 int32_t* refs, uint32_t* flags, void* ws, cudaStream_t st) {
  const cudaError_t e = launch_pdl(pages_reserve_kernel, 1, kPlanThreads, 0, st, c.B, max_pages_of(c, page_rows), num_pages,
                                   page_rows, rows, table, refs, flags, page_ws(ws, c.B, num_pages));
  note_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_pages_fork(const medusa_cfg& c, void* Kp, void* Vp, int num_pages, int page_rows, int n_layers,
                              size_t pool_layer_elems, int n, const int32_t* src, const int32_t* dst, int32_t* table,
                              int32_t* L, int32_t* refs, uint32_t* flags, void* ws, cudaStream_t st) {
  const PageWs w = page_ws(ws, c.B, num_pages);
  cudaError_t e = launch_pdl(pages_fork_kernel, 1, kPlanThreads, 0, st, c.B, max_pages_of(c, page_rows), num_pages, page_rows,
                             n, src, dst, table, L, refs, flags, w);
  note_launches(1);
  if (e != cudaSuccess) return e;
  const int per16 = 16 / elt_of(c), row_vec = c.D / per16;
  const size_t items = (size_t)n * n_layers * 2 * c.Hkv;
  e = launch_pdl(pages_fork_copy_kernel, (unsigned)(items < kCopyGrid ? items : kCopyGrid), kCopyThreads, 0, st,
                 static_cast<uint4*>(Kp), static_cast<uint4*>(Vp), pool_layer_elems / per16, page_rows * row_vec, row_vec,
                 c.Hkv, n_layers, n, w);
  note_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_pages_free(const medusa_cfg& c, int num_pages, int page_rows, int n, const int32_t* seqs, int32_t* table,
                              int32_t* L, int32_t* refs, cudaStream_t st) {
  const cudaError_t e = launch_pdl(pages_free_kernel, n < kCopyGrid ? n : kCopyGrid, 256, 0, st, c.B,
                                   max_pages_of(c, page_rows), num_pages, n, seqs, table, L, refs);
  note_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_pages_compact(const medusa_cfg& c, void* Kp, void* Vp, int num_pages, int page_rows, int n_layers,
                                 size_t pool_layer_elems, int32_t* table, int32_t* refs, int32_t* page_map, int32_t* n_live,
                                 void* ws, cudaStream_t st) {
  const PageWs w = page_ws(ws, c.B, num_pages);
  cudaError_t e =
      launch_pdl(pages_compact_plan_kernel, 1, kPlanThreads, 0, st, num_pages, refs, page_map, n_live, w);
  note_launches(1);
  if (e != cudaSuccess) return e;
  const int per16 = 16 / elt_of(c);
  const int page_vec = c.Hkv * page_rows * (c.D / per16);
  // at most half of the pages move; and every table entry is looked at
  const size_t entries = (size_t)c.B * max_pages_of(c, page_rows), pieces = (page_vec + kCopyVec - 1) / kCopyVec;
  const size_t most = (size_t)(num_pages / 2) * n_layers * 2 * pieces, look = (entries + kCopyThreads - 1) / kCopyThreads;
  const size_t want = most > look ? most : look;
  e = launch_pdl(pages_compact_move_kernel, (unsigned)(want < kCopyGrid ? want : kCopyGrid), kCopyThreads, 0, st, static_cast<uint4*>(Kp), static_cast<uint4*>(Vp),
                 pool_layer_elems / per16, page_vec, n_layers, table, entries, num_pages,
                 static_cast<const int32_t*>(page_map), w);
  note_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_kv_store_paged(const medusa_cfg& c, const void* K, const void* V, int T, int64_t k_stride, int64_t v_stride,
                                  const int32_t* cu, const int32_t* start, void* Kp, void* Vp, int num_pages, int page_rows,
                                  const int32_t* table, cudaStream_t st) {
  const int per16 = 16 / elt_of(c);
  const cudaError_t e = launch_pdl(
      kv_store_paged_kernel, (unsigned)(((int64_t)T + kStoreRows - 1) / kStoreRows), kCopyThreads, 0, st, static_cast<const uint4*>(K),
      static_cast<const uint4*>(V), T, k_stride / per16, v_stride / per16, cu, start, c.B, static_cast<uint4*>(Kp),
      static_cast<uint4*>(Vp), num_pages, page_rows, table, max_pages_of(c, page_rows), c.Hkv, c.D / per16);
  note_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace medusa
