// Attention of new tokens over the pages of a cache: what its kernels share.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/medusa.h"

namespace medusa {

struct ChunkArgs {
  const int32_t* cu;      // [B + 1]
  const int32_t* start;   // [B], or NULL: 0
  const int32_t* table;   // [B][max_pages]
  int B, T, Hq, Hkv;
  int L_cap, page_rows, max_pages, num_pages;
  int window, sinks;      // row p sees keys j <= p with j > p - window or j < sinks
  int64_t q_stride;
  float scale_log2;
};

size_t chunk_workspace(const medusa_cfg& c, int T);
cudaError_t launch_chunk_attention(const medusa_cfg& c, const void* Q, const void* Kp, const void* Vp, void* O, const ChunkArgs& a,
                                   void* ws, cudaStream_t st);

}  // namespace medusa
