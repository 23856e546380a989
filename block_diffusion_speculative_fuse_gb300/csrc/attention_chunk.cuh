// Shared by the kernels over ragged chunks of rows (attention_chunk.cu,
// attention_mass.cu): the rows and lengths of a request.
#pragma once
#include "common.cuh"
#include "kernels.h"
#include "tc05.cuh"

namespace dflash {

// Of request r: its first row, its rows, its cached positions (their own among
// them).  Rows outside [0, T) or in falling order count as none (site `site`), a
// length beyond the page table as the table's (site + 1); both are recorded.
struct ChunkRequest {
  int start, n, ctx;
  __device__ ChunkRequest() : start(0), n(0), ctx(0) {}
  __device__ ChunkRequest(const int32_t* row_start, const int32_t* ctx_len, int r, int T, int max_pages,
                          int* status, int site) {
    start = __ldg(row_start + r);
    const int end = __ldg(row_start + r + 1);
    ctx = max(__ldg(ctx_len + r), 0);
    n = end - start;
    if (start < 0 || end > T || end < start) {
      raise_status(status, DFLASH_ERR_CAPACITY, site);
      start = n = 0;
    }
    if (ctx > max_pages * 16) {
      raise_status(status, DFLASH_ERR_CAPACITY, site + 1);
      ctx = max_pages * 16;
    }
  }
};

}  // namespace dflash
