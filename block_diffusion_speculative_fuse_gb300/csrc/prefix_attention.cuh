// Shared by the kernels of dflash_attention_prefix: how a call's work is cut
// up, and where its partial results lie.
//
// Entities.  The keys of a call are the prefixes of its groups (entities 0 ..
// ng-1, each seen by all rows of the group) and what follows, request by
// request (entities ng .. ng+batch-1).  Rows of a prefix: (request of the
// group, block row, query head of the KV head); of a request: (block row,
// query head).  An entity's rows are cut into tiles, its keys into chunks, and
// (entity, KV head, row tile) is a unit.
//
// The lengths are on the device, so the host cannot deal out the keys.  Every
// worker of a kernel derives the same list from them: all chunks of all units
// in order, cut into equal ranges, one per worker, wherever a unit ends.  A
// unit's part in one range is a segment; each leaves a partial (O, m, l) for
// the unit's rows.  Segment number = unit + worker is unique and below units +
// workers, which fixes its slot.  A last kernel joins the partials of each
// row in order.
//
// A prefix is cut short to whole pages that every row of the group sees
// (causal rows near its end, short requests), so prefix chunks need no mask.
#pragma once
#include "common.cuh"
#include "kernels.h"

namespace dflash {

constexpr int kMaxPrefixBatch = 1024;

struct PrefixList {            // one kernel's share of the work
  int chunk_keys;              // keys per chunk
  int tile_rows;               // rows per unit
  int workers;
  int prefix_tiles;            // row tiles of a prefix (0: not this kernel's)
  int suffix_tiles;            // row tiles of a request (0: not this kernel's)
  int* off;                    // [entities + 1] first chunk of each entity (written for the merge)
  float* part_o;               // [units + workers][tile_rows][d]
  float* part_ml;              // [units + workers][tile_rows][2]
};

struct PrefixParams {
  const uint16_t* q;           // [batch][n][hq][d]
  int batch, n, group, ng, hq, hkv, causal;
  float scale_log2;            // scale * log2(e)
  const uint16_t* pool;        // layer base
  const int32_t* page_table;
  int max_pages, n_pages;
  const int32_t *ctx_len, *prefix_len;
  uint16_t* out;
  float* lse;
  int32_t* status;
  int* cut;                    // [ng] prefix keys used (written for the merge)
  PrefixList list[2];          // small tiles (mma.sync), large tiles (tcgen05)
};

__device__ __forceinline__ int clamped_ctx(const PrefixParams& p, int r) {
  return min(max(__ldcg(p.ctx_len + r), 0), p.max_pages * 16);
}
// Units before entity e of the list (for the slots).
__device__ __forceinline__ int units_before(const PrefixParams& p, const PrefixList& L, int e) {
  return p.hkv * (min(e, p.ng) * L.prefix_tiles + max(e - p.ng, 0) * L.suffix_tiles);
}
__device__ __forceinline__ int entity_tiles(const PrefixParams& p, const PrefixList& L, int e) {
  return e < p.ng ? L.prefix_tiles : L.suffix_tiles;
}

// The list, by all threads of a CTA: cut[ng] (keys of each group's prefix),
// live[ng] (a request of the group whose table is read for it), off[ne + 1].
// scratch: 33 ints.
__device__ __forceinline__ void prefix_plan(const PrefixParams& p, const PrefixList& L, int* cut,
                                            int* live, int* off, int* scratch) {
  const int tid = threadIdx.x, nt = blockDim.x;
  for (int g = tid; g < p.ng; g += nt) {
    cut[g] = p.group > 1 ? min(max(__ldcg(p.prefix_len + g), 0), p.max_pages * 16) : 0;
    live[g] = p.batch;
  }
  __syncthreads();
  for (int r = tid; r < p.batch; r += nt) {
    const int raw = __ldcg(p.ctx_len + r);
    if (raw > p.max_pages * 16 && blockIdx.x == 0) raise_status(p.status, DFLASH_ERR_CAPACITY, 522);
    const int c = clamped_ctx(p, r);
    if (c > 0) {
      atomicMin(&cut[r / p.group], p.causal ? max(0, c - p.n + 1) : c);
      atomicMin(&live[r / p.group], r);
    }
  }
  __syncthreads();
  for (int g = tid; g < p.ng; g += nt) cut[g] = live[g] < p.batch ? cut[g] & ~15 : 0;
  __syncthreads();
  // exclusive scan of the entities' chunks, thread t taking a run of them
  const int ne = p.ng + p.batch;
  const int per = (ne + nt - 1) / nt;
  auto chunks = [&](int e) {
    int keys;
    if (e < p.ng) {
      keys = cut[e];
    } else {
      const int c = clamped_ctx(p, e - p.ng);
      keys = max(0, c - cut[(e - p.ng) / p.group]);
    }
    return (keys + L.chunk_keys - 1) / L.chunk_keys * p.hkv * entity_tiles(p, L, e);
  };
  const int e0 = min(ne, tid * per), e1 = min(ne, e0 + per);
  int sum = 0;
  for (int e = e0; e < e1; ++e) sum += chunks(e);
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, inc, o);
    if (tid % 32 >= o) inc += x;
  }
  if (tid % 32 == 31) scratch[tid / 32] = inc;
  __syncthreads();
  int run = inc - sum;
  for (int w = 0; w < tid / 32; ++w) run += scratch[w];
  for (int e = e0; e < e1; ++e) {
    off[e] = run;
    run += chunks(e);
  }
  if (tid == nt - 1) off[ne] = run;  // the last thread's run ends at the total
  __syncthreads();
  if (blockIdx.x == 0) {
    for (int e = tid; e <= ne; e += nt) L.off[e] = off[e];
    for (int g = tid; g < p.ng; g += nt) p.cut[g] = cut[g];
  }
}

__device__ __forceinline__ int chunks_per_worker(int total, int workers) {
  return max(1, (total + workers - 1) / workers);
}

// The entity that holds chunk c (off[e] <= c < off[e + 1]).
__device__ __forceinline__ int find_entity(const int* off, int ne, int c) {
  int lo = 0, hi = ne;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (off[mid] <= c) lo = mid;
    else hi = mid;
  }
  return lo;
}

}  // namespace dflash
