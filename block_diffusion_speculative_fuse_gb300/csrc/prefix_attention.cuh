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
// worker of a kernel derives the same list from them: all units in order, each
// with a cost of unit_cost plus chunk_cost for every chunk, cut into ranges of
// equal cost, one per worker; a chunk belongs to the worker in whose range its
// cost starts.  A unit's part in one range is a segment; each leaves a partial
// (O, m, l) for the unit's rows.  From one segment to the next the unit goes up, or
// the worker, so the rows of the units before plus the worker times the rows of the
// largest unit fix a place for it that no other segment's overlaps.  A last kernel
// joins the partials of each row in order.
//
// A prefix is cut short to whole pages that every row of the group sees
// (causal rows near its end, short requests), so prefix chunks need no mask.
#pragma once
#include "common.cuh"
#include "kernels.h"
#include "tc05.cuh"

namespace dflash {

constexpr int kMaxPrefixBatch = 1024;

struct PrefixList {            // one kernel's share of the work
  int chunk_shift;             // log2 of the keys per chunk
  int tile_rows;               // rows per unit
  int prefix_rows, suffix_rows;  // of a unit's partial: tile_rows, or less in a single tile
  int worker_rows;             // the larger of them, of those that there are
  int workers;
  int prefix_tiles;            // row tiles of a prefix (0: not this kernel's)
  int suffix_tiles;            // row tiles of a request (0: not this kernel's)
  int unit_cost;               // see above; a range is at least one chunk's cost
  int prefix_cost, suffix_cost;  // of a chunk: log2
  int prefix_split, suffix_split;  // large tiles: at most 128 rows (see there)
  int* off;                    // [entities + 1] cost before each entity (written for the join)
  int* unit;                   // [entities + 1] cost of one of its units; last: of a worker's range
  float* part_o;               // [rows of all units + workers * worker_rows][d]
  float* part_ml;              // [the same][2]
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
  unsigned inv_n, inv_G, inv_group;  // for n, hq / hkv and group: 2^32 / d rounded up (0 for d = 1)
  PrefixList list[2];          // small tiles (mma.sync), large tiles (tcgen05)
};

// First row of the partial that `worker` leaves for unit ul of entity e.
__device__ __forceinline__ size_t part_row(const PrefixParams& p, const PrefixList& L, int e, int ul, int worker) {
  const size_t before = static_cast<size_t>(p.hkv * min(e, p.ng) * L.prefix_tiles + (e < p.ng ? ul : 0)) * L.prefix_rows;
  const size_t own = e < p.ng ? 0 : static_cast<size_t>(p.hkv * (e - p.ng) * L.suffix_tiles + ul) * L.suffix_rows;
  return before + own + static_cast<size_t>(worker) * L.worker_rows;
}
__device__ __forceinline__ int entity_tiles(const PrefixParams& p, const PrefixList& L, int e) {
  return e < p.ng ? L.prefix_tiles : L.suffix_tiles;
}

// x / d by its rounded-up inverse: exact while x * d < 2^32 (rows of an entity
// stay below 2^19 with d up to 32, requests and groups below 2^11).
__device__ __forceinline__ int inv_div(int x, unsigned inv) {
  return inv == 0 ? x : static_cast<int>(__umulhi(static_cast<unsigned>(x), inv));
}

// a / b for 0 <= a, 0 < b and a quotient below 2^20, by way of a float quotient
// that is off by one at most.
__device__ __forceinline__ int small_div(int a, int b) {
  int q = static_cast<int>(__fdividef(static_cast<float>(a), static_cast<float>(b)));
  const int r = a - q * b;
  if (r < 0) --q;
  if (r >= b) ++q;
  return q;
}

__device__ __forceinline__ int chunk_cost(const PrefixParams& p, const PrefixList& L, int e) {
  return e < p.ng ? L.prefix_cost : L.suffix_cost;
}

__device__ __forceinline__ int cost_per_worker(const PrefixList& L, int total) {
  return max(1 << max(L.prefix_cost, L.suffix_cost), (total + L.workers - 1) / L.workers);
}

// What every CTA works out first, in shared memory.
struct PrefixPlan {
  int* ctx;      // [batch] context lengths, within the page table
  int* cut;      // [ng] keys of each group's prefix
  int* live;     // [ng] a request of the group whose page-table row is read for it
  int* off;      // [entities + 1] cost before each entity
  int* unit;     // [entities] cost of one of its units
  int* scratch;  // [32]
  __host__ __device__ static int ints(int batch, int ng) { return 3 * batch + 4 * ng + 33; }
  __device__ PrefixPlan(int* mem, int batch, int ng)
      : ctx(mem), cut(ctx + batch), live(cut + ng), off(live + ng), unit(off + ng + batch + 1),
        scratch(unit + ng + batch) {}
};

// The list, by all threads of a CTA.
__device__ __forceinline__ void prefix_plan(const PrefixParams& p, int list, const PrefixPlan& pl) {
  const PrefixList& L = p.list[list];
  const int tid = threadIdx.x, nt = blockDim.x;
  const int cap = p.max_pages * 16;
  for (int r = tid; r < p.batch; r += nt) {
    const int raw = __ldcg(p.ctx_len + r);
    if (raw > cap && blockIdx.x == 0) raise_status(p.status, DFLASH_ERR_CAPACITY, 522);
    pl.ctx[r] = min(max(raw, 0), cap);
  }
  for (int g = tid; g < p.ng; g += nt) {
    pl.cut[g] = p.group > 1 ? min(max(__ldcg(p.prefix_len + g), 0), cap) : 0;
    pl.live[g] = p.batch;
  }
  __syncthreads();
  if (p.group > 1) {
    for (int r = tid; r < p.batch; r += nt) {
      const int c = pl.ctx[r], g = inv_div(r, p.inv_group);
      if (c > 0) {
        atomicMin(&pl.cut[g], p.causal ? max(0, c - p.n + 1) : c);
        atomicMin(&pl.live[g], r);
      }
    }
    __syncthreads();
    for (int g = tid; g < p.ng; g += nt) pl.cut[g] = pl.live[g] < p.batch ? pl.cut[g] & ~15 : 0;
    __syncthreads();
  }
  // exclusive scan of the entities' costs, thread t taking a run of them
  const int ne = p.ng + p.batch;
  const int per = (ne + nt - 1) / nt;
  auto cost = [&](int e) {
    const int keys = e < p.ng ? pl.cut[e] : max(0, pl.ctx[e - p.ng] - pl.cut[inv_div(e - p.ng, p.inv_group)]);
    const int n = (keys + (1 << L.chunk_shift) - 1) >> L.chunk_shift;
    const int unit = n > 0 ? L.unit_cost + (n << chunk_cost(p, L, e)) : 0;
    pl.unit[e] = unit;
    return unit * p.hkv * entity_tiles(p, L, e);
  };
  const int e0 = min(ne, tid * per), e1 = min(ne, e0 + per);
  int sum = 0;
  for (int e = e0; e < e1; ++e) sum += cost(e);
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, inc, o);
    if (tid % 32 >= o) inc += x;
  }
  if (tid % 32 == 31) pl.scratch[tid / 32] = inc;
  __syncthreads();
  int run = inc - sum;
  for (int w = 0; w < tid / 32; ++w) run += pl.scratch[w];
  for (int e = e0; e < e1; ++e) {
    pl.off[e] = run;
    run += pl.unit[e] * p.hkv * entity_tiles(p, L, e);
  }
  if (tid == nt - 1) pl.off[ne] = run;  // the last thread's run ends at the total
  __syncthreads();
  if (blockIdx.x == 0) {
    for (int e = tid; e <= ne; e += nt) {
      L.off[e] = pl.off[e];
      L.unit[e] = e < ne ? pl.unit[e] : cost_per_worker(L, pl.off[ne]);
    }
  }
}

// The entity in whose cost c lies (off[e] <= c < off[e + 1]).
__device__ __forceinline__ int find_entity(const int* off, int ne, int c) {
  int lo = 0, hi = ne;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (off[mid] <= c) lo = mid;
    else hi = mid;
  }
  return lo;
}

// A worker's segments, one after the other.
struct Segments {
  int c, end;          // cost still to do
  int e;               // entity
  int ul;              // unit of the entity: head * tiles + tile
  int chunk0, chunk1;  // the segment's chunks
  int nch;             // the unit's
  __device__ Segments(const PrefixList& L, const int* off, int ne, int worker) {
    const int total = off[ne];
    const int per = cost_per_worker(L, total);
    const long long lo = static_cast<long long>(worker) * per;
    c = lo < total ? static_cast<int>(lo) : total;
    end = min(total - c, per) + c;
    e = c < end ? find_entity(off, ne, c) : 0;
  }
  __device__ bool next(const PrefixParams& p, const PrefixList& L, const PrefixPlan& pl) {
    while (c < end) {
      while (pl.off[e + 1] <= c) ++e;
      const int cw = chunk_cost(p, L, e), half = (1 << cw) - 1;
      const int unit = pl.unit[e];
      nch = (unit - L.unit_cost) >> cw;
      ul = small_div(c - pl.off[e], unit);
      const int first = pl.off[e] + ul * unit + L.unit_cost;  // where its chunks start
      // chunks whose start lies in [c, end)
      chunk0 = c > first ? (c - first + half) >> cw : 0;
      chunk1 = end > first ? min(nch, (end - first + half) >> cw) : 0;
      c = first - L.unit_cost + unit;
      if (chunk0 < chunk1) return true;
    }
    return false;
  }
};

// The workers [w0, w1] that have chunks of unit ul of entity e (off_e: the cost
// before the entity, unit: of one unit, per: of a worker's range).
__device__ __forceinline__ void unit_workers(const PrefixParams& p, const PrefixList& L, int e, int ul, int off_e,
                                             int unit, int per, int* w0, int* w1) {
  *w0 = small_div(off_e + ul * unit + L.unit_cost, per);
  *w1 = small_div(off_e + (ul + 1) * unit - (1 << chunk_cost(p, L, e)), per);
}

// Row `row` of an entity: its block row, and its vector of q and out
// ([batch][n][hq]); false past the entity's rows.
struct RowMap {
  int req0, n, G, hq, kvh, rows;
  unsigned inv_n, inv_G;
  __device__ RowMap(const PrefixParams& p, int e, int kv_head)
      : req0(e < p.ng ? e * p.group : e - p.ng), n(p.n), G(p.hq / p.hkv), hq(p.hq), kvh(kv_head),
        rows((e < p.ng ? p.group : 1) * p.n * (p.hq / p.hkv)), inv_n(p.inv_n), inv_G(p.inv_G) {}
  __device__ __forceinline__ bool at(int row, int* i, size_t* vec) const {
    if (row >= rows) return false;
    const int bi = inv_div(row, inv_G), h = row - bi * G;
    const int r = inv_div(bi, inv_n);
    *i = bi - r * n;
    *vec = (static_cast<size_t>(req0) * n + bi) * hq + kvh * G + h;
    return true;
  }
};

// Large tiles (prefix_attention_tc05.cu).  map: the pool as [rows / 8][d / 64][8
// rows][64 columns], box one 16-row page.
constexpr int kTcCtas = 152;
cudaError_t prefix_tc_launch(const CUtensorMap& map, int group0, int oob_group, const PrefixParams& p,
                             int d, cudaStream_t s);

}  // namespace dflash
