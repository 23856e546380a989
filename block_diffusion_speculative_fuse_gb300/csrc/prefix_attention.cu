// Attention over the paged cache for batches whose requests share a prefix:
// the small-tile kernel and the join of the partial results.
//
//   s_j = scale q.k_j, o = sum_j exp(s_j) v_j / sum_j exp(s_j)
//
// over the keys a row sees, with a running maximum and sum per row (in the
// exp2 domain, fp32).  See prefix_attention.cuh for how the work is cut up.
//
// Small tiles (mma.sync, 16 rows).  With one token per request a unit has at
// most 16 rows, 16 flop per key byte: the bound is bytes, and the many short
// ranges favour independent workers over large tiles.  A worker is one warp:
// a page (16 keys) is a step of two m16n8 score tiles and one k16 step of the
// product with V, fed by the warp's own ring of pages through cp.async, with
// no barrier between warps.  32 requests of 1024 own keys, 8 KV heads of 128:
// 68 MB in 16 us (22 alone from cold), 4.2 TB/s; a warp's range is 13 pages, so
// the plan and the ring's start are a third of it.
#include <climits>

#include "attention.cuh"
#include "common.cuh"
#include "kernels.h"
#include "prefix_attention.cuh"

namespace dflash {

namespace {

constexpr int kSmallWarps = 8;
constexpr int kSmallCtas = 152;    // one per SM
constexpr int kSmallRows = 16;
// An entity with more rows per KV head goes to the large tiles (the lengths are
// not known here).  Small / large, us a call, 8 KV heads of 128: a prefix of 8192
// keys, 32 rows 24.3 / 27.2, 48 rows 27.7 / 28.5, 128 rows 41.4 / 30.3; 16 or 32
// requests' own keys, 32 rows of 64 keys 13.2 / 23.8, of 600 keys 37.1 / 36.0, of
// 2048 keys 49.5 / 35.4, 64 rows of 2048 keys 88.3 / 38.0.  At 17 to 32 rows the
// small tiles lose with the length, because the second tile of 16 rows fetches the
// keys again: 32 requests, 32 rows, 608 keys 29.7 / 33.3, 2048 keys 90.2 / 60.5,
// 16384 keys 616 / 325.
constexpr int kTcMinRows = 32;

template <int D>
struct SmallCfg {
  static constexpr int PAGE = 16 * D * 2;          // bytes of one page of K or V
  static constexpr int STAGES = D == 128 ? 3 : 6;  // pages in flight per warp
  static constexpr int RING = STAGES * 2 * PAGE;
};

// 16 bytes global -> shared (zeros when bytes is 0) under an L2 policy.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(bytes), "l"(policy)
               : "memory");
}

template <int D>
__global__ void __launch_bounds__(kSmallWarps * 32, 1) prefix_small_kernel(const PrefixParams p) {
  using C = SmallCfg<D>;
  extern __shared__ __align__(128) uint8_t smem[];
  const PrefixList& L = p.list[0];
  const int ne = p.ng + p.batch;
  const PrefixPlan pl(reinterpret_cast<int*>(smem + kSmallWarps * C::RING), p.batch, p.ng);
  // After the large-tile kernel there is nothing to wait for: this one starts
  // only when every CTA of that one has waited for what came before (it lets its
  // dependents go after that), and the two share no memory.  So the first CTAs
  // start here while the last still work there.
  const bool behind_tc = p.list[1].workers > 0;
  griddep_launch_dependents();
  if (!behind_tc) griddep_wait();
  prefix_plan(p, 0, pl);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int worker = blockIdx.x * kSmallWarps + warp;
  uint8_t* ring = smem + warp * C::RING;
  const uint32_t ring_a = smem_u32(ring);
  const size_t head_elems = 16 * D;
  const size_t page_elems = static_cast<size_t>(2) * p.hkv * head_elems;
  const int tq = lane % 4, tg = lane / 4;
  // Shared-memory offsets of a lane.  A page row's 16-byte pieces are permuted by
  // XOR with the row's low bits; an even step along a row, or whole rows, then
  // only flips bits of the first offset, or adds to it.
  constexpr int RPI = 32 / (D / 8);  // rows of a page that one load instruction covers
  const uint32_t ld_off = swz<D>(lane / (D / 8), lane % (D / 8));
  const uint32_t k_off = swz<D>((lane & 7) + (lane >> 4) * 8, (lane >> 3) & 1);
  const uint32_t v_off = swz<D>((lane & 7) + ((lane >> 3) & 1) * 8, lane >> 4);
  const uint32_t q_off = v_off;
  const uint64_t pol = l2_policy_evict_first();  // keys are read once, or by neighbouring workers at once

  Segments seg(L, pl.off, ne, worker);
  while (seg.next(p, L, pl)) {
    // ---- the segment: unit (e, kvh, tile), its pages [pg0, pg1)
    const int e = seg.e, pg0 = seg.chunk0, pg1 = seg.chunk1;
    const int tiles = entity_tiles(p, L, e);
    const int kvh = small_div(seg.ul, tiles), tile = seg.ul - kvh * tiles;
    const size_t slot_row = part_row(p, L, e, seg.ul, worker);
    const bool pre = e < p.ng;
    const int req_t = pre ? pl.live[e] : e - p.ng;               // whose table row
    const int page0 = pre ? 0 : pl.cut[inv_div(e - p.ng, p.inv_group)] / 16;
    const int ctx = pre ? pl.cut[e] : pl.ctx[e - p.ng];  // keys at or past it take no part
    const int common = pre || !p.causal ? ctx : ctx - p.n + 1;  // keys before it are seen by all rows
    const int32_t* table = p.page_table + static_cast<size_t>(req_t) * p.max_pages + page0;
    const RowMap map(p, e, kvh);

    // ---- the query rows to the ring's last stage (free until the second page
    // is done), and the limits of rows tg, tg + 8 of the tile
    int lim[2];
    {
      const uint32_t qs = ring_a + (C::STAGES - 1) * (2 * C::PAGE);
#pragma unroll
      for (int i = 0; i < C::PAGE / 512; ++i) {
        int bi;
        size_t vec = 0;
        const bool ok = map.at(tile * kSmallRows + i * RPI + lane / (D / 8), &bi, &vec);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(qs + (ld_off ^ ((i * RPI & 7) << 4)) + i * 512),
                     "l"(p.q + (ok ? vec : 0) * D + lane % (D / 8) * 8), "r"(ok ? 16 : 0)
                     : "memory");
      }
      cp_async_commit();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        int i = 0;
        size_t vec;
        const bool ok = map.at(tile * kSmallRows + tg + 8 * h, &i, &vec);
        lim[h] = !ok ? 0 : pre ? INT_MAX : p.causal ? ctx - p.n + i + 1 : ctx;
      }
    }

    // ---- page ids, 32 at a time, one per lane
    int ids = 0, left = 0;  // ids not yet used: lanes [32 - left, 32)
    int pg_ids = pg0;
    auto page_id = [&]() {
      if (left == 0) {
        const int j = pg_ids + lane;
        ids = j < pg1 ? __ldcg(table + j) : 0;
        if (ids < 0 || ids >= p.n_pages) {
          raise_status(p.status, DFLASH_ERR_CAPACITY, 521);
          ids = -1;
        }
        pg_ids += 32;
        left = 32;
      }
      return __shfl_sync(0xffffffffu, ids, 32 - left--);
    };
    int st_load = 0, st_use = 0;  // ring positions
    auto load_page = [&]() {
      const int id = page_id();
      const uint16_t* k = p.pool + (id < 0 ? 0 : id) * page_elems + kvh * head_elems + lane * 8;
      const uint16_t* v = k + p.hkv * head_elems;
      const uint32_t st = ring_a + st_load * (2 * C::PAGE);
      st_load = st_load == C::STAGES - 1 ? 0 : st_load + 1;
      const int bytes = id < 0 ? 0 : 16;
#pragma unroll
      for (int i = 0; i < C::PAGE / 512; ++i) {  // 16-byte piece i * 32 + lane of the page
        const uint32_t o = st + (ld_off ^ ((i * RPI & 7) << 4)) + i * 512;
        copy16(o, k + i * 256, bytes, pol);
        copy16(o + C::PAGE, v + i * 256, bytes, pol);
      }
    };

    float o[D / 8][4];
    float m_r[2] = {-INFINITY, -INFINITY}, l_r[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    // keys that both of this thread's rows see without a mask
    const int clear = min(min(lim[0], lim[1]), ctx);

#pragma unroll
    for (int s = 0; s < C::STAGES - 1; ++s) {
      if (pg0 + s < pg1) load_page();
      cp_async_commit();
    }
    uint32_t qf[D / 16][4];
    cp_async_wait<C::STAGES - 1>();
    __syncwarp();
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
      ldsm_x4(ring_a + (C::STAGES - 1) * (2 * C::PAGE) + (q_off ^ (kk << 5)), qf[kk][0], qf[kk][1], qf[kk][2], qf[kk][3]);
    __syncwarp();
    for (int pg = pg0; pg < pg1; ++pg) {
      if (pg + C::STAGES - 1 < pg1) load_page();
      cp_async_commit();
      cp_async_wait<C::STAGES - 1>();
      __syncwarp();
      const uint32_t kb = ring_a + st_use * (2 * C::PAGE);
      const uint32_t vb = kb + C::PAGE;
      st_use = st_use == C::STAGES - 1 ? 0 : st_use + 1;
      const int key0 = (page0 + pg) * 16;
      if (key0 + 16 > common) {
        // 0 * V must be 0.  Positions at or past the context hold whatever was
        // there; of those that only some rows see, what is not finite goes, and
        // the rows that see it get a NaN by way of l
        int bad = INT_MAX;
        for (int i = lane; i < 16 * (D / 8); i += 32) {
          const int key = key0 + i / (D / 8);
          if (key < common) continue;
          const uint32_t at = vb + swz<D>(i / (D / 8), i % (D / 8));
          if (key < ctx) {
            if (!bf16_not_finite(ld_shared_u4(at))) continue;
            bad = min(bad, key);
          }
          st_shared_u4(at, make_uint4(0u, 0u, 0u, 0u));
        }
        bad = __reduce_min_sync(0xffffffffu, bad);
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (lim[h] > bad) l_r[h] = __int_as_float(0x7FFFFFFF);
        __syncwarp();
      }
      // S = Q K^T: keys 0-7 and 8-15, each in two independent sums
      float s[2][2][4];
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i / 8][i / 4 % 2][i % 4] = 0.f;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        uint32_t b0, b1, b2, b3;
        ldsm_x4(kb + (k_off ^ (kk << 5)), b0, b1, b2, b3);
        mma16816(s[kk & 1][0], qf[kk], b0, b1);
        mma16816(s[kk & 1][1], qf[kk], b2, b3);
      }
      // scale, mask, maximum of rows tg and tg + 8
      float x[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          x[h][j] = (s[0][j / 2][2 * h + j % 2] + s[1][j / 2][2 * h + j % 2]) * p.scale_log2;
      if (__any_sync(0xffffffffu, key0 + 16 > clear)) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int key = key0 + (j / 2) * 8 + tq * 2 + j % 2;
            if (key >= lim[h] || key >= ctx) x[h][j] = -INFINITY;
          }
      }
      float mx[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        mx[h] = fmaxf(fmaxf(x[h][0], x[h][1]), fmaxf(x[h][2], x[h][3]));
        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
      }
      // the reference maximum moves, and O and l with it, only when exceeded by
      // 2^8 (P stays below 2^8; its rounding to bf16, the type of V, is relative:
      // the output is off by 2.2e-3 rms of its values where the rounding of the
      // output alone makes 1.7e-3)
      const bool up0 = mx[0] > m_r[0] + 8.f, up1 = mx[1] > m_r[1] + 8.f;
      if (__any_sync(0xffffffffu, up0 || up1)) {
        const float f0 = up0 ? ex2(m_r[0] - mx[0]) : 1.f, f1 = up1 ? ex2(m_r[1] - mx[1]) : 1.f;
        if (up0) m_r[0] = mx[0];
        if (up1) m_r[1] = mx[1];
        l_r[0] *= f0;
        l_r[1] *= f1;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          o[i][0] *= f0;
          o[i][1] *= f0;
          o[i][2] *= f1;
          o[i][3] *= f1;
        }
      }
      uint32_t a[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float ref = m_r[h] == -INFINITY ? 0.f : m_r[h];
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[h][j] = ex2(x[h][j] - ref);
          sum += x[h][j];
        }
        l_r[h] += sum;  // this thread's keys only
        a[h] = bf16x2(x[h][0], x[h][1]);
        a[2 + h] = bf16x2(x[h][2], x[h][3]);
      }
#pragma unroll
      for (int nd = 0; nd < D / 8; nd += 2) {
        uint32_t b0, b1, b2, b3;
        ldsm_x4_t(vb + (v_off ^ (nd << 4)), b0, b1, b2, b3);
        mma16816(o[nd], a, b0, b1);
        mma16816(o[nd + 1], a, b2, b3);
      }
      __syncwarp();  // all lanes are done with the stage before it is refilled
    }

    // ---- partial of the segment
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float l = l_r[h];
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      const int row = tile * kSmallRows + tg + 8 * h;
      if (row < map.rows) {
        const size_t ps = slot_row + tg + 8 * h;
        float* dst = L.part_o + ps * D;
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
          *reinterpret_cast<float2*>(dst + i * 8 + tq * 2) = make_float2(o[i][2 * h], o[i][2 * h + 1]);
        if (tq == 0) *reinterpret_cast<float2*>(L.part_ml + ps * 2) = make_float2(m_r[h], l);
      }
    }
  }
  if (behind_tc) griddep_wait();  // the join waits for this kernel, and so for both
}

// Joins the partials of each vector (row, query head): WPV warps per vector,
// warp `sub` taking the partials sub, sub + WPV, ...; the order is fixed.  The
// bound is the latency of a few dependent loads, so there are two levels only:
// the lists' offsets, once per CTA (loaded by every warp they were hot spots of
// L2, up to 6 us of a call), then (m, l) and O, four rows at a time.  1024
// vectors of about 25 partials: 6 us; 16384 of about 4: 12 us.
template <int D, int WPV>
__global__ void __launch_bounds__(256, 5) prefix_join_kernel(const PrefixParams p) {
  constexpr int VEC = D / 32;  // columns per lane
  __shared__ float so[8][D];
  __shared__ float sml[8][2];
  __shared__ int head[8];  // of the CTA's request: see below
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int row_q = blockIdx.y;  // request * n + block row
  const int req = inv_div(row_q, p.inv_n), i = row_q - req * p.n;
  const int gi = inv_div(req, p.inv_group), se = p.ng + req;
  const PrefixList& P = p.list[p.list[0].prefix_tiles > 0 ? 0 : 1];
  const PrefixList& S = p.list[p.list[0].suffix_tiles > 0 ? 0 : 1];
  griddep_launch_dependents();
  griddep_wait();
  if (threadIdx.x < 7) {
    const int* src[7] = {S.off + se, S.unit + se, S.unit + p.ng + p.batch, p.ctx_len + req,
                         P.off + gi, P.unit + gi, P.unit + p.ng + p.batch};
    const int* from = src[0];
#pragma unroll
    for (int j = 1; j < 7; ++j) from = threadIdx.x == j ? src[j] : from;
    head[threadIdx.x] = threadIdx.x < 4 || P.prefix_tiles > 0 ? __ldcg(from) : 0;
  }
  __syncthreads();
  const int h = blockIdx.x * (8 / WPV) + warp / WPV, sub = warp % WPV;
  const bool on = h < p.hq;
  const int vec = row_q * p.hq + h;
  float m = -INFINITY, l = 0.f, acc[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) acc[j] = 0.f;
  if (on) {
    const int G = p.hq / p.hkv;
    const int kvh = inv_div(h, p.inv_G), g = h - kvh * G;
    const int so_ = head[0], su = head[1], sper = head[2], po = head[4], pu = head[5], pper = head[6];
    const int ctx = min(max(head[3], 0), p.max_pages * 16);
    const bool sees = (p.causal ? ctx - p.n + i + 1 : ctx) > 0;
    int np = 0, nsu = 0;
    size_t p_at = 0, s_at = 0;  // partial rows of the first worker
    if (sees && pu > 0) {
      const int row = ((req - gi * p.group) * p.n + i) * G + g;
      const int tile = row / P.tile_rows, ul = kvh * P.prefix_tiles + tile;
      int w0, w1;
      unit_workers(p, P, gi, ul, po, pu, pper, &w0, &w1);
      np = w1 - w0 + 1;
      p_at = part_row(p, P, gi, ul, w0) + row - tile * P.tile_rows;
    }
    if (sees && su > 0) {
      const int row = i * G + g;
      const int tile = row / S.tile_rows, ul = kvh * S.suffix_tiles + tile;
      int w0, w1;
      unit_workers(p, S, se, ul, so_, su, sper, &w0, &w1);
      nsu = w1 - w0 + 1;
      s_at = part_row(p, S, se, ul, w0) + row - tile * S.tile_rows;
    }
    const int parts = np + nsu;
    for (int b = sub; b < parts; b += 32 * WPV) {
      const int mine = b + lane * WPV;  // this lane's partial
      const int cnt = min(32, (parts - b + WPV - 1) / WPV);
      auto at = [&](int k, const PrefixList** L) {  // row of partial k in its list's buffers
        const bool pre = k < np;
        *L = pre ? &P : &S;
        return pre ? p_at + static_cast<size_t>(k) * P.worker_rows : s_at + static_cast<size_t>(k - np) * S.worker_rows;
      };
      float v[4][VEC];
      auto load4 = [&](int j0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
          for (int t = 0; t < VEC; ++t) v[j][t] = 0.f;
          if (j0 + j < cnt) {
            const PrefixList* L;
            const size_t ps = at(b + (j0 + j) * WPV, &L);
            const float* src = L->part_o + ps * D;
            if constexpr (VEC == 4) {
              const float4 x = __ldcg(reinterpret_cast<const float4*>(src) + lane);
              v[j][0] = x.x, v[j][1] = x.y, v[j][2] = x.z, v[j][3] = x.w;
            } else {
              const float2 x = __ldcg(reinterpret_cast<const float2*>(src) + lane);
              v[j][0] = x.x, v[j][1] = x.y;
            }
          }
        }
      };
      float ms = -INFINITY, ls = 0.f;
      if (mine < parts) {
        const PrefixList* L;
        const size_t ps = at(mine, &L);
        const float2 x = __ldcg(reinterpret_cast<const float2*>(L->part_ml + ps * 2));
        ms = x.x;
        ls = x.y;
      }
      load4(0);
      // -inf: the row saw none of that segment's keys, and no O was written
      const float mn = fmaxf(m, warp_max(ms));
      const float ref = mn == -INFINITY ? 0.f : mn;
      const float w = ms == -INFINITY ? 0.f : exp2f(ms - ref);
      const float f0 = exp2f(m - ref);
      l = l * f0 + warp_sum(ls * w);
#pragma unroll
      for (int j = 0; j < VEC; ++j) acc[j] *= f0;
      m = mn;
      for (int j0 = 0; j0 < cnt; j0 += 4) {
        if (j0 > 0) load4(j0);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float wj = __shfl_sync(0xffffffffu, w, (j0 + j) & 31);
          if (j0 + j < cnt && wj > 0.f) {
#pragma unroll
            for (int t = 0; t < VEC; ++t) acc[t] = fmaf(v[j][t], wj, acc[t]);
          }
        }
      }
    }
  }
  if (WPV > 1) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) so[warp][lane * VEC + j] = acc[j];
    if (lane == 0) {
      sml[warp][0] = m;
      sml[warp][1] = l;
    }
    __syncthreads();
    if (sub != 0 || !on) return;
    float mn = m;
    for (int w = 1; w < WPV; ++w) mn = fmaxf(mn, sml[warp + w][0]);
    if (mn > -INFINITY) {
      const float f0 = exp2f(m - mn);
      l *= f0;
#pragma unroll
      for (int j = 0; j < VEC; ++j) acc[j] *= f0;
      for (int w = 1; w < WPV; ++w) {
        const float f1 = exp2f(sml[warp + w][0] - mn);
        l = fmaf(sml[warp + w][1], f1, l);
#pragma unroll
        for (int j = 0; j < VEC; ++j) acc[j] = fmaf(so[warp + w][lane * VEC + j], f1, acc[j]);
      }
      m = mn;
    }
  }
  if (!on) return;
  const bool any = m > -INFINITY;
  const float inv = any ? 1.f / l : 0.f;
  uint16_t* dst = p.out + static_cast<size_t>(vec) * D + lane * VEC;
  if constexpr (VEC == 4)
    __stcs(reinterpret_cast<uint2*>(dst), make_uint2(bf16x2(acc[0] * inv, acc[1] * inv), bf16x2(acc[2] * inv, acc[3] * inv)));
  else
    __stcs(reinterpret_cast<uint32_t*>(dst), bf16x2(acc[0] * inv, acc[1] * inv));
  if (p.lse != nullptr && lane == 0)
    p.lse[vec] = any ? (m + log2f(l)) * 0.693147180559945309f : -INFINITY;
}

cudaError_t launch_pdl(const void* fn, dim3 grid, int block, size_t smem, void** args, cudaStream_t s) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  count_launch();
  return cudaLaunchKernelExC(&cfg, fn, args);
}

template <int D>
cudaError_t run_small(const PrefixParams& p, void** args, cudaStream_t s) {
  const size_t smem = kSmallWarps * SmallCfg<D>::RING + PrefixPlan::ints(p.batch, p.ng) * sizeof(int);
  const void* fn = reinterpret_cast<const void*>(prefix_small_kernel<D>);
  static thread_local int allowed = -1;
  const cudaError_t e = allow_smem(fn, kSmallWarps * SmallCfg<D>::RING + PrefixPlan::ints(kMaxPrefixBatch, kMaxPrefixBatch) * 4, &allowed);
  if (e != cudaSuccess) return e;
  return launch_pdl(fn, dim3(kSmallCtas), kSmallWarps * 32, smem, args, s);
}

template <int D>
cudaError_t run_join(const PrefixParams& p, void** args, cudaStream_t s) {
  const int rows = p.batch * p.n;
  // Few vectors have many partials each: more warps per vector.  The call with
  // one / four warps: 32 vectors 35.7 / 17.6 us, 2048 34.7 / 33.8, 4096 39.0 / 42.5,
  // 16384 81.5 / 106.9.
  if (rows * p.hq >= 4096)
    return launch_pdl(reinterpret_cast<const void*>(prefix_join_kernel<D, 1>), dim3((p.hq + 7) / 8, rows), 256, 0, args, s);
  return launch_pdl(reinterpret_cast<const void*>(prefix_join_kernel<D, 4>), dim3((p.hq + 1) / 2, rows), 256, 0, args, s);
}

}  // namespace

// Row tiles and workers of the two lists.
void prefix_attention_shape(PrefixParams* p) {
  const int G = p->hq / p->hkv;
  const int rows_p = p->group * p->n * G, rows_s = p->n * G;
  p->ng = p->batch / p->group;
  const bool tc_p = p->group > 1 && rows_p > kTcMinRows, tc_s = rows_s > kTcMinRows;
  PrefixList& S = p->list[0];
  S.chunk_shift = 4;
  S.tile_rows = kSmallRows;
  S.prefix_tiles = tc_p || p->group == 1 ? 0 : (rows_p + kSmallRows - 1) / kSmallRows;
  S.suffix_tiles = tc_s ? 0 : (rows_s + kSmallRows - 1) / kSmallRows;
  S.workers = S.prefix_tiles + S.suffix_tiles > 0 ? kSmallCtas * kSmallWarps : 0;
  S.prefix_cost = S.suffix_cost = 0;
  PrefixList& T = p->list[1];
  T.chunk_shift = 7;
  T.tile_rows = 256;
  T.prefix_tiles = tc_p ? (rows_p + 255) / 256 : 0;
  T.suffix_tiles = tc_s ? (rows_s + 255) / 256 : 0;
  T.workers = T.prefix_tiles + T.suffix_tiles > 0 ? kTcCtas : 0;
  // up to 128 rows leave half of a tile's tensor work to do
  T.prefix_split = rows_p <= 128;
  T.suffix_split = rows_s <= 128;
  T.prefix_cost = T.prefix_split ? 0 : 1;
  T.suffix_cost = T.suffix_split ? 0 : 1;
  // a segment's fixed cost (Q, the pipeline's start, the partial) is about that of
  // ten chunks of half a tile (a block verify with 0, 10, 20: 318, 152, 168 us)
  T.unit_cost = 10;
  for (PrefixList& L : p->list) {
    L.prefix_rows = L.prefix_tiles == 0 ? 0 : L.prefix_tiles > 1 ? L.tile_rows : rows_p;
    L.suffix_rows = L.suffix_tiles == 0 ? 0 : L.suffix_tiles > 1 ? L.tile_rows : rows_s;
    L.worker_rows = L.prefix_rows > L.suffix_rows ? L.prefix_rows : L.suffix_rows;
  }
  auto inverse = [](int d) { return d > 1 ? static_cast<unsigned>((1ull << 32) / d + 1) : 0u; };
  p->inv_n = inverse(p->n);
  p->inv_G = inverse(G);
  p->inv_group = inverse(p->group);
}

cudaError_t prefix_attention_launch(const PrefixParams& p, int d, const CUtensorMap* map, int group0,
                                    int oob_group, cudaStream_t s) {
  void* args[] = {const_cast<PrefixParams*>(&p)};
  cudaError_t e = cudaSuccess;
  if (p.list[1].workers > 0) e = prefix_tc_launch(*map, group0, oob_group, p, d, s);
  if (e == cudaSuccess && p.list[0].workers > 0) e = d == 128 ? run_small<128>(p, args, s) : run_small<64>(p, args, s);
  if (e != cudaSuccess) return e;
  return d == 128 ? run_join<128>(p, args, s) : run_join<64>(p, args, s);
}

}  // namespace dflash
