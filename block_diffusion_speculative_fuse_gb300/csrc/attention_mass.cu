// The attention weight that each cached key receives from the last rows of its request:
//
//   mass[j] (+)= sum over rows i and the query heads of j's KV head: exp(scale q_i . k_j - lse_i)
//
// over the rows that see j.  The rows' lse is known, so this is one product and one
// exponential per (row, key), without a running maximum, and keys are independent.
//
// The product is taken the other way round, D = K Q^T (M = 128 keys, N = 128 rows): in
// TMEM a key is a lane, so the sum over rows is a thread's own, in registers, without
// exchange or atomics, and a key whose K is not finite spoils its own sum alone.
//
// A unit is 256 keys of one request and KV head, two planes of 128, and all rows in tiles
// of 128 / G rows of the call (G query heads each).  Persistent CTAs take a range of
// units each where there are few rows, and otherwise groups of units in turn (w, w + 152,
// ...), so that causal units, the later the fewer rows, even out (8 x 16384 keys, 32
// rows: ranges 50 us, in turn 53); units in a row share Q where there is one tile.  Per tile
// and plane one D, in two stages each, which the plane's four warps sum up.
//
// Bound: with the usual window of rows (32 rows of 4 heads, one tile) K's bytes: 8
// requests of 16384 keys 46 us, 5.9 TB/s with 6 us of start-up, 32 of them 176 us, 6.2
// TB/s (169 with the same inputs again); 8 rows take as long as 32.  With many tiles 512 rows
// of 8 requests of 16848 keys 488 us, 1.14 PFLOP/s: a warp waits for each 32 columns of D before
// it works on them, with two warps to a scheduler, and Q comes from L2 again for every 256 keys (2.2
// GB, 4.6 TB/s); which of the two it is has not been measured.
#include <climits>

#include "attention_chunk.cuh"

namespace dflash {

namespace {

constexpr int kThreads = 384;   // warps 0-7 sums, 8 TMA, 9 products, 10 lse, 11 plan
constexpr int kWarps = kThreads / 32;
constexpr int kKeys = 128;      // of a plane
constexpr int kUnits = 4;       // planned ahead
constexpr int kWorkers = 152;

template <int D>
struct Cfg {
  static constexpr int HALVES = D / 64;
  static constexpr int PAGE = 16 * D * 2;
  static constexpr int PLANE = kKeys * D * 2;
  static constexpr int Q_TILE = 128 * D * 2;
  static constexpr int SLOTS = D == 128 ? 4 : 8;   // planes of K
};
constexpr int kQ = 2;           // Q tiles (and their lse) in shared memory

struct Unit {
  int k0;                  // first key; -1: the end
  int ctx, r, h;
  int token0, rows;        // the rows that weigh: first of the call, how many
  int base;                // row i of them sees keys up to base + i
  int t0, tiles;           // tiles [t0, tiles) see some of the keys
  int load, release;       // Q is loaded for this unit; is not used after it
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    mass_kernel(const __grid_constant__ CUtensorMap kv_map, const __grid_constant__ CUtensorMap q_map,
                const __grid_constant__ MassParams p, int group0, int oob_group) {
  using C = Cfg<D>;
  constexpr int SLOTS = C::SLOTS;
  extern __shared__ __align__(1024) uint8_t sm[];
  uint8_t* ring = sm + kQ * C::Q_TILE;
  float* lse_s = reinterpret_cast<float*>(ring + SLOTS * C::PLANE);  // [kQ][128] -lse / ln 2
  uint64_t* k_full = reinterpret_cast<uint64_t*>(lse_s + kQ * 128);
  uint64_t* k_free = k_full + SLOTS;
  uint64_t* q_full = k_free + SLOTS;     // [kQ]
  uint64_t* q_free = q_full + kQ;
  uint64_t* l_full = q_free + kQ;        // [kQ] lse
  uint64_t* l_free = l_full + kQ;
  uint64_t* d_full = l_free + kQ;        // [2 planes][2 stages]
  uint64_t* d_free = d_full + 4;
  uint64_t* drain = d_free + 4;
  uint64_t* u_full = drain + 1;          // [kUnits]
  uint64_t* u_free = u_full + kUnits;
  Unit* units = reinterpret_cast<Unit*>(u_free + kUnits);
  int* groups = reinterpret_cast<int*>(units + kUnits);   // [kUnits][16] K's 8-row groups in the map, by page
  int* scratch = groups + kUnits * 16;                    // [kWarps]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(scratch + kWarps);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* before = const_cast<int*>(abort_flag) + 1;         // [batch + 1] units of the requests before

  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid / 32, 0), lane = tid % 32;
  if (tid == 0) {
#pragma unroll 1
    for (int s = 0; s < SLOTS; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_free[s], 1);
    }
#pragma unroll 1
    for (int s = 0; s < kQ; ++s) {
      mbar_init(&q_full[s], 1);
      mbar_init(&q_free[s], 1);
      mbar_init(&l_full[s], 1);
      mbar_init(&l_free[s], 8);
    }
#pragma unroll 1
    for (int s = 0; s < 4; ++s) {
      mbar_init(&d_full[s], 1);
      mbar_init(&d_free[s], 4);
    }
#pragma unroll 1
    for (int s = 0; s < kUnits; ++s) {
      mbar_init(&u_full[s], 1);
      mbar_init(&u_free[s], 11);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    before[0] = 0;
    fence_barrier_init();
    tma_prefetch_desc(&kv_map);
    tma_prefetch_desc(&q_map);
  }
  if (warp == 9) tmem_alloc(tmem_slot, 512);
  griddep_wait();
  auto request = [&](int r) { return ChunkRequest(p.row_start, p.ctx_len, r, p.T, p.max_pages, p.status, 561); };
  // units of a request and KV head; a length beyond the sums' room counts as that
  auto length = [&](const ChunkRequest& q) { return static_cast<int>(min(static_cast<int64_t>(q.ctx), p.ld_mass)); };
  {
    int sum = 0;
#pragma unroll 1
    for (int base = 0; base < p.batch; base += kThreads) {
      const int r = base + tid;
      int v = 0;
      if (r < p.batch) {
        const ChunkRequest q = request(r);
        if (q.ctx > p.ld_mass) raise_status(p.status, DFLASH_ERR_CAPACITY, 564);
        v = (length(q) + 2 * kKeys - 1) / (2 * kKeys) * p.hkv;
      }
      int upto = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      __syncthreads();
      if (lane == 31) scratch[warp] = upto;
      __syncthreads();
      const int part = lane < kWarps ? scratch[lane] : 0;
      const int lead = __reduce_add_sync(0xffffffffu, lane < warp ? part : 0);
      if (r < p.batch) before[r + 1] = sum + lead + upto;
      sum += __reduce_add_sync(0xffffffffu, part);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_launch_dependents();   // (this CTA has its TMEM)
  const uint32_t tmem = *tmem_slot;

  // The next unit, for a whole warp; false at the end.  A role that gives up on a wait
  // goes on through the units without working on them.
  int taken = 0;
  bool ok = true;
  auto next_unit = [&](Unit* u) {
    const int at = taken % kUnits;
    if (!__all_sync(0xffffffffu, mbar_wait_for(&u_full[at], (taken / kUnits) & 1, nullptr, 4 * kWaitLimitNs))) return false;
    const int w = lane < sizeof(Unit) / 4 ? reinterpret_cast<const int*>(units + at)[lane] : 0;
#pragma unroll
    for (int j = 0; j < sizeof(Unit) / 4; ++j) reinterpret_cast<int*>(u)[j] = __shfl_sync(0xffffffffu, w, j);
    return u->k0 >= 0;
  };
  auto unit_done = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(&u_free[taken % kUnits]);
    ++taken;
  };
  auto give_up = [&](int site) {
    ok = false;
    *abort_flag = 1;
    if (lane == 0) raise_status(p.status, DFLASH_ERR_TIMEOUT, site);
  };
  auto wait = [&](uint64_t* bar, int parity, int site) {
    if (__all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag))) return true;
    give_up(site);
    return false;
  };
  // tiles whose Q goes through the ring for a unit
  auto tiles_of = [](const Unit& u) { return u.tiles - u.t0; };
  auto planes_of = [](const Unit& u) { return u.ctx - u.k0 > kKeys ? 2 : 1; };
  Unit u;

  if (warp == 11) {
    // ------------------------------------------------ plan
    const int all = before[p.batch];
    // with one or two tiles units cost the same: a range each; otherwise groups in turn
    const int w = blockIdx.x;
    const int start = p.few ? static_cast<int>(static_cast<int64_t>(all) * w / kWorkers) : 0;
    const int group = p.few ? static_cast<int>(static_cast<int64_t>(all) * (w + 1) / kWorkers) - start
                            : min(8, max(1, all / (kWorkers * 8)));
    int count = 0, r = 0, loaded = -1;
    ChunkRequest q;
    bool more = true;
#pragma unroll 1
    for (int64_t base = p.few ? start : w * group; more; base = p.few ? all : base + kWorkers * group) {
#pragma unroll 1
      for (int j = 0; j < max(group, 1) && more; ++j) {
        const int64_t at = group > 0 ? base + j : all;
        Unit x;
        x.k0 = -1;
        if (at < all) {
          // the request: groups go up, so the search goes on from the last one
          while (before[r + 1] <= at) {
            const int64_t hit = r + 1 + lane;
            const unsigned above = __ballot_sync(0xffffffffu, hit >= p.batch || before[min(static_cast<int>(hit), p.batch - 1) + 1] > at);
            r += above ? __ffs(above) : 32;
          }
          if (loaded != r) {
            q = request(r);
            loaded = r;
          }
          const int len = length(q), blocks = (len + 2 * kKeys - 1) / (2 * kKeys);
          const int local = static_cast<int>(at) - before[r], h = local / blocks, b = local - h * blocks;
          x.k0 = b * 2 * kKeys;
          x.ctx = len;
          x.r = r;
          x.h = h;
          x.rows = p.last > 0 ? min(p.last, q.n) : q.n;
          x.token0 = q.start + q.n - x.rows;
          x.base = q.ctx - x.rows;
          x.tiles = (x.rows + p.tokens - 1) / p.tokens;
          x.t0 = p.causal ? min(max(0, x.k0 - x.base) / p.tokens, x.tiles) : 0;
          const bool one = x.tiles == 1;
          x.load = !(one && j > 0 && b > 0);
          x.release = !(one && j + 1 < group && b + 1 < blocks);
        }
        more = x.k0 >= 0;
        const int slot = count % kUnits;
        int grp = oob_group;
        if (more && x.tiles > x.t0 && lane < 16 && x.k0 / 16 + lane < (x.ctx + 15) / 16) {
          const int id = __ldcg(p.page_table + static_cast<size_t>(x.r) * p.max_pages + x.k0 / 16 + lane);
          if (id >= 0 && id < p.n_pages) grp = group0 + (id * 2 * p.hkv + x.h) * 2;
          else raise_status(p.status, DFLASH_ERR_CAPACITY, 563);
        }
        if (count >= kUnits && !__all_sync(0xffffffffu, mbar_wait_for(&u_free[slot], (count / kUnits + 1) & 1, nullptr,
                                                                      4 * kWaitLimitNs))) {
          give_up(568);
          more = false;
          break;
        }
        if (lane < 16) groups[slot * 16 + lane] = grp;
        if (lane == 0) units[slot] = x;
        __syncwarp();
        if (lane == 0) mbar_arrive(&u_full[slot]);
        __syncwarp();
        ++count;
      }
    }
  } else if (warp == 8) {
    // ------------------------------------------------ TMA producer
    const uint64_t pol = l2_policy_evict_normal(), pol_k = l2_policy_evict_first();
    int at = 0, qn = 0;
    Cursor cur, qc;
    while (next_unit(&u)) {
      if (ok && tiles_of(u) > 0) {
        const int planes = planes_of(u), *grp = groups + taken % kUnits * 16;
        // the first tile's Q goes before the keys, the others after
        auto load_q = [&](int t) {
          if (qn >= kQ && !wait(&q_free[qc.slot], qc.parity ^ 1, 565)) return;
          if (lane == 0) {
            mbar_arrive_expect_tx(&q_full[qc.slot], C::HALVES * p.tokens * p.G * 128);
#pragma unroll
            for (int b = 0; b < C::HALVES; ++b)
              tma_load_3d(sm + qc.slot * C::Q_TILE + b * (128 * 128), &q_map, b * 64, u.h * p.G, u.token0 + t * p.tokens,
                          &q_full[qc.slot], pol);
          }
          __syncwarp();
          ++qn;
          qc.advance(kQ);
        };
        if (u.load) load_q(u.t0);
#pragma unroll 1
        for (int k = 0; ok && k < planes; ++k) {
          const int st = cur.slot;
          int y[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = grp[k * 8 + i];
          if (at >= SLOTS && !wait(&k_free[st], cur.parity ^ 1, 565)) break;
          if (elect_one()) {
            mbar_arrive_expect_tx(&k_full[st], C::PLANE);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              tma_load_4d(smem_u32(ring + st * C::PLANE + i * C::PAGE), &kv_map, y[i], &k_full[st], pol_k);
          }
          __syncwarp();
          ++at;
          cur.advance(SLOTS);
        }
#pragma unroll 1
        for (int t = u.t0 + 1; ok && t < u.tiles; ++t) load_q(t);
      }
      unit_done();
    }
    // copies still in flight after an abort land before the CTA exits
    if (lane == 0) {
#pragma unroll 1
      for (int j = max(0, at - SLOTS); j < at; ++j) mbar_wait(&k_full[j % SLOTS], (j / SLOTS) & 1, nullptr);
#pragma unroll 1
      for (int j = max(0, qn - kQ); j < qn; ++j) mbar_wait(&q_full[j % kQ], (j / kQ) & 1, nullptr);
    }
  } else if (warp == 9) {
    // ------------------------------------------------ products
    constexpr uint32_t idesc = umma_idesc_bf16(kKeys, 128);
    constexpr uint32_t GS = C::HALVES * 1024;  // between 8-row groups of a plane
    const uint32_t q_addr = smem_u32(sm), ring_addr = smem_u32(ring);
    Cursor cur, qc;
    int dn = 0;          // D stages used
    bool held = false;   // the tile at qc is there already
    while (next_unit(&u)) {
      if (ok && tiles_of(u) > 0) {
        const int planes = planes_of(u);
        int slot[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          slot[k] = cur.slot;
          if (k < planes) {
            if (ok) wait(&k_full[cur.slot], cur.parity, 566);
            cur.advance(SLOTS);
          }
        }
#pragma unroll 1
        for (int t = u.t0; ok && t < u.tiles; ++t) {
          if (!held && !wait(&q_full[qc.slot], qc.parity, 566)) break;
          const int stage = dn & 1;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            if (k >= planes || !ok) continue;
            if (dn >= 2 && !wait(&d_free[k * 2 + stage], (dn / 2 + 1) & 1, 566)) break;
            tc_fence_after();
            const uint32_t a = desc_lo(ring_addr + slot[k] * C::PLANE, 16), b = desc_lo(q_addr + qc.slot * C::Q_TILE, 16);
            if (elect_one()) {
#pragma unroll
              for (int j = 0; j < D / 16; ++j)
                umma_ss(tmem + (k * 2 + stage) * 128, desc_of(a + (j / 4) * (1024 / 16) + (j % 4) * 2, desc_hi(GS)),
                        desc_of(b + (j / 4) * (128 * 128 / 16) + (j % 4) * 2, desc_hi(1024)), idesc, j > 0 ? 1u : 0u);
              umma_commit(&d_full[k * 2 + stage]);
              if (t + 1 == u.tiles) umma_commit(&k_free[slot[k]]);
            }
            __syncwarp();
          }
          // a plane that is not there: its stage passes unused
          if (planes == 1 && ok) {
            if (dn < 2 || wait(&d_free[2 + stage], (dn / 2 + 1) & 1, 566))
              if (lane == 0) mbar_arrive(&d_full[2 + stage]);
          }
          ++dn;
          const bool keep = u.tiles == 1 && !u.release;
          held = keep;
          if (!keep) {
            if (elect_one()) umma_commit(&q_free[qc.slot]);
            __syncwarp();
            qc.advance(kQ);
          }
        }
      }
      unit_done();
    }
    // the products in flight end before their memory is given back
    if (!ok && dn > 0) {
      if (elect_one()) umma_commit(drain);
      __syncwarp();
      mbar_wait(drain, 0, nullptr);
    }
  } else if (warp == 10) {
    // ------------------------------------------------ lse of the rows
    Cursor qc;
    int qn = 0;
    while (next_unit(&u)) {
      if (u.load) {
#pragma unroll 1
        for (int t = u.t0; ok && t < u.tiles; ++t) {
          if (qn >= kQ && !wait(&l_free[qc.slot], qc.parity ^ 1, 567)) break;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int row = j * 32 + lane, tok = row / p.G, token = t * p.tokens + tok;
            float x = 0.f;
            if (tok < p.tokens && token < u.rows)
              x = -1.44269504088896340736f * __ldg(p.lse + static_cast<size_t>(u.token0 + token) * p.hq + u.h * p.G + row - tok * p.G);
            lse_s[qc.slot * 128 + row] = x;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&l_full[qc.slot]);
          ++qn;
          qc.advance(kQ);
        }
      }
      unit_done();
    }
  } else {
    // ------------------------------------------------ sums: a thread per key
    const int plane = warp / 4, lane128 = warp % 4 * 32 + lane;
    const uint32_t d_addr = tmem + (static_cast<uint32_t>(warp % 4 * 32) << 16) + plane * 256;
    Cursor qc;
    int dn = 0;
    bool held = false;
    while (next_unit(&u)) {
      const int key = u.k0 + plane * kKeys + lane128;
      float* out = p.mass + (static_cast<int64_t>(u.r) * p.hkv + u.h) * p.ld_mass + key;
      float old = 0.f;
      if (p.accumulate && key < u.ctx) old = *out;
      float sum = 0.f, lost = 0.f;   // of the tiles, and what its last rounding added
#pragma unroll 1
      for (int t = u.t0; t < u.tiles; ++t) {
        const int stage = dn & 1;
        float2 a0 = make_float2(0.f, 0.f), a1 = a0;
        if (ok && !held) wait(&l_full[qc.slot], qc.parity, 569);
        if (ok) wait(&d_full[plane * 2 + stage], (dn / 2) & 1, 569);
        tc_fence_after();
        // columns [c0, c1) see this key
        const int c1 = min(u.rows - t * p.tokens, p.tokens) * p.G;
        int c0 = 0;
        if (p.causal) c0 = min(max(0, key - u.base - t * p.tokens), p.tokens) * p.G;
        const bool whole = __all_sync(0xffffffffu, c0 == 0);
        const float2 sc = make_float2(p.scale_log2, p.scale_log2);
        const float4* ls = reinterpret_cast<const float4*>(lse_s + qc.slot * 128);
        // Whole groups of 32 columns have no tests: as selects in the same loop they cost as
        // much again as the sums (same inputs again, 8 x 16384 keys 50 us instead of 46, all of
        // 512 rows 621 instead of 480).
        int c = 0;
        if (whole) {
#pragma unroll 1
          for (; c + 32 <= c1; c += 32) {
            uint32_t x[32];
            tmem_ld32_nowait(d_addr + stage * 128 + c, x);
            tmem_wait_ld(x);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float4 l4 = ls[c / 4 + j];
              const float2 s0 = fma2(make_float2(__uint_as_float(x[4 * j]), __uint_as_float(x[4 * j + 1])), sc, make_float2(l4.x, l4.y));
              const float2 s1 = fma2(make_float2(__uint_as_float(x[4 * j + 2]), __uint_as_float(x[4 * j + 3])), sc, make_float2(l4.z, l4.w));
              a0 = add2(a0, make_float2(ex2(s0.x), ex2(s0.y)));
              a1 = add2(a1, make_float2(ex2(s1.x), ex2(s1.y)));
            }
          }
        }
#pragma unroll 1
        for (; c < c1; c += 16) {
          uint32_t x[16];
          tmem_ld16_raw(d_addr + stage * 128 + c, x);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float4 l4 = ls[c / 4 + j];
            const float2 s0 = fma2(make_float2(__uint_as_float(x[4 * j]), __uint_as_float(x[4 * j + 1])), sc, make_float2(l4.x, l4.y));
            const float2 s1 = fma2(make_float2(__uint_as_float(x[4 * j + 2]), __uint_as_float(x[4 * j + 3])), sc, make_float2(l4.z, l4.w));
            auto seen = [&](int i, float v) { return c + 4 * j + i >= c0 && c + 4 * j + i < c1 ? ex2(v) : 0.f; };
            a0 = add2(a0, make_float2(seen(0, s0.x), seen(1, s0.y)));
            a1 = add2(a1, make_float2(seen(2, s1.x), seen(3, s1.y)));
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&d_free[plane * 2 + stage]);
        // A tile's weights add up by themselves, the tiles' sums with their roundings carried along
        // (Kahan): in one running sum a key that 24576 rows of 16 heads see lost 1.2e-3.
        const float more = (a0.x + a0.y) + (a1.x + a1.y) - lost, next = sum + more;
        lost = (next - sum) - more;
        sum = next;
        ++dn;
        const bool keep = u.tiles == 1 && !u.release;
        held = keep;
        if (!keep) {
          if (lane == 0) mbar_arrive(&l_free[qc.slot]);
          qc.advance(kQ);
        }
      }
      if (key < u.ctx && (u.tiles > 0 || !p.accumulate)) *out = old + sum;
      unit_done();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

template <int D>
cudaError_t launch(const MassParams& p, const CUtensorMap& kv_map, const CUtensorMap& q_map, int group0,
                   int oob_group, cudaStream_t s) {
  using C = Cfg<D>;
  constexpr int fixed = kQ * C::Q_TILE + C::SLOTS * C::PLANE + kQ * 128 * 4 +
                        (2 * C::SLOTS + 4 * kQ + 9 + 2 * kUnits) * 8 + kUnits * (sizeof(Unit) + 64) + (kWarps + 2) * 4;
  constexpr int most = fixed + (kMaxMassBatch + 1) * 4;
  static_assert(most <= 227 * 1024, "fits");
  static thread_local int allowed = -1;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(mass_kernel<D>), most, &allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kWorkers);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = fixed + (p.batch + 1) * 4;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  count_launch();
  return cudaLaunchKernelEx(&cfg, mass_kernel<D>, kv_map, q_map, p, group0, oob_group);
}

}  // namespace

cudaError_t attention_mass_launch(const MassParams& p, int d, const CUtensorMap& kv_map, const CUtensorMap& q_map,
                                  int group0, int oob_group, cudaStream_t s) {
  return d == 128 ? launch<128>(p, kv_map, q_map, group0, oob_group, s)
                  : launch<64>(p, kv_map, q_map, group0, oob_group, s);
}

}  // namespace dflash
