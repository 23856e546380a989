// Attention over the paged cache for batches whose requests share a prefix:
// the large-tile kernel (tcgen05), for entities of more than 32 rows per KV
// head (prefixes of a batch, block verifies).
//
// One persistent CTA per SM works through its segments (prefix_attention.cuh).
// A unit is 256 rows in two tiles of 128, A and B, which read the same keys,
// 128 a chunk: per chunk and tile
//   S = Q K^T   (M = 128, N = 128, K = d)   TMEM, 128 columns
//   O += P V    (M = 128, N = d, K = 128)   TMEM, d columns
// issued in the order S_A S_B | PV_A S_A' PV_B S_B' | ..., so that the tensor
// cores work on one tile while the other's warps form P = exp2(S - m).  P
// replaces S in TMEM (bf16, the A operand of the second product).  An entity of
// at most 128 rows has no second tile: there A takes the even chunks and B the
// odd ones, over the same Q, and the two states are joined at the end.
//
// Softmax: a thread per row (warps 0-3 tile A, 4-7 tile B), no exchange
// between threads.  The row's reference maximum is raised, and O rescaled,
// only when a chunk exceeds it by more than 2^8, which after the first chunks
// is rare; P then stays below 2^8, exact enough in bf16 (relative rounding; the
// products want P in V's type, and a second term of P would be half as many products
// again: the output is off by 2.3e-3 rms of its values, of which 1.7e-3 are its own
// rounding), and l is summed in fp32.
//
// Keys arrive by TMA, one 4 KB box per page and plane, as [8-row group][column
// half][8 rows][128 B]: the 8-row groups of a 128-key plane then lie at one
// distance, which is what both the K-major (K) and the MN-major (V)
// descriptors need; a box per column half would double the boxes, and the SM's
// TMA unit spends a fixed time on each.  K and V planes of 32 KB (d = 128) go
// through one ring in the order in which the MMAs use them, each released by
// the MMA that read it last.
//
// 0 * V must be 0, so before its product the issuing warp goes over the part of V
// that a row may not see (clean_v): past the context it puts zeros; among the keys
// of the block's own rows it puts them for what is not finite, and the rows that do
// see such a key get a NaN in the end.  A block verify takes 130.3 us without and
// 131.1 with it; done by the softmax warps, which have no registers to spare, 134.
//
// Bound: with 256 rows (a block verify: 16384 shared keys, 2048 rows on each of
// 8 KV heads, and 512 own keys for 64 rows of 32 requests) the products: a chunk's
// four take 1.05 us of the tensor pipe and, S reading Q and K, P V reading V, the
// loads writing both, 256 KB or 1.05 us of shared memory; it comes every 1.4-1.5
// us, 112 us in all, 1.25 PFLOP/s.  The loads are never waited for, and a tile's
// softmax, 0.7 us, runs under the other's products; the hand-overs between them
// are the rest.  With up to 128 rows (a decode of the same prefix: 67 MB in 20 us,
// 3.4 TB/s) the pipeline's start in each CTA's one or two segments of about seven
// chunks.  One tile over alternating chunks there takes 53 us a call where two
// tiles, half of them empty, take 59.
#include <climits>

#include "common.cuh"
#include "kernels.h"
#include "prefix_attention.cuh"

namespace dflash {

namespace {

constexpr int kTcThreads = 320;   // warps 0-7 softmax, 8 TMA, 9 MMA
constexpr int kChunk = 128;
constexpr float kRaise = 8.f;     // log2

template <int D>
struct TcCfg {
  static constexpr int HALVES = D / 64;
  static constexpr int PAGE = 16 * D * 2;
  static constexpr int PLANE = kChunk * D * 2;           // K or V of a chunk
  static constexpr int Q_TILE = 128 * D * 2;             // [HALVES][128 rows][128 B]
  static constexpr int MAX_SLOTS = D == 128 ? 5 : 10;
  // two tiles each: + 128 * tile; P (64 columns) takes the upper half of S
  static constexpr uint32_t S_COL = 0, P_COL = 64, O_COL = 256;
};

// One thread issues the products, and an M = N = 128, K = 16 step takes the
// tensor pipe 64 cycles: building both 64-bit descriptors anew for each step
// took that thread 150.  Only the address field changes from step to step, so
// the steps add constants to a low word (address >> 4, leading offset) and join
// it with a constant high word (stride between 8-row groups, version, swizzle).
// And its whole warp runs the loop, with one lane elected for the instructions
// themselves: the descriptors then stay in uniform registers, where the
// instruction wants them (a block verify 147 -> 129 us).
__device__ __forceinline__ uint64_t desc_of(uint32_t lo, uint32_t hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
  return d;
}
__device__ __forceinline__ constexpr uint32_t desc_hi(uint32_t group_stride) {
  return (group_stride >> 4) | (1u << 14) | (2u << 29);  // bits 32-45, 46, 61-63: SWIZZLE_128B
}
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t leading) {
  return (addr >> 4) | ((leading >> 4) << 16);
}
// A and B in shared memory
__device__ __forceinline__ void umma_ss(uint32_t tmem_d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// A in TMEM (lane = row, two bf16 of K per column)
__device__ __forceinline__ void umma_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem_d),
      "r"(tmem_a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(r))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)), "l"(reinterpret_cast<uint64_t&>(c)));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(r))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return r;
}
// 4-D tiled load (coordinates innermost first).
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int w, uint64_t* bar,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %2, %2, %3}], [%4], %5;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(w), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

// Position in the ring: the slot and the parity of its present round.  (Slot
// numbers by division cost the issuing thread 600 cycles a chunk.)
struct Cursor {
  int slot = 0, parity = 0;
  __device__ __forceinline__ void advance(int slots) {
    if (++slot == slots) {
      slot = 0;
      parity ^= 1;
    }
  }
};

// Place of a segment's planes in the ring's order (n chunks): two tiles per
// chunk K0 V0 K1 V1 ...; split K0 K1 V0 K2 V1 K3 ...
__device__ __forceinline__ int place_k(bool split, int c) { return split ? c + max(0, c - 1) : 2 * c; }
// Of a V plane (one warp): makes the keys [first, live) finite and those from live
// to the end of its page zero.  The lane's first key that was not finite, else
// kChunk.  Not inlined: its code in the issuing warp's loop made a block verify 3
// to 15 us longer even where it was not run.
template <int D>
__device__ __noinline__ int clean_v(uint8_t* plane, int first, int live) {
  constexpr int HALVES = TcCfg<D>::HALVES, PIECES = HALVES * 8;  // 16-byte pieces of a key
  auto piece = [&](int i) {
    const int key = i / PIECES, half = i / 8 % HALVES;
    return reinterpret_cast<uint4*>(plane + (key / 8) * (HALVES * 1024) + half * 1024 + (key % 8) * 128 +
                                    (((i ^ key) & 7) << 4));
  };
  const int lane = threadIdx.x % 32;
  const int i0 = max(first, 0) * PIECES + lane, i1 = min(live, kChunk) * PIECES;
  bool found = false;
#pragma unroll 8
  for (int i = i0; i < i1; i += 32) found |= bf16_not_finite(*piece(i));
  int bad = kChunk;
  if (__any_sync(0xffffffffu, found)) {
#pragma unroll 1
    for (int i = i0; i < i1; i += 32) {
      if (!bf16_not_finite(*piece(i))) continue;
      bad = min(bad, i / PIECES);
      *piece(i) = make_uint4(0u, 0u, 0u, 0u);
    }
  }
#pragma unroll 1
  for (int i = max(live, 0) * PIECES + lane; i < min((live + 15) & ~15, kChunk) * PIECES; i += 32)
    *piece(i) = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  __syncwarp();
  return bad;
}

template <int D>
__global__ void __launch_bounds__(kTcThreads, 1)
    prefix_tc_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ PrefixParams p,
                     int group0, int oob_group, int slots) {
  using C = TcCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~static_cast<uintptr_t>(1023));
  uint8_t* ring = sm + 2 * C::Q_TILE;
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + slots * C::PLANE);
  uint64_t* empty = full + C::MAX_SLOTS;
  uint64_t* s_full = empty + C::MAX_SLOTS;  // [2] S of a tile is complete (and the PV before it)
  uint64_t* p_full = s_full + 2;            // [2][2] P of a tile is in TMEM: upper, lower 64 keys
  uint64_t* q_full = p_full + 4;            // Q of the segment is in shared memory
  uint64_t* o_full = q_full + 1;            // all of the segment's products are complete; bad_key
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(o_full + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* bad_key = abort_flag + 1;   // the segment's first key with a V that is not finite
  const PrefixList& L = p.list[1];
  const int ne = p.ng + p.batch;
  const PrefixPlan pl(reinterpret_cast<int*>(tmem_slot + 4), p.batch, p.ng);

  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  if (tid == 0) {
    for (int s = 0; s < slots; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s_full[t], 1);
      mbar_init(&p_full[2 * t], 4);
      mbar_init(&p_full[2 * t + 1], 4);
    }
    mbar_init(q_full, 8);
    mbar_init(o_full, 2);
    *abort_flag = 0;
    *bad_key = INT_MAX;
    fence_barrier_init();
    tma_prefetch_desc(&map);
  }
  if (warp == 9) tmem_alloc(tmem_slot, 512);
  griddep_wait();
  griddep_launch_dependents();
  prefix_plan(p, 1, pl);  // ends with a barrier
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int worker = blockIdx.x;
  Segments seg(L, pl.off, ne, worker);

  if (warp == 8) {
    // ------------------------------------------------ TMA producer
    // keys that other row tiles read too stay as they may; those read once leave
    // first (kept, they pushed the next kernels' code out of L2: 8 us a call)
    const uint64_t pol = L.prefix_tiles > 1 ? l2_policy_evict_normal() : l2_policy_evict_first();
    int at = 0;                                   // planes requested so far
    Cursor cur;
    bool ok = true;
    while (ok && seg.next(p, L, pl)) {
      const int e = seg.e, n = seg.chunk1 - seg.chunk0;
      const bool pre = e < p.ng, split = pre ? L.prefix_split : L.suffix_split;
      const int kvh = small_div(seg.ul, entity_tiles(p, L, e));
      const int page0 = (pre ? 0 : pl.cut[inv_div(e - p.ng, p.inv_group)] / 16) + seg.chunk0 * 8;
      const int pages_end = pre ? pl.cut[e] / 16 : (pl.ctx[e - p.ng] + 15) / 16;
      const int npg = min(n * 8, pages_end - page0);
      const int32_t* table = p.page_table + static_cast<size_t>(pre ? pl.live[e] : e - p.ng) * p.max_pages + page0;
      // lane -> 8-row group of its page's K plane in the map, 32 pages a time,
      // the next 32 requested ahead
      auto ids_of = [&](int b) {
        const int j = b * 32 + lane;
        return j < npg ? max(__ldcg(table + j), -1) : -2;  // -2: past the segment
      };
      auto check = [&](int id) {
        if (id >= 0 && id < p.n_pages) return group0 + (id * 2 * p.hkv + kvh) * 2;
        if (id != -2) raise_status(p.status, DFLASH_ERR_CAPACITY, 521);
        return oob_group;
      };
      int kb = 0, vb = 0;  // 32-page batch held for K, for V
      int next_id = ids_of(1);
      int kg = check(ids_of(0)), vg = kg;
      int k = 0, v = 0;
      for (int i = 0; i < 2 * n; ++i, ++at, cur.advance(slots)) {
        const bool is_k = k < n && place_k(split, k) == i;
        const int c = is_k ? k++ : v++;
        if (is_k) {
          if (c / 4 != kb) {  // K runs ahead: V's batch is the previous one until it follows
            kb = c / 4;
            kg = check(next_id);
            next_id = ids_of(kb + 1);
          }
        } else if (c / 4 != vb) {
          vb = c / 4;
          vg = kg;
        }
        // V's batch may lag one behind K's; K is at most two chunks ahead
        const int grp = __shfl_sync(0xffffffffu, is_k ? kg : vg, (c % 4) * 8 + lane % 8);
        const int st = cur.slot;
        int go = 1;
        if (lane == 0) {
          if (at >= slots && !mbar_wait(&empty[st], cur.parity ^ 1, abort_flag)) {
            *abort_flag = 1;
            raise_status(p.status, DFLASH_ERR_TIMEOUT, 523);
            go = 0;
          } else {
            mbar_arrive_expect_tx(&full[st], C::PLANE);
          }
        }
        if (!__shfl_sync(0xffffffffu, go, 0)) {
          ok = false;
          break;
        }
        if (lane < 8) {
          const int y = grp == oob_group || is_k ? grp : grp + p.hkv * 2;
          tma_load_4d(smem_u32(ring + st * C::PLANE + lane * C::PAGE), &map, y, &full[st], pol);
        }
      }
    }
    // copies still in flight after an abort land before the CTA exits
    if (lane == 0)
      for (int i = max(0, at - slots); i < at; ++i) mbar_wait(&full[i % slots], (i / slots) & 1, nullptr);
  } else if (warp == 9) {
    // ------------------------------------------------ MMA issuer
    {
      constexpr uint32_t idesc_s = umma_idesc_bf16(128, kChunk);
      constexpr uint32_t idesc_pv = umma_idesc_bf16(128, D) | (1u << 16);  // V MN-major
      constexpr uint32_t GS = C::HALVES * 1024;  // between 8-row groups of a plane
      const uint32_t q_addr = smem_u32(sm), ring_addr = smem_u32(ring);
      int segs = 0;
      int np[2] = {0, 0};  // parity of the next P of each tile
      int bad = INT_MAX;   // see above
      bool ok = true;
      Cursor cur;          // the next plane: they are used in the order they arrive
      auto commit = [&](uint64_t* bar) {
        if (elect_one()) umma_commit(bar);
        __syncwarp();
      };
      // the end of a segment
      auto finish = [&]() {
        bad = __reduce_min_sync(0xffffffffu, bad);
        if (lane == 0) {
          *bad_key = bad;
          mbar_arrive(o_full);
        }
        commit(o_full);
      };
      // waits for the next plane and takes it: its slot, or -1
      auto take = [&]() {
        const int st = cur.slot;
        const bool r = __all_sync(0xffffffffu, mbar_wait(&full[st], cur.parity, abort_flag));
        cur.advance(slots);
        return r ? st : -1;
      };
      auto issue_s = [&](int tile, int q_tile, int st) {
        const uint32_t q = desc_lo(q_addr + q_tile * C::Q_TILE, 16);
        const uint32_t k = desc_lo(ring_addr + st * C::PLANE, 16);
        if (elect_one()) {
#pragma unroll
          for (int j = 0; j < D / 16; ++j)
            umma_ss(tmem + C::S_COL + tile * 128, desc_of(q + (j / 4) * (128 * 128 / 16) + (j % 4) * 2, desc_hi(1024)),
                    desc_of(k + (j / 4) * (1024 / 16) + (j % 4) * 2, desc_hi(GS)), idesc_s, j > 0 ? 1u : 0u);
          umma_commit(&s_full[tile]);
        }
        __syncwarp();
      };
      // waits for the tile's P, half by half, and issues O += P V
      auto issue_pv = [&](int tile, int st, bool accumulate) {
        const uint32_t v = desc_lo(ring_addr + st * C::PLANE, 1024);
        const uint32_t o = tmem + C::O_COL + tile * 128, pa = tmem + C::P_COL + tile * 128;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!__all_sync(0xffffffffu, mbar_wait(&p_full[2 * tile + h], np[tile], abort_flag))) return false;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int j = (1 - h) * 4 + i;  // the upper keys first
              umma_ts(o, pa + j * 8, desc_of(v + j * (C::PAGE / 16), desc_hi(GS)), idesc_pv,
                      h + i > 0 ? 1u : accumulate ? 1u : 0u);
            }
          }
          __syncwarp();
        }
        np[tile] ^= 1;
        return true;
      };
      int tail = INT_MAX;  // from this key of the segment on V is gone over
      const int hidden = p.causal ? p.n - 1 : 0;
      auto clean = [&](int c, int st) {
        if ((c + 1) * kChunk > tail) {
          const int first = tail - c * kChunk;
          const int b = clean_v<D>(ring + st * C::PLANE, first, first + hidden);
          if (b < kChunk) bad = min(bad, c * kChunk + b);
        }
      };
      while (ok && seg.next(p, L, pl)) {
        const int n = seg.chunk1 - seg.chunk0;
        const bool split = seg.e < p.ng ? L.prefix_split : L.suffix_split;
        tail = bad = INT_MAX;
        if (seg.e >= p.ng) {  // (a prefix is whole pages that all rows see)
          const int r = seg.e - p.ng, ctx = pl.ctx[r];
          if (hidden > 0 || ctx % 16) tail = ctx - hidden - pl.cut[inv_div(r, p.inv_group)] - seg.chunk0 * kChunk;
        }
        ok = __all_sync(0xffffffffu, mbar_wait(q_full, segs++ & 1, abort_flag));
        if (!ok) break;
        tc_fence_after();
        if (split) {
          for (int c = 0; ok && c < min(2, n); ++c) {
            const int ik = take();
            ok = ik >= 0;
            if (!ok) break;
            issue_s(c, 0, ik);
            commit(&empty[ik]);
          }
          for (int c = 0; ok && c < n; ++c) {
            const int t = c & 1, iv = take();
            if (iv >= 0) clean(c, iv);
            ok = iv >= 0 && issue_pv(t, iv, c >= 2);
            if (!ok) break;
            commit(&empty[iv]);
            if (c + 2 < n) {
              const int ik = take();
              ok = ik >= 0;
              if (!ok) break;
              issue_s(t, 0, ik);
              commit(&empty[ik]);
            }
          }
        } else {
          int ik = take();
          ok = ik >= 0;
          if (ok) {
            issue_s(0, 0, ik);
            issue_s(1, 1, ik);
            commit(&empty[ik]);
          }
          for (int c = 0; ok && c < n; ++c) {
            const bool more = c + 1 < n;
            const int iv = take();
            if (iv >= 0) clean(c, iv);
            ok = iv >= 0 && issue_pv(0, iv, c > 0);
            if (!ok) break;
            if (more) {
              ik = take();
              ok = ik >= 0;
              if (!ok) break;
              issue_s(0, 0, ik);
            }
            ok = issue_pv(1, iv, c > 0);
            if (!ok) break;
            commit(&empty[iv]);
            if (more) {
              issue_s(1, 1, ik);
              commit(&empty[ik]);
            }
          }
        }
        if (ok) finish();
      }
      if (!ok) {
        *abort_flag = 1;
        if (lane == 0) raise_status(p.status, DFLASH_ERR_TIMEOUT, 524);
        // the products in flight end before their memory is given back
        finish();
        mbar_wait(o_full, (segs - 1) & 1, nullptr);
      }
    }
  } else {
    // ------------------------------------------------ softmax: a thread per row
    const int tile = warp / 4;
    const int r128 = (warp % 4) * 32 + lane;  // row of the tile, TMEM lane
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp % 4) * 32) << 16);
    const uint32_t s_addr = lane_base + C::S_COL + tile * 128;
    const uint32_t o_addr = lane_base + C::O_COL + tile * 128;
    // After a wait that gave up, a warp goes on through the segments without
    // waiting, so that all warps meet at the same named barriers; the results
    // are void (the status word says so).
    int segs = 0, ns = 0;
    bool ok = true;
    while (seg.next(p, L, pl)) {
      const int e = seg.e, n = seg.chunk1 - seg.chunk0;
      const bool pre = e < p.ng, split = pre ? L.prefix_split : L.suffix_split;
      const int tiles = entity_tiles(p, L, e);
      const int kvh = small_div(seg.ul, tiles), row0 = (seg.ul - kvh * tiles) * L.tile_rows;
      const RowMap rows(p, e, kvh);
      // ---- Q of the segment (split: A's warps load it for both)
      if (tile == 0 || !split) {
        // piece c of rows r0, r0 + RS, ...; eight loads in flight
        constexpr int CH = D / 8, RS = 128 / CH;
        const int c = tid % CH, r0 = tid % 128 / CH;
#pragma unroll 1
        for (int b = 0; b < 128; b += 8 * RS) {
          uint4 x[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            int ri;
            size_t vec;
            x[j] = make_uint4(0u, 0u, 0u, 0u);
            if (rows.at(row0 + tile * 128 + b + j * RS + r0, &ri, &vec))
              x[j] = __ldcg(reinterpret_cast<const uint4*>(p.q + vec * D + c * 8));
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int r = b + j * RS + r0;
            *reinterpret_cast<uint4*>(sm + tile * C::Q_TILE + (c / 8) * (128 * 128) + r * 128 +
                                      (((c % 8) ^ (r & 7)) << 4)) = x[j];
          }
        }
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
      // keys this row sees, from the segment's first
      const int my_row = row0 + (split ? r128 : tile * 128 + r128);
      int lim = 0;
      {
        int ri = 0;
        size_t vec;
        const bool real = rows.at(my_row, &ri, &vec);
        const int base = (pre ? 0 : pl.cut[inv_div(e - p.ng, p.inv_group)]) + seg.chunk0 * kChunk;
        const int ctx = pre ? pl.cut[e] : pl.ctx[e - p.ng];
        lim = (real && !pre && p.causal ? ctx - p.n + ri + 1 : ctx) - base;
      }
      float m = -INFINITY, l = 0.f;
      for (int c = split ? tile : 0; ok && c < n; c += split ? 2 : 1) {
        if (!__all_sync(0xffffffffu, mbar_wait(&s_full[tile], ns++ & 1, abort_flag))) {
          ok = false;
          break;
        }
        tc_fence_after();
        // the row's maximum; in a chunk that ends past this row's keys the
        // scores beyond them become -inf, here and in TMEM
        const bool masked = __any_sync(0xffffffffu, (c + 1) * kChunk > lim);
        uint32_t x[4][32];
#pragma unroll
        for (int j = 0; j < 4; ++j) tmem_ld32_nowait(s_addr + j * 32, x[j]);
        tmem_wait_ld(x[0]);
#pragma unroll
        for (int j = 1; j < 4; ++j) tmem_regs_ready(x[j]);
        if (masked) {
          const int left = lim - c * kChunk;
#pragma unroll
          for (int j = 0; j < 128; ++j)
            if (j >= left) x[j / 32][j % 32] = 0xFF800000u;
          tmem_st32(s_addr, x[0]);
          tmem_st32(s_addr + 32, x[1]);
          tmem_wait_st();
        }
        float mx4[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          mx4[j] = fmaxf(__uint_as_float(x[j][0]), __uint_as_float(x[j][1]));
#pragma unroll
          for (int i = 2; i < 32; i += 2)
            mx4[j] = fmaxf(mx4[j], fmaxf(__uint_as_float(x[j][i]), __uint_as_float(x[j][i + 1])));
        }
        const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
        const float mc = mx * p.scale_log2;
        const bool raise = mc > m + kRaise;
        const bool rescale = raise && m != -INFINITY;
        if (__any_sync(0xffffffffu, rescale)) {
          // S is complete, so the PV before it is too: O may be read
          const float alpha = rescale ? ex2(m - mc) : 1.f;
#pragma unroll 1
          for (int q = 0; q < D / 32; ++q) {
            uint32_t o[32];
            tmem_ld32_nowait(o_addr + q * 32, o);
            tmem_wait_ld(o);
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
            tmem_st32(o_addr + q * 32, o);
            tmem_wait_st();
          }
          l *= alpha;
        }
        if (raise) m = mc;
        // P = exp2(scale S - m) in bf16.  The upper 64 keys first, still in
        // registers: the product with V starts on them while the lower 64,
        // read again from TMEM, are formed.
        const float neg = m == -INFINITY ? 0.f : -m;
        const float2 sc2 = make_float2(p.scale_log2, p.scale_log2), neg2 = make_float2(neg, neg);
        float2 la = make_float2(0.f, 0.f), lb = la;
        auto form = [&](const uint32_t (&y)[32], uint32_t* pk) {
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            float2 t = fma2(make_float2(__uint_as_float(y[2 * j]), __uint_as_float(y[2 * j + 1])), sc2, neg2);
            t.x = ex2(t.x);
            t.y = ex2(t.y);
            if (j & 1) lb = add2(lb, t);
            else la = add2(la, t);
            pk[j] = bf16x2(t.x, t.y);
          }
        };
        const uint32_t p_addr = lane_base + C::P_COL + tile * 128;
#pragma unroll
        for (int h = 1; h >= 0; --h) {
          uint32_t pk[32];
          if (h == 0) {
            tmem_wait_ld(x[0]);
            tmem_regs_ready(x[1]);
          }
          form(x[2 * h], pk);
          form(x[2 * h + 1], pk + 16);
          tmem_st32(p_addr + h * 32, pk);
          if (h == 1) {
            tmem_ld32_nowait(s_addr, x[0]);
            tmem_ld32_nowait(s_addr + 32, x[1]);
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[2 * tile + 1 - h]);
        }
        l += (la.x + la.y) + (lb.x + lb.y);
      }
      if (ok && !__all_sync(0xffffffffu, mbar_wait(o_full, segs & 1, abort_flag))) ok = false;
      ++segs;
      tc_fence_after();
      if (lim > *bad_key) l = __int_as_float(0x7FFFFFFF);
      // ---- partial of the segment.  O goes through shared memory (the Q
      // tiles are free now: a quarter of one for each warp's 32 rows, half a row
      // at a time) so that rows are written to global memory whole.  Split: B
      // hands its state to A's warp with the same rows, which joins the two.
      constexpr int COLS = D / 2, PIECES = COLS / 4;  // half a row; its 16-byte pieces
      constexpr int STAGE = 32 * COLS * 4;
      static_assert(8 * STAGE <= 2 * C::Q_TILE, "stages fit the Q tiles");
      const bool have = !split || tile < n;  // split: this tile had a chunk
      uint8_t* stage = sm + warp * STAGE;
      uint8_t* stage_b = sm + (4 + warp % 4) * STAGE;
      auto pair_sync = [&]() { asm volatile("bar.sync %0, 64;" ::"r"(1 + warp % 4) : "memory"); };
      float wa = 1.f, wb = 0.f;
      if (split) {
        if (tile == 1) *reinterpret_cast<float2*>(stage + lane * 8) = make_float2(have ? m : -INFINITY, l);
        pair_sync();
        if (tile == 0) {
          const float2 b = *reinterpret_cast<const float2*>(stage_b + lane * 8);
          const float mn = fmaxf(m, b.x);
          const float ref = mn == -INFINITY ? 0.f : mn;
          wa = ex2(m - ref);
          wb = ex2(b.x - ref);
          l = l * wa + b.y * wb;
          m = mn;
        }
        pair_sync();
      }
      const size_t slot_row = part_row(p, L, e, seg.ul, worker);
      const int first = (split ? 0 : tile * 128) + (warp % 4) * 32;  // the warp's first row in the unit
      const int rows_here = min(32, rows.rows - row0 - first);
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        uint32_t o[COLS / 32][32];
        if (have) {
#pragma unroll
          for (int j = 0; j < COLS / 32; ++j) tmem_ld32_nowait(o_addr + half * COLS + j * 32, o[j]);
          tmem_wait_ld(o[0]);
#pragma unroll
          for (int j = 1; j < COLS / 32; ++j) tmem_regs_ready(o[j]);
        } else {
#pragma unroll
          for (int j = 0; j < COLS; ++j) o[j / 32][j % 32] = 0u;
        }
        auto at16 = [&](uint8_t* base, int r, int piece) {
          return reinterpret_cast<uint4*>(base + r * (COLS * 4) + ((piece ^ (r & (PIECES - 1))) << 4));
        };
        auto put = [&]() {
#pragma unroll
          for (int j = 0; j < PIECES; ++j)
            *at16(stage, lane, j) = make_uint4(o[j / 8][j % 8 * 4], o[j / 8][j % 8 * 4 + 1], o[j / 8][j % 8 * 4 + 2],
                                               o[j / 8][j % 8 * 4 + 3]);
        };
        if (split) {
          if (tile == 1) put();
          pair_sync();
          if (tile == 0) {
#pragma unroll
            for (int j = 0; j < PIECES; ++j) {
              const uint4 b = *at16(stage_b, lane, j);
              const uint32_t x[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
              for (int t = 0; t < 4; ++t) {
                uint32_t& y = o[j / 8][j % 8 * 4 + t];
                y = __float_as_uint(__uint_as_float(y) * wa + __uint_as_float(x[t]) * wb);
              }
            }
          }
          pair_sync();  // B may put its next half
        }
        if (tile == 0 || !split) {
          put();
          __syncwarp();
          for (int r = lane / PIECES; r < rows_here; r += 32 / PIECES)
            *reinterpret_cast<uint4*>(L.part_o + (slot_row + first + r) * D + half * COLS + (lane % PIECES) * 4) =
                *at16(stage, r, lane % PIECES);
          __syncwarp();
        }
      }
      if ((tile == 0 || !split) && lane < rows_here)
        *reinterpret_cast<float2*>(L.part_ml + (slot_row + first + lane) * 2) = make_float2(m, l);
      // the next Q overwrites the stages: all of the tiles' warps are done
      asm volatile("bar.sync 5, 256;" ::: "memory");
      tc_fence_before();
    }
    if (!ok) {
      *abort_flag = 1;
      if (lane == 0) raise_status(p.status, DFLASH_ERR_TIMEOUT, 525);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

template <int D>
cudaError_t launch(const CUtensorMap& map, int group0, int oob_group, const PrefixParams& p, cudaStream_t s) {
  using C = TcCfg<D>;
  constexpr int kMax = 227 * 1024;
  // barriers and flags, the plan, slack for the alignment
  const int fixed = (2 * C::MAX_SLOTS + 8) * 8 + 16 + PrefixPlan::ints(p.batch, p.ng) * 4 + 1024;
  int slots = (kMax - fixed - 2 * C::Q_TILE) / C::PLANE;
  if (slots > C::MAX_SLOTS) slots = C::MAX_SLOTS;
  const int smem = fixed + 2 * C::Q_TILE + slots * C::PLANE;
  static thread_local int allowed = -1;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(prefix_tc_kernel<D>), kMax, &allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kTcCtas);
  cfg.blockDim = dim3(kTcThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  count_launch();
  return cudaLaunchKernelEx(&cfg, prefix_tc_kernel<D>, map, p, group0, oob_group, slots);
}

}  // namespace

cudaError_t prefix_tc_launch(const CUtensorMap& map, int group0, int oob_group, const PrefixParams& p,
                             int d, cudaStream_t s) {
  return d == 128 ? launch<128>(map, group0, oob_group, p, s) : launch<64>(map, group0, oob_group, p, s);
}

}  // namespace dflash
