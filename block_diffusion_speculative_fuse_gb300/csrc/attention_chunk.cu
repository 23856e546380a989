// Attention of a ragged batch of new rows (single tokens, chunks of prompts, whole
// prompts) to the paged cache.
#include <climits>

#include "attention_chunk.cuh"

namespace dflash {

namespace {

constexpr int kThreads = 384;     // warps 0-7 softmax, 8 TMA, 9 products, 10 V's values, 11 idle
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88;  // of a thread
constexpr int kChunk = 128;       // keys
constexpr float kRaise = 8.f;     // log2
// Cost of a unit, in keys that one tile goes over (two tiles: twice the keys):
constexpr int kUnitCost = 300;    // its start and end
constexpr int kWorkerCost = 512;  // the least share of a worker
constexpr int kLeast = 2;         // chunks of a piece of a unit

template <int D>
struct Cfg {
  static constexpr int HALVES = D / 64;
  static constexpr int PAGE = 16 * D * 2;
  static constexpr int PLANE = kChunk * D * 2;           // K or V of a chunk
  static constexpr int Q_TILE = 128 * D * 2;             // [HALVES][128 rows][128 B]
  static constexpr int SLOTS = D == 128 ? 4 : 8;
  static constexpr int STAGE = 32 * 128;                 // of a softmax warp: 32 rows of 128 B
  static constexpr uint32_t S_COL = 0, P_COL = 64, O_COL = 256;
  static constexpr int FIXED = 2 * Q_TILE + SLOTS * PLANE + 8 * STAGE;
  static constexpr int SMEM = FIXED + 3072;
};

// A place in the work: requests, their KV heads, their row units, chunks of keys.
struct Place {
  int r, h, i, c;
};

// What a worker leaves for the join.
struct WorkerRecord {
  int cont, ends;            // its first piece continues a unit; and ends it
  int head;                  // its last piece begins a unit that others continue
  int token0, tokens, kvh;   // that unit's first row of the call, its rows, its head
  int pad[2];
};

// Units of a request: `per` rows (tokens) each; a last one of at most half as many has
// one tile.
struct Units {
  int n, ctx, per, half, tiles;
  bool causal;
  __device__ Units(const ChunkRequest& q, int tokens, int causal_)
      : n(q.n), ctx(q.ctx), per(2 * tokens), half(tokens), tiles((q.n + 2 * tokens - 1) / (2 * tokens)),
        causal(causal_) {}
  __device__ int rows(int i) const { return min(per, n - i * per); }
  __device__ bool split(int i) const { return n - i * per <= half; }
  // keys that the unit's last row sees
  __device__ int keys(int i) const { return causal ? max(0, ctx - n + min(n, (i + 1) * per)) : ctx; }
  __device__ int chunks(int i) const { return (keys(i) + kChunk - 1) / kChunk; }
  // cost of units [0, k), k < tiles: keys in closed form
  __device__ long long cost(int k) const {
    long long s = static_cast<long long>(kUnitCost) * k;
    if (!causal) return s + 2ll * k * ctx;
    const long long base = ctx - n;
    const long long skip = base < 0 ? min(static_cast<long long>(k), -base / per) : 0;  // units that see nothing
    return s + 2 * ((k - skip) * base + per * (static_cast<long long>(k) * (k + 1) - skip * (skip + 1)) / 2);
  }
  __device__ long long total() const {
    return tiles == 0 ? 0 : cost(tiles - 1) + kUnitCost + static_cast<long long>(split(tiles - 1) ? 1 : 2) * keys(tiles - 1);
  }
  // the unit and chunk at which a boundary at cost x of [0, total()) cuts
  __device__ void find(long long x, int* i, int* c) const {
    int lo = 0, hi = tiles - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (cost(mid) <= x) lo = mid;
      else hi = mid - 1;
    }
    *i = lo;
    const int all = chunks(lo);
    const long long at = (x - cost(lo) - kUnitCost) / (split(lo) ? 1 : 2);
    int cut = static_cast<int>(max(0ll, at + kChunk / 2) / kChunk);
    // no pieces below kLeast chunks
    if (all < 2 * kLeast) cut = 2 * cut <= all ? 0 : all;
    else if (cut < kLeast) cut = 0;
    else if (cut > all - kLeast) cut = all;
    *c = cut;
  }
};

__device__ __forceinline__ ChunkRequest request(const ChunkParams& p, int r) {
  return ChunkRequest(p.row_start, p.ctx_len, r, p.T, p.max_pages, p.status, 551);
}

// Start and end of a worker's range, by all threads of the CTA; ends with a barrier.
// scratch: kThreads / 32 + 1 words of 64 bits.
__device__ void find_range(const ChunkParams& p, int worker, int workers, Place* out, long long* scratch) {
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  auto cost_of = [&](int r) {
    return r < p.batch ? Units(request(p, r), p.tokens, p.causal).total() * p.hkv : 0ll;
  };
  auto inclusive = [&](long long v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    return v;
  };
  long long mine = 0;
  for (int r = tid; r < p.batch; r += kThreads) mine += cost_of(r);
  mine = inclusive(mine);
  if (lane == 31) scratch[warp] = mine;
  if (tid < 2) out[tid] = Place{p.batch, 0, 0, 0};
  __syncthreads();
  long long all = 0;
  for (int w = 0; w < kThreads / 32; ++w) all += scratch[w];
  const long long used = min(static_cast<long long>(workers), (all + kWorkerCost - 1) / kWorkerCost);
  __syncthreads();
  if (worker < used) {
    const long long x[2] = {all * worker / used, all * (worker + 1) / used};
    long long before = 0;
    for (int base = 0; base < p.batch; base += kThreads) {
      const long long v = cost_of(base + tid), upto = inclusive(v);
      if (lane == 31) scratch[warp] = upto;
      __syncthreads();
      long long at = before + upto - v;
      for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) at += scratch[w];
        before += scratch[w];
      }
      for (int j = 0; j < 2; ++j)
        if (v > 0 && x[j] >= at && x[j] < at + v) {
          const Units u(request(p, base + tid), p.tokens, p.causal);
          const long long one = v / p.hkv;
          const int h = static_cast<int>((x[j] - at) / one);
          Place pl{base + tid, h, 0, 0};
          u.find(x[j] - at - h * one, &pl.i, &pl.c);
          out[j] = pl;
        }
      __syncthreads();
    }
  }
  __syncthreads();
}

// Walks a worker's range piece by piece: of unit (r, h, i) the chunks [c0, c1).
struct Pieces {
  Place at, end;
  int c0, c1, all;   // of the piece; chunks of its unit
  ChunkRequest q;
  int loaded;
  __device__ Pieces(const Place* range) : at(range[0]), end(range[1]), c0(0), c1(0), all(0), loaded(-1) {}
  __device__ bool past() const {
    if (at.r != end.r) return at.r > end.r;
    if (at.h != end.h) return at.h > end.h;
    if (at.i != end.i) return at.i > end.i;
    return at.c >= end.c;
  }
  int r, h, i;
  __device__ bool next(const ChunkParams& p) {
    while (at.r < p.batch && !past()) {
      if (loaded != at.r) {
        q = request(p, at.r);
        loaded = at.r;
      }
      const Units u(q, p.tokens, p.causal);
      if (at.i >= u.tiles) {  // the request's next head, or the next request
        at.i = at.c = 0;
        if (u.tiles == 0 || ++at.h >= p.hkv) {
          at.h = 0;
          ++at.r;
        }
        continue;
      }
      r = at.r, h = at.h, i = at.i, c0 = at.c;
      all = u.chunks(i);
      const bool here = r == end.r && h == end.h && i == end.i;
      c1 = here ? end.c : all;
      ++at.i;
      at.c = 0;
      if (c0 >= c1 && !(all == 0 && !here)) continue;
      return true;
    }
    return false;
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_kernel(const __grid_constant__ CUtensorMap kv_map, const __grid_constant__ CUtensorMap q_map,
                 const __grid_constant__ ChunkParams p, int group0, int oob_group) {
  using C = Cfg<D>;
  constexpr int SLOTS = C::SLOTS;
  extern __shared__ __align__(1024) uint8_t sm[];
  uint8_t* ring = sm + 2 * C::Q_TILE;
  uint8_t* stages = ring + SLOTS * C::PLANE;
  float2* exch = reinterpret_cast<float2*>(stages + 8 * C::STAGE);  // [256] (m, l) of a row
  uint64_t* full = reinterpret_cast<uint64_t*>(exch + 256);
  uint64_t* empty = full + SLOTS;
  uint64_t* clean = empty + SLOTS;          // the plane's V has been gone over
  uint64_t* s_full = clean + SLOTS;         // [2] S of a tile is complete (and the PV before it)
  uint64_t* p_full = s_full + 2;            // [2][2] P of a tile is in TMEM: upper, lower 64 keys
  uint64_t* q_full = p_full + 4;            // Q of the piece is in shared memory
  uint64_t* q_free = q_full + 1;            // its last S is complete
  uint64_t* o_full = q_free + 1;            // all of the piece's products are complete; bad
  long long* scratch = reinterpret_cast<long long*>(o_full + 1);  // [kThreads / 32]
  Place* range = reinterpret_cast<Place*>(scratch + kThreads / 32);  // [2]
  volatile int* bad = reinterpret_cast<volatile int*>(range + 2);    // [16] first key with a V that is not finite
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(const_cast<int*>(bad) + 16);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  static_assert(256 * 8 + (3 * SLOTS + 9) * 8 + kThreads / 32 * 8 + 2 * 16 + 18 * 4 <= 3072, "fits");

  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  if (tid == 0) {
    for (int s = 0; s < SLOTS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 2);
      mbar_init(&clean[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s_full[t], 1);
      mbar_init(&p_full[2 * t], 4);
      mbar_init(&p_full[2 * t + 1], 4);
    }
    mbar_init(q_full, 1);
    mbar_init(q_free, 1);
    mbar_init(o_full, 2);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&kv_map);
    tma_prefetch_desc(&q_map);
  }
  if (warp == 9) tmem_alloc(tmem_slot, 512);
  griddep_wait();
  griddep_launch_dependents();
  const int worker = blockIdx.x;
  find_range(p, worker, gridDim.x, range, scratch);  // ends with a barrier
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  Pieces seg(range);

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == 8) {
      // ------------------------------------------------ TMA producer
      const uint64_t pol = l2_policy_evict_normal();
      int at = 0, segs = 0;                        // planes, pieces requested so far
      Cursor cur;
      bool ok = true;
      while (ok && seg.next(p)) {
        const int n = seg.c1 - seg.c0;
        if (n == 0) continue;
        const Units u(seg.q, p.tokens, p.causal);
        const bool split = u.split(seg.i);
        const int page0 = seg.c0 * 8;
        const int npg = min(n * 8, (u.keys(seg.i) + 15) / 16 - page0);
        const int32_t* table = p.page_table + static_cast<size_t>(seg.r) * p.max_pages + page0;
        // lane -> 8-row group of its page's K plane in the map, 32 pages a time,
        // the next 32 requested ahead
        auto ids_of = [&](int b) {
          const int j = b * 32 + lane;
          return j < npg ? max(__ldcg(table + j), -1) : -2;  // -2: past the piece
        };
        auto check = [&](int id) {
          if (id >= 0 && id < p.n_pages) return group0 + (id * 2 * p.hkv + seg.h) * 2;
          if (id != -2) raise_status(p.status, DFLASH_ERR_CAPACITY, 553);
          return oob_group;
        };
        int kb = 0, vb = 0;  // 32-page batch held for K, for V
        int next_id = ids_of(1);
        int kg = check(ids_of(0)), vg = kg;
        int k = 0, v = 0;
        for (int j = 0; j < 2 * n; ++j, ++at, cur.advance(SLOTS)) {
          // planes in the order of their use: K0 V0 K1 V1 ..., one tile K0 K1 V0 K2 V1 ...
          const bool is_k = k < n && (split ? k + max(0, k - 1) : 2 * k) == j;
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
          const int grp = __shfl_sync(0xffffffffu, is_k ? kg : vg, (c % 4) * 8 + lane % 8);
          const int st = cur.slot;
          int go = 1;
          if (lane == 0) {
            if (at >= SLOTS && !mbar_wait(&empty[st], cur.parity ^ 1, abort_flag)) go = 0;
            if (go && j == 0 && segs > 0 && !mbar_wait(q_free, (segs - 1) & 1, abort_flag)) go = 0;
            if (go) {
              mbar_arrive_expect_tx(&full[st], C::PLANE);
            } else {
              *abort_flag = 1;
              raise_status(p.status, DFLASH_ERR_TIMEOUT, 554);
            }
          }
          if (!__shfl_sync(0xffffffffu, go, 0)) {
            ok = false;
            break;
          }
          if (lane < 8) {
            const int y = grp == oob_group || is_k ? grp : grp + p.hkv * 2;
            tma_load_4d(smem_u32(ring + st * C::PLANE + lane * C::PAGE), &kv_map, y, &full[st], pol);
          }
          if (j == 0) {  // Q of the piece: [tile][column half], `tokens` rows of G heads each
            if (lane == 0) {
              const int boxes = (split ? 1 : 2) * C::HALVES;
              mbar_arrive_expect_tx(q_full, boxes * p.tokens * p.G * 128);
              for (int b = 0; b < boxes; ++b)
                tma_load_3d(sm + b * (128 * 128), &q_map, b % C::HALVES * 64, seg.h * p.G,
                            seg.q.start + seg.i * u.per + b / C::HALVES * p.tokens, q_full, pol);
            }
            __syncwarp();
            ++segs;
          }
        }
      }
      // copies still in flight after an abort land before the CTA exits
      if (lane == 0) {
        for (int j = max(0, at - SLOTS); j < at; ++j) mbar_wait(&full[j % SLOTS], (j / SLOTS) & 1, nullptr);
        if (segs > 0) mbar_wait(q_full, (segs - 1) & 1, nullptr);
      }
    } else if (warp == 9) {
      // ------------------------------------------------ products
      constexpr uint32_t idesc_s = umma_idesc_bf16(128, kChunk);
      constexpr uint32_t idesc_pv = umma_idesc_bf16(128, D) | (1u << 16);  // V MN-major
      constexpr uint32_t GS = C::HALVES * 1024;  // between 8-row groups of a plane
      const uint32_t q_addr = smem_u32(sm), ring_addr = smem_u32(ring);
      int segs = 0;
      int np[2] = {0, 0};  // parity of the next P of each tile
      bool ok = true;
      Cursor cur;          // the next plane: they are used in the order they arrive
      auto commit = [&](uint64_t* bar) {
        if (elect_one()) umma_commit(bar);
        __syncwarp();
      };
      auto finish = [&]() {
        if (lane == 0) mbar_arrive(o_full);
        commit(o_full);
      };
      // waits for the next plane and takes it: its slot, or -1
      auto take = [&](bool is_v) {
        const int st = cur.slot;
        bool r = mbar_wait(&full[st], cur.parity, abort_flag);
        if (r && is_v) r = mbar_wait(&clean[st], cur.parity, abort_flag);
        cur.advance(SLOTS);
        return __all_sync(0xffffffffu, r) ? st : -1;
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
      while (ok && seg.next(p)) {
        const int n = seg.c1 - seg.c0;
        if (n == 0) continue;
        const bool split = Units(seg.q, p.tokens, p.causal).split(seg.i);
        ok = __all_sync(0xffffffffu, mbar_wait(q_full, segs++ & 1, abort_flag));
        if (!ok) break;
        if (split) {
          for (int c = 0; ok && c < min(2, n); ++c) {
            const int ik = take(false);
            ok = ik >= 0;
            if (!ok) break;
            tc_fence_after();
            issue_s(c, 0, ik);
            commit(&empty[ik]);
            if (c + 1 == n) commit(q_free);
          }
          for (int c = 0; ok && c < n; ++c) {
            const int t = c & 1, iv = take(true);
            ok = iv >= 0 && issue_pv(t, iv, c >= 2);
            if (!ok) break;
            commit(&empty[iv]);
            if (c + 2 < n) {
              const int ik = take(false);
              ok = ik >= 0;
              if (!ok) break;
              issue_s(t, 0, ik);
              commit(&empty[ik]);
            }
            if (c + 3 == n) commit(q_free);
          }
        } else {
          int ik = take(false);
          ok = ik >= 0;
          if (ok) {
            tc_fence_after();
            issue_s(0, 0, ik);
            issue_s(1, 1, ik);
            commit(&empty[ik]);
            if (n == 1) commit(q_free);
          }
          for (int c = 0; ok && c < n; ++c) {
            const bool more = c + 1 < n;
            const int iv = take(true);
            ok = iv >= 0 && issue_pv(0, iv, c > 0);
            if (!ok) break;
            if (more) {
              ik = take(false);
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
              if (c + 2 == n) commit(q_free);
            }
          }
        }
        if (ok) finish();
      }
      if (!ok) {
        *abort_flag = 1;
        if (lane == 0) raise_status(p.status, DFLASH_ERR_TIMEOUT, 555);
        // the products in flight end before their memory is given back
        finish();
        mbar_wait(o_full, (segs - 1) & 1, nullptr);
      }
    } else if (warp == 10) {
      // ------------------------------------------------ V's values
      int segs = 0;
      bool ok = true;
      Cursor cur;
      while (ok && seg.next(p)) {
        const int n = seg.c1 - seg.c0;
        if (n == 0) continue;
        const Units u(seg.q, p.tokens, p.causal);
        const bool split = u.split(seg.i);
        // keys from the piece's first one: all rows see those before `first`, none those from `live` on
        const int live = u.keys(seg.i) - seg.c0 * kChunk;
        const int first = u.causal ? max(0, u.ctx - u.n + seg.i * u.per + 1) - seg.c0 * kChunk : live;
        int found = INT_MAX;
        if (lane == 0) bad[segs % 16] = INT_MAX;
        int k = 0, v = 0;
        for (int j = 0; j < 2 * n; ++j) {
          const bool is_k = k < n && (split ? k + max(0, k - 1) : 2 * k) == j;
          const int c = is_k ? k++ : v++;
          const int st = cur.slot;
          ok = __all_sync(0xffffffffu, mbar_wait(&full[st], cur.parity, abort_flag));
          if (!ok) break;
          cur.advance(SLOTS);
          if (!is_k && (c + 1) * kChunk > first) {
            const int b = clean_v<D>(ring + st * C::PLANE, first - c * kChunk, live - c * kChunk);
            if (b < kChunk) found = min(found, c * kChunk + b);
          }
          if (j == 2 * n - 1) {
            found = __reduce_min_sync(0xffffffffu, found);
            if (lane == 0) bad[segs % 16] = found;
          }
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&clean[st]);
            mbar_arrive(&empty[st]);
          }
        }
        ++segs;
      }
      if (!ok) {
        *abort_flag = 1;
        if (lane == 0) raise_status(p.status, DFLASH_ERR_TIMEOUT, 556);
      }
    }
  } else {
    // ------------------------------------------------ softmax: a thread per row
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int tile = warp / 4;
    const int r128 = (warp % 4) * 32 + lane;  // row of the tile, TMEM lane
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp % 4) * 32) << 16);
    const uint32_t s_addr = lane_base + C::S_COL + tile * 128;
    const uint32_t o_addr = lane_base + C::O_COL + tile * 128;
    uint8_t* stage = stages + warp * C::STAGE;
    // row / G for rows below 128
    const int inv_G = 65536 / p.G + 1;
    WorkerRecord rec = {};
    // After a wait that gave up, a warp goes on through the pieces without
    // waiting, so that all warps meet at the same named barriers; the results
    // are void (the status word says so).
    int segs = 0, ns = 0;
    bool ok = true, first_piece = true;
    while (seg.next(p)) {
      const int n = seg.c1 - seg.c0;
      const Units u(seg.q, p.tokens, p.causal);
      const bool split = u.split(seg.i);
      const int tokens = u.rows(seg.i);                    // of the unit
      const int token0 = seg.q.start + seg.i * u.per;      // its first row of the call
      if (first_piece && seg.c0 > 0) {
        rec.cont = 1;
        rec.ends = seg.c1 == seg.all;
      }
      if (seg.c0 == 0 && seg.c1 < seg.all) {
        rec.head = 1;
        rec.token0 = token0;
        rec.tokens = tokens;
        rec.kvh = seg.h;
      }
      first_piece = false;
      // keys this row sees, from the piece's first
      const int tok = r128 * inv_G >> 16;                  // of the tile
      const int my_token = (split ? 0 : tile * u.half) + tok;
      const bool real = tok < u.half && my_token < tokens;
      int lim = INT_MAX;   // rows that do not exist see whatever lies there
      if (real) lim = (u.causal ? max(0, u.ctx - u.n + seg.i * u.per + my_token + 1) : u.ctx) - seg.c0 * kChunk;
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
      if (n > 0) {
        if (ok && !__all_sync(0xffffffffu, mbar_wait(o_full, segs & 1, abort_flag))) ok = false;
        if (lim > bad[segs % 16]) l = __int_as_float(0x7FFFFFFF);
        ++segs;
        tc_fence_after();
      }
      // ---- result of the piece.  One tile: the two states are joined, A's warps
      // taking the lower half of the columns, B's the upper.
      const bool have = n > (split ? tile : 0);
      float wa = have ? 1.f : 0.f, wb = 0.f;   // weights of this tile's O and the other's
      auto pair_sync = [&]() { asm volatile("bar.sync %0, 64;" ::"r"(1 + warp % 4) : "memory"); };
      if (split) {
        exch[tile * 128 + r128] = make_float2(m, l);
        pair_sync();
        const float2 y = exch[(1 - tile) * 128 + r128];
        const float mn = fmaxf(m, y.x), ref = mn == -INFINITY ? 0.f : mn;
        wa = have ? ex2(m - ref) : 0.f;
        wb = n > 1 - tile ? ex2(y.x - ref) : 0.f;
        // (the same order of summation in both tiles' warps)
        const float mine = l * wa, other = y.y * wb;
        l = tile == 0 ? mine + other : other + mine;
        m = mn;
      }
      const bool whole = seg.c0 == 0 && seg.c1 == seg.all;
      const int row0 = (split ? 0 : tile * 128) + (warp % 4) * 32;   // the warp's first row in the unit
      constexpr int HALF = D / 2;
      const int col0 = split ? tile * HALF : 0, cols = split ? HALF : D;
      const float inv = whole ? (m == -INFINITY ? 0.f : 1.f / l) : 1.f;
      const float fa = wa * inv, fb = wb * inv;
      const size_t slot = 2 * static_cast<size_t>(worker) + (seg.c0 > 0 ? 0 : 1);
#pragma unroll 1
      for (int cc = col0; cc < col0 + cols; cc += 32) {
        uint32_t o[32];
        const bool use_a = n > 0 && (!split || have), use_b = split && n > 1 - tile;
        if (use_a) {
          tmem_ld32_nowait(o_addr + cc, o);
          tmem_wait_ld(o);
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(fa == 0.f ? 0.f : __uint_as_float(o[j]) * fa);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = 0u;
        }
        if (use_b) {
          uint32_t y[32];
          tmem_ld32_nowait(lane_base + C::O_COL + (1 - tile) * 128 + cc, y);
          tmem_wait_ld(y);
#pragma unroll
          for (int j = 0; j < 32; ++j)
            o[j] = __float_as_uint(__uint_as_float(o[j]) + (fb == 0.f ? 0.f : __uint_as_float(y[j]) * fb));
        }
        // through shared memory, so that whole lines are written
        auto at16 = [&](int r, int piece) { return reinterpret_cast<uint4*>(stage + r * 128 + ((piece ^ (r & 7)) << 4)); };
        if (whole) {  // bf16: 32 columns are four pieces
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t w[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) w[t] = bf16x2(__uint_as_float(o[8 * j + 2 * t]), __uint_as_float(o[8 * j + 2 * t + 1]));
            *at16(lane, j) = make_uint4(w[0], w[1], w[2], w[3]);
          }
          __syncwarp();
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const int r = b * 8 + lane / 4, rt = (warp % 4) * 32 + r, t = rt * inv_G >> 16;
            const int token = (split ? 0 : tile * u.half) + t;
            if (t < u.half && token < tokens)
              *reinterpret_cast<uint4*>(p.out + static_cast<size_t>(token0 + token) * p.ld_out +
                                        (seg.h * p.G + rt - t * p.G) * D + cc + lane % 4 * 8) = *at16(r, lane % 4);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) *at16(lane, j) = make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
          __syncwarp();
#pragma unroll
          for (int b = 0; b < 8; ++b) {
            const int r = b * 4 + lane / 8, rt = (warp % 4) * 32 + r, t = rt * inv_G >> 16;
            if (t < u.half && (split ? 0 : tile * u.half) + t < tokens)
              *reinterpret_cast<uint4*>(p.part_o + (slot * p.slot_rows + row0 + r) * D + cc + lane % 8 * 4) =
                  *at16(r, lane % 8);
          }
        }
        __syncwarp();
      }
      if (real && (!split || tile == 0)) {
        if (!whole) {
          *reinterpret_cast<float2*>(p.part_ml + (slot * p.slot_rows + row0 + lane) * 2) = make_float2(m, l);
        } else if (p.lse != nullptr) {
          p.lse[static_cast<size_t>(token0 + my_token) * p.hq + seg.h * p.G + r128 - tok * p.G] =
              m == -INFINITY ? -INFINITY : (m + log2f(l)) * 0.693147180559945309f;
        }
      }
      // both tiles' O have been read before either's next product
      if (split) pair_sync();
      tc_fence_before();
    }
    if (!ok) {
      *abort_flag = 1;
      if (lane == 0) raise_status(p.status, DFLASH_ERR_TIMEOUT, 557);
    }
    if (tid == 0) reinterpret_cast<WorkerRecord*>(p.records)[worker] = rec;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

// Joins the pieces of the units that were cut: a CTA takes 32 rows of the unit that
// worker blockIdx.x began; a warp per row.
constexpr int kJoinRows = 32;
template <int D>
__global__ void __launch_bounds__(256) chunk_join_kernel(const __grid_constant__ ChunkParams p, int workers) {
  constexpr int VEC = D / 32;
  __shared__ int list[kChunkWorkers + 1], count[8], last;
  griddep_wait();
  griddep_launch_dependents();
  const WorkerRecord* recs = reinterpret_cast<const WorkerRecord*>(p.records);
  const int w = blockIdx.x, tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const WorkerRecord head = recs[w];
  if (!head.head) return;
  if (tid == 0) {
    last = workers - 1;
    list[0] = 2 * w + 1;
  }
  __syncthreads();
  int cont = 0;
  if (tid > w && tid < workers) {
    cont = recs[tid].cont;
    if (cont && recs[tid].ends) atomicMin(&last, tid);
  }
  __syncthreads();
  cont = cont && tid <= last;
  const unsigned votes = __ballot_sync(0xffffffffu, cont);
  if (lane == 0) count[warp] = __popc(votes);
  __syncthreads();
  int parts = 1;
  for (int j = 0; j < 8; ++j) {
    if (j == warp && cont) list[parts + __popc(votes & ((1u << lane) - 1))] = 2 * tid;
    parts += count[j];
  }
  __syncthreads();
  constexpr int MOST = (kChunkWorkers + 1 + 31) / 32;
#pragma unroll 1
  for (int row = blockIdx.y * kJoinRows + warp; row < min((blockIdx.y + 1) * kJoinRows, p.slot_rows); row += 8) {
    const int rt = row % 128, t = rt / p.G, token = row / 128 * p.tokens + t;
    if (t >= p.tokens || token >= head.tokens) continue;
    float ms[MOST], ls[MOST], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int j = 0; j < MOST; ++j) {
      ms[j] = -INFINITY, ls[j] = 0.f;
      if (j * 32 + lane < parts) {
        const float2 y = __ldcg(reinterpret_cast<const float2*>(p.part_ml + (static_cast<size_t>(list[j * 32 + lane]) * p.slot_rows + row) * 2));
        ms[j] = y.x, ls[j] = y.y;
      }
      m = fmaxf(m, ms[j]);
    }
    m = warp_max(m);
    float acc[VEC] = {};
#pragma unroll
    for (int j = 0; j < MOST; ++j) {
      const float weight = ms[j] == -INFINITY ? 0.f : exp2f(ms[j] - m);
      l += warp_sum(weight == 0.f ? 0.f : ls[j] * weight);
      const int here = min(32, parts - j * 32);
#pragma unroll 4
      for (int i = 0; i < here; ++i) {
        const float wi = __shfl_sync(0xffffffffu, weight, i);
        const float* src = p.part_o + (static_cast<size_t>(list[j * 32 + i]) * p.slot_rows + row) * D + lane * VEC;
        float v[VEC];
        if constexpr (VEC == 4) {
          const float4 y = __ldcg(reinterpret_cast<const float4*>(src));
          v[0] = y.x, v[1] = y.y, v[2] = y.z, v[3] = y.w;
        } else {
          const float2 y = __ldcg(reinterpret_cast<const float2*>(src));
          v[0] = y.x, v[1] = y.y;
        }
        if (wi > 0.f) {
#pragma unroll
          for (int k = 0; k < VEC; ++k) acc[k] = fmaf(v[k], wi, acc[k]);
        }
      }
    }
    const bool any = m > -INFINITY;
    const float inv = any ? 1.f / l : 0.f;
    const int head_of_row = head.kvh * p.G + rt - t * p.G;
    uint16_t* dst = p.out + static_cast<size_t>(head.token0 + token) * p.ld_out + head_of_row * D + lane * VEC;
    if constexpr (VEC == 4)
      *reinterpret_cast<uint2*>(dst) = make_uint2(bf16x2(acc[0] * inv, acc[1] * inv), bf16x2(acc[2] * inv, acc[3] * inv));
    else
      *reinterpret_cast<uint32_t*>(dst) = bf16x2(acc[0] * inv, acc[1] * inv);
    if (p.lse != nullptr && lane == 0)
      p.lse[static_cast<size_t>(head.token0 + token) * p.hq + head_of_row] =
          any ? (m + log2f(l)) * 0.693147180559945309f : -INFINITY;
  }
}

template <int D>
cudaError_t launch(const ChunkParams& p, const CUtensorMap& kv_map, const CUtensorMap& q_map, int group0,
                   int oob_group, cudaStream_t s) {
  static thread_local int allowed = -1;
  const bool first = allowed < 0;
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(chunk_kernel<D>), Cfg<D>::SMEM, &allowed);
  if (e == cudaSuccess && first) {
    // the warpgroups' shares come out of what the block is launched with
    cudaFuncAttributes a;
    e = cudaFuncGetAttributes(&a, chunk_kernel<D>);
    if (e == cudaSuccess && a.numRegs * kThreads < 256 * kSoftmaxRegs + 128 * kOtherRegs)
      e = cudaErrorInvalidConfiguration;
    if (e != cudaSuccess) allowed = -1;
  }
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kChunkWorkers);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Cfg<D>::SMEM;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  count_launch();
  e = cudaLaunchKernelEx(&cfg, chunk_kernel<D>, kv_map, q_map, p, group0, oob_group);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(kChunkWorkers, (p.slot_rows + kJoinRows - 1) / kJoinRows);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  count_launch();
  return cudaLaunchKernelEx(&cfg, chunk_join_kernel<D>, p, kChunkWorkers);
}

}  // namespace

cudaError_t attention_chunk_launch(const ChunkParams& p, int d, const CUtensorMap& kv_map,
                                   const CUtensorMap& q_map, int group0, int oob_group, cudaStream_t s) {
  return d == 128 ? launch<128>(p, kv_map, q_map, group0, oob_group, s)
                  : launch<64>(p, kv_map, q_map, group0, oob_group, s);
}

}  // namespace dflash
