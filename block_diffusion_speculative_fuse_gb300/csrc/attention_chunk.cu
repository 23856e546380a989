// Attention of a ragged batch of new rows (single tokens, chunks of prompts, whole
// prompts) to the paged cache.
//
//   out_i = sum_j p_ij v_j,  p_ij = exp(s_ij - lse_i),  s_ij = scale q_i . k_j
//
// A unit is the rows of up to 2 * (128 / G) tokens of a request for one KV head (G query
// heads to each, so a tile of 128 rows reads a key once for all of them): two tiles of
// 128 rows, A and B, over the same keys, 128 a chunk.  Per chunk and tile
//   S = Q K^T   (M = 128, N = 128, K = d)   TMEM, 128 columns
//   O += P V    (M = 128, N = d, K = 128)   TMEM, d columns
// in the order S_A S_B | PV_A S_A' PV_B S_B' | ..., so that the tensor pipe has one tile's
// products while the other's warps form P = exp2(S - m); P replaces S in TMEM (bf16, the A
// operand of the second product).  A unit whose rows fit one tile (single tokens) takes
// turns instead: A the even chunks, B the odd ones, over the same Q, joined at its end.
//
// Softmax: two threads to a row, 64 keys each, all of them in registers at once.  The
// row's reference maximum m is raised, and O rescaled, only when a chunk exceeds it by more
// than 2^8: after the first chunks that is rare, so the two threads' warps exchange a
// vote per chunk (one barrier with a reduction) and their maxima only when it carries.  P
// stays below 2^8, and l is summed in fp32 before P is rounded to bf16, the type that the product with
// bf16 V takes (a second term of P would be half as many products again).
//
// Work.  Lengths are on the device, so every CTA (one per SM) adds up the same costs over
// the requests, in closed form, and takes the range of equal cost that is its own; a planning
// warp walks it and hands pieces (chunks of a unit) to the others.  A unit that lies in one range
// is written by its CTA; the pieces of one that was cut leave partial (O, m, l), joined
// in order by a second kernel or, where rows are few, by the CTA that finishes last.
//
// Values that a row must not see.  S is replaced by -inf, and 0 * V must be 0: a warp goes
// over the planes of V whose keys not all of a unit's rows see, before their product:
// zeros past the last row's keys, and for what is not finite (the rows that do
// see it get a NaN by way of O's factor; l, and with it lse, does not depend on V).
//
// Bound (times with inputs that change from call to call): with whole units the products and
// their issue.  4096 rows of 32 heads behind 28672 keys (134 MB, more than L2) 1.19 to 1.28 ms by
// box and clock, 1.73 to 1.61 PFLOP/s, in two rounds; behind 126976 5.18 ms, 1.67 PFLOP/s,
// in eight.  A chunk of both tiles takes some 2800
// cycles: its products 2048 of the tensor pipe and, at 128 bytes a cycle, 2048 of shared memory (S
// reads Q and K, P V reads V, the loads write both); a tile's softmax 1100 under the other's
// products.  For short prompts the units' ends: 8 x 1024 rows take 84 us, 52 of them chunks; the
// softmax warps read and store O themselves, and the next unit's P waits for them.  For
// single tokens the keys' bytes: 32 requests of 3100 to 6200 keys 96 us, 6.1 TB/s; one
// request of 4096 keys 16 us, of which the keys' bytes are 2.5: plan, first loads and join are
// chains of loads, and code that is not yet in the instruction cache.  Beside whole units a CTA
// with single tokens takes 1800 cycles for each of its chunks (77 GB/s an SM; with d = 64
// as many): the chain of S, softmax and P V, and their issue.  That softmax goes over all 128
// rows of the tile, though only G of them are a token's.
//
// That cache decides more than arithmetic here.  All roles' code together has to stay
// in it: with the polls of 20 waits unrolled (172 KB of instructions instead of 77) a
// unit's end took 5000 cycles instead of 2500 and 8 x 1024 rows 107 us instead of 86.
#include <climits>

#include "attention_chunk.cuh"

namespace dflash {

namespace {

constexpr int kThreads = 640;     // warps 0-15 softmax, 16 TMA, 17 products, 18 V's values, 19 plan
constexpr int kWarps = kThreads / 32;
constexpr int kSoftmaxRegs = 104, kOtherRegs = 64;  // of a thread
constexpr int kChunk = 128;       // keys
constexpr float kRaise = 8.f;     // log2
constexpr int kPieces = 4;        // planned ahead
// Costs are counted in 64 keys that one tile of 128 rows goes over (32 bits).
constexpr int kUnitCost = 10;     // a unit's start and end
constexpr int kSplitCost = 3;     // of a chunk with one tile (2, 3, 4: a mixed batch, same inputs again, 238, 235, 254 us)
constexpr int kWorkerCost = 8;    // the least share of a worker
// Keys that several row units read should stay in L2 from one unit to the next.  Where those
// of all requests do not fit, the workers take the work in rounds (phases), each of fewer
// heads or requests: the units that run at a time then read the same keys.  One round against
// up to 8 (same inputs again, before the loads were quicker, which gave both 5 %): 4096 rows behind 28672 keys 1.37 ->
// 1.29 ms, behind 126976 keys 6.24 -> 5.41, 8 x 2048 rows behind 15000 3.24 -> 2.88, 1000 rows
// behind 131072 1.59 -> 1.39.
constexpr int kResident = 5760;   // in 64 keys of one head of 64: 90 MB
constexpr int kPhaseCost = 400;   // the least share of a worker in a phase (100, 200, 400: no difference)
constexpr int kLeast = 3;         // chunks of a piece of a unit (2, 3, 4: 8 prompts of 1024 rows 88,
                                  // 85, 85 us, one row of 4096 keys 16.1, 16.4, 17.2)

template <int D>
struct Cfg {
  static constexpr int HALVES = D / 64;
  static constexpr int PAGE = 16 * D * 2;
  static constexpr int PLANE = kChunk * D * 2;           // K or V of a chunk
  static constexpr int Q_TILE = 128 * D * 2;             // [HALVES][128 rows][128 B]
  static constexpr int SLOTS = D == 128 ? 5 : 10;
  static constexpr uint32_t S_COL = 0, O_COL = 256;      // + 128 * tile
  static constexpr int FIXED = 2 * Q_TILE + SLOTS * PLANE;
  static constexpr int PLAN = (D == 128 ? 3 : 4) * 1024;                  // all else, behind the tiles
  static constexpr int SMEM = FIXED + PLAN;
};

// A place in the work: requests, their KV heads, their row units, chunks of keys.
struct Place {
  int r, h, i, c;
  int x;            // cost of everything before the request's units of this head
};

// The deal: range v, of used * phases, starts at share * v + rest * v / (used * phases);
// worker w has the ranges w, w + used, ... (one where there is one phase).
struct Deal {
  int share, rest, used, phases;
  int keys;   // in units of 64, of the requests that have several row units
  ChunkRequest q;   // of the first range's start
  __device__ int start(int v) const { return share * v + rest * v / (used * phases); }
};

// Chunks [c0, c0 + n) of a unit, for all warps of the CTA.
struct Piece {
  int n, c0;               // n -1: the end
  int keys;                // that the unit's last row sees
  int see, step;           // keys that its row k sees: max(0, see + k * step)
  int r, h, token0, tokens;  // request, KV head, first row of the call, rows
  int split, begins, ends;   // one tile; the piece is the unit's first, its last
  int x, all;              // of a unit with one tile: cost of everything before it; its chunks
  int range, first;        // whose piece it is; the range's first
};

// What a range leaves for the join.
struct RangeRecord {
  int cont, ends;            // its first piece continues a unit; and ends it
  int head;                  // its last piece begins a unit that others continue
  int token0, tokens, kvh;   // that unit's first row of the call, its rows, its head
  int pad[2];
};

// Units of a request: `per` rows (tokens) each; a last one of at most half as many has
// one tile.
struct Units {
  int n, ctx, per, tiles, causal;
  __device__ Units(const ChunkRequest& q, int tokens, int causal_)
      : n(q.n), ctx(q.ctx), per(2 * tokens), tiles((q.n + 2 * tokens - 1) / (2 * tokens)), causal(causal_) {}
  __device__ bool split(int i) const { return 2 * (n - i * per) <= per; }
  // keys that the unit's last row sees
  __device__ int keys(int i) const { return causal ? max(0, ctx - n + min(n, (i + 1) * per)) : ctx; }
  __device__ int chunks(int i) const { return (keys(i) + kChunk - 1) / kChunk; }
  // cost of units [0, k), k < tiles, from the sum of their keys in closed form
  __device__ int cost(int k) const {
    long long s = static_cast<long long>(k) * ctx;
    if (causal) {
      const int base = ctx - n, skip = base < 0 ? min(k, -base / per) : 0;  // units that see nothing
      s = static_cast<long long>(k - skip) * base +
          per * (static_cast<long long>(k) * (k + 1) - static_cast<long long>(skip) * (skip + 1)) / 2;
    }
    return kUnitCost * k + static_cast<int>(s >> 5);
  }
  static __device__ int unit_cost(int keys, bool split) {
    return kUnitCost + (split ? keys / kChunk * kSplitCost : keys >> 5);
  }
  __device__ int total() const {
    return tiles == 0 ? 0 : cost(tiles - 1) + unit_cost(keys(tiles - 1), split(tiles - 1));
  }
  // the unit and chunk at which a boundary at cost x of [0, total()) cuts
  __device__ void find(int x, int* i, int* c) const {
    int lo = 0, hi = tiles - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (cost(mid) <= x) lo = mid;
      else hi = mid - 1;
    }
    *i = lo;
    *c = cut(x - cost(lo), chunks(lo), split(lo));
  }
  // the chunk at which a boundary at cost x of the unit cuts
  static __device__ int cut(int x, int all, bool split) {
    const int at = max(0, x - kUnitCost);
    int cut = split ? (at + kSplitCost / 2) / kSplitCost : at / 4 + (at % 4 > 1);
    // no pieces below kLeast chunks
    if (all < 2 * kLeast) cut = 2 * cut <= all ? 0 : all;
    else if (cut < kLeast) cut = 0;
    else if (cut > all - kLeast) cut = all;
    return cut;
  }
};

__device__ __forceinline__ ChunkRequest request(const ChunkParams& p, int r) {
  return ChunkRequest(p.row_start, p.ctx_len, r, p.T, p.max_pages, p.status, 551);
}

// Start and end of a worker's ranges, by all threads of the CTA; ends with a barrier.
// scratch: kWarps words.
__device__ void find_range(const ChunkParams& p, int worker, int workers, Place* out, int* scratch, Deal* deal) {
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  if (tid < 2 * kChunkPhases) out[tid] = Place{p.batch, 0, 0, 0, 0};
  if (tid == 0) *deal = Deal{0, 0, 0, 1, 0, ChunkRequest()};
  int all = 0;
  Deal d{0, 0, 0, 1, 0, ChunkRequest()};
  // a first round adds up the costs, a second finds the boundaries
#pragma unroll 1
  for (int round = 0; round < 2; ++round) {
    int before = 0;
#pragma unroll 1
    for (int base = 0; base < p.batch; base += kThreads) {
      const int r = base + tid;
      const ChunkRequest q = r < p.batch ? request(p, r) : ChunkRequest();
      const Units u(q, p.tokens, p.causal);
      const int one = u.total(), v = one * p.hkv;
      int upto = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      __syncthreads();
      if (lane == 31) scratch[warp] = upto;
      if (p.phases > 1 && round == 0 && u.tiles > 1) atomicAdd(&deal->keys, q.ctx / 64);
      __syncthreads();
      int at = before + upto - v;
      const int part = lane < kWarps ? scratch[lane] : 0;
      at += __reduce_add_sync(0xffffffffu, lane < warp ? part : 0);
      before += __reduce_add_sync(0xffffffffu, part);
      if (round == 0 && p.batch <= kThreads) {  // the sum is known at once
        round = 1;
        all = before;
      }
      if (round == 1) {
        if (base == 0) {
          d.used = min(workers, (all + kWorkerCost - 1) / kWorkerCost);
          if (worker >= d.used) break;
          if (d.used == workers)
            while (d.phases < p.phases && d.phases * kResident <= static_cast<int64_t>(deal->keys) * p.hkv * p.halves &&
                   all >= 2 * d.phases * workers * kPhaseCost)
              d.phases *= 2;   // (by twos, so that a phase is whole heads more often)
          d.share = all / (d.used * d.phases);
          d.rest = all - d.share * (d.used * d.phases);
        }
#pragma unroll 1
        for (int j = 0; j < 2 * d.phases; ++j) {
          const int x = d.start(worker + j / 2 * d.used + j % 2) - at;
          if (x < 0 || x >= v) continue;
          Place pl{r, x / one, 0, 0, 0};
          if (j == 0) deal->q = q;
          pl.x = at + pl.h * one;
          u.find(x - pl.h * one, &pl.i, &pl.c);
          out[j] = pl;
        }
      }
    }
    if (round == 0) all = before;
  }
  if (tid == 0) {
    deal->share = d.share;
    deal->rest = d.rest;
    deal->used = d.used;
    deal->phases = d.phases;
  }
  __syncthreads();
}

// A barrier of `threads` threads; and one that tells whether any of them says so.
__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ bool named_any(int id, int threads, bool mine) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %3, 0;\n\t"
      "bar.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(threads), "r"(static_cast<uint32_t>(mine))
      : "memory");
  return r != 0;
}

// 32 bytes, in one instruction where they are aligned to their size.
__device__ __forceinline__ void store_32(void* dst, const uint32_t* w, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// Row `row` of a unit with one tile, whose list[0] pieces lie in the slots list[1 ..]; a warp.
template <int D>
__device__ __forceinline__ void join_row(const ChunkParams& p, const int* list, int row, int token0, int kvh) {
  constexpr int VEC = D / 32;
  const int lane = threadIdx.x % 32, parts = list[0];
  float m = -INFINITY, l = 0.f, acc[VEC] = {};
#pragma unroll 1
  for (int j = 0; j < parts; j += 32) {
    float2 ml = make_float2(-INFINITY, 0.f);
    if (j + lane < parts)
      ml = __ldcg(reinterpret_cast<const float2*>(p.part_ml) + static_cast<size_t>(list[1 + j + lane]) * p.slot_rows + row);
    const float mn = fmaxf(m, warp_max(ml.x)), ref = mn == -INFINITY ? 0.f : mn;
    const float weight = ex2(ml.x - ref), old = ex2(m - ref);
    l = l * old + warp_sum(ml.y * weight);
#pragma unroll
    for (int k = 0; k < VEC; ++k) acc[k] *= old;
    m = mn;
    const int here = min(32, parts - j);
#pragma unroll 4
    for (int i = 0; i < here; ++i) {
      const float wi = __shfl_sync(0xffffffffu, weight, i);
      const float* src = p.part_o + (static_cast<size_t>(list[1 + j + i]) * p.slot_rows + row) * D + lane * VEC;
      if constexpr (VEC == 4) {
        const float4 y = __ldcg(reinterpret_cast<const float4*>(src));
        acc[0] = fmaf(y.x, wi, acc[0]);
        acc[1] = fmaf(y.y, wi, acc[1]);
        acc[2] = fmaf(y.z, wi, acc[2]);
        acc[3] = fmaf(y.w, wi, acc[3]);
      } else {
        const float2 y = __ldcg(reinterpret_cast<const float2*>(src));
        acc[0] = fmaf(y.x, wi, acc[0]);
        acc[1] = fmaf(y.y, wi, acc[1]);
      }
    }
  }
  const bool any = m > -INFINITY;
  const float inv = any ? 1.f / l : 0.f;
  const int token = row / p.G, qh = kvh * p.G + row - token * p.G;
  uint16_t* dst = p.out + (token0 + token) * p.ld_out + qh * D + lane * VEC;
  if constexpr (VEC == 4)
    *reinterpret_cast<uint2*>(dst) = make_uint2(bf16x2(acc[0] * inv, acc[1] * inv), bf16x2(acc[2] * inv, acc[3] * inv));
  else
    *reinterpret_cast<uint32_t*>(dst) = bf16x2(acc[0] * inv, acc[1] * inv);
  if (p.lse != nullptr && lane == 0)
    p.lse[static_cast<int64_t>(token0 + token) * p.hq + qh] = any ? (m + log2f(l)) * 0.693147180559945309f : -INFINITY;
}

__device__ __forceinline__ void scale2(uint32_t* x, float f) {
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %2};\n\t"
      "mul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "+r"(x[0]), "+r"(x[1])
      : "r"(__float_as_uint(f)));
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_kernel(const __grid_constant__ CUtensorMap kv_map, const __grid_constant__ CUtensorMap q_map,
                 const __grid_constant__ ChunkParams p, int group0, int oob_group) {
  using C = Cfg<D>;
  constexpr int SLOTS = C::SLOTS;
  extern __shared__ __align__(1024) uint8_t sm[];
  uint8_t* ring = sm + 2 * C::Q_TILE;
  float* exch = reinterpret_cast<float*>(ring + SLOTS * C::PLANE);  // [2 tiles][2 halves][128 rows]
  uint64_t* full = reinterpret_cast<uint64_t*>(exch + 512);
  uint64_t* empty = full + SLOTS;
  uint64_t* clean = empty + SLOTS;          // the plane's V has been gone over
  uint64_t* s_full = clean + SLOTS;         // [2] S of a tile is complete (and the PV before it)
  uint64_t* p_full = s_full + 2;            // [2][2] P of a tile is in TMEM: of each 64 keys the first 32, the others
  uint64_t* q_full = p_full + 4;            // Q of the piece is in shared memory
  uint64_t* q_free = q_full + 1;            // its last S is complete
  uint64_t* o_full = q_free + 1;            // all of the piece's products are complete, bad is written
  uint64_t* piece_full = o_full + 1;        // [kPieces]
  uint64_t* piece_free = piece_full + kPieces;
  Piece* pieces = reinterpret_cast<Piece*>(piece_free + kPieces);  // [kPieces]
  Place* range = reinterpret_cast<Place*>(pieces + kPieces);       // [kChunkPhases][2]
  Deal* deal = reinterpret_cast<Deal*>(range + 2 * kChunkPhases);
  int* scratch = reinterpret_cast<int*>(deal + 1);                 // [kWarps]
  volatile int* bad = reinterpret_cast<volatile int*>(scratch + kWarps);  // [kPieces] first key with a V that is not finite
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(const_cast<int*>(bad) + kPieces);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  static_assert(512 * 4 + (3 * SLOTS + 9 + 2 * kPieces) * 8 + kPieces * sizeof(Piece) + 2 * kChunkPhases * sizeof(Place) +
                        sizeof(Deal) +
                        (kWarps + kPieces + 2) * 4 <= Cfg<D>::PLAN, "fits");

  // (one lane's word for it, so that the compiler knows roles and pieces to be the
  // warp's and keeps what depends on them in uniform registers)
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid / 32, 0), lane = tid % 32;
  if (tid == 0) {
#pragma unroll 1
    for (int s = 0; s < SLOTS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 2);
      mbar_init(&clean[s], 1);
    }
#pragma unroll 1
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s_full[t], 1);
      mbar_init(&p_full[2 * t], 8);
      mbar_init(&p_full[2 * t + 1], 8);
    }
#pragma unroll 1
    for (int t = 0; t < kPieces; ++t) {
      mbar_init(&piece_full[t], 1);
      mbar_init(&piece_free[t], 19);
    }
    mbar_init(q_full, 1);
    mbar_init(q_free, 1);
    mbar_init(o_full, 2);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&kv_map);
    tma_prefetch_desc(&q_map);
  }
  if (warp == 17) tmem_alloc(tmem_slot, 512);
  griddep_wait();
  const int worker = blockIdx.x;
  find_range(p, worker, gridDim.x, range, scratch, deal);  // ends with a barrier
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_launch_dependents();   // (this CTA has its TMEM)
  const uint32_t tmem = *tmem_slot;

  // The next piece, for a whole warp; false at the end.  A role that gives up on a
  // wait says so (give_up) and goes on through the pieces without working on them,
  // so that all warps meet at the same barriers and every piece is handed back.
  int taken = 0;
  bool ok = true;
  auto next_piece = [&](Piece* pc) {
    const int at = taken % kPieces;
    if (!__all_sync(0xffffffffu, mbar_wait_for(&piece_full[at], (taken / kPieces) & 1, nullptr, 4 * kWaitLimitNs)))
      return false;
    int w = lane < sizeof(Piece) / 4 ? reinterpret_cast<const int*>(pieces + at)[lane] : 0;
#pragma unroll
    for (int j = 0; j < sizeof(Piece) / 4; ++j) reinterpret_cast<int*>(pc)[j] = __shfl_sync(0xffffffffu, w, j);
    return pc->n >= 0;
  };
  auto give_up = [&](int site) {
    ok = false;
    *abort_flag = 1;
    if (lane == 0) raise_status(p.status, DFLASH_ERR_TIMEOUT, site);
  };
  auto piece_done = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(&piece_free[taken % kPieces]);
    ++taken;
  };
  // A plane's chunk in the order of their use: K0 V0 K1 V1 ..., one tile K0 K1 V0 K2 V1 ...
  auto is_key = [](bool split, int n, int k, int j) { return k < n && (split ? k + max(0, k - 1) : 2 * k) == j; };

  if (warp >= 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == 19) {
      // ------------------------------------------------ plan: the worker's range, piece by piece
      Place at = range[0], end = range[1];
      ChunkRequest q = deal->q;
      int loaded = at.r, count = 0, phase = 0;
      bool last = false, first_piece = true;
      while (!last) {
        Piece pc;
        pc.n = -1;
        while (true) {
          const bool same = at.r == end.r, there = same && at.h == end.h && at.i == end.i;
          if (at.r >= p.batch || at.r > end.r ||
              (same && (at.h > end.h || (at.h == end.h && (at.i > end.i || (there && at.c >= end.c)))))) {
            if (++phase < deal->phases) {   // the next range
              at = range[2 * phase];
              end = range[2 * phase + 1];
              loaded = -1;
              first_piece = true;
              continue;
            }
            last = true;
            break;
          }
          if (loaded != at.r) {
            q = request(p, at.r);
            loaded = at.r;
          }
          const Units u(q, p.tokens, p.causal);
          if (at.i >= u.tiles) {  // the request's next head, or the next request
            at.i = at.c = 0;
            at.x += u.total();
            if (u.tiles == 0 || ++at.h >= p.hkv) {
              at.h = 0;
              ++at.r;
            }
            continue;
          }
          const int all = u.chunks(at.i), c0 = at.c, c1 = there ? end.c : all;
          const int i = at.i++;
          at.c = 0;
          if (c0 >= c1 && all > 0) continue;
          const int first = u.ctx - u.n + i * u.per + 1;
          pc.n = c1 - c0;
          pc.c0 = c0;
          pc.keys = u.keys(i);
          pc.see = u.causal ? first : u.ctx;
          pc.step = u.causal;
          pc.r = at.r;
          pc.h = at.h;
          pc.token0 = q.start + i * u.per;
          pc.tokens = min(u.per, u.n - i * u.per);
          pc.split = u.split(i);
          pc.begins = c0 == 0;
          pc.ends = c1 == all;
          pc.x = at.x;
          pc.all = all;
          pc.range = worker + phase * deal->used;
          pc.first = first_piece;
          first_piece = false;
          break;
        }
        const int slot = count % kPieces;
        if (count >= kPieces && !__all_sync(0xffffffffu, mbar_wait_for(&piece_free[slot], (count / kPieces + 1) & 1,
                                                                       nullptr, 4 * kWaitLimitNs))) {
          give_up(558);
          break;
        }
        if (lane == 0) {
          pieces[slot] = pc;
          mbar_arrive(&piece_full[slot]);
        }
        __syncwarp();
        ++count;
      }
    } else if (warp == 16) {
      // ------------------------------------------------ TMA producer
      const uint64_t pol = l2_policy_evict_normal();
      int at = 0, segs = 0;                        // planes, pieces requested so far
      Cursor cur;
      Piece pc;
      while (next_piece(&pc)) {
        const int n = ok ? pc.n : 0, page0 = pc.c0 * 8;
        const int npg = min(n * 8, (pc.keys + 15) / 16 - page0);
        const int32_t* table = p.page_table + static_cast<size_t>(pc.r) * p.max_pages + page0;
        // lane -> 8-row group of its page's K plane in the map, 32 pages a time,
        // the next 32 requested ahead
        auto ids_of = [&](int b) {
          const int j = b * 32 + lane;
          return j < npg ? max(__ldcg(table + j), -1) : -2;  // -2: past the piece
        };
        auto check = [&](int id) {
          if (id >= 0 && id < p.n_pages) return group0 + (id * 2 * p.hkv + pc.h) * 2;
          if (id != -2) raise_status(p.status, DFLASH_ERR_CAPACITY, 553);
          return oob_group;
        };
        int kb = 0, vb = 0;  // 32-page batch held for K, for V
        int next_id = ids_of(1);
        int kg = check(ids_of(0)), vg = kg;
        int k = 0, v = 0;
#pragma unroll 1
        for (int j = 0; j < 2 * n; ++j, ++at, cur.advance(SLOTS)) {
          const bool is_k = is_key(pc.split, n, k, j);
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
          const int grp = is_k || vg == oob_group ? (is_k ? kg : vg) : vg + p.hkv * 2;
          int y[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(0xffffffffu, grp, (c % 4) * 8 + i);
          const int st = cur.slot;
          bool go = mbar_wait(&empty[st], cur.parity ^ 1, abort_flag);   // (the first SLOTS pass)
          if (j == 0 && segs > 0) go = go && mbar_wait(q_free, (segs - 1) & 1, abort_flag);
          if (!__all_sync(0xffffffffu, go)) {
            give_up(554);
            break;
          }
          // (eight lanes with a load each take turns, and longer: 1300 cycles a plane, not 700)
          if (elect_one()) {
            mbar_arrive_expect_tx(&full[st], C::PLANE);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              tma_load_4d(smem_u32(ring + st * C::PLANE + i * C::PAGE), &kv_map, y[i], &full[st], pol);
          }
          __syncwarp();
          if (j == 0) {  // Q of the piece: [tile][column half], `tokens` rows of G heads each
            if (lane == 0) {
              const int boxes = (pc.split ? 1 : 2) * C::HALVES;
              mbar_arrive_expect_tx(q_full, boxes * p.tokens * p.G * 128);
#pragma unroll 1
              for (int b = 0; b < boxes; ++b)
                tma_load_3d(sm + b * (128 * 128), &q_map, b % C::HALVES * 64, pc.h * p.G,
                            pc.token0 + b / C::HALVES * p.tokens, q_full, pol);
            }
            __syncwarp();
            ++segs;
          }
        }
        piece_done();
      }
      // copies still in flight after an abort land before the CTA exits
      if (lane == 0) {
#pragma unroll 1
        for (int j = max(0, at - SLOTS); j < at; ++j) mbar_wait(&full[j % SLOTS], (j / SLOTS) & 1, nullptr);
        if (segs > 0) mbar_wait(q_full, (segs - 1) & 1, nullptr);
      }
    } else if (warp == 17) {
      // ------------------------------------------------ products
      constexpr uint32_t idesc_s = umma_idesc_bf16(128, kChunk);
      constexpr uint32_t idesc_pv = umma_idesc_bf16(128, D) | (1u << 16);  // V MN-major
      constexpr uint32_t GS = C::HALVES * 1024;  // between 8-row groups of a plane
      const uint32_t q_addr = smem_u32(sm), ring_addr = smem_u32(ring);
      int segs = 0;
      int np = 0;          // parity of the next P of each tile (bits)
      Cursor cur;          // the next plane: they are used in the order they arrive
      Piece pc;
      auto commit = [&](uint64_t* bar) {
        if (elect_one()) umma_commit(bar);
        __syncwarp();
      };
      auto finish = [&]() {
        if (lane == 0) mbar_arrive(o_full);
        commit(o_full);
      };
      // waits for the next plane and takes it: its slot, or -1
      auto take = [&](bool cleaned) {
        const int st = cur.slot;
        bool r = mbar_wait(&full[st], cur.parity, abort_flag);
        if (cleaned) r = r && mbar_wait(&clean[st], cur.parity, abort_flag);
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
      // waits for the tile's P, part by part, and issues O += P V
      auto issue_pv = [&](int tile, int st, bool accumulate) {
        const uint32_t v = desc_lo(ring_addr + st * C::PLANE, 1024);
        const uint32_t o = tmem + C::O_COL + tile * 128, pa = tmem + C::S_COL + tile * 128;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          if (!__all_sync(0xffffffffu, mbar_wait(&p_full[2 * tile + g], (np >> tile) & 1, abort_flag))) return false;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int j = (i / 2) * 4 + 2 * g + i % 2;  // 16 keys
              umma_ts(o, pa + (j / 4) * 64 + (j % 4) * 8, desc_of(v + j * (C::PAGE / 16), desc_hi(GS)), idesc_pv,
                      g + i > 0 ? 1u : accumulate ? 1u : 0u);
            }
          }
          __syncwarp();
        }
        np ^= 1 << tile;
        return true;
      };
      while (next_piece(&pc)) {
        const int n = pc.n;
        if (n == 0 || !ok) {
          piece_done();
          continue;
        }
        // two tiles: S_A S_B | PV_A S_A' PV_B S_B' | ...; one tile takes turns over
        // the chunks: S_0 S_1 | PV_0 S_2 | PV_1 S_3 | ...
        ok = __all_sync(0xffffffffu, mbar_wait(q_full, segs++ & 1, abort_flag));
        const int lead = pc.split ? min(2, n) : 1;
        // chunks from here on have keys that not all rows see
        const int clean0 = max(0, pc.see) / kChunk - pc.c0;
        int ik = -1;
#pragma unroll 1
        for (int c = 0; ok && c < lead; ++c) {
          ik = take(false);
          ok = ik >= 0;
          if (!ok) break;
          tc_fence_after();
          issue_s(c, 0, ik);
          if (!pc.split) issue_s(1, 1, ik);
          commit(&empty[ik]);
          if (c + 1 == n) commit(q_free);
        }
#pragma unroll 1
        for (int c = 0; ok && c < n; ++c) {
          const int t = pc.split ? c & 1 : 0;
          const bool more = c + lead < n && (!pc.split || n > 1);
          // (the last one in any case: what the value warp found in the piece is then written
          // down before its last product, whose completion is what the softmax waits for)
          const int iv = take(c >= clean0 || c + 1 == n);
          ok = iv >= 0 && issue_pv(t, iv, pc.split ? c >= 2 : c > 0);
          if (!ok) break;
          if (pc.split) commit(&empty[iv]);
          if (more) {
            ik = take(false);
            ok = ik >= 0;
            if (!ok) break;
            issue_s(t, 0, ik);
          }
          if (!pc.split) {
            ok = issue_pv(1, iv, c > 0);
            if (!ok) break;
            commit(&empty[iv]);
            if (more) issue_s(1, 1, ik);
          }
          if (more) {
            commit(&empty[ik]);
            if (c + lead + 1 == n) commit(q_free);
          }
        }
        if (ok) finish();
        else give_up(555);
        piece_done();
      }
      if (!ok) {
        // the products in flight end before their memory is given back
        finish();
        mbar_wait(o_full, (segs - 1) & 1, nullptr);
      }
    } else {
      // ------------------------------------------------ V's values
      Cursor cur;
      Piece pc;
      while (next_piece(&pc)) {
        const int n = ok ? pc.n : 0;
        // keys from the piece's first one: all rows see those before `first`, none those from `live` on
        const int live = pc.keys - pc.c0 * kChunk;
        const int first = max(0, pc.see) - pc.c0 * kChunk;
        int found = INT_MAX, k = 0, v = 0;
#pragma unroll 1
        for (int j = 0; j < 2 * n; ++j) {
          const bool is_k = is_key(pc.split, n, k, j);
          const int c = is_k ? k++ : v++;
          const int st = cur.slot;
          if (!__all_sync(0xffffffffu, mbar_wait(&full[st], cur.parity, abort_flag))) {
            give_up(556);
            break;
          }
          cur.advance(SLOTS);
          if (!is_k && (c + 1) * kChunk > first) {
            const int b = clean_v<D>(ring + st * C::PLANE, first - c * kChunk, live - c * kChunk);
            if (b < kChunk) found = min(found, c * kChunk + b);
          }
          if (j == 2 * n - 1) {
            found = __reduce_min_sync(0xffffffffu, found);
            if (lane == 0) bad[taken % kPieces] = found;
          }
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&clean[st]);
            mbar_arrive(&empty[st]);
          }
        }
        piece_done();
      }
    }
  } else {
    // ------------------------------------------------ softmax: two threads per row, each
    // for 64 of a chunk's keys and half of O's columns
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int tile = warp / 8, half = warp / 4 % 2, quad = warp % 4;
    const int r128 = quad * 32 + lane;        // row of the tile, TMEM lane
    const int pair = 1 + tile * 4 + quad;     // barrier of the two halves' warps
    const int four = 9 + quad;                // and of both tiles'
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t s_addr = lane_base + C::S_COL + tile * 128 + half * 64;
    const uint32_t o_addr = lane_base + C::O_COL + tile * 128;
    float* mine = exch + (tile * 2 + half) * 128 + r128;
    const float* theirs = exch + (tile * 2 + 1 - half) * 128 + r128;
    const int inv_G = 65536 / p.G + 1;        // row / G for rows below 128
    const int tok = r128 * inv_G >> 16;       // of the tile
    int segs = 0, ns = 0;
    Piece pc;
    RangeRecord* records = reinterpret_cast<RangeRecord*>(p.records);
    if (tid < p.phases) records[worker + tid * kChunkWorkers] = RangeRecord{};
    __syncwarp();
    while (next_piece(&pc)) {
      const int n = pc.n;
      if (tid == 0) {
        RangeRecord* rec = records + pc.range;
        if (pc.first) {
          rec->cont = !pc.begins;
          rec->ends = !pc.begins && pc.ends;
        }
        if (pc.begins && !pc.ends) {
          rec->head = 1;
          rec->token0 = pc.token0;
          rec->tokens = pc.tokens;
          rec->kvh = pc.h;
        }
      }
      // keys this row sees, from the half's first of the piece
      const int my_token = (pc.split ? 0 : tile * p.tokens) + tok;
      const bool real = tok < p.tokens && my_token < pc.tokens;
      int lim = 1 << 30;   // rows that do not exist see whatever lies there
      if (real) lim = max(0, pc.see + my_token * pc.step) - pc.c0 * kChunk - half * 64;
      float m = -INFINITY, l = 0.f;
#pragma unroll 1
      for (int c = pc.split ? tile : 0; c < n; c += pc.split ? 2 : 1) {
        if (ok && !__all_sync(0xffffffffu, mbar_wait(&s_full[tile], ns++ & 1, abort_flag))) give_up(557);
        tc_fence_after();
        uint32_t x[2][32];
        tmem_ld32_nowait(s_addr, x[0]);
        tmem_ld32_nowait(s_addr + 32, x[1]);
        const int left = lim - c * kChunk;
        tmem_wait_ld(x[0]);
        tmem_regs_ready(x[1]);
        // keys past this row's count -inf
        if (__any_sync(0xffffffffu, left < 64)) {
#pragma unroll
          for (int j = 0; j < 64; ++j)
            if (j >= left) x[j / 32][j % 32] = 0xFF800000u;
        }
        float mx4[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          mx4[j] = fmaxf(__uint_as_float(x[j / 2][j % 2 * 16]), __uint_as_float(x[j / 2][j % 2 * 16 + 1]));
#pragma unroll
          for (int i = 2; i < 16; i += 2)
            mx4[j] = fmaxf(mx4[j], fmaxf(__uint_as_float(x[j / 2][j % 2 * 16 + i]),
                                         __uint_as_float(x[j / 2][j % 2 * 16 + i + 1])));
        }
        float mc = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * p.scale_log2;
        // the reference is raised, for both halves, where one exceeds it by more than kRaise
        if (named_any(pair, 64, mc > m + kRaise)) {
          *mine = mc;
          named_sync(pair, 64);
          mc = fmaxf(mc, *theirs);
          const bool raise = mc > m + kRaise, rescale = raise && m != -INFINITY;
          if (__any_sync(0xffffffffu, rescale)) {
            // S is complete, so the PV before it is too: O may be read
            const float alpha = rescale ? ex2(m - mc) : 1.f;
#pragma unroll 1
            for (int q = half * (D / 32); q < (half + 1) * (D / 32); ++q) {
              uint32_t o[16];
              tmem_ld16_raw(o_addr + q * 16, o);
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
              tmem_st16(o_addr + q * 16, o);
            }
            tmem_wait_st();
            l *= alpha;
          }
          if (raise) m = mc;
        }
        // P = exp2(scale S - m) in bf16 takes the place of S
        const float neg = m == -INFINITY ? 0.f : -m;
        const float2 sc2 = make_float2(p.scale_log2, p.scale_log2), neg2 = make_float2(neg, neg);
        float2 la = make_float2(0.f, 0.f), lb = la;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          uint32_t pk[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            float2 t = fma2(make_float2(__uint_as_float(x[g][2 * j]), __uint_as_float(x[g][2 * j + 1])), sc2, neg2);
            t.x = ex2(t.x);
            t.y = ex2(t.y);
            if (j & 1) lb = add2(lb, t);
            else la = add2(la, t);
            pk[j] = bf16x2(t.x, t.y);
          }
          tmem_st16(s_addr + g * 16, pk);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[2 * tile + g]);
        }
        l += (la.x + la.y) + (lb.x + lb.y);
      }
      bool spoilt = false;   // the row sees a V that is not finite: its result is NaN, its lse is not
      if (n > 0) {
        if (ok && !__all_sync(0xffffffffu, mbar_wait(o_full, segs & 1, abort_flag))) give_up(557);
        spoilt = lim + half * 64 > bad[taken % kPieces];
        ++segs;
        tc_fence_after();
      }
      // ---- result of the piece: the halves' l; one tile: the tiles' states too
      named_sync(pair, 64);
      *mine = l;
      named_sync(pair, 64);
      l = half == 0 ? l + *theirs : *theirs + l;
      const bool have = n > (pc.split ? tile : 0), have_b = pc.split && n > 1 - tile;
      float wa = have ? 1.f : 0.f, wb = 0.f;   // weights of this tile's O and the other's
      if (pc.split) {
        named_sync(four, 128);
        *mine = half == 0 ? m : l;
        named_sync(four, 128);
        const float om = exch[(1 - tile) * 256 + r128], ol = exch[(1 - tile) * 256 + 128 + r128];
        const float mn = fmaxf(m, om), ref = mn == -INFINITY ? 0.f : mn;
        wa = have ? ex2(m - ref) : 0.f;
        wb = have_b ? ex2(om - ref) : 0.f;
        const float a = l * wa, b = ol * wb;
        l = tile == 0 ? a + b : b + a;   // (the same order in both tiles' warps)
        m = mn;
      }
      const bool whole = pc.begins && pc.ends;
      const float inv = spoilt ? __int_as_float(0x7FFFFFFF) : whole ? (m == -INFINITY ? 0.f : 1.f / l) : 1.f;
      const float fa = wa * inv, fb = wb * inv;
      const int row0 = pc.split ? 0 : tile * 128;      // the tile's first in the unit
      const size_t slot_row = (2 * static_cast<size_t>(pc.range) + (pc.begins ? 1 : 0)) * p.slot_rows + row0 + r128;
      const int64_t out_row = (pc.token0 + my_token) * p.ld_out + (pc.h * p.G + r128 - tok * p.G) * D;
      // One tile: a quarter of the columns for each of the four warps of its rows.  16 columns
      // at a time, in few instructions: they are not in the instruction cache when a unit
      // ends, and 2.4 KB of them, 32 columns unrolled, took 3700 cycles the first time round
      // and 500 the second.  A thread writes its own row, 32 bytes an instruction (16
      // bytes, half a sector, were the limit of short units).
      const int cols = pc.split ? D / 4 : D / 2, col0 = pc.split ? (tile * 2 + half) * cols : half * cols;
#pragma unroll 1
      for (int cc = col0; cc < col0 + cols; cc += 16) {
        uint32_t o[16];
        if (have) {
          tmem_ld16_raw(o_addr + cc, o);
#pragma unroll
          for (int j = 0; j < 16; j += 2) scale2(o + j, fa);
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) o[j] = 0u;
        }
        if (have_b) {
          uint32_t y[16];
          tmem_ld16_raw(lane_base + C::O_COL + (1 - tile) * 128 + cc, y);
#pragma unroll
          for (int j = 0; j < 16; ++j)
            o[j] = __float_as_uint(fmaf(__uint_as_float(y[j]), fb, __uint_as_float(o[j])));
        }
        if (real && whole) {
          uint32_t w[8];
#pragma unroll
          for (int t = 0; t < 8; ++t) w[t] = bf16x2(__uint_as_float(o[2 * t]), __uint_as_float(o[2 * t + 1]));
          store_32(p.out + out_row + cc, w, p.wide);
        } else if (real) {
          store_32(p.part_o + slot_row * D + cc, o, true);
          store_32(p.part_o + slot_row * D + cc + 8, o + 8, true);
        }
        __syncwarp();
      }
      if (real && half == 0 && (!pc.split || tile == 0)) {
        if (!whole)
          *reinterpret_cast<float2*>(p.part_ml + slot_row * 2) = make_float2(m, l);
        else if (p.lse != nullptr)
          p.lse[static_cast<size_t>(pc.token0 + my_token) * p.hq + pc.h * p.G + r128 - tok * p.G] =
              m == -INFINITY ? -INFINITY : (m + log2f(l)) * 0.693147180559945309f;
      }
      // both tiles' O have been read before either's next product
      if (pc.split) named_sync(four, 128);
      tc_fence_before();
      if (p.fused && !whole) {
        // ---- the last of the unit's pieces joins them, a row to a warp
        __threadfence();
        named_sync(13, 512);
        if (tid == 0) {
          int* done = p.status + 64 + pc.r * p.hkv + pc.h;   // chunks that are done (left at 0)
          scratch[0] = atomicAdd(done, n) + n == pc.all;
          if (scratch[0]) *done = 0;
        }
        named_sync(13, 512);
        if (scratch[0]) {
          __threadfence();
          int* list = reinterpret_cast<int*>(exch);
          if (warp == 0) {
            // the workers in whose ranges it lies
            const Deal d = *deal;   // (one phase: keys are read once)
            const int end_x = pc.x + Units::unit_cost(pc.keys, true);
            int parts = 0;
#pragma unroll 1
            for (int w0 = 0; w0 < d.used; w0 += 32) {
              const int w = w0 + lane, x0 = d.start(w), x1 = d.start(w + 1);
              const int lo = x0 <= pc.x ? 0 : Units::cut(x0 - pc.x, pc.all, true);
              const int hi = w + 1 >= d.used || x1 >= end_x ? pc.all : Units::cut(x1 - pc.x, pc.all, true);
              const bool has = w < d.used && x0 < end_x && x1 > pc.x && lo < hi;
              const unsigned votes = __ballot_sync(0xffffffffu, has);
              if (has) list[1 + parts + __popc(votes & ((1u << lane) - 1))] = lo > 0 ? 2 * w : 2 * w + 1;
              parts += __popc(votes);
            }
            if (lane == 0) list[0] = parts;
          }
          named_sync(13, 512);
#pragma unroll 1
          for (int row = warp; row < pc.tokens * p.G; row += 16) join_row<D>(p, list, row, pc.token0, pc.h);
        }
        named_sync(13, 512);
      }
      piece_done();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 17) tmem_dealloc(tmem, 512);
}

// Joins the pieces of the units that were cut: a CTA takes 32 rows of the units that
// worker blockIdx.x began, a warp four of them, whose pieces are read together.
constexpr int kJoinRows = 32;
template <int D>
__global__ void __launch_bounds__(256) chunk_join_kernel(const __grid_constant__ ChunkParams p) {
  __shared__ int list[kChunkWorkers * kChunkPhases], count[8], last;
  griddep_wait();
  griddep_launch_dependents();
  const RangeRecord* recs = reinterpret_cast<const RangeRecord*>(p.records);
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int ranges = kChunkWorkers * p.phases, mine = blockIdx.x + lane * kChunkWorkers;
  unsigned heads = __ballot_sync(0xffffffffu, mine < ranges && recs[mine].head);  // of its ranges
#pragma unroll 1
  for (; heads != 0; heads &= heads - 1) {
    const int w = blockIdx.x + (__ffs(heads) - 1) * kChunkWorkers;
    const RangeRecord head = recs[w];
    if (tid == 0) {
      last = INT_MAX;
      list[0] = 2 * w + 1;
    }
    int parts = 1;
    // the ranges that continue the unit, in order, up to the one that ends it
#pragma unroll 1
    for (int base = w + 1; base < ranges; base += 256) {
      const int v = base + tid;
      bool cont = v < ranges && recs[v].cont;
      const bool ends = cont && recs[v].ends;
      __syncthreads();
      if (ends) atomicMin(&last, v);
      __syncthreads();
      cont = cont && v <= last;
      const unsigned votes = __ballot_sync(0xffffffffu, cont);
      if (lane == 0) count[warp] = __popc(votes);
      __syncthreads();
      for (int j = 0; j < 8; ++j) {
        if (j == warp && cont) list[parts + __popc(votes & ((1u << lane) - 1))] = 2 * v;
        parts += count[j];
      }
      if (last != INT_MAX) break;
    }
    __syncthreads();
    // a warp's four rows, eight lanes to each; a lane has 4 columns of every 32
    constexpr int COLS = D / 32;
    const int row = blockIdx.y * kJoinRows + warp * 4 + lane / 8, rt = row % 128, t = rt / p.G;
    const int token = row / 128 * p.tokens + t;
    if (row < p.slot_rows && t < p.tokens && token < head.tokens) {
      float m = -INFINITY, l = 0.f, acc[COLS][4] = {};
#pragma unroll 2
      for (int part = 0; part < parts; ++part) {
        const size_t at = static_cast<size_t>(list[part]) * p.slot_rows + row;
        const float2 y = __ldcg(reinterpret_cast<const float2*>(p.part_ml) + at);
        float4 v[COLS];
#pragma unroll
        for (int i = 0; i < COLS; ++i) v[i] = __ldcg(reinterpret_cast<const float4*>(p.part_o + at * D) + i * 8 + lane % 8);
        const float mn = fmaxf(m, y.x), ref = mn == -INFINITY ? 0.f : mn, a = ex2(m - ref), b = ex2(y.x - ref);
        l = l * a + y.y * b;
#pragma unroll
        for (int i = 0; i < COLS; ++i) {
          acc[i][0] = fmaf(v[i].x, b, acc[i][0] * a);
          acc[i][1] = fmaf(v[i].y, b, acc[i][1] * a);
          acc[i][2] = fmaf(v[i].z, b, acc[i][2] * a);
          acc[i][3] = fmaf(v[i].w, b, acc[i][3] * a);
        }
        m = mn;
      }
      const bool any = m > -INFINITY;
      const float inv = any ? 1.f / l : 0.f;
      const int qh = head.kvh * p.G + rt - t * p.G;
      uint16_t* dst = p.out + static_cast<int64_t>(head.token0 + token) * p.ld_out + qh * D + lane % 8 * 4;
#pragma unroll
      for (int i = 0; i < COLS; ++i)
        *reinterpret_cast<uint2*>(dst + i * 32) =
            make_uint2(bf16x2(acc[i][0] * inv, acc[i][1] * inv), bf16x2(acc[i][2] * inv, acc[i][3] * inv));
      if (p.lse != nullptr && lane % 8 == 0)
        p.lse[static_cast<int64_t>(head.token0 + token) * p.hq + qh] =
            any ? (m + log2f(l)) * 0.693147180559945309f : -INFINITY;
    }
    __syncthreads();
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
    if (e == cudaSuccess && a.numRegs * kThreads < 512 * kSoftmaxRegs + 128 * kOtherRegs)
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
  // no unit of fewer than 2 * kLeast chunks is cut
  if (e != cudaSuccess || p.fused || p.max_pages * 16ll <= (2 * kLeast - 1) * kChunk) return e;
  cfg.gridDim = dim3(kChunkWorkers, (p.slot_rows + kJoinRows - 1) / kJoinRows);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  count_launch();
  return cudaLaunchKernelEx(&cfg, chunk_join_kernel<D>, p);
}

}  // namespace

bool attention_chunk_fits(const ChunkParams& p) {
  const double units = p.T / (2 * p.tokens) + static_cast<double>(p.batch);
  return units * p.hkv * (kUnitCost + p.max_pages * 0.5 + 1) < 1073741824.0;
}

cudaError_t attention_chunk_launch(const ChunkParams& p, int d, const CUtensorMap& kv_map,
                                   const CUtensorMap& q_map, int group0, int oob_group, cudaStream_t s) {
  return d == 128 ? launch<128>(p, kv_map, q_map, group0, oob_group, s)
                  : launch<64>(p, kv_map, q_map, group0, oob_group, s);
}

}  // namespace dflash
