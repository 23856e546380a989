// Draws under per-row temperature, top-k, top-p and min-p.
//
//   w_i = exp((z_i - m) / T), m = max z; tokens ordered by (z desc, index asc)
//   K = first top_k, P = shortest prefix of K with mass >= top_p mass(K),
//   M = {(z - m)/T >= ln min_p}; all three are prefixes of that order, so the
//   kept set is {z > v} plus the tokens with z = v up to an index.  The token
//   is the smallest index with a * S < C over the kept weights in index order.
//
// A few rows, or rows that fit: one thread-block cluster per row, each CTA with
// its slice of the logits in shared memory, so the row is read from memory once
// however many passes follow.  Many long rows: one CTA per row, which reads the
// row again in every pass (the rows in flight fit L2); that saves the cluster's
// barriers, which cost a row as much as its arithmetic (both sides' times are at
// the rule, in sample_filtered_launch).
//
// Weights.  2^-t with t = (m - z) log2(e) / T is evaluated as an integer with
// 45 fractional bits: t as an unevaluated float pair, t = j/16 + r with a table
// of 2^(-j/16) (P. T. P. Tang's table-driven scheme) and the Taylor series of
// exp(-r ln 2), all as float pairs; relative error 2^-35 per weight and without
// bias, so a row's sum is good to about 1e-12.  Sixteen entries, because a
// warp's lanes then read them without bank conflicts; with 64, and a series
// shorter by a term, the loads took as long as the arithmetic.
// fp64 would do, but its rate here is a sixty-fourth of fp32's.  Integer sums
// are exact: results do not depend on how the row is split or in which order
// atomics arrive.
//
// Selection without a sort.  Over 1023 equal steps of t in [0, 46) the tokens
// are counted, and their distances from the step's middle summed (two shared-
// memory atomics per logit): to first order that is the step's mass, so every
// prefix's mass is known within 2e-4, which leaves one or two steps that can hold
// the border of top-p (one for top-k).  (From the counts alone it would be 3 %:
// on flat logits a quarter of all tokens.)  Those steps' tokens, the candidates,
// go to a list if they are few, where each counts what precedes it; otherwise
// they are first split by their exact 32-bit key, eight bits a pass, with the
// exact masses.  A border that falls on many equal logits is settled by
// counting them in index order.
// And where the steps up to top-k's border hold no more tokens than the list,
// one CTA settles the whole row from a list of those.
//
// Bound: 512 rows of 151936 under top-p take 428 us, 0.7 TB/s.  A row's 95 us on
// its SM are 8 for the maximum, 19 for the counts, 47 for the weights and 20 for
// the border and the draw.  The weights are bound by instruction issue (about 75
// each, at nearly one a cycle); the rest is not: the one CTA of 1024 threads on an
// SM has nothing to run under its barriers and loads, so that over the kernel 52 %
// of the issue slots are used, and 512 rows on 152 SMs are 3.4 rounds run as four.
// Cheaper weights (fp32's 2^-22) would halve the 47 but move borders that 64-bit
// arithmetic puts elsewhere.  Under top-k 50, settled from the list, they take 197
// us (214 with top-p), under top-k 1000 364 (403).  For a few
// rows the latency of the passes, each ending in a cluster barrier: one row of
// 151936 takes 31 us under top-p alone, about ten passes, and 17 under top-k 50
// and top-p, five passes and a list (26 without the list); 32 rows with mixed
// settings 48 us.
#include <cfloat>
#include <climits>
#include <cmath>

#include "common.cuh"
#include "kernels.h"

namespace dflash {

namespace {

typedef unsigned long long u64;

constexpr int kBins = 1024;          // the last is the tail (t >= 46)
constexpr int kList = 256;           // candidates settled in the list
constexpr int kMaxWarps = 32;
constexpr int kKeyBins = 256;        // of a pass over the candidates' keys
constexpr float kMaxLog2 = 46.f;     // weights below 2^-46 count as 0
constexpr int kMaxCluster = 8;
static_assert(kMaxSampleVocab / kMaxCluster * 4 + 28672 <= 227 * 1024, "a slice fits shared memory");

struct Shared {
  float tab[32];                     // 2^(-j/16) as float pairs: high parts, then low parts
  u64 list[2 * kList];               // candidates: orders, weights
  unsigned hist[kBins];              // counts by step
  unsigned dist[kBins];              // sums of (distance + 1/2) * 2^13: 32 bits hold a whole row's
  unsigned keys[5][kKeyBins];        // counts; masses in limbs
  u64 xch[2][kMaxCluster][2];        // exchanged values, one row per rank of the cluster
  unsigned xch32[2][kMaxCluster][2];
  u64 wred[kMaxWarps][2];
  u64 wscan[kMaxWarps];
  u64 wadd[kMaxWarps];               // kept candidates' mass, by the warp that owns their index
  unsigned wred32[kMaxWarps][2];
  float f0[kMaxWarps], f1[kMaxWarps];
  float tot0, tot1;
  float ch, cl, scale;               // log2(e)/T as a float pair; bins per unit of z
  double inv_T, min_p_z, ln_S;       // 1/T; T ln min_p; ln of the kept mass
  unsigned key_m;                    // smallest key that min_p keeps
  int b_lo, b_hi;
  int found;
  unsigned found_n;
  u64 before;
  unsigned list_n;                   // rank 0: candidates listed
  unsigned cand_n;                   // candidates kept aside
  unsigned above_n;                  // tokens of K above them
  unsigned border_key;               // the list's answer
  int border_index;
};

// 2^(-j/16) for the kernel, made on the host
struct WeightTable {
  float e[32];
};

struct Weights {
  const float* tab;
  float m, ch, cl, scale;
  unsigned unit;                     // bits of 2^23 (2^22: 44 fractional bits)
};

// increasing integer key of a float (no NaN); -0 and +0 share one
__device__ __forceinline__ unsigned key_of(float z) {
  const unsigned u = __float_as_uint(z + 0.f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float of_key(unsigned k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
}

// Roundings to an integer are made by adding 1.5 * 2^23 (for magnitudes below
// 2^22): the conversion instructions run at an eighth of the rate of an add and
// set the pace otherwise.
constexpr float kMagic = 12582912.f;
__device__ __forceinline__ int magic_int(float x_plus_magic) {
  return __float_as_int(x_plus_magic) - 0x4B400000;
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

constexpr float kLastStep = kMagic + (kBins - 2);
// The step of t nearest to the logit's, non-decreasing as z falls.
__device__ __forceinline__ int bin_of(const Weights& w, float z) {
  const float k = fmaf(w.m - z, w.scale, kMagic);  // one rounding: every pass has the same steps
  return k <= kLastStep ? magic_int(k) : kBins - 1;
}

// Two fp32 operations in one instruction.
struct F2 {
  u64 v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ F2 f2(float a) { return f2(a, a); }
__device__ __forceinline__ void un2(F2 x, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x.v)); }
__device__ __forceinline__ F2 add(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 mul(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

// A weight in two parts, hi 2^-23 + lo 2^-45, as the bits of floats whose last
// place is one unit: sums of a few hundred may be taken of the bits, modulo 2^32
// (hi <= 2^23, |lo| <= 2^21).
constexpr unsigned kHiBits = 0x4B000000u, kLoBits = 0x4B400000u;  // of hi = 0, lo = 0
struct Parts {
  unsigned hi, lo;
  // n: number of weights summed
  __device__ __forceinline__ u64 sum(unsigned n) const {
    return (static_cast<u64>(hi - n * kHiBits) << 22) + static_cast<u64>(static_cast<long long>(static_cast<int>(lo - n * kLoBits)));
  }
};

// The weights of two logits z <= m that are not in the tail; without `take`, a
// weight of 0.  All that is written as a product stays one (none is only added
// to), so that every place this is compiled into gives the same bits.
__device__ __forceinline__ void weight_parts(const Weights& w, float z0, float z1, bool take0, bool take1, Parts* p0, Parts* p1) {
  const F2 neg = f2(-1.f), magic = f2(kMagic);
  const F2 z = f2(take0 ? z0 : w.m, take1 ? z1 : w.m);
  // z - m = d + dl exactly
  const F2 d = add(z, f2(-w.m));
  const F2 b = add(d, f2(w.m));
  const F2 dl = add(fma(b, neg, z), fma(fma(b, neg, d), neg, f2(-w.m)));
  // -t = t - e
  const F2 t = mul(d, f2(w.ch));
  F2 e = fma(d, f2(-w.ch), t);
  e = fma(d, f2(-w.cl), e);
  e = fma(dl, f2(-w.ch), e);
  // k = 16 n + j nearest to 16 t; r = k / 16 - t
  const F2 kx = fma(t, f2(-16.f), magic);
  const F2 r = fma(add(kx, f2(-kMagic)), f2(1.f / 16.f), t);
  float k[2];
  un2(kx, k[0], k[1]);
  float th_[2], tl_[2], sc_[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const unsigned kb = __float_as_uint(k[i]);
    th_[i] = w.tab[kb & 15];
    tl_[i] = w.tab[16 + (kb & 15)];
    // 2^(23 - n), or 0 (of the bits that make kMagic, the shifts leave nothing)
    sc_[i] = __uint_as_float((i == 0 ? take0 : take1) ? w.unit - ((kb >> 4) << 23) : 0u);
  }
  const F2 th = f2(th_[0], th_[1]), tl = f2(tl_[0], tl_[1]), sc = f2(sc_[0], sc_[1]);
  // u = (r - e) ln 2 = uh - ul
  constexpr double LN2 = 0.693147180559945309;
  constexpr float LH = static_cast<float>(LN2), LL = static_cast<float>(LN2 - static_cast<double>(LH));
  const F2 uh = mul(r, f2(LH));
  F2 ul = fma(r, f2(-LH), uh);
  ul = fma(r, f2(-LL), ul);
  ul = fma(e, f2(LH), ul);
  // exp(u) - 1 = uh - tail = v + vl
  const F2 sq = mul(uh, uh);
  const F2 q = fma(uh, fma(uh, fma(uh, f2(-1.f / 120.f), f2(-1.f / 24.f)), f2(-1.f / 6.f)), f2(-0.5f));
  const F2 tail = fma(sq, q, fma(fma(sq, f2(0.5f), uh), ul, ul));
  const F2 v = fma(tail, neg, uh);
  const F2 vl = fma(tail, neg, fma(v, neg, uh));
  // (th + tl) exp(u) = s + sl
  const F2 s = fma(th, v, th);
  F2 sl = fma(th, v, fma(s, neg, th));
  sl = fma(tl, v, sl);
  sl = add(fma(th, vl, sl), tl);
  // in units of 2^-23, and what is left in units of 2^-45
  const F2 top = f2(8388608.f);
  const F2 hi = fma(s, sc, top);
  const F2 lo = fma(fma(sl, sc, fma(s, sc, fma(hi, neg, top))), f2(0x1p22f), magic);
  float x0, x1;
  un2(hi, x0, x1);
  p0->hi = __float_as_uint(x0);
  p1->hi = __float_as_uint(x1);
  un2(lo, x0, x1);
  p0->lo = __float_as_uint(x0);
  p1->lo = __float_as_uint(x1);
}
__device__ __forceinline__ u64 weight_of(const Weights& w, float z) {
  Parts p, q;
  weight_parts(w, z, z, true, true, &p, &q);
  return p.sum(1);
}

__device__ __forceinline__ u64 shfl_xor64(u64 v, int o) { return __shfl_xor_sync(0xffffffffu, v, o); }

__device__ __forceinline__ void st_cluster_u64(const void* smem, uint32_t rank, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(dsmem_map(smem_u32(smem), rank)), "l"(v)
               : "memory");
}
__device__ __forceinline__ u64 ld_cluster_u64(const void* smem, uint32_t rank) {
  u64 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(dsmem_map(smem_u32(smem), rank)) : "memory");
  return v;
}
__device__ __forceinline__ unsigned ld_cluster_u32(const void* smem, uint32_t rank) {
  unsigned v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(dsmem_map(smem_u32(smem), rank)) : "memory");
  return v;
}

__device__ __forceinline__ void st_cluster_u32(const void* smem, uint32_t rank, unsigned v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(dsmem_map(smem_u32(smem), rank)), "r"(v) : "memory");
}
__device__ __forceinline__ unsigned add_cluster_u32(const void* smem, uint32_t rank, unsigned v) {
  unsigned r;
  asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(r) : "r"(dsmem_map(smem_u32(smem), rank)), "r"(v) : "memory");
  return r;
}

// (key, index) as one number that orders tokens: larger key first, then lower
// index.
__device__ __forceinline__ u64 order_of(unsigned key, int i) {
  return (static_cast<u64>(~key) << 32) | static_cast<unsigned>(i);
}

struct Border {
  unsigned key;
  int index;  // tokens with this key are in up to this index
};

// The row's work, shared by all threads of the cluster.  HELD: the slice is in
// shared memory; otherwise (one CTA per row) it is read from the logits.
template <int kThreads, bool HELD>
struct Row {
  [[maybe_unused]] static constexpr int kWarps = kThreads / 32;
  [[maybe_unused]] static constexpr int BPT = kBins / kThreads;  // steps of t per thread
  [[maybe_unused]] static constexpr unsigned kCand = HELD ? 512 : 4096;  // candidates a CTA keeps aside
  // A weight (46 bits) is summed per key in limbs of 16 bits when the CTA has a
  // slice, of fewer than 2^16 logits, and of 12 bits when it has the row: 32
  // bits hold a limb's sum.
  [[maybe_unused]] static constexpr int kLimbs = HELD ? 3 : 4, kLimbBits = HELD ? 16 : 12;
  Shared* sh;
  u64 *cand_order, *cand_w;  // [kCand]
  const float* vals;   // this CTA's slice (HELD: padded with -inf to kWarps * cs)
  int n_loc;           // its logits
  bool vec;            // its address is 16-byte aligned
  int cs;              // logits per warp (a multiple of 128)
  int base;            // index of the slice's first logit
  int nc, rank;        // CTAs of the cluster, this one's rank
  int par;             // exchange buffer
  Weights w;

  __device__ void barrier() const {
    if (HELD && nc > 1) cluster_sync();
    else __syncthreads();
  }

  // Four logits from slice offset o on.
  __device__ __forceinline__ float4 four(int o) const {
    if constexpr (HELD) return *reinterpret_cast<const float4*>(vals + o);
    float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    if (vec && o + 3 < n_loc) {
      v = __ldcg(reinterpret_cast<const float4*>(vals + o));
    } else {
      if (o < n_loc) v.x = __ldcg(vals + o);
      if (o + 1 < n_loc) v.y = __ldcg(vals + o + 1);
      if (o + 2 < n_loc) v.z = __ldcg(vals + o + 2);
      if (o + 3 < n_loc) v.w = __ldcg(vals + o + 3);
    }
    return v;
  }

  // Sums of two values and the least and largest of two keys, over the
  // cluster.  The CTAs' own sums stay in sh->xch[buffer][rank], the warps' in
  // sh->wred; the buffer alternates, and the barrier of the reduction in
  // between separates its uses.
  __device__ void reduce(u64& s0, u64& s1, unsigned& lo, unsigned& hi) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s0 += shfl_xor64(s0, o);
      s1 += shfl_xor64(s1, o);
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) {
      sh->wred[warp][0] = s0;
      sh->wred[warp][1] = s1;
      sh->wred32[warp][0] = lo;
      sh->wred32[warp][1] = hi;
    }
    __syncthreads();
    if (warp == 0) {
      const bool in = lane < kWarps;
      s0 = in ? sh->wred[lane][0] : 0;
      s1 = in ? sh->wred[lane][1] : 0;
      lo = in ? sh->wred32[lane][0] : ~0u;
      hi = in ? sh->wred32[lane][1] : 0u;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        s0 += shfl_xor64(s0, o);
        s1 += shfl_xor64(s1, o);
      }
      lo = __reduce_min_sync(0xffffffffu, lo);
      hi = __reduce_max_sync(0xffffffffu, hi);
      if (lane < nc) {
        if (nc > 1) {
          st_cluster_u64(&sh->xch[par][rank][0], lane, s0);
          st_cluster_u64(&sh->xch[par][rank][1], lane, s1);
          st_cluster_u32(&sh->xch32[par][rank][0], lane, lo);
          st_cluster_u32(&sh->xch32[par][rank][1], lane, hi);
        } else {
          sh->xch[par][0][0] = s0;
          sh->xch[par][0][1] = s1;
          sh->xch32[par][0][0] = lo;
          sh->xch32[par][0][1] = hi;
        }
      }
    }
    barrier();
    s0 = s1 = 0;
    lo = ~0u;
    hi = 0;
    for (int r = 0; r < nc; ++r) {
      s0 += sh->xch[par][r][0];
      s1 += sh->xch[par][r][1];
      lo = min(lo, sh->xch32[par][r][0]);
      hi = max(hi, sh->xch32[par][r][1]);
    }
    par ^= 1;
  }

  // Calls f(four logits, index of the first) for this thread's logits; a warp's
  // 128 at a time, the next on their way.
  template <typename F>
  __device__ __forceinline__ void each4(F f) const {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int end = (warp + 1) * cs;
    int o = warp * cs + lane * 4;
    if constexpr (HELD) {
      for (; o < end; o += 128) f(four(o), base + o);
    } else {
      for (; o + 3 * 128 < end; o += 4 * 128) {
        const float4 v0 = four(o), v1 = four(o + 128), v2 = four(o + 256), v3 = four(o + 384);
        f(v0, base + o);
        f(v1, base + o + 128);
        f(v2, base + o + 256);
        f(v3, base + o + 384);
      }
      for (; o < end; o += 128) f(four(o), base + o);
    }
  }
  // Calls f(z, index) for each of them.
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    each4([&](const float4& v, int i) {
      f(v.x, i);
      f(v.y, i + 1);
      f(v.z, i + 2);
      f(v.w, i + 3);
    });
  }

  // Inclusive scan over the threads of the CTA.
  __device__ u64 scan(u64 v) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 x = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += x;
    }
    if (lane == 31) sh->wscan[warp] = v;
    __syncthreads();
    u64 x = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) x += i < warp ? sh->wscan[i] : 0;
    __syncthreads();
    return v + x;
  }
  __device__ void scan2f(float& a, float& b) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
      if (lane >= o) a += x, b += y;
    }
    if (lane == 31) sh->f0[warp] = a, sh->f1[warp] = b;
    __syncthreads();
    float x = 0.f, y = 0.f;
    for (int i = 0; i < warp; ++i) x += sh->f0[i], y += sh->f1[i];
    a += x;
    b += y;
    __syncthreads();
  }

  // Where, in index order, the running sum of value(z, index) reaches `need`
  // (1 <= need <= the total).  The caller has just reduced the threads' sums as
  // reduce()'s first value through buffer `buf`; returns true on one thread of
  // the cluster, with the index and its logit.
  template <typename F>
  __device__ bool locate(int buf, u64 need, F value, int* index, float* logit) {
    for (int r = 0; r < rank; ++r) {
      const u64 x = sh->xch[buf][r][0];
      if (need <= x) return false;   // an earlier CTA's
      need -= x;
    }
    if (need > sh->xch[buf][rank][0]) return false;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    for (int i = 0; i < warp; ++i) {
      const u64 x = sh->wred[i][0];
      if (need <= x) return false;
      need -= x;
    }
    if (need > sh->wred[warp][0]) return false;
    // this warp's: 128 logits at a time
    for (int o = warp * cs + lane * 4; o < (warp + 1) * cs; o += 128) {
      const float4 v = four(o);
      const float zs[4] = {v.x, v.y, v.z, v.w};
      u64 x[4], sum = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) sum += (x[j] = value(zs[j], base + o + j));
      u64 inc = sum;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const u64 y = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += y;
      }
      const u64 all = __shfl_sync(0xffffffffu, inc, 31);
      if (need <= all) {
        u64 c = inc - sum;
        if (!(c < need && need <= inc)) return false;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          c += x[j];
          if (need <= c) {
            *index = base + o + j;
            *logit = zs[j];
            return true;
          }
        }
        return false;
      }
      need -= all;
    }
    return false;
  }

  // Adds a token to the list in rank 0's shared memory.
  __device__ __forceinline__ void push(u64 order, u64 weight) {
    u64 *orders = sh->list, *weights = sh->list + kList;
    if (nc > 1) {
      const unsigned at = add_cluster_u32(&sh->list_n, 0, 1);
      if (at < kList) {
        st_cluster_u64(&orders[at], 0, order);
        st_cluster_u64(&weights[at], 0, weight);
      }
    } else {
      const unsigned at = atomicAdd(&sh->list_n, 1u);
      if (at < kList) {
        orders[at] = order;
        weights[at] = weight;
      }
    }
  }

  // Sums of two values over the threads of this CTA.
  __device__ void sum_cta(u64& s0, u64& s1) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s0 += shfl_xor64(s0, o);
      s1 += shfl_xor64(s1, o);
    }
    __syncthreads();
    if (lane == 0) {
      sh->wred[warp][0] = s0;
      sh->wred[warp][1] = s1;
    }
    __syncthreads();
    s0 = s1 = 0;
    for (int i = 0; i < kWarps; ++i) {
      s0 += sh->wred[i][0];
      s1 += sh->wred[i][1];
    }
  }

  // Of the admitted logits with this key, the index of the c-th in index
  // order (INT_MAX if there are no more than c).
  template <typename In>
  __device__ int border_index(unsigned key, u64 c, In in) {
    const float z = of_key(key);
    auto tie = [&](float x, int i) -> u64 { return x == z && in(x, i) ? 1 : 0; };
    u64 all = 0, none = 0;
    unsigned lo = 0, hi = 0;
    each([&](float x, int i) { all += tie(x, i); });
    const int buf = par;
    reduce(all, none, lo, hi);
    if (c >= all) {
      __syncthreads();
      return INT_MAX;
    }
    int idx;
    float dummy;
    unsigned cut = 0x7FFFFFFFu;
    if (locate(buf, c, tie, &idx, &dummy)) cut = static_cast<unsigned>(idx);
    __syncthreads();
    u64 z0 = 0, z1 = 0;
    unsigned top = 0;
    reduce(z0, z1, cut, top);
    return static_cast<int>(cut);
  }

  // The border of a prefix in (key descending, index ascending) order: the
  // token at which the running sum (of counts, or of masses) reaches `need`,
  // among n candidates; `above` is the sum before them.  The candidates are the
  // logits with keys in [lo, hi] that in(z, index) admits, or, `aside`, what the
  // CTAs hold in cand_order, cand_w (masses only).
  template <bool MASS, typename In>
  __device__ Border border(unsigned n, unsigned lo, unsigned hi, u64 need, u64 above, bool aside, In in) {
    const int tid = threadIdx.x;
    // f(order, weight) for this CTA's candidates with keys in [lo, hi]
    auto candidates = [&](auto f) {
      if (aside) {
        for (unsigned j = tid; j < sh->cand_n; j += kThreads) {
          const u64 o = cand_order[j];
          const unsigned key = ~static_cast<unsigned>(o >> 32);
          if (key >= lo && key <= hi) f(o, cand_w[j]);
        }
      } else {
        each([&](float z, int i) {
          const unsigned key = key_of(z);
          if (key < lo || key > hi || !in(z, i)) return;
          f(order_of(key, i), MASS ? weight_of(w, z) : 1ull);
        });
      }
    };
    while (n > kList && lo < hi) {
      const int shift = max(0, 32 - __clz(hi - lo) - 8);
      if (tid < kKeyBins)
        for (int j = 0; j <= kLimbs; ++j) sh->keys[j][tid] = 0;
      if (tid == 0) sh->found = -1;
      __syncthreads();
      candidates([&](u64 o, u64 x) {
        const unsigned b = (hi - ~static_cast<unsigned>(o >> 32)) >> shift;
        atomicAdd(&sh->keys[0][b], 1u);
        if (MASS) {
#pragma unroll
          for (int j = 0; j < kLimbs; ++j)
            atomicAdd(&sh->keys[1 + j][b], static_cast<unsigned>(x >> (j * kLimbBits)) & ((1u << kLimbBits) - 1));
        }
      });
      barrier();
      u64 v = 0;
      unsigned cn = 0;
      if (tid < kKeyBins) {
#pragma unroll
        for (int j = 0; j < (MASS ? 1 + kLimbs : 1); ++j) {
          u64 x = 0;
          for (int r = 0; r < nc; ++r) x += nc > 1 ? ld_cluster_u32(&sh->keys[j][tid], r) : sh->keys[j][tid];
          if (j == 0) cn = static_cast<unsigned>(x);
          else v += x << (kLimbBits * (j - 1));
        }
        if (!MASS) v = cn;
      }
      const u64 inc = above + scan(v);
      if (v > 0 && need <= inc && inc - v < need) {
        sh->found = tid;
        sh->found_n = cn;
        sh->before = inc - v;
      }
      barrier();  // also: the bins may be cleared again
      const int b = sh->found;
      const u64 before = sh->before;
      const unsigned bn = sh->found_n;
      __syncthreads();
      if (b < 0) return Border{lo, INT_MAX};  // the sums end below `need`: all candidates
      above = before;
      n = bn;
      hi -= static_cast<unsigned>(b) << shift;
      const unsigned span = (1u << shift) - 1;
      lo = hi - lo > span ? hi - span : lo;
    }
    if (n > kList) {  // one key
      const u64 wk = MASS ? max(weight_of(w, of_key(lo)), 1ull) : 1;
      return Border{lo, border_index(lo, need > above ? (need - above + wk - 1) / wk : 1, in)};
    }
    // ---- the list, in rank 0's shared memory
    u64* orders = sh->list;
    u64* weights = sh->list + kList;
    candidates([&](u64 o, u64 x) { push(o, x); });
    barrier();
    if (rank == 0) {
      // TPC threads per candidate, each summing a part of what precedes it
      constexpr int TPC = kThreads / kList;
      const unsigned cnt = min(sh->list_n, static_cast<unsigned>(kList));
      const int c = tid / TPC;
      const bool on = c < static_cast<int>(cnt);
      const u64 mine = on ? orders[c] : 0, wm = on ? weights[c] : 0;
      u64 before = 0, all = 0;
      for (unsigned j = tid % TPC; j < cnt; j += TPC) {
        const u64 x = weights[j];
        all += x;
        before += orders[j] < mine ? x : 0;
      }
#pragma unroll
      for (int o = TPC / 2; o > 0; o >>= 1) {
        before += shfl_xor64(before, o);
        all += shfl_xor64(all, o);
      }
      // the first to reach `need`, or the last of all
      if (on && tid % TPC == 0 && above + before < need && (above + before + wm >= need || before + wm == all)) {
        const unsigned bk = ~static_cast<unsigned>(mine >> 32), bi = static_cast<unsigned>(mine);
        for (int r = 0; r < nc; ++r) {
          if (nc > 1) {
            st_cluster_u32(&sh->border_key, r, bk);
            st_cluster_u32(&sh->border_index, r, bi);
          } else {
            sh->border_key = bk;
            sh->border_index = static_cast<int>(bi);
          }
        }
      }
      __syncthreads();
      if (tid == 0) sh->list_n = 0;  // for the next border
    }
    barrier();
    return Border{sh->border_key, sh->border_index};
  }
};

template <int kThreads, bool HELD>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads)
    sample_filtered_kernel(const __grid_constant__ SampleFilteredParams p,
                           const __grid_constant__ WeightTable table, int nc, int slice, int cs) {
  extern __shared__ __align__(16) uint8_t smem[];
  Shared* sh = reinterpret_cast<Shared*>(smem);
  u64* cand = reinterpret_cast<u64*>(smem + (sizeof(Shared) + 15) / 16 * 16);
  float* vals = reinterpret_cast<float*>(cand + 2 * Row<kThreads, HELD>::kCand);
  griddep_launch_dependents();
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int row = blockIdx.x / nc, rank = blockIdx.x % nc;
  const int V = p.vocab;

  Row<kThreads, HELD> R;
  constexpr int BPT = Row<kThreads, HELD>::BPT;
  R.sh = sh;
  R.cand_order = cand;
  R.cand_w = cand + R.kCand;
  R.cs = cs;
  R.base = rank * slice;
  R.nc = nc;
  R.rank = rank;
  R.par = 0;
  if (tid < 32) sh->tab[tid] = table.e[tid];
  if (tid == 0) sh->list_n = 0;
  if (tid < kMaxWarps) sh->wadd[tid] = 0;
  griddep_wait();

  // ---- settings (used after the first reduction)
  const float T = p.temperature[row];
  const float Tc = fminf(fmaxf(T, 1e-30f), 1e30f);  // (0 and bad values are dealt with below)
  const int k = p.top_k != nullptr ? p.top_k[row] : 0;
  const float tp = p.top_p != nullptr ? p.top_p[row] : 1.f;
  const float mp = p.min_p != nullptr ? p.min_p[row] : 0.f;
  const double a = p.a[row];

  // (fp64 is slow here: one thread, before the logits have arrived)
  if (tid == 32) {
    const double Td = Tc;
    if (mp > 0.f) sh->min_p_z = Td * log(fmin(static_cast<double>(mp), 1.0));
    sh->inv_T = 1.0 / Td;
  }

  // ---- the logits' maximum, and the slice to shared memory
  R.n_loc = max(0, min(slice, V - rank * slice));
  R.vals = p.logits + row * p.ld + static_cast<int64_t>(rank) * slice;
  R.vec = (reinterpret_cast<uintptr_t>(R.vals) & 15) == 0;
  float mx = -INFINITY;  // NaN as soon as one logit is
  Row<kThreads, false> src;
  src.vals = R.vals;
  src.n_loc = R.n_loc;
  src.vec = R.vec;
  src.cs = cs;
  src.base = 0;
  src.each4([&](const float4& v, int o) {
    if constexpr (HELD) *reinterpret_cast<float4*>(vals + o) = v;
    mx = max_nan(mx, max_nan(max_nan(v.x, v.y), max_nan(v.z, v.w)));
  });
  if constexpr (HELD) R.vals = vals;
  if (tid == kThreads - 1) {
    // log2(e)/T as a float pair: the quotient, then that of its remainder
    constexpr double L2E = 1.44269504088896340736;
    constexpr float LH = static_cast<float>(L2E), LL = static_cast<float>(L2E - static_cast<double>(LH));
    const float ch = LH / Tc;
    sh->ch = ch;
    sh->cl = (fmaf(-ch, Tc, LH) + LL) / Tc;
    sh->scale = ch * ((kBins - 1) / kMaxLog2);
  }
  R.barrier();  // every CTA of the cluster runs before its shared memory is written
  u64 nans = mx != mx ? 1 : 0, none = 0;
  unsigned least = 0, top = mx != mx ? 0 : key_of(mx);
  R.reduce(nans, none, least, top);
  const float m = of_key(top);

  if (!(T >= 0.f && T <= FLT_MAX) || tp != tp || mp != mp || !(a >= 0.0 && a < 1.0) || nans != 0 ||
      !(m >= -FLT_MAX && m <= FLT_MAX)) {
    if (rank == 0 && tid == 0) {
      p.token[row] = -1;
      if (p.n_kept != nullptr) p.n_kept[row] = 0;
      if (p.logprob != nullptr) p.logprob[row] = 0.f;
      raise_status(p.status, DFLASH_ERR_INVALID_ARG, 541);
    }
    return;  // the whole cluster
  }
  if (T == 0.f) {
    unsigned first = ~0u, none = 0;
    u64 z0 = 0, z1 = 0;
    R.each([&](float z, int i) {
      if (z == m) first = min(first, static_cast<unsigned>(i));
    });
    R.reduce(z0, z1, first, none);
    if (rank == 0 && tid == 0) {
      p.token[row] = static_cast<int32_t>(first);
      if (p.n_kept != nullptr) p.n_kept[row] = 1;
      if (p.logprob != nullptr) p.logprob[row] = 0.f;
    }
    return;
  }
  if (mp > 0.f) {
    if (tid == 0) {
      // the smallest float z with z - m >= T ln min_p, by its key: from the nearest
      // float in steps that double until it is between two of them, then by halves
      // (where m and T ln min_p cancel, the differences of up to 10^9 floats round to
      // the same double)
      const double lim = sh->min_p_z, md = m;
      auto ok = [&](unsigned key) { return static_cast<double>(of_key(key)) - md >= lim; };
      unsigned lo = key_of(-FLT_MAX), hi = top;  // (m itself passes)
      unsigned at = min(max(key_of(static_cast<float>(fmax(md + lim, -static_cast<double>(FLT_MAX)))), lo), hi);
      const bool down = ok(at);
      if (down) hi = at;
      else lo = at + 1;
      for (unsigned step = 1; lo < hi; step *= 2) {
        at = down ? hi - min(step, hi - lo) : lo + min(step - 1, hi - 1 - lo);
        const bool in = ok(at);
        if (in) hi = at;
        else lo = at + 1;
        if (in != down) break;
      }
      while (lo < hi) {
        at = lo + (hi - lo) / 2;
        if (ok(at)) hi = at;
        else lo = at + 1;
      }
      sh->key_m = lo;
    }
    __syncthreads();
  }
  R.w.tab = sh->tab;
  R.w.m = m;
  R.w.ch = sh->ch;
  R.w.cl = sh->cl;
  R.w.scale = sh->scale;
  // (sums of weights stay below 2^64: one bit less for the longest rows)
  const bool longest = V > (1 << 18);
  R.w.unit = __float_as_uint(longest ? 0x1p22f : 0x1p23f);

  // the kept set: keys above v, and key v up to index vi
  unsigned v = mp > 0.f ? sh->key_m : 0;
  int vi = INT_MAX;
  auto narrow = [&](const Border& b) {
    if (b.key > v || (b.key == v && b.index < vi)) {
      v = b.key;
      vi = b.index;
      return true;
    }
    return false;
  };
  const bool use_k = k > 0 && k < V;
  const bool use_p = tp < 1.f;
  // a top-p border that decides: the mass of what this thread keeps for sure,
  // and the bins that hold the rest
  u64 sure = 0;
  bool aside = true;
  int p_lo = kBins, p_hi = -1;
  if (use_k || use_p) {
    // ---- counts by t
    for (int j = tid; j < kBins; j += kThreads) sh->hist[j] = sh->dist[j] = 0;
    __syncthreads();
    auto count2 = [&](float z0, float z1) {
      // bin_of's steps, two at a time, and the distances
      const F2 dh = fma(f2(z0, z1), f2(-1.f), f2(m)), sc = f2(R.w.scale);
      const F2 k = fma(dh, sc, f2(kMagic));
      const F2 d = fma(fma(dh, sc, fma(k, f2(-1.f), f2(kMagic))), f2(8192.f), f2(kMagic + 4096.f));
      float k_[2], d_[2];
      un2(k, k_[0], k_[1]);
      un2(d, d_[0], d_[1]);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (!(k_[j] <= kLastStep)) continue;
        const int b = magic_int(k_[j]);
        atomicAdd(&sh->hist[b], 1u);
        if (use_p) atomicAdd(&sh->dist[b], static_cast<unsigned>(magic_int(d_[j])));
      }
    };
    R.each4([&](const float4& v4, int) {
      count2(v4.x, v4.y);
      count2(v4.z, v4.w);
    });
    R.barrier();
    unsigned cnt[BPT], cum[BPT];
    float dist[BPT];
#pragma unroll
    for (int j = 0; j < BPT; ++j) {
      cnt[j] = 0;
      dist[j] = 0.f;
    }
    if constexpr (BPT == 2) {
      for (int r = 0; r < nc; ++r) {
        const u64 c = nc > 1 ? ld_cluster_u64(&sh->hist[2 * tid], r) : *reinterpret_cast<const u64*>(&sh->hist[2 * tid]);
        const u64 d = nc > 1 ? ld_cluster_u64(&sh->dist[2 * tid], r) : *reinterpret_cast<const u64*>(&sh->dist[2 * tid]);
        cnt[0] += static_cast<unsigned>(c);
        cnt[1] += static_cast<unsigned>(c >> 32);
        dist[0] += static_cast<float>(static_cast<unsigned>(d));
        dist[1] += static_cast<float>(static_cast<unsigned>(d >> 32));
      }
    } else {
      cnt[0] = sh->hist[tid];
      dist[0] = static_cast<float>(sh->dist[tid]);
    }
    unsigned all = cnt[0];
    if constexpr (BPT == 2) all += cnt[1];
    cum[BPT - 1] = static_cast<unsigned>(R.scan(all));
    if constexpr (BPT == 2) cum[0] = cum[1] - cnt[1];
    if (tid == 0) sh->found = -1;
    __syncthreads();

    // ---- top-k
    Border bk = {0, INT_MAX};
    int k_bin = kBins - 1;  // bin of K's border (kBins - 1: in the tail, or none)
    if (use_k) {
      const unsigned ku = k;
#pragma unroll
      for (int j = 0; j < BPT; ++j)
        if (cnt[j] > 0 && cum[j] >= ku && cum[j] - cnt[j] < ku) {
          sh->found = BPT * tid + j;
          sh->found_n = cnt[j];
          sh->before = cum[j] - cnt[j];
        }
      __syncthreads();
      const int f = sh->found;
      const unsigned fn = sh->found_n;
      const u64 before = sh->before;
      __syncthreads();
      if (f >= 0) {
        k_bin = f;
        if (before + fn <= kList) {
          // K is among a few tokens: rank 0 settles the row from a list of them
          R.each([&](float z, int i) {
            if (bin_of(R.w, z) <= f) R.push(order_of(key_of(z), i), weight_of(R.w, z));
          });
          R.barrier();
          if (rank != 0) return;
          const u64* orders = sh->list;
          u64* weights = sh->list + kList;
          constexpr int TPC = kThreads / kList;  // threads per token, each summing a part
          const int c = tid / TPC, cnt = static_cast<int>(sh->list_n);
          const bool on = c < cnt, one = tid % TPC == 0;
          const u64 mine = on ? orders[c] : 0, wm = on ? weights[c] : 0;
          u64 mass = 0;  // of what precedes it
          unsigned pos = 0;
          for (int j = tid % TPC; j < cnt; j += TPC) {
            const bool less = orders[j] < mine;
            mass += less ? weights[j] : 0;
            pos += less;
          }
#pragma unroll
          for (int o = TPC / 2; o > 0; o >>= 1) {
            mass += shfl_xor64(mass, o);
            pos += __shfl_xor_sync(0xffffffffu, pos, o);
          }
          bool keep = on && pos < ku;
          u64 M = keep && one ? wm : 0, none = 0;
          R.sum_cta(M, none);
          if (use_p) {
            u64 need = static_cast<u64>(ceil(static_cast<double>(fmaxf(tp, 0.f)) * static_cast<double>(M)));
            keep = keep && mass < max(min(need, M), 1ull);
          }
          const unsigned key = ~static_cast<unsigned>(mine >> 32), idx = static_cast<unsigned>(mine);
          keep = keep && key >= v;
          u64 S = keep && one ? wm : 0, kept = keep && one ? 1 : 0;
          R.sum_cta(S, kept);  // (its barriers: all weights have been read)
          if (on && one && !keep) weights[c] = 0;
          if (tid == kThreads - 32 && p.logprob != nullptr)
            sh->ln_S = log(static_cast<double>(S) * (longest ? 0x1p-44 : 0x1p-45));
          __syncthreads();
          u64 sum = 0;  // of the kept up to it, in index order
          for (int j = tid % TPC; j < cnt; j += TPC) sum += static_cast<unsigned>(orders[j]) <= idx ? weights[j] : 0;
#pragma unroll
          for (int o = TPC / 2; o > 0; o >>= 1) sum += shfl_xor64(sum, o);
          const u64 need = min(static_cast<u64>(a * static_cast<double>(S)) + 1, S);
          if (keep && one && need <= sum && sum - wm < need) {
            p.token[row] = static_cast<int32_t>(idx);
            if (p.n_kept != nullptr) p.n_kept[row] = static_cast<int32_t>(kept);
            if (p.logprob != nullptr)
              p.logprob[row] =
                  static_cast<float>((static_cast<double>(of_key(key)) - static_cast<double>(m)) * sh->inv_T - sh->ln_S);
          }
          return;
        }
        unsigned lo = 0, hi = ~0u;
        if (fn > kList) {  // the keys of its tokens
          lo = ~0u;
          hi = 0;
          R.each([&](float z, int) {
            if (bin_of(R.w, z) != f) return;
            lo = min(lo, key_of(z));
            hi = max(hi, key_of(z));
          });
          u64 z0 = 0, z1 = 0;
          R.reduce(z0, z1, lo, hi);
        }
        bk = R.template border<false>(fn, lo, hi, ku, before, false, [&](float z, int) { return bin_of(R.w, z) == f; });
      }
    }
    auto in_k = [&](float z, int i) {
      const unsigned key = key_of(z);
      return key > bk.key || (key == bk.key && i <= bk.index);
    };
    narrow(bk);

    // ---- top-p
    if (use_p) {
      // bounds of every prefix's mass.  A step's mass relative to its middle is
      // sum exp(-c d), c = step ln 2, |d| <= 1/2: n - c sum d, and more by at most
      // n (c/2)^2 / 2 = 1.2e-4 n; the sum's quantisation and fp32 are far below.
      // K's last step, of which only a part counts, by its edges.
      constexpr float step = kMaxLog2 / (kBins - 1), c = step * 0.69314718f;
      float low[BPT], high[BPT], li = 0.f, hi_ = 0.f;
      unsigned part[BPT];
#pragma unroll
      for (int j = 0; j < BPT; ++j) {
        const int b = BPT * tid + j;
        const float mid = exp2f(-b * step);
        part[j] = b < k_bin ? cnt[j] : 0;
        low[j] = fmaf(-c, dist[j] * (1.f / 8192.f) - 0.5f * cnt[j], static_cast<float>(cnt[j])) * mid * (1.f - 3e-5f);
        high[j] = low[j] * (1.f + 2e-4f);
        if (b >= k_bin || part[j] == 0) low[j] = high[j] = 0.f;
        if (b == k_bin && b < kBins - 1) {
          part[j] = k - (cum[j] - cnt[j]);
          low[j] = part[j] * mid * (1.f - 0.5f * c);
          high[j] = part[j] * mid * (1.f + 0.51f * c);
        }
        li += low[j];
        hi_ += high[j];
      }
      R.scan2f(li, hi_);
      if (tid == kThreads - 1) {
        sh->tot0 = li;
        sh->tot1 = hi_;
        sh->b_lo = sh->b_hi = kBins - 2;
        sh->found_n = 0;
        sh->cand_n = 0;
      }
      __syncthreads();
      const float q = fmaxf(tp, 0.f);
#pragma unroll
      for (int j = BPT - 1; j >= 0; --j) {
        if (part[j] > 0 && hi_ * (1.f + 1e-5f) >= q * sh->tot0) atomicMin(&sh->b_lo, BPT * tid + j);
        if (part[j] > 0 && li >= q * sh->tot1 * (1.f + 1e-5f)) atomicMin(&sh->b_hi, BPT * tid + j);
        li -= low[j];
        hi_ -= high[j];
      }
      __syncthreads();
      p_lo = sh->b_lo;
      p_hi = sh->b_hi;
      // the candidates, by count, and the tokens above them
#pragma unroll
      for (int j = 0; j < BPT; ++j) {
        const int b = BPT * tid + j;
        if (b >= p_lo && b <= p_hi && part[j] > 0) atomicAdd(&sh->found_n, part[j]);
        if (b == p_lo) sh->above_n = cum[j] - cnt[j];
      }
      __syncthreads();
      const unsigned n_cand = sh->found_n;
      __syncthreads();
      // K's mass, and the mass above the steps in question; their tokens go aside
      // (the sums' parts fit 32 bits: a thread has at most 384 logits, or 256 of 45 bits)
      Parts sum = {0, 0}, above = {0, 0};
      unsigned pairs = 0, n_above = 0;
      unsigned lo = ~0u, hi = 0;
      bool overflow = false;
      // steps as bin_of's magic sums, two at a time
      const float f_lo = kMagic + p_lo, f_hi = kMagic + p_hi;
      const F2 neg = f2(-1.f, -1.f), m2 = f2(m, m), sc2 = f2(R.w.scale, R.w.scale), magic = f2(kMagic, kMagic);
      auto put_aside = [&](float z, int i, u64 x) {
        const unsigned key = key_of(z);
        lo = min(lo, key);
        hi = max(hi, key);
        const unsigned at = atomicAdd(&sh->cand_n, 1u);
        if (at < R.kCand) {
          R.cand_order[at] = order_of(key, i);
          R.cand_w[at] = x;
        } else {
          overflow = true;
        }
      };
      auto pair = [&](float z0, float z1, int i) {
        float f0, f1;
        un2(fma(fma(f2(z0, z1), neg, m2), sc2, magic), f0, f1);
        bool t0 = f0 <= kLastStep, t1 = f1 <= kLastStep;
        if (use_k) {
          t0 = t0 && in_k(z0, i);
          t1 = t1 && in_k(z1, i + 1);
        }
        if (!t0 && !t1) return;
        Parts x0, x1;
        weight_parts(R.w, z0, z1, t0, t1, &x0, &x1);
        sum.hi += x0.hi + x1.hi;
        sum.lo += x0.lo + x1.lo;
        ++pairs;
        if (f0 < f_lo) {
          above.hi += x0.hi;
          above.lo += x0.lo;
          ++n_above;
        }
        if (f1 < f_lo) {
          above.hi += x1.hi;
          above.lo += x1.lo;
          ++n_above;
        }
        // (rarely) a candidate
        const bool c0 = t0 && f0 >= f_lo && f0 <= f_hi, c1 = t1 && f1 >= f_lo && f1 <= f_hi;
        if (c0 || c1) {
          if (c0) put_aside(z0, i, x0.sum(1));
          if (c1) put_aside(z1, i + 1, x1.sum(1));
        }
      };
      R.each4([&](const float4& v4, int i) {
        pair(v4.x, v4.y, i);
        pair(v4.z, v4.w, i + 2);
      });
      u64 M = sum.sum(2 * pairs), A = above.sum(n_above);
      sure = A;
      R.reduce(M, A, lo, hi);
      if (n_cand > R.kCand) {  // some CTA may have had more than it can keep aside
        u64 spilt = overflow ? 1 : 0, zero = 0;
        unsigned none_lo = 0, none_hi = 0;
        R.reduce(spilt, zero, none_lo, none_hi);
        aside = spilt == 0;
      }
      u64 need = static_cast<u64>(ceil(static_cast<double>(q) * static_cast<double>(M)));
      if (need > M) need = M;
      if (need <= A) need = A + 1;
      if (!narrow(R.template border<true>(n_cand, lo, hi, need, A, aside, in_k))) p_lo = kBins;
    }
  }
  const bool by_p = p_lo < kBins;  // top-p's border is the kept set's

  // ---- the draw
  auto value = [&](float z, int i) -> u64 {
    const unsigned key = key_of(z);
    if (key < v || (key == v && i > vi) || bin_of(R.w, z) >= kBins - 1) return 0;
    return weight_of(R.w, z);
  };
  u64 mine = by_p ? sure : 0, kept = 0;
  if (by_p && aside) {
    // what lies above p_lo is in `sure` already, nothing below p_hi is kept, and
    // the rest is aside
    if (rank == 0 && tid == 0) kept = sh->above_n;
    for (unsigned j = tid; j < sh->cand_n; j += kThreads) {
      const u64 o = R.cand_order[j];
      const unsigned key = ~static_cast<unsigned>(o >> 32);
      const int i = static_cast<int>(static_cast<unsigned>(o));
      if (key > v || (key == v && i <= vi)) {
        ++kept;
        atomicAdd(&sh->wadd[(i - R.base) / cs], R.cand_w[j]);
      }
    }
    __syncthreads();
    if (lane == 0) mine += sh->wadd[warp];
  } else {
    R.each4([&](const float4& v4, int i) {
      const float zs[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
      for (int j = 0; j < 4; j += 2) {
        bool take[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const unsigned key = key_of(zs[j + t]);
          const bool in = zs[j + t] > -INFINITY && (key > v || (key == v && i + j + t <= vi));
          kept += in;
          const int b = bin_of(R.w, zs[j + t]);
          take[t] = in && b < kBins - 1 && (!by_p || b >= p_lo);
        }
        if (!take[0] && !take[1]) continue;
        Parts x0, x1;
        weight_parts(R.w, zs[j], zs[j + 1], take[0], take[1], &x0, &x1);
        mine += x0.sum(1) + x1.sum(1);
      }
    });
  }
  const int buf = R.par;
  u64 S = mine;
  unsigned none0 = 0, none1 = 0;
  R.reduce(S, kept, none0, none1);
  u64 need = static_cast<u64>(a * static_cast<double>(S)) + 1;
  if (need > S) need = S;
  int idx;
  float z;
  if (tid == kThreads - 32 && p.logprob != nullptr)
    sh->ln_S = log(static_cast<double>(S) * (longest ? 0x1p-44 : 0x1p-45));  // one token: exactly 0
  const bool here = R.locate(buf, need, value, &idx, &z);
  __syncthreads();
  if (here) {
    p.token[row] = idx;
    if (p.n_kept != nullptr) {
      if (k > 0 && kept > static_cast<u64>(k)) kept = k;  // K's border lies in the tail
      p.n_kept[row] = static_cast<int32_t>(kept);
    }
    if (p.logprob != nullptr)
      p.logprob[row] = static_cast<float>((static_cast<double>(z) - static_cast<double>(m)) * sh->inv_T - sh->ln_S);
  }
}

const WeightTable& weight_table() {
  static const WeightTable t = [] {
    WeightTable x;
    for (int j = 0; j < 16; ++j) {
      const double e = std::exp2(-j / 16.0);
      x.e[j] = static_cast<float>(e);
      x.e[16 + j] = static_cast<float>(e - static_cast<double>(x.e[j]));
    }
    return x;
  }();
  return t;
}

}  // namespace

template <int kThreads, bool HELD>
static cudaError_t launch_sample(const SampleFilteredParams& p, int nc, cudaStream_t s) {
  constexpr int kWarps = kThreads / 32;
  const int slice = ((p.vocab + nc - 1) / nc + 3) / 4 * 4;
  const int cs = (slice + kWarps * 128 - 1) / (kWarps * 128) * 128;
  const size_t smem = (sizeof(Shared) + 15) / 16 * 16 + 16 * Row<kThreads, HELD>::kCand +
                      (HELD ? static_cast<size_t>(kWarps) * cs * 4 : 0);
  static thread_local int allowed = -1;
  const cudaError_t e =
      allow_smem(reinterpret_cast<const void*>(sample_filtered_kernel<kThreads, HELD>), 227 * 1024, &allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = nc;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.rows) * nc);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  count_launch();
  return cudaLaunchKernelEx(&cfg, sample_filtered_kernel<kThreads, HELD>, p, weight_table(), nc, slice, cs);
}

cudaError_t sample_filtered_launch(const SampleFilteredParams& p, cudaStream_t s) {
  // CTAs per row: a slice of at most kSlice logits, so that two CTAs fit an SM;
  // more, down to kMinSlice logits, while the rows leave SMs without work (one row
  // of 32000: slices of 16000 21.6 us, of 8000 17.7, of 4000 no faster; nor are
  // clusters of 16: one row of 151936 26.7 us to 27.3 with 8, nine rows 35.9 to 29.2)
  constexpr int kSlice = 20480, kMinSlice = 4096, kSms = 152;
  int nc = 1;
  while (nc < kMaxCluster && ((p.vocab + nc - 1) / nc > kSlice ||
                              (2 * nc * p.rows <= 2 * kSms && p.vocab / (2 * nc) >= kMinSlice)))
    nc *= 2;
  // Clusters take time in proportion to the rows; whole-row CTAs, 152 at a time,
  // that of 85 rows per round.  Clusters / whole rows, top-p alone: 151936 tokens,
  // 48 rows 81 / 116 us, 80 rows 117 / 123, 96 rows 134 / 126, 170 rows 218 / 220,
  // 200 rows 253 / 223, 512 rows 614 / 434; 50000 tokens, 76 rows 50 / 50, 120 rows
  // 65 / 51.  Clusters of two stay ahead (32000 tokens, 600 rows: 130 / 140).
  const int rounds = (p.rows + kSms - 1) / kSms;
  if (nc > 2 && p.rows > 85 * rounds) return launch_sample<1024, false>(p, 1, s);
  return launch_sample<512, true>(p, nc, s);
}

}  // namespace dflash
