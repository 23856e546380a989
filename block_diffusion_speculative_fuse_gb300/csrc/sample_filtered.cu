// Draws under per-row temperature, top-k, top-p and min-p.
//
//   w_i = exp((z_i - m) / T), m = max z; tokens ordered by (z desc, index asc)
//   K = first top_k, P = shortest prefix of K with mass >= top_p mass(K),
//   M = {(z - m)/T >= ln min_p}; all three are prefixes of that order, so the
//   kept set is {z > v} plus the tokens with z = v up to an index.  The token
//   is the smallest index with a * S < C over the kept weights in index order.
//
// One thread-block cluster per row; each CTA keeps its slice of the logits in
// shared memory, so the row is read from HBM once however many passes follow.
//
// Weights.  2^-t with t = (m - z) log2(e) / T is evaluated as a 46-bit integer
// (45 fractional bits): t as an unevaluated float pair, t = j/64 + r with a
// table of 2^(-j/64) (P. T. P. Tang's table-driven scheme) and the Taylor
// series of exp(-r ln 2), the parts added in fixed point; relative error
// 2^-35 per weight and without bias, so a row's sum is good to about 1e-12.
// fp64 would do, but its rate here is a sixty-fourth of fp32's.  Integer sums
// are exact: results do not depend on how the row is split or in which order
// atomics arrive.
//
// Selection without a sort.  A histogram of counts over 1023 equal steps of t
// in [0, 46) (one shared-memory atomic per logit) bounds the mass of every
// prefix within 3 %, which leaves a few bins that can hold the border of top-p
// (one bin for top-k).  Only their tokens are then split by their exact
// 32-bit key, ten bits a pass, with the exact masses; a border that falls on
// equal logits is settled by counting them in index order.
#include <cfloat>
#include <climits>

#include "common.cuh"
#include "kernels.h"

namespace dflash {

namespace {

typedef unsigned long long u64;

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 1024;          // one per thread; the last is the tail (t >= 46)
constexpr float kMaxLog2 = 46.f;     // weights below 2^-46 count as 0
constexpr int kMaxCluster = 8;
constexpr int kMaxSlice = 49152;     // logits per CTA (192 KB)

struct Shared {
  float4 tab[64];                    // 2^(-j/64): float pair, then the integer 2^(45-j/64) in two words
  u64 mass[kBins];
  unsigned hist[kBins];
  u64 xch[2][kMaxCluster][4];        // exchanged values, one row per rank of the cluster
  u64 wred[kWarps][4];
  u64 blk[4];
  float f0[kWarps], f1[kWarps];
  float ch, cl, scale;               // log2(e)/T as a float pair; bins per unit of z
  unsigned key_m;                    // smallest key that min_p keeps
  int b_lo, b_hi;
  int found;
  u64 before;
};

struct Weights {
  const float4* tab;
  float m, ch, cl, scale;
  int extra;                         // 1: 44 fractional bits
};

// increasing integer key of a float (no NaN)
__device__ __forceinline__ unsigned key_of(float z) {
  const unsigned u = __float_as_uint(z);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float of_key(unsigned k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
}

__device__ __forceinline__ int bin_of(const Weights& w, float z) {
  const float x = (w.m - z) * w.scale;
  return x < static_cast<float>(kBins - 1) ? static_cast<int>(x) : kBins - 1;
}

// the weight of logit z <= m, not in the tail
__device__ __forceinline__ u64 weight_of(const Weights& w, float z) {
  // m - z = dh + dl exactly
  const float dh = w.m - z;
  const float bb = dh - w.m;
  const float dl = (w.m - (dh - bb)) + (-z - bb);
  const float t = dh * w.ch;
  float e = fmaf(dh, w.ch, -t);
  e = fmaf(dh, w.cl, e);
  e = fmaf(dl, w.ch, e);
  const float k64 = rintf(t * 64.f);
  const int k = static_cast<int>(k64);
  const float r = fmaf(k64, -1.f / 64.f, t);
  // u = -(r + e) ln 2 = -(uh + ul)
  constexpr float LH = 0.693147180559945309f;
  constexpr float LL = static_cast<float>(0.693147180559945309 - static_cast<double>(LH));
  float uh = r * LH;
  float ul = fmaf(r, LH, -uh);
  ul = fmaf(r, LL, ul);
  ul = fmaf(e, LH, ul);
  uh = -uh;
  ul = -ul;
  const float s = (uh * uh) * fmaf(uh, fmaf(uh, 1.f / 24.f, 1.f / 6.f), 0.5f);
  const float tail = s + fmaf(uh, ul, ul);  // exp(u) - 1 = uh + tail
  const float4 tj = w.tab[k & 63];
  const u64 fix = (static_cast<u64>(__float_as_uint(tj.w)) << 32) | __float_as_uint(tj.z);
  const float ph = tj.x * uh;
  float low = fmaf(tj.x, uh, -ph);
  low = fmaf(tj.y, uh, low);
  low = fmaf(tj.x, tail, low);
  const float a = rintf(ph * 0x1p30f);
  low += fmaf(a, -0x1p-30f, ph);
  const long long R = static_cast<long long>(fix) + (static_cast<long long>(static_cast<int>(a)) << 15) +
                      __float2int_rn(low * 0x1p45f);
  const int n = (k >> 6) + w.extra;
  return (static_cast<u64>(R) + ((1ull << n) >> 1)) >> n;
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

enum Op { kSum, kMax, kMin };
template <Op op>
__device__ __forceinline__ u64 combine(u64 a, u64 b) {
  return op == kSum ? a + b : op == kMax ? (a > b ? a : b) : (a < b ? a : b);
}

// The row's work, shared by all threads of the cluster.
struct Row {
  Shared* sh;
  const float* vals;   // this CTA's slice, padded with -inf to 32 * cs
  int cs;              // logits per warp (a multiple of 128)
  int base;            // index of the slice's first logit
  int nc, rank;        // CTAs of the cluster, this one's rank
  int par;             // exchange buffer
  Weights w;

  __device__ void barrier() const {
    if (nc > 1) cluster_sync();
    else __syncthreads();
  }

  // Reduces one value per thread over the cluster.  The CTAs' own values stay
  // in sh->xch[buffer][rank][slot]; the buffer alternates, and the barrier of
  // the exchange in between separates its uses.
  template <Op op0, Op op1>
  __device__ void reduce2(u64& v0, u64& v1) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      v0 = combine<op0>(v0, shfl_xor64(v0, o));
      v1 = combine<op1>(v1, shfl_xor64(v1, o));
    }
    if (lane == 0) {
      sh->wred[warp][0] = v0;
      sh->wred[warp][1] = v1;
    }
    __syncthreads();
    if (warp == 0) {
      v0 = sh->wred[lane][0];
      v1 = sh->wred[lane][1];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        v0 = combine<op0>(v0, shfl_xor64(v0, o));
        v1 = combine<op1>(v1, shfl_xor64(v1, o));
      }
      if (lane < nc) {
        if (nc > 1) {
          st_cluster_u64(&sh->xch[par][rank][0], lane, v0);
          st_cluster_u64(&sh->xch[par][rank][1], lane, v1);
        } else {
          sh->xch[par][0][0] = v0;
          sh->xch[par][0][1] = v1;
        }
      }
    }
    barrier();
    v0 = sh->xch[par][0][0];
    v1 = sh->xch[par][0][1];
    for (int r = 1; r < nc; ++r) {
      v0 = combine<op0>(v0, sh->xch[par][r][0]);
      v1 = combine<op1>(v1, sh->xch[par][r][1]);
    }
    par ^= 1;
  }

  // Calls f(z, index) for this thread's logits; a warp's 128 logits at a time.
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    for (int o = warp * cs + lane * 4; o < (warp + 1) * cs; o += 128) {
      const float4 v = *reinterpret_cast<const float4*>(vals + o);
      f(v.x, base + o);
      f(v.y, base + o + 1);
      f(v.z, base + o + 2);
      f(v.w, base + o + 3);
    }
  }

  // Inclusive scan over the threads of the CTA.
  __device__ u64 scan(u64 v) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 x = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += x;
    }
    if (lane == 31) sh->wred[warp][2] = v;
    __syncthreads();
    if (warp == 0) {
      u64 x = sh->wred[lane][2];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const u64 y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      sh->wred[lane][2] = x;
    }
    __syncthreads();
    if (warp > 0) v += sh->wred[warp - 1][2];
    __syncthreads();
    return v;
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
  // reduce2's first value through buffer `buf`; returns true on one thread of
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
      const float4 v = *reinterpret_cast<const float4*>(vals + o);
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

  // Border search by key.  The candidates are the logits with keys in [lo,
  // hi] that in(z, index) admits; `base_sum` is what lies above them.  Finds
  // the key at which the running sum (of counts, or of masses) in descending
  // key order reaches `need`; *sum_above = the sum strictly above that key.
  template <bool MASS, typename In>
  __device__ unsigned border_key(unsigned lo, unsigned hi, u64 need, u64 base_sum, In in,
                                 u64* sum_above) {
    while (lo < hi) {
      const int shift = max(0, 32 - __clz(hi - lo) - 10);
      sh->mass[threadIdx.x] = 0;
      sh->hist[threadIdx.x] = 0;
      if (threadIdx.x == 0) sh->found = -1;
      __syncthreads();
      each([&](float z, int i) {
        const unsigned k = key_of(z);
        if (k < lo || k > hi || !in(z, i)) return;
        const unsigned b = (hi - k) >> shift;
        if (MASS) atomicAdd(&sh->mass[b], weight_of(w, z));
        else atomicAdd(&sh->hist[b], 1u);
      });
      barrier();
      u64 v = 0;
      for (int r = 0; r < nc; ++r) {
        if (MASS) v += nc > 1 ? ld_cluster_u64(&sh->mass[threadIdx.x], r) : sh->mass[threadIdx.x];
        else v += nc > 1 ? ld_cluster_u32(&sh->hist[threadIdx.x], r) : sh->hist[threadIdx.x];
      }
      const u64 inc = base_sum + scan(v);
      if (v > 0 && need <= inc && inc - v < need) {
        sh->found = threadIdx.x;
        sh->before = inc - v;
      }
      barrier();  // also: the bins may be cleared again
      const int b = sh->found;
      const u64 before = sh->before;
      __syncthreads();
      if (b < 0) break;  // the sums end below `need`: all candidates
      base_sum = before;
      hi -= static_cast<unsigned>(b) << shift;
      const unsigned span = (1u << shift) - 1;
      lo = hi - lo > span ? hi - span : lo;
    }
    *sum_above = base_sum;
    return lo;
  }

  // Of the admitted logits with this key, the index of the c-th in index
  // order (INT_MAX if there are no more than c).
  template <typename In>
  __device__ int border_index(unsigned key, u64 c, In in) {
    const float z = of_key(key);
    auto tie = [&](float x, int i) -> u64 { return x == z && in(x, i) ? 1 : 0; };
    u64 mine = 0, none = 0;
    each([&](float x, int i) { mine += tie(x, i); });
    const int buf = par;
    u64 all = mine;
    reduce2<kSum, kSum>(all, none);
    if (c >= all) {
      __syncthreads();
      return INT_MAX;
    }
    int idx;
    float dummy;
    u64 cut = ~0ull, zero = 0;
    if (locate(buf, c, tie, &idx, &dummy)) cut = static_cast<u64>(idx);
    __syncthreads();
    reduce2<kMin, kSum>(cut, zero);
    return static_cast<int>(cut);
  }
};

__global__ void __launch_bounds__(kThreads) sample_filtered_kernel(const SampleFilteredParams p,
                                                                   int nc, int slice, int cs) {
  extern __shared__ __align__(16) uint8_t smem[];
  Shared* sh = reinterpret_cast<Shared*>(smem);
  float* vals = reinterpret_cast<float*>(smem + (sizeof(Shared) + 15) / 16 * 16);
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int row = blockIdx.x / nc, rank = blockIdx.x % nc;
  const int V = p.vocab;

  Row R;
  R.sh = sh;
  R.vals = vals;
  R.cs = cs;
  R.base = rank * slice;
  R.nc = nc;
  R.rank = rank;
  R.par = 0;

  if (tid < 64) {
    // 2^(-j/64) in 64 bits (64 threads, once)
    const double t = exp2(-tid / 64.0);
    const float hi = static_cast<float>(t);
    const u64 fix = static_cast<u64>(t * 0x1p45 + 0.5);
    sh->tab[tid] = make_float4(hi, static_cast<float>(t - static_cast<double>(hi)),
                               __uint_as_float(static_cast<unsigned>(fix)),
                               __uint_as_float(static_cast<unsigned>(fix >> 32)));
  }
  // ---- the slice to shared memory; -0 becomes +0, so that the zeros tie
  const int n_loc = max(0, min(slice, V - rank * slice));
  const float* src = p.logits + row * p.ld + static_cast<int64_t>(rank) * slice;
  const bool vec = (reinterpret_cast<uintptr_t>(src) & 15) == 0;
  float mx = -INFINITY;
  unsigned finite = 0;
  bool bad = false;
  for (int o = warp * cs + lane * 4; o < (warp + 1) * cs; o += 128) {
    float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    if (vec && o + 3 < n_loc) {
      v = __ldcs(reinterpret_cast<const float4*>(src + o));
    } else {
      if (o < n_loc) v.x = __ldcs(src + o);
      if (o + 1 < n_loc) v.y = __ldcs(src + o + 1);
      if (o + 2 < n_loc) v.z = __ldcs(src + o + 2);
      if (o + 3 < n_loc) v.w = __ldcs(src + o + 3);
    }
    v.x += 0.f, v.y += 0.f, v.z += 0.f, v.w += 0.f;
    *reinterpret_cast<float4*>(vals + o) = v;
    bad |= !(v.x <= FLT_MAX && v.y <= FLT_MAX && v.z <= FLT_MAX && v.w <= FLT_MAX);
    mx = fmaxf(mx, fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)));
    finite += (v.x > -INFINITY) + (v.y > -INFINITY) + (v.z > -INFINITY) + (v.w > -INFINITY);
  }
  R.barrier();  // every CTA of the cluster runs before its shared memory is written
  u64 top = key_of(mx), n_fin = finite + (bad ? 1ull << 40 : 0);
  R.reduce2<kMax, kSum>(top, n_fin);
  const float m = of_key(static_cast<unsigned>(top));

  // ---- settings
  const float T = p.temperature[row];
  const int k = p.top_k != nullptr ? p.top_k[row] : 0;
  const float tp = p.top_p != nullptr ? p.top_p[row] : 1.f;
  const float mp = p.min_p != nullptr ? p.min_p[row] : 0.f;
  const double a = p.a[row];
  if (!(T >= 0.f && T <= FLT_MAX) || tp != tp || mp != mp || !(a >= 0.0 && a < 1.0) || n_fin == 0 ||
      n_fin >> 40) {
    if (rank == 0 && tid == 0) {
      p.token[row] = -1;
      if (p.n_kept != nullptr) p.n_kept[row] = 0;
      if (p.logprob != nullptr) p.logprob[row] = 0.f;
      raise_status(p.status, DFLASH_ERR_INVALID_ARG, 541);
    }
    return;  // the whole cluster
  }
  if (T == 0.f) {
    u64 first = ~0ull, none = 0;
    R.each([&](float z, int i) {
      if (z == m && static_cast<u64>(i) < first) first = i;
    });
    R.reduce2<kMin, kSum>(first, none);
    if (rank == 0 && tid == 0) {
      p.token[row] = static_cast<int32_t>(first);
      if (p.n_kept != nullptr) p.n_kept[row] = 1;
      if (p.logprob != nullptr) p.logprob[row] = 0.f;
    }
    return;
  }
  const double Td = fmax(static_cast<double>(T), 1e-30);
  if (tid == 0) {
    const double c = 1.44269504088896340736 / Td;
    sh->ch = static_cast<float>(c);
    sh->cl = static_cast<float>(c - static_cast<double>(sh->ch));
    sh->scale = static_cast<float>(c * ((kBins - 1) / static_cast<double>(kMaxLog2)));
    // smallest float z with (z - m) / T >= ln min_p
    unsigned km = 0;
    if (mp > 0.f) {
      const double lim = log(static_cast<double>(mp)), md = m;
      float z = static_cast<float>(fmin(fmax(md + Td * lim, -static_cast<double>(FLT_MAX)), md));
      auto ok = [&](float x) { return (static_cast<double>(x) - md) / Td >= lim; };
      unsigned kz = key_of(z);
      const unsigned kmax = key_of(m), kmin = key_of(-FLT_MAX);
      while (kz < kmax && !ok(of_key(kz))) ++kz;
      while (kz > kmin && ok(of_key(kz - 1))) --kz;
      km = kz;
    }
    sh->key_m = km;
  }
  __syncthreads();
  R.w.tab = sh->tab;
  R.w.m = m;
  R.w.ch = sh->ch;
  R.w.cl = sh->cl;
  R.w.scale = sh->scale;
  R.w.extra = V > (1 << 18) ? 1 : 0;

  // the kept set: keys above v, and key v up to index i
  unsigned v = sh->key_m;
  int vi = INT_MAX;
  const bool use_k = k > 0 && static_cast<u64>(k) < n_fin;
  const bool use_p = tp < 1.f;
  if (use_k || use_p) {
    // ---- counts by t
    sh->hist[tid] = 0;
    __syncthreads();
    R.each([&](float z, int) {
      const int b = bin_of(R.w, z);
      if (b < kBins - 1) atomicAdd(&sh->hist[b], 1u);
    });
    R.barrier();
    u64 cnt = 0;
    for (int r = 0; r < nc; ++r) cnt += nc > 1 ? ld_cluster_u32(&sh->hist[tid], r) : sh->hist[tid];
    const u64 cum = R.scan(cnt);
    if (tid == 0) sh->found = -1;
    R.barrier();

    // ---- top-k
    unsigned vk = 0;
    int ik = INT_MAX, bk = kBins - 1;  // bin of K's border (kBins - 1: in the tail, or none)
    if (use_k) {
      if (cnt > 0 && cum >= static_cast<u64>(k) && cum - cnt < static_cast<u64>(k)) {
        sh->found = tid;
        sh->before = cum - cnt;
      }
      __syncthreads();
      bk = sh->found < 0 ? kBins - 1 : sh->found;
      const u64 before = sh->before;
      __syncthreads();
      if (bk < kBins - 1) {
        u64 lo = ~0ull, hi = 0;
        R.each([&](float z, int) {
          if (bin_of(R.w, z) == bk) {
            const u64 key = key_of(z);
            lo = key < lo ? key : lo;
            hi = key > hi ? key : hi;
          }
        });
        R.reduce2<kMin, kMax>(lo, hi);
        auto any = [](float, int) { return true; };
        u64 above;
        vk = R.border_key<false>(static_cast<unsigned>(lo), static_cast<unsigned>(hi), k, before, any, &above);
        ik = R.border_index(vk, k - above, any);
      }
    }
    auto in_k = [&](float z, int i) {
      const unsigned key = key_of(z);
      return key > vk || (key == vk && i <= ik);
    };
    if (vk > v || (vk == v && ik < vi)) v = vk, vi = ik;

    // ---- top-p
    if (use_p) {
      // bounds of every prefix's mass from the counts (K's last bin in part)
      constexpr float step = kMaxLog2 / (kBins - 1);
      u64 part = cnt;
      if (bk < kBins - 1) part = tid < bk ? cnt : tid == bk ? k - (cum - cnt) : 0;
      if (tid == kBins - 1) part = 0;
      const float c = static_cast<float>(part);
      float low = c * exp2f(-(tid + 1) * step * 1.0001f), high = c * exp2f(-tid * step * 0.9999f);
      R.scan2f(low, high);
      if (tid == kThreads - 1) {
        sh->f0[0] = low;
        sh->f1[0] = high;
        sh->b_lo = sh->b_hi = kBins - 2;
      }
      __syncthreads();
      const float q = fmaxf(tp, 0.f);
      if (part > 0 && high >= q * sh->f0[0] * 0.999f) atomicMin(&sh->b_lo, tid);
      if (part > 0 && low >= q * sh->f1[0] * 1.001f) atomicMin(&sh->b_hi, tid);
      __syncthreads();
      const int b_lo = sh->b_lo, b_hi = sh->b_hi;
      __syncthreads();
      // K's mass, and the mass above the bins in question
      u64 M = 0, A = 0, lo = ~0ull, hi = 0;
      R.each([&](float z, int i) {
        const int b = bin_of(R.w, z);
        if (b >= kBins - 1 || !in_k(z, i)) return;
        const u64 x = weight_of(R.w, z);
        M += x;
        if (b < b_lo) A += x;
        else if (b <= b_hi) {
          const u64 key = key_of(z);
          lo = key < lo ? key : lo;
          hi = key > hi ? key : hi;
        }
      });
      R.reduce2<kSum, kSum>(M, A);
      R.reduce2<kMin, kMax>(lo, hi);
      const double want = ceil(static_cast<double>(q) * static_cast<double>(M));
      u64 need = static_cast<u64>(want);
      if (need > M) need = M;
      if (need <= A) need = A + 1;
      u64 above;
      const unsigned vp = R.border_key<true>(static_cast<unsigned>(lo), static_cast<unsigned>(hi), need, A,
                                             in_k, &above);
      const u64 wp = weight_of(R.w, of_key(vp));
      const u64 c_ties = need > above ? (need - above + wp - 1) / max(wp, 1ull) : 1;
      const int ip = R.border_index(vp, c_ties, in_k);
      // a tie cut by K and not by P stays cut by K
      if (vp > v || (vp == v && ip < vi)) v = vp, vi = ip;
    }
  }

  // ---- the draw
  auto value = [&](float z, int i) -> u64 {
    const unsigned key = key_of(z);
    if (key < v || (key == v && i > vi) || bin_of(R.w, z) >= kBins - 1) return 0;
    return weight_of(R.w, z);
  };
  u64 mine = 0, kept = 0;
  R.each([&](float z, int i) {
    const unsigned key = key_of(z);
    if (z > -INFINITY && (key > v || (key == v && i <= vi))) {
      ++kept;
      if (bin_of(R.w, z) < kBins - 1) mine += weight_of(R.w, z);
    }
  });
  const int buf = R.par;
  u64 S = mine;
  R.reduce2<kSum, kSum>(S, kept);
  u64 need = static_cast<u64>(a * static_cast<double>(S)) + 1;
  if (need > S) need = S;
  int idx;
  float z;
  if (R.locate(buf, need, value, &idx, &z)) {
    p.token[row] = idx;
    if (p.n_kept != nullptr) {
      if (k > 0 && kept > static_cast<u64>(k)) kept = k;  // K's border lies in the tail
      p.n_kept[row] = static_cast<int32_t>(kept);
    }
    if (p.logprob != nullptr)
      p.logprob[row] = static_cast<float>((static_cast<double>(z) - static_cast<double>(m)) / Td -
                                          log(ldexp(static_cast<double>(S), R.w.extra - 45)));
  }
}

}  // namespace

cudaError_t sample_filtered_launch(const SampleFilteredParams& p, cudaStream_t s) {
  // CTAs per row: a slice of at most kSlice logits, so that two CTAs fit an SM;
  // more (down to kMinSlice logits) while the rows leave SMs without work
  constexpr int kSlice = 24576, kMinSlice = 4096, kResident = 2 * 152;
  int nc = 1;
  while (nc < kMaxCluster && ((p.vocab + nc - 1) / nc > kSlice ||
                              (2 * nc * p.rows <= kResident && p.vocab / (2 * nc) >= kMinSlice)))
    nc *= 2;
  const int slice = ((p.vocab + nc - 1) / nc + 3) / 4 * 4;
  const int cs = (slice + kWarps * 128 - 1) / (kWarps * 128) * 128;
  const size_t smem = (sizeof(Shared) + 15) / 16 * 16 + static_cast<size_t>(kWarps) * cs * 4;
  static thread_local int allowed = -1;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(sample_filtered_kernel), 227 * 1024, &allowed);
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
  return cudaLaunchKernelEx(&cfg, sample_filtered_kernel, p, nc, slice, cs);
}

}  // namespace dflash
