// Log probability and rank of given tokens, entropy and the best alternatives of rows
// of logits.
//
//   t_i = (z_i - m) / T, m = max z;  S = sum exp(t_i);
//   logprob = t_id - ln S;  entropy = ln S - sum exp(t_i) t_i / S;
//   rank = #{z_j > z_id} + #{z_j = z_id, j < id}.
//
// One pass over the row.  Every thread keeps a running maximum and, relative to it, S
// and the entropy's sum, both rescaled when the maximum rises (after a few groups of
// vectors that is rare); sums go group, thread, warp, CTA, so a row of 2^17 logits adds
// up over some forty fp32 roundings.  Exponents are formed as (z - m) c, not as z c - m c,
// whose second product's rounding all weights would share.
//
// The alternatives need no sort and no second pass: a thread also keeps the maximum of
// each of its groups of 16 logits.  The n-th largest of the threads'
// maxima bounds the n-th largest logit from below, so only groups that reach it are read
// again, about n of them, and what reaches it there is ranked by counting.  Where
// too many do (plateaus of equal logits), the n-th largest is found by digits of its key,
// with a pass over the slice for each, and equals are taken in order of their index.
//
// Rows are a CTA each, two CTAs to an SM; fewer rows than that are cut over clusters.
//
// Bound: 2048 fp32 rows of 151936 the loads: 197 us without alternatives, 6.3 TB/s, 221
// with five: the phases behind a row's pass take its SM 4 us, in which only the other
// CTA's loads are in flight.  bf16 rows instruction issue, 162 us, 3.8 TB/s (without
// alternatives 139, 4.5).  One row
// (a cluster of 8) 10.8 us, the latency of five phases.
#include <cfloat>
#include <climits>

#include "common.cuh"
#include "kernels.h"
#include "tc05.cuh"

namespace dflash {

namespace {

constexpr int kThreads = 512;
constexpr int kGroup = 16;         // logits that a thread reads together
constexpr int kCandidates = 1024, kGroups = 512;   // places for candidates, and for groups that hold some
constexpr int kMaxCluster = 8;
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.693147180559945309f;

struct Stats {
  float m, s, e;   // maximum, sum of 2^t, sum of 2^t t (t in base 2, relative to m)
  int better;
};

// Ordered as floats are; -0 and +0 alike.
__device__ __forceinline__ uint32_t key_of(float z) {
  const uint32_t b = __float_as_uint(z + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
// 1 where z <= border does not hold (NaN on either side included), else 0.
__device__ __forceinline__ float not_at_most(float z, float border) {
  float r;
  asm("set.gtu.f32.f32 %0, %1, %2;" : "=f"(r) : "f"(z), "f"(border));
  return r;
}
__device__ __forceinline__ bool before(float za, int ia, float zb, int ib) {
  return za > zb || (za == zb && ia < ib);
}

// x's sums relative to the maximum m >= x.m.
__device__ __forceinline__ void rebase(Stats& x, float m, float c) {
  if (x.m == -INFINITY) {   // nothing, or NaN
    x.e = x.s;
  } else {
    const float d = (x.m - m) * c, w = ex2(d);
    x.e = w * (x.e + x.s * fmaxf(d, -200.f));
    x.s *= w;
  }
  x.m = m;
}
// The lanes' sums together, to all lanes.
__device__ __forceinline__ void warp_join(Stats& x, float c) {
  rebase(x, warp_max(x.m), c);
  x.s = warp_sum(x.s);
  x.e = warp_sum(x.e);
  x.better = __reduce_add_sync(0xffffffffu, x.better);
}

__device__ __forceinline__ void st_cluster(uint32_t addr, float4 v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
               : "memory");
}

template <bool HALF>
struct Row {
  static constexpr int PER = HALF ? 8 : 4;   // logits of a 16-byte vector
  static constexpr int UNROLL = kGroup / PER;
  const uint8_t* base;   // of vector 0 (the row may start inside it)
  int shift, vocab;      // logits of vector 0 before the row
  __device__ Row(const ScoreParams& p, int row) : vocab(p.vocab) {
    const uint8_t* at = reinterpret_cast<const uint8_t*>(p.logits) + static_cast<int64_t>(row) * p.ld * (HALF ? 2 : 4);
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(at) & 15);
    base = at - off;
    shift = off / (HALF ? 2 : 4);
  }
  __device__ int vectors() const { return (shift + vocab + PER - 1) / PER; }
  __device__ int first(int v) const { return v * PER - shift; }   // index of its first logit
  // logits outside the row count -inf (and are not read)
  __device__ uint4 load(int v) const {
    const int i = first(v);
    if (i >= 0 && i + PER <= vocab) return __ldg(reinterpret_cast<const uint4*>(base) + v);
    return edge(v);
  }
  // A row's first and last vector.  Out of line: what a row's phases run once has to stay in
  // the instruction cache beside the pass.
  __device__ __noinline__ uint4 edge(int v) const {
    uint32_t w[4] = {};
    for (int j = 0; j < PER; ++j) {
      const int i = first(v) + j;
      const bool in = i >= 0 && i < vocab;
      if (HALF) {
        const uint32_t x = in ? __ldg(reinterpret_cast<const uint16_t*>(base) + v * 8 + j) : 0xFF80u;
        w[j / 2] |= x << (j % 2 * 16);
      } else {
        w[j % 4] = in ? __ldg(reinterpret_cast<const uint32_t*>(base) + v * 4 + j) : 0xFF800000u;
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  static __device__ uint4 none() {
    constexpr uint32_t w = HALF ? 0xFF80FF80u : 0xFF800000u;
    return make_uint4(w, w, w, w);
  }
  static __device__ void unpack(uint4 v, float* z) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (HALF) {
        z[2 * j] = __uint_as_float(w[j] << 16);
        z[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
      } else {
        z[j] = __uint_as_float(w[j]);
      }
    }
  }
  __device__ float at(int i) const {
    if (HALF) return bf2f(__ldg(reinterpret_cast<const uint16_t*>(base) + shift + i));
    return __ldg(reinterpret_cast<const float*>(base) + shift + i);
  }
};

// The `n` best of vectors [v0, v1) into list (unordered) where more of them reach a bound
// than fit there: returns how many (n, or all that are above -inf).
template <bool HALF>
__device__ __noinline__ int many_equal(const Row<HALF>& row, int v0, int v1, int n, float2* list, int* scratch,
                                       int* count, int* bins) {
  constexpr int PER = Row<HALF>::PER;
  const int tid = threadIdx.x;
  // key of the n-th largest, eight bits a pass
  uint32_t prefix = 0, mask = 0;
  int above = 0;   // logits with larger keys
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) bins[tid] = 0;
    __syncthreads();
    for (int v = v0 + tid; v < v1; v += kThreads) {
      float z[PER];
      Row<HALF>::unpack(row.load(v), z);
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const uint32_t k = key_of(z[j]);
        if (z[j] > -INFINITY && (k & mask) == prefix) atomicAdd(&bins[k >> shift & 255], 1);
      }
    }
    __syncthreads();
    if (tid == 0) {
      int b = 255, sum = above;
      while (b > 0 && sum + bins[b] < n) sum += bins[b--];
      scratch[0] = b;
      scratch[1] = sum;
    }
    __syncthreads();
    prefix |= static_cast<uint32_t>(scratch[0]) << shift;
    mask |= 255u << shift;
    above = scratch[1];
    __syncthreads();
  }
  // those above it, then the equals in order of their index until there are n
  if (tid == 0) *count = 0;
  __syncthreads();
  for (int v = v0 + tid; v < v1; v += kThreads) {
    float z[PER];
    Row<HALF>::unpack(row.load(v), z);
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if (z[j] > -INFINITY && key_of(z[j]) > prefix)
        list[atomicAdd(count, 1)] = make_float2(z[j], __int_as_float(row.first(v) + j));
  }
  __syncthreads();
  int have = *count;
  for (int b = v0; b < v1 && have < n; b += kThreads) {
    float z[PER];
    Row<HALF>::unpack(b + tid < v1 ? row.load(b + tid) : Row<HALF>::none(), z);
    int mine = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) mine += z[j] > -INFINITY && key_of(z[j]) == prefix;
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, o);
      if (tid % 32 >= o) upto += y;
    }
    __syncthreads();
    if (tid % 32 == 31) scratch[tid / 32] = upto;
    __syncthreads();
    int at = have + upto - mine;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < tid / 32) at += scratch[w];
      have += scratch[w];
    }
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if (z[j] > -INFINITY && key_of(z[j]) == prefix) {
        if (at < n) list[at] = make_float2(z[j], __int_as_float(row.first(b + tid) + j));
        ++at;
      }
  }
  __syncthreads();
  return min(have, n);
}

template <bool HALF>
__global__ void __launch_bounds__(kThreads, 2) score_kernel(const __grid_constant__ ScoreParams p, int cluster) {
  using R = Row<HALF>;
  constexpr int PER = R::PER, kUnroll = R::UNROLL;
  // upper halves of the keys of the groups' maxima, [groups][kThreads] (only for
  // alternatives): what shared memory takes is missing to L1, which holds the loads in flight
  extern __shared__ uint16_t group_max[];
  __shared__ float2 list[kCandidates];
  __shared__ float2 best[kMaxCluster * kMaxScoreTop];   // of all slices (rank 0's)
  __shared__ float4 slices[kMaxCluster];                // their statistics (rank 0's)
  __shared__ float thread_max[kThreads];
  __shared__ int scratch[kThreads / 32], bins[256], group_list[kGroups], count, reaching, bound;
  __shared__ Stats warps[kThreads / 32];
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int rank = cluster > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int r = blockIdx.x / cluster;
  // (a CTA's shared memory may be written to by others once it runs)
  if (cluster > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  griddep_wait();
  griddep_launch_dependents();
  const R row(p, r);
  const int vectors = row.vectors(), slice = (vectors + cluster - 1) / cluster;
  const int v0 = min(rank * slice, vectors), v1 = min(v0 + slice, vectors);
  const int groups = (v1 - v0 + kThreads * kUnroll - 1) / (kThreads * kUnroll);
  uint4 raw[kUnroll];
  auto fetch = [&](int g) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int v = v0 + (g * kUnroll + u) * kThreads + tid;
      raw[u] = v < v1 ? row.load(v) : R::none();
    }
  };
  int id = p.ids != nullptr ? __ldg(p.ids + r) : -1;
  const bool bad_id = id >= p.vocab;
  if (bad_id || id < 0) id = -1;
  const float zid = id >= 0 ? row.at(id) : INFINITY;
  // !(z <= below) counts equals before the token, -inf too
  const float below = zid == -INFINITY ? __int_as_float(0x7FFFFFFF) : nextafterf(zid, -INFINITY);
  float T = p.temperature != nullptr ? __ldg(p.temperature + r) : 1.f;
  const bool bad_T = !(T > 0.f) || T == INFINITY;
  T = bad_T ? 1.f : fminf(fmaxf(T, 1e-30f), 1e30f);
  const float c = kLog2e / T;

  // Groups [whole0, whole1) lie inside the row and the slice for all threads.
  const int whole0 = v0 == 0 && row.shift > 0 ? 1 : 0;
  const int whole1 = max(min(v1, (row.shift + row.vocab) / PER) - v0, 0) / (kThreads * kUnroll);
  auto whole = [&](int g) { return g >= whole0 && g < whole1; };
  // ---- the pass
  Stats st = {-INFINITY, 0.f, 0.f, 0};
  float better = 0.f;   // (a thread has fewer than 2^24 logits)
#pragma unroll 1
  for (int g = -1; g < groups; ++g) {   // (-1: only the first loads)
    float z[kGroup];
    if (g >= 0) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) R::unpack(raw[u], z + u * PER);
    }
    if (whole(g + 1)) {
      const uint4* at = reinterpret_cast<const uint4*>(row.base) + v0 + (g + 1) * (kUnroll * kThreads) + tid;
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) raw[u] = __ldg(at + u * kThreads);
    } else if (g + 1 < groups) {
      fetch(g + 1);
    }
    if (g < 0) continue;
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < kGroup; ++j) top = fmaxf(top, z[j]);
    if (p.n_top > 0) group_max[g * kThreads + tid] = static_cast<uint16_t>(key_of(top) >> 16);
    if (top > st.m) {
      if (st.m > -INFINITY) {
        const float d = (st.m - top) * c, w = ex2(d);
        st.e = w * (st.e + st.s * fmaxf(d, -200.f));
        st.s *= w;
      }
      st.m = top;
    }
    if (st.m == -INFINITY) {   // nothing yet (NaN is no maximum)
#pragma unroll
      for (int j = 0; j < kGroup; ++j)
        if (z[j] != z[j]) st.s = z[j];
    } else {
      float2 s = make_float2(0.f, 0.f), e = s;
      const float2 m2 = make_float2(-st.m, -st.m), c2 = make_float2(c, c);
#pragma unroll
      for (int j = 0; j < kGroup; j += 2) {
        const float2 t = mul2(add2(make_float2(z[j], z[j + 1]), m2), c2);
        const float2 w = make_float2(ex2(t.x), ex2(t.y));
        s = add2(s, w);
        e = fma2(w, make_float2(fmaxf(t.x, -200.f), fmaxf(t.y, -200.f)), e);
      }
      st.s += s.x + s.y;
      st.e += e.x + e.y;
    }
    if (id >= 0) {
      // all of the group before the token or all behind it, or a vector at a time
      const int i0 = row.first(v0 + g * (kUnroll * kThreads) + tid), i1 = i0 + (kUnroll - 1) * kThreads * PER + PER;
      if (whole(g) && (i1 <= id || i0 > id)) {
        const float border = i0 > id ? zid : below;
        float2 n2 = make_float2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < kGroup; j += 2)
          n2 = add2(n2, make_float2(not_at_most(z[j], border), not_at_most(z[j + 1], border)));
        better += n2.x + n2.y;
      } else {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          const int v = v0 + (g * kUnroll + u) * kThreads + tid, i = row.first(v);
          // (not the vector that holds the token, nor the one in which the row starts)
          if (v >= v1 || i < 0 || (i <= id && id < i + PER)) continue;
          const float border = i > id ? zid : below;
#pragma unroll
          for (int j = 0; j < PER; ++j) better += not_at_most(z[u * PER + j], border);
        }
      }
    }
  }
  st.better = static_cast<int>(better);
  if (id >= 0 && tid < 2 * PER) {   // those two, a logit to a thread
    const int own = (id + row.shift) / PER, v = tid < PER ? own : 0, i = row.first(v) + tid % PER;
    if ((tid < PER || (own > 0 && row.shift > 0)) && v >= v0 && v < v1 && i >= 0 && i < row.vocab && i != id)
      st.better += !(row.at(i) <= (i > id ? zid : below));
  }
  if (p.n_top > 0) thread_max[tid] = st.m;

  // ---- the CTA's statistics
  if (cluster > 1) {
    __syncwarp();
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  }
  warp_join(st, c);
  if (lane == 0) warps[warp] = st;
  if (tid == 0) count = reaching = 0;
  __syncthreads();
  if (warp == 0) {
    Stats a = lane < kThreads / 32 ? warps[lane] : Stats{-INFINITY, 0.f, 0.f, 0};
    warp_join(a, c);
    if (lane == 0) {
      const float4 v = make_float4(a.m, a.s, a.e, __int_as_float(a.better));
      if (rank == 0) slices[0] = v;
      else st_cluster(dsmem_map(smem_u32(&slices[rank]), 0), v);
    }
  }

  // ---- the slice's best
  int mine = 0;   // entries of this slice
  const int n = p.n_top;
  if (n > 0) {
    if (warp == 1) {
      // the n-th largest of the threads' maxima, by the upper 16 bits of its key
      uint32_t k[kThreads / 32], lo = ~0u, hi = 0;
#pragma unroll
      for (int j = 0; j < kThreads / 32; ++j) {
        k[j] = key_of(thread_max[j * 32 + lane]) >> 16;
        lo = min(lo, k[j]);
        hi = max(hi, k[j]);
      }
      lo = __reduce_min_sync(0xffffffffu, lo);
      hi = __reduce_max_sync(0xffffffffu, hi);
      // (bits above the first in which they differ are all of them's)
      const int bits = 32 - __clz(lo ^ hi);
      uint32_t least = hi >> bits << bits;
#pragma unroll 1
      for (int b = bits - 1; b >= 0; --b) {
        const uint32_t y = least | 1u << b;
        int many = 0;
#pragma unroll
        for (int j = 0; j < kThreads / 32; ++j) many += k[j] >= y;
        if (__reduce_add_sync(0xffffffffu, many) >= n) least = y;
      }
      if (lane == 0) bound = static_cast<int>(least);
    }
    __syncthreads();
    const uint32_t least = static_cast<uint32_t>(bound);
    auto reaches = [&](float z) { return z > -INFINITY && key_of(z) >> 16 >= least; };
    // the groups that reach it, then their logits, sixteen lanes to a group
#pragma unroll 1
    for (int g = 0; g < groups; ++g)
      if (group_max[g * kThreads + tid] >= least) {
        const int at = atomicAdd(&reaching, 1);
        if (at < kGroups) group_list[at] = g * kThreads + tid;
      }
    __syncthreads();
    const int many = reaching;
#pragma unroll 1
    for (int x = warp * 2 + lane / 16; x < min(many, kGroups); x += kThreads / 16) {
      const int gt = group_list[x], g = gt / kThreads, l = lane % 16;
      const int v = v0 + (g * kUnroll + l / PER) * kThreads + gt - g * kThreads, i = row.first(v) + l % PER;
      if (v >= v1 || i < 0 || i >= row.vocab) continue;
      const float z = row.at(i);
      if (!reaches(z)) continue;
      const int at = atomicAdd(&count, 1);
      if (at < kCandidates) list[at] = make_float2(z, __int_as_float(i));
    }
    __syncthreads();
    int found = count;
    if (found > kCandidates || many > kGroups) found = many_equal<HALF>(row, v0, v1, n, list, scratch, &count, bins);
    // each counts what precedes it
    mine = min(found, n);
    for (int a = tid; a < found; a += kThreads) {
      const float2 x = list[a];
      int place = 0;
      for (int b = 0; b < found; ++b) {
        const float2 y = list[b];
        place += before(y.x, __float_as_int(y.y), x.x, __float_as_int(x.y));
      }
      if (place < n) {
        const int slot = rank * kMaxScoreTop + place;
        if (rank == 0) {
          best[slot] = x;
        } else {
          asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(dsmem_map(smem_u32(&best[slot]), 0)), "f"(x.x),
                       "f"(x.y)
                       : "memory");
        }
      }
    }
    // the places that this slice leaves empty
    for (int a = mine + tid; a < n; a += kThreads) {
      const int slot = rank * kMaxScoreTop + a;
      if (rank == 0) {
        best[slot] = make_float2(-INFINITY, __int_as_float(-1));
      } else {
        asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(dsmem_map(smem_u32(&best[slot]), 0)),
                     "f"(-INFINITY), "f"(__int_as_float(-1))
                     : "memory");
      }
    }
  }
  if (cluster > 1) cluster_sync();
  else __syncthreads();
  if (rank != 0) return;

  // ---- the row's results
  Stats a = {-INFINITY, 0.f, 0.f, 0};
  if (lane < cluster) {
    const float4 v = slices[lane];
    a = Stats{v.x, v.y, v.z, __float_as_int(v.w)};
  }
  warp_join(a, c);
  const bool bad = bad_T || a.m == -INFINITY || a.m == INFINITY || !(a.s > 0.f);
  const float nan = __int_as_float(0x7FC00000), ln_s = logf(a.s);
  if (tid == 0) {
    if (bad || bad_id) raise_status(p.status, DFLASH_ERR_INVALID_ARG, bad ? 571 : 572);
    if (p.logprob != nullptr) p.logprob[r] = bad || bad_id ? nan : id >= 0 ? (zid - a.m) / T - ln_s : 0.f;
    if (p.rank != nullptr) p.rank[r] = bad || id < 0 ? -1 : a.better;
    if (p.entropy != nullptr) p.entropy[r] = bad ? nan : fmaxf(ln_s - kLn2 * (a.e / a.s), 0.f);
  }
  for (int x = tid; x < cluster * n; x += kThreads) {
    const float2 v = best[x / n * kMaxScoreTop + x % n];
    const int i = __float_as_int(v.y);
    int place = 0;
    if (cluster == 1) place = x;
    else
      for (int k = 0; k < cluster; ++k)
      {   // a slice's are in order: how many precede this one
        int lo = 0, hi = n;
        while (lo < hi) {
          const int mid = (lo + hi) / 2;
          const float2 w = best[k * kMaxScoreTop + mid];
          const int j = __float_as_int(w.y);
          if (j >= 0 && (i < 0 || before(w.x, j, v.x, i))) lo = mid + 1;
          else hi = mid;
        }
        place += lo;
      }
    // empty places come after all others, in any order
    if (i < 0 && cluster > 1) {
      for (int y = 0; y < x; ++y) place += __float_as_int(best[y / n * kMaxScoreTop + y % n].y) < 0;
    }
    if (place < n) {
      p.top_id[static_cast<size_t>(r) * n + place] = bad ? -1 : i;
      p.top_logprob[static_cast<size_t>(r) * n + place] =
          bad ? nan : i < 0 ? -INFINITY : (v.x - a.m) / T - ln_s;
    }
  }
}

template <bool HALF>
cudaError_t launch(const ScoreParams& p, cudaStream_t s) {
  constexpr int PER = Row<HALF>::PER, kUnroll = Row<HALF>::UNROLL;
  const int vectors = p.vocab / PER + 2;
  // Rows are cut until the CTAs fill the machine twice, down to one group a thread.
  int cluster = 1;
  while (cluster < kMaxCluster && static_cast<int64_t>(p.rows) * cluster * 2 <= 304 &&
         vectors / (2 * cluster) >= kThreads * kUnroll)
    cluster *= 2;
  const int slice = (vectors + cluster - 1) / cluster;
  const int groups = (slice + kThreads * kUnroll - 1) / (kThreads * kUnroll);
  const int smem = p.n_top > 0 ? groups * kThreads * 2 : 0;
  const void* fn = reinterpret_cast<const void*>(score_kernel<HALF>);
  static thread_local int allowed = -1;
  const cudaError_t e = allow_smem(fn, 64 * 1024, &allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.rows) * cluster);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  count_launch();
  return cudaLaunchKernelEx(&cfg, score_kernel<HALF>, p, cluster);
}

}  // namespace

cudaError_t score_tokens_launch(const ScoreParams& p, bool half, cudaStream_t s) {
  return half ? launch<true>(p, s) : launch<false>(p, s);
}

}  // namespace dflash
