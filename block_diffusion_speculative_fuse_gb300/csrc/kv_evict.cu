// Eviction from a paged cache: of each request and KV head the positions with the largest
// accumulated attention weight are kept and moved together, in order, into other pages.
//
// Two kernels.  The first marks the pages that are read and written, so that a target page
// named twice, or read by the same call, is found before anything is moved, and
// finds the kept positions: the border's 32-bit key by three digits of 11, 11 and 10 bits (a
// histogram in shared memory each; the first holds sign, exponent and two bits, so that
// masses, whose exponents lie together, do not all meet in one counter), then one pass that
// numbers what is above it and the first equals in order of position.  One CTA per request
// and head, or a cluster, each CTA a slice of the positions, where there are few.  The second
// copies whole vectors.
//
// Bound: the copy's bytes where there are many requests: 32 x 8192 positions to 2048 in
// 111 us, of which the copy is 83, 6.4 TB/s.  For one request the choice: 98304
// positions of 8 heads take 46 us (40 with the same inputs again), 20 of them for three digits (each a pass over 6144
// positions a CTA, a barrier of 16 CTAs and an exchange of 96 counts) and the numbering.
#include <climits>

#include "common.cuh"
#include "kernels.h"

namespace dflash {

namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kCached = 24576;   // positions of a CTA whose keys stay in shared memory
constexpr int kBins = 2048, kCoarse = 64;
constexpr int kMaxCluster = 16;
constexpr int kCopyThreads = 256;
constexpr int kCopies = 8;       // loads of a thread in flight

// Kept positions of request r, and its length; errors are recorded by `tell`.
struct Request {
  int ctx, keep;
  __device__ Request(const EvictParams& p, int r, bool tell) {
    ctx = max(__ldg(p.ctx_len + r), 0);
    const int room = static_cast<int>(min(static_cast<int64_t>(p.src_max_pages) * 16, p.ld_mass));
    if (ctx > room) {
      if (tell) raise_status(p.status, DFLASH_ERR_CAPACITY, 581);
      ctx = room;
    }
    keep = min(max(__ldg(p.keep + r), 0), ctx);
    const int place = static_cast<int>(min(static_cast<int64_t>(p.dst_max_pages) * 16, p.ld_kept));
    if (keep > place) {
      if (tell) raise_status(p.status, DFLASH_ERR_CAPACITY, 582);
      keep = place;
    }
  }
};

// Marks the pages of a request (bit 0: written by the call, bit 1: read by it).
__device__ void mark_pages(const EvictParams& p, int r, const Request& q) {
  auto mark = [&](int id, unsigned bit) {
    const unsigned old = atomicOr(p.owner + id, bit);
    if (old & (bit == 1 ? 3u : 1u)) {
      raise_status(p.status, DFLASH_ERR_INVALID_ARG, 584);
      *p.conflict = 1;
    }
  };
  for (int i = threadIdx.x; i < (q.keep + 15) / 16; i += blockDim.x) {
    const int id = __ldg(p.dst_table + static_cast<size_t>(r) * p.dst_max_pages + i);
    if (id < 0 || id >= p.dst_pages) raise_status(p.status, DFLASH_ERR_CAPACITY, 583);
    else mark(id, 1);
  }
  if (!p.same_pool || q.keep == 0) return;
  for (int i = threadIdx.x; i < (q.ctx + 15) / 16; i += blockDim.x) {
    const int id = __ldg(p.src_table + static_cast<size_t>(r) * p.src_max_pages + i);
    if (id >= 0 && id < p.dst_pages) mark(id, 2);
  }
}

// Ordered as masses are, NaN last; -0 and +0 alike.
__device__ __forceinline__ uint32_t key_of(float m) {
  if (m != m) return 0u;
  const uint32_t b = __float_as_uint(m + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__global__ void __launch_bounds__(kThreads, 2) evict_select_kernel(const __grid_constant__ EvictParams p, int cluster,
                                                                         int cached) {
  extern __shared__ uint32_t cache[];   // keys of the slice, where they fit (cached)
  __shared__ uint32_t bins[2][kBins], coarse[2][kCoarse];
  __shared__ int gathered[kMaxCluster * kCoarse], warps[2][kWarps], found[2];
  __shared__ int2 slice_counts;   // of this CTA's slice: above the border, equal
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int rank = cluster > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int unit = blockIdx.x / cluster, r = unit / p.hkv, h = unit % p.hkv;
  const bool first = h == 0 && rank == 0;
  const Request q(p, r, first && tid == 0);
  griddep_launch_dependents();
  if (first) {
    if (tid == 0 && p.new_len != nullptr) p.new_len[r] = q.keep;
    mark_pages(p, r, q);
  }
  if (q.keep == 0) return;   // (the whole cluster)
  const int slice = (q.ctx + cluster - 1) / cluster;
  const int j0 = min(rank * slice, q.ctx), j1 = min(j0 + slice, q.ctx);
  const float* mass = p.mass + (static_cast<int64_t>(r) * p.hkv + h) * p.ld_mass;
  const int safe0 = p.sink, safe1 = q.ctx - min(p.recent, q.ctx);
  auto key = [&](float m, int j) { return j < safe0 || j >= safe1 ? 0xFFFFFFFFu : key_of(m); };
  const bool fits = j1 - j0 <= cached;
  auto sum_of_lower = [&](int v) {   // of the warps before; v: lane w has warp w's
    return static_cast<int>(__reduce_add_sync(0xffffffffu, lane < warp ? v : 0));
  };
  // Of n <= 64 counts in every CTA of the cluster, at `mine`: their sums, to gathered[0, n).
  auto gather = [&](const uint32_t* mine, int n) {
    __syncthreads();
    for (int x = tid; x < cluster * n; x += kThreads) {
      const int c = x / n;
      int v;
      if (cluster == 1) v = mine[x];
      else
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(dsmem_map(smem_u32(mine + x - c * n), c)));
      gathered[x] = v;
    }
    __syncthreads();
    int v = 0;
    if (tid < n)
      for (int c = 0; c < cluster; ++c) v += gathered[c * n + tid];
    __syncthreads();
    if (tid < n) gathered[tid] = v;
    __syncthreads();
  };
  // Of gathered[0, n), from the last down: the one in which the need-th of them lies and
  // how many lie above it (found), by the first warp.
  auto search = [&](int n, int need) {
    if (warp == 0) {
      const int hi = n - 1 - 2 * lane;   // two to a lane (n = 64), or one
      const int a = n == 64 ? gathered[hi] : gathered[n - 1 - lane], b = n == 64 ? gathered[hi - 1] : 0;
      int upto = a + b;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      const int before = upto - a - b;
      if (before < need && before + a >= need) {
        found[0] = n == 64 ? hi : n - 1 - lane;
        found[1] = before;
      } else if (before + a < need && upto >= need) {
        found[0] = hi - 1;
        found[1] = before + a;
      }
    }
    __syncthreads();
  };
  uint32_t border = 0;
  int equals = 0;                 // kept of those at the border
  const bool all = q.keep >= q.ctx;
  if (!all) {
    uint32_t prefix = 0, mask = 0;
    int need = q.keep;            // of the positions with this prefix
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 1023 : 2047;
      uint32_t* mine = bins[pass & 1];
      for (int b = tid; b < kBins; b += kThreads) mine[b] = 0;
      __syncthreads();
      // four positions of a thread at once; the first pass leaves their keys behind
#pragma unroll 1
      for (int at = tid; at < j1 - j0; at += 4 * kThreads) {
        uint32_t k[4];
        if (pass > 0 && fits) {
#pragma unroll
          for (int i = 0; i < 4; ++i) k[i] = cache[min(at + i * kThreads, j1 - j0 - 1)];
        } else {
          float m[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) m[i] = __ldg(mass + min(j0 + at + i * kThreads, j1 - 1));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            k[i] = key(m[i], j0 + at + i * kThreads);
            if (fits && at + i * kThreads < j1 - j0) cache[at + i * kThreads] = k[i];
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (at + i * kThreads < j1 - j0 && (k[i] & mask) == prefix) atomicAdd(&mine[k[i] >> shift & bits], 1u);
      }
      __syncthreads();
      // sums of 32 bins, so that other CTAs' need not all be read: a warp adds up four
#pragma unroll
      for (int i = 0; i < kCoarse / kWarps; ++i) {
        const int c = warp * (kCoarse / kWarps) + i;
        const int sum = __reduce_add_sync(0xffffffffu, mine[c * 32 + lane]);
        if (lane == 0) coarse[pass & 1][c] = sum;
      }
      if (cluster > 1) cluster_sync();
      else __syncthreads();
      gather(coarse[pass & 1], kCoarse);
      search(kCoarse, need);
      const int c = found[0];
      need -= found[1];
      gather(mine + c * 32, 32);
      search(32, need);
      if (warp == 0) {   // of this slice: what lies above the digit, and at it
        const uint32_t* co = coarse[pass & 1];
        int over = (lane > c ? co[lane] : 0) + (lane + 32 > c ? co[lane + 32] : 0);
        if (lane > found[0]) over += mine[c * 32 + lane];
        over = __reduce_add_sync(0xffffffffu, over);
        if (lane == 0) slice_counts = make_int2((pass == 0 ? 0 : slice_counts.x) + over, mine[c * 32 + found[0]]);
      }
      prefix |= static_cast<uint32_t>(c * 32 + found[0]) << shift;
      mask |= static_cast<uint32_t>(bits) << shift;
      need -= found[1];
      __syncthreads();
    }
    border = prefix;
    equals = need;
  }
  // where this slice's kept positions go: count, then number them in order
  int above0 = all ? j0 : 0, equal0 = 0;
  if (!all && cluster > 1) {
    cluster_sync();
    int2 v[kMaxCluster];
#pragma unroll
    for (int x = 0; x < kMaxCluster; ++x) {
      v[x] = make_int2(0, 0);
      if (x < rank)
        asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];"
                     : "=r"(v[x].x), "=r"(v[x].y)
                     : "r"(dsmem_map(smem_u32(&slice_counts), x)));
    }
#pragma unroll
    for (int x = 0; x < kMaxCluster; ++x) {
      above0 += v[x].x;
      equal0 += v[x].y;
    }
  }
  int32_t* kept = p.kept + (static_cast<int64_t>(r) * p.hkv + h) * p.ld_kept;
  float* mass_out = p.mass_out == nullptr ? nullptr : p.mass_out + (static_cast<int64_t>(r) * p.hkv + h) * p.ld_mass;
  __syncthreads();
#pragma unroll 1
  for (int base = j0; base < j1; base += 4 * kThreads) {
    // four positions in a row to a thread; counts above and at the border in one word
    const int first_j = base + 4 * tid;
    uint32_t k[4];
    float m[4];
    int mine = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = first_j + i;
      m[i] = __ldg(mass + min(j, j1 - 1));
      k[i] = fits && !all ? cache[min(j, j1 - 1) - j0] : key(m[i], j);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = first_j + i;
      if (j >= j1) continue;
      if (all || k[i] > border) mine += 1;
      else if (k[i] == border) mine += 1 << 16;
    }
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    int* counts = warps[(base - j0) / (4 * kThreads) & 1];
    if (lane == 31) counts[warp] = upto;
    __syncthreads();
    const int part = lane < kWarps ? counts[lane] : 0;
    const int before = sum_of_lower(part) + upto - mine, whole = __reduce_add_sync(0xffffffffu, part);
    int a = above0 + (before & 0xFFFF), e = equal0 + (before >> 16);
    above0 += whole & 0xFFFF;
    equal0 += whole >> 16;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = first_j + i;
      if (j >= j1) break;
      const bool above = all || k[i] > border, equal = !above && k[i] == border;
      if (above || (equal && e < equals)) {
        const int at = a + min(e, equals);
        if (at < q.keep) {
          kept[at] = j;
          if (mass_out != nullptr) mass_out[at] = m[i];
        }
      }
      a += above;
      e += equal;
    }
  }
  // (others may still read this CTA's counts)
  if (cluster > 1) cluster_sync();
}

// VEC: 16-byte pieces of a cached vector of one plane.  A warp moves 32 positions: its
// lanes look up a source and a target each, then copy them together, 32 / VEC
// vectors an instruction.
template <int VEC>
__global__ void __launch_bounds__(kCopyThreads, 4) evict_copy_kernel(const __grid_constant__ EvictParams p) {
  constexpr int AT_ONCE = 32 / VEC;
  const int r = blockIdx.z, h = blockIdx.y, lane = threadIdx.x % 32;
  const int i0 = (blockIdx.x * (kCopyThreads / 32) + threadIdx.x / 32) * 32;
  griddep_wait();
  const Request q(p, r, false);
  if (i0 >= q.keep) return;
  if (*reinterpret_cast<volatile int*>(p.conflict)) return;
  const int i = i0 + lane;
  const size_t plane = static_cast<size_t>(p.hkv) * 16;      // vectors between planes
  long long from = -1, to = -1;                              // plane 0's vectors
  if (i < q.keep) {
    const int j = __ldcg(p.kept + (static_cast<int64_t>(r) * p.hkv + h) * p.ld_kept + i);
    const int src = __ldg(p.src_table + static_cast<size_t>(r) * p.src_max_pages + j / 16);
    const int dst = __ldg(p.dst_table + static_cast<size_t>(r) * p.dst_max_pages + i / 16);
    if (src >= 0 && src < p.src_pages) from = static_cast<long long>(src * plane * p.planes + h * 16 + j % 16);
    else raise_status(p.status, DFLASH_ERR_CAPACITY, 585);
    if (dst >= 0 && dst < p.dst_pages) to = static_cast<long long>(dst * plane * p.planes + h * 16 + i % 16);
  }
  const int piece = lane % VEC, sub = lane / VEC;
#pragma unroll 1
  for (int pl = 0; pl < p.planes; ++pl) {
    const size_t off = pl * plane;
#pragma unroll
    for (int b = 0; b < 32 / AT_ONCE; b += kCopies) {
      constexpr int N = kCopies < 32 / AT_ONCE ? kCopies : 32 / AT_ONCE;
      uint4 x[N];
      long long t[N];
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int l = (b + k) * AT_ONCE + sub;
        const long long f = __shfl_sync(0xffffffffu, from, l);
        t[k] = __shfl_sync(0xffffffffu, to, l);
        x[k] = make_uint4(0u, 0u, 0u, 0u);
        if (f >= 0) x[k] = __ldcs(reinterpret_cast<const uint4*>(p.src_pool) + (f + off) * VEC + piece);
      }
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (t[k] >= 0) reinterpret_cast<uint4*>(p.dst_pool)[(t[k] + off) * VEC + piece] = x[k];
    }
    if (p.dst_scales != nullptr && to >= 0) p.dst_scales[to + off] = from >= 0 ? __ldg(p.src_scales + from + off) : 1.f;
  }
}

template <int VEC>
cudaError_t launch_copy(const EvictParams& p, cudaStream_t s) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((p.ld_kept + kCopyThreads - 1) / kCopyThreads), p.hkv, p.batch);
  cfg.blockDim = dim3(kCopyThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  count_launch();
  return cudaLaunchKernelEx(&cfg, evict_copy_kernel<VEC>, p);
}

}  // namespace

cudaError_t kv_evict_launch(const EvictParams& p, int vector_bytes, cudaStream_t s) {
  cudaError_t e = cudaMemsetAsync(p.conflict, 0, 256 + static_cast<size_t>(p.dst_pages) * 4, s);
  if (e != cudaSuccess) return e;
  // slices of at least 2048 positions, until the CTAs fill the machine
  int cluster = 1;
  while (cluster < kMaxCluster && static_cast<int64_t>(p.batch) * p.hkv * cluster * 2 <= 304 &&
         p.ld_mass / (2 * cluster) >= 2048)
    cluster *= 2;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.batch) * p.hkv * cluster);
  cfg.blockDim = dim3(kThreads);
  const int64_t slice = (p.ld_mass + cluster - 1) / cluster;
  const int cached = slice <= kCached ? static_cast<int>(slice) : 0;
  cfg.dynamicSmemBytes = cached * 4;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  static thread_local int allowed = -1;
  const int was = allowed;
  e = allow_smem(reinterpret_cast<const void*>(evict_select_kernel), kCached * 4, &allowed);
  if (e == cudaSuccess && allowed != was) {   // clusters of 16 are more than every device has to offer
    e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) allowed = -1;
  }
  if (e != cudaSuccess) return e;
  count_launch();
  e = cudaLaunchKernelEx(&cfg, evict_select_kernel, p, cluster, cached);
  if (e != cudaSuccess) return e;
  return vector_bytes == 256 ? launch_copy<16>(p, s) : vector_bytes == 128 ? launch_copy<8>(p, s) : launch_copy<4>(p, s);
}

}  // namespace dflash
