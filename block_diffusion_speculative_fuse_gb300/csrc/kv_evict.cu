// Eviction from a paged cache: of each request and KV head the positions with the largest
// accumulated attention weight are kept and moved together, in order, into other pages.
//
// Three kernels.  The first marks the pages that are read and written, so that a target page
// named twice, or read by the same call, is found before anything is moved.  The second
// finds the kept positions: the border's 32-bit key by three digits of 11, 11 and 10 bits (a
// histogram in shared memory each; the first holds sign, exponent and two bits, so that
// masses, whose exponents lie together, do not all meet in one counter), then one pass that
// numbers what is above it and the first equals in order of position.  One CTA per request
// and head, or a cluster, each CTA a slice of the positions, where there are few.  The third
// copies, a target page of a head at a time; source vectors are whole lines, and
// a thread has eight of their pieces in flight.
//
// Bound: the copy's bytes.
#include <climits>

#include "common.cuh"
#include "kernels.h"

namespace dflash {

namespace {

constexpr int kThreads = 1024;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int kCopyThreads = 256;
constexpr int kCopies = 8;       // pieces of a thread, all in flight

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

// bit 0: written by the call, bit 1: read by it
__global__ void evict_check_kernel(const __grid_constant__ EvictParams p) {
  const int r = blockIdx.x;
  const Request q(p, r, threadIdx.x == 0);
  if (threadIdx.x == 0 && p.new_len != nullptr) p.new_len[r] = q.keep;
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

__global__ void __launch_bounds__(kThreads, 1) evict_select_kernel(const __grid_constant__ EvictParams p, int cluster) {
  __shared__ uint32_t bins[2][kBins];
  __shared__ int warps[2][kThreads / 32], found[2];
  __shared__ int2 slice_counts;   // of this CTA's slice: above the border, equal
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int rank = cluster > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int unit = blockIdx.x / cluster, r = unit / p.hkv, h = unit % p.hkv;
  const Request q(p, r, false);
  if (q.keep == 0) return;   // (the whole cluster)
  const float* mass = p.mass + (static_cast<int64_t>(r) * p.hkv + h) * p.ld_mass;
  const int slice = (q.ctx + cluster - 1) / cluster;
  const int j0 = min(rank * slice, q.ctx), j1 = min(j0 + slice, q.ctx);
  const int safe0 = p.sink, safe1 = q.ctx - min(p.recent, q.ctx);
  auto key_at = [&](int j, float* m) {
    *m = __ldg(mass + j);
    return j < safe0 || j >= safe1 ? 0xFFFFFFFFu : key_of(*m);
  };
  auto sync_all = [&]() {
    if (cluster > 1) cluster_sync();
    else __syncthreads();
  };
  uint32_t border = 0;
  int equals = 0;                 // kept of those at it
  if (q.keep < q.ctx) {
    uint32_t prefix = 0, mask = 0;
    int need = q.keep;            // of the positions with this prefix
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 1023 : 2047;
      uint32_t* mine = bins[pass & 1];
      for (int b = tid; b < kBins; b += kThreads) mine[b] = 0;
      __syncthreads();
#pragma unroll 4
      for (int j = j0 + tid; j < j1; j += kThreads) {
        float m;
        const uint32_t k = key_at(j, &m);
        if ((k & mask) == prefix) atomicAdd(&mine[k >> shift & bits], 1u);
      }
      sync_all();
      // counts of the two largest bins first: thread t has bins 2047 - 2 t and the one below
      const int hi = kBins - 1 - 2 * tid;
      int a = 0, b = 0;
      for (int c = 0; c < cluster; ++c) {
        if (cluster == 1) {
          a = mine[hi];
          b = mine[hi - 1];
        } else {
          uint2 v;
          asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];"
                       : "=r"(v.x), "=r"(v.y)
                       : "r"(dsmem_map(smem_u32(&mine[hi - 1]), c))
                       : "memory");
          b += v.x;
          a += v.y;
        }
      }
      int upto = a + b;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      if (lane == 31) warps[0][warp] = upto;
      __syncthreads();
      const int part = warps[0][lane];
      const int before = __reduce_add_sync(0xffffffffu, lane < warp ? part : 0) + upto - a - b;
      if (before < need && before + a >= need) {
        found[0] = hi;
        found[1] = before;
      } else if (before + a < need && before + a + b >= need) {
        found[0] = hi - 1;
        found[1] = before + a;
      }
      __syncthreads();
      prefix |= static_cast<uint32_t>(found[0]) << shift;
      mask |= static_cast<uint32_t>(bits) << shift;
      need -= found[1];
    }
    border = prefix;
    equals = need;
  }
  // where this slice's kept positions go: count, then number them in order
  int above0 = 0, equal0 = 0;
  if (q.keep < q.ctx && cluster > 1) {
    int above = 0, equal = 0;
    for (int j = j0 + tid; j < j1; j += kThreads) {
      float m;
      const uint32_t k = key_at(j, &m);
      above += k > border;
      equal += k == border;
    }
    above = __reduce_add_sync(0xffffffffu, above);
    equal = __reduce_add_sync(0xffffffffu, equal);
    __syncthreads();
    if (lane == 0) {
      warps[0][warp] = above;
      warps[1][warp] = equal;
    }
    __syncthreads();
    if (warp == 0) {
      above = __reduce_add_sync(0xffffffffu, warps[0][lane]);
      equal = __reduce_add_sync(0xffffffffu, warps[1][lane]);
      if (lane == 0) slice_counts = make_int2(above, equal);
    }
    cluster_sync();
    for (int c = 0; c < rank; ++c) {
      int2 v;
      asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];"
                   : "=r"(v.x), "=r"(v.y)
                   : "r"(dsmem_map(smem_u32(&slice_counts), c))
                   : "memory");
      above0 += v.x;
      equal0 += v.y;
    }
  }
  int32_t* kept = p.kept + (static_cast<int64_t>(r) * p.hkv + h) * p.ld_kept;
  float* mass_out = p.mass_out == nullptr ? nullptr : p.mass_out + (static_cast<int64_t>(r) * p.hkv + h) * p.ld_mass;
  const bool all = q.keep >= q.ctx;
  if (all) above0 = j0;
#pragma unroll 1
  for (int base = j0; base < j1; base += kThreads) {
    const int j = base + tid;
    float m = 0.f;
    uint32_t k = 0;
    if (j < j1) k = key_at(j, &m);
    const bool above = j < j1 && (all || k > border), equal = j < j1 && !all && k == border;
    const unsigned va = __ballot_sync(0xffffffffu, above), ve = __ballot_sync(0xffffffffu, equal);
    __syncthreads();
    if (lane == 0) {
      warps[0][warp] = __popc(va);
      warps[1][warp] = __popc(ve);
    }
    __syncthreads();
    const unsigned lower = (1u << lane) - 1;
    const int pa = warps[0][lane], pe = warps[1][lane];
    const int a = above0 + __reduce_add_sync(0xffffffffu, lane < warp ? pa : 0) + __popc(va & lower);
    const int e = equal0 + __reduce_add_sync(0xffffffffu, lane < warp ? pe : 0) + __popc(ve & lower);
    above0 += __reduce_add_sync(0xffffffffu, pa);
    equal0 += __reduce_add_sync(0xffffffffu, pe);
    if (above || (equal && e < equals)) {
      const int at = a + min(e, equals);
      if (at < q.keep) {
        kept[at] = j;
        if (mass_out != nullptr) mass_out[at] = m;
      }
    }
  }
  // (others may still read this CTA's counts)
  if (cluster > 1) cluster_sync();
}

// VEC: 16-byte pieces of a cached vector of one plane.
template <int VEC>
__global__ void __launch_bounds__(kCopyThreads) evict_copy_kernel(const __grid_constant__ EvictParams p) {
  constexpr int ROWS = kCopyThreads / VEC;   // vectors at once
  const int r = blockIdx.z, h = blockIdx.y;
  if (*p.conflict) return;
  const Request q(p, r, false);
  const int32_t* kept = p.kept + (static_cast<int64_t>(r) * p.hkv + h) * p.ld_kept;
  const int planes = p.planes, per = kCopies / planes;   // positions of a thread
  const int piece = threadIdx.x % VEC, first = blockIdx.x * ROWS * per + threadIdx.x / VEC;
  if (blockIdx.x * ROWS * per >= q.keep) return;
  const size_t plane = static_cast<size_t>(p.hkv) * 16;      // vectors between planes
  uint4 x[kCopies];
  float sc[kCopies];
  size_t to[kCopies];
  bool on[kCopies];
#pragma unroll
  for (int k = 0; k < kCopies; ++k) {
    const int i = first + k / planes * ROWS;
    on[k] = i < q.keep && k / planes < per;
    if (!on[k]) continue;
    const int j = __ldg(kept + i);
    const int from = __ldg(p.src_table + static_cast<size_t>(r) * p.src_max_pages + j / 16);
    const int dest = __ldg(p.dst_table + static_cast<size_t>(r) * p.dst_max_pages + i / 16);
    const size_t in = k % planes * plane + h * 16;
    x[k] = make_uint4(0u, 0u, 0u, 0u);
    sc[k] = 1.f;
    if (from >= 0 && from < p.src_pages) {
      const size_t v = static_cast<size_t>(from) * planes * plane + in + j % 16;
      x[k] = __ldg(reinterpret_cast<const uint4*>(p.src_pool) + v * VEC + piece);
      if (p.src_scales != nullptr && piece == 0) sc[k] = __ldg(p.src_scales + v);
    } else if (piece == 0) {
      raise_status(p.status, DFLASH_ERR_CAPACITY, 585);
    }
    on[k] = dest >= 0 && dest < p.dst_pages;
    to[k] = static_cast<size_t>(dest) * planes * plane + in + i % 16;
  }
#pragma unroll
  for (int k = 0; k < kCopies; ++k) {
    if (!on[k]) continue;
    reinterpret_cast<uint4*>(p.dst_pool)[to[k] * VEC + piece] = x[k];
    if (p.dst_scales != nullptr && piece == 0) p.dst_scales[to[k]] = sc[k];
  }
}

template <int VEC>
void launch_copy(const EvictParams& p, cudaStream_t s) {
  const int64_t rows = kCopyThreads / VEC * (kCopies / p.planes);
  count_launch();
  evict_copy_kernel<VEC><<<dim3(static_cast<unsigned>((p.ld_kept + rows - 1) / rows), p.hkv, p.batch), kCopyThreads, 0, s>>>(p);
}

}  // namespace

cudaError_t kv_evict_launch(const EvictParams& p, int vector_bytes, cudaStream_t s) {
  cudaError_t e = cudaMemsetAsync(p.conflict, 0, 256 + static_cast<size_t>(p.dst_pages) * 4, s);
  if (e != cudaSuccess) return e;
  count_launch();
  evict_check_kernel<<<p.batch, 256, 0, s>>>(p);
  // slices of at least 4096 positions, until the CTAs fill the machine
  int cluster = 1;
  while (cluster < kMaxCluster && static_cast<int64_t>(p.batch) * p.hkv * cluster * 2 <= 152 &&
         p.ld_mass / (2 * cluster) >= 4096)
    cluster *= 2;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.batch) * p.hkv * cluster);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  count_launch();
  e = cudaLaunchKernelEx(&cfg, evict_select_kernel, p, cluster);
  if (e != cudaSuccess) return e;
  if (vector_bytes == 256) launch_copy<16>(p, s);
  else if (vector_bytes == 128) launch_copy<8>(p, s);
  else launch_copy<4>(p, s);
  return cudaGetLastError();
}

}  // namespace dflash
