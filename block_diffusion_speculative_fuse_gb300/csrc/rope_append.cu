// Rotation of q and k by their positions and append of k, v to the paged
// cache, in one launch.
//
// For every head vector x of a row at position pos (after an optional RMSNorm
// with a gain): pair p of its first rot_dim components turns by
// phi = pos * f_p,
//   (a, b) -> mscale * (a cos phi - b sin phi, a sin phi + b cos phi),
// the pair being (p, p + rot/2) or, interleaved, (2p, 2p+1).
//
// The angle: f_p / 2pi is held as a 64-bit fraction of a turn, so that
// pos * f_p modulo one turn is one integer multiplication modulo 2^64, exact
// up to the fraction's last bit (2^-64 of a turn per position); the upper 32
// bits, as a float in half turns, go to sincospif.  The error (2e-7 rad) is
// that of the conversion to float at any position (2^30 of them: 2^-34 of a
// turn, 4e-10 rad, more).
//
// Bound: bytes.  Each thread owns two 16-byte pieces (of bf16) of a head
// vector, chosen so that both members of its eight pairs are its own: no
// exchange but the row sums of the norm (and the maximum for an E4M3 scale)
// among the head's D/16 threads.  One CTA of 128 threads per row, eight to an SM;
// the row's sines and cosines are made while its first loads are on their way,
// once for all heads, and passed through shared memory.  8192 rows of 32 + 8 + 8
// heads of 128: bf16 37 us, 5.4 TB/s; fp32 47 us, 6.4 TB/s (four CTAs to an SM 56
// us; loads of up to four head vectors ahead of the work on them no faster).  Whole
// calls: bf16 40 us, into an E4M3 cache 46, of fp32 52, into two terms 54.  A
// row alone: 3 us, the latency of its two dependent loads and a launch.
#include "common.cuh"
#include "kernels.h"

namespace dflash {

namespace {

constexpr int kThreads = 128;

// 8 consecutive elements, as loaded and as floats
template <typename In>
struct Raw8;
template <>
struct Raw8<uint16_t> {
  uint4 v;
  __device__ __forceinline__ void load(const uint16_t* p) { v = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[2 * j] = __uint_as_float(w[j] << 16);
      x[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  }
};
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p + 4));
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
};
__device__ __forceinline__ void load8(const uint16_t* p, float (&x)[8]) {
  Raw8<uint16_t> r;
  r.v = __ldg(reinterpret_cast<const uint4*>(p));
  r.get(x);
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(bf16x2(x[0], x[1]), bf16x2(x[2], x[3]),
                                            bf16x2(x[4], x[5]), bf16x2(x[6], x[7]));
}
// the low terms bf16(x - bf16(x))
__device__ __forceinline__ void store8_lo(uint16_t* p, const float (&x)[8]) {
  float y[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) y[j] = x[j] - bf2f(f2bf(x[j]));
  store8(p, y);
}

template <int D, typename In>
__global__ void __launch_bounds__(kThreads, 8) rope_append_kernel(const __grid_constant__ RopeAppendParams p) {
  constexpr int TPH = D / 16;          // threads per head vector
  constexpr int HPR = kThreads / TPH;  // head vectors per round
  // (cos, sin) of pair 8 s + 2 i + b at [i][s][b]: thread s of a head reads its
  // eight pairs as four vectors, neighbours next to each other
  __shared__ float4 cs[4][8];
  griddep_launch_dependents();
  griddep_wait();
  const int t = blockIdx.x;
  const int rot = p.rot_dim, half = rot / 2;
  const int heads_q = p.q != nullptr ? p.hq : 0;
  const int heads = heads_q + 2 * p.hkv;
  // the two 8-element pieces of this thread: a rotated pair of pieces, or two
  // neighbours (interleaved pairs, and everything past rot_dim)
  const int sub = threadIdx.x % TPH;
  const bool split = !p.interleaved && sub < rot / 16;
  const int c0 = (split ? sub : 2 * sub) * 8;
  const int c1 = split ? c0 + half : c0 + 8;
  const int pos = __ldcg(p.row_pos + t), req = __ldcg(p.row_req + t);

  bool first = true;
  long long page = -1;
  // all threads of the CTA run the same number of rounds (barrier, shuffles)
  for (int h0 = 0; h0 < heads; h0 += HPR) {
    const int head = h0 + threadIdx.x / TPH;
    const bool on = head < heads;
    const bool is_q = head < heads_q;
    const int hk = head - heads_q;
    const bool is_v = !is_q && hk >= p.hkv;
    const int h = is_q ? head : is_v ? hk - p.hkv : hk;
    Raw8<In> r0, r1;
    if (on) {
      const In* src = is_q   ? static_cast<const In*>(p.q) + t * p.ld_q + h * D
                      : is_v ? static_cast<const In*>(p.v) + t * p.ld_v + h * D
                             : static_cast<const In*>(p.k) + t * p.ld_k + h * D;
      r0.load(src + c0);
      r1.load(src + c1);
    }
    if (first) {
      first = false;
      if (pos < 0) return;  // the whole CTA
      // where the row's K and V go
      if (req >= 0 && req < p.n_req && pos / 16 < p.max_pages)
        page = __ldcg(p.page_table + static_cast<size_t>(req) * p.max_pages + pos / 16);
      if (page >= p.n_pages) page = -1;
      if (page < 0 && threadIdx.x == 0) raise_status(p.status, DFLASH_ERR_CAPACITY, 501);
      if (threadIdx.x < half) {
        const unsigned long long phase = static_cast<unsigned long long>(pos) * p.turns[threadIdx.x];
        float s, c;
        sincospif(static_cast<float>(static_cast<int>(phase >> 32)) * 0x1p-31f, &s, &c);
        const int pair = threadIdx.x;
        reinterpret_cast<float2*>(&cs[pair / 2 % 4][pair / 8])[pair % 2] = make_float2(c * p.mscale, s * p.mscale);
      }
      __syncthreads();
    }
    float x[8], y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = y[j] = 0.f;
    if (on) {
      r0.get(x);
      r1.get(y);
    }
    const uint16_t* gain = is_v ? nullptr : is_q ? p.q_norm : p.k_norm;
    if (p.q_norm != nullptr || p.k_norm != nullptr) {
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], fmaf(y[j], y[j], ss));
#pragma unroll
      for (int o = TPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (gain != nullptr) {
        const float r = rsqrtf(ss * (1.f / D) + p.eps);
        float g0[8], g1[8];
        load8(gain + c0, g0);
        load8(gain + c1, g1);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          x[j] = x[j] * r * g0[j];
          y[j] = y[j] * r * g1[j];
        }
      }
    }
    if (!is_v && sub < (half + 7) / 8) {
      float2 w[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 v = cs[i][sub];
        w[2 * i] = make_float2(v.x, v.y);
        w[2 * i + 1] = make_float2(v.z, v.w);
      }
      if (split) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float a = x[j], b = y[j];
          x[j] = a * w[j].x - b * w[j].y;
          y[j] = fmaf(a, w[j].y, b * w[j].x);
        }
      } else if (p.interleaved) {
        // rot_dim is a multiple of 16: all of a thread's pairs turn, or none
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const float a = x[j], b = x[j + 1], c = y[j], d = y[j + 1];
          const float2 u0 = w[j / 2], u1 = w[4 + j / 2];
          x[j] = a * u0.x - b * u0.y;
          x[j + 1] = fmaf(a, u0.y, b * u0.x);
          y[j] = c * u1.x - d * u1.y;
          y[j + 1] = fmaf(c, u1.y, d * u1.x);
        }
      }
    }
    if (on && is_q) {
      uint16_t* o = p.q_out + t * p.ld_qo + h * D;
      store8(o + c0, x);
      store8(o + c1, y);
    }
    if (p.pool8 != nullptr) {
      // E4M3 codes of the bf16-rounded vector, scale = amax / 448 (1 for a
      // zero vector), the code decided from the fp32 quotient
      float am = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        x[j] = bf2f(f2bf(x[j]));
        y[j] = bf2f(f2bf(y[j]));
        am = fmaxf(am, fmaxf(fabsf(x[j]), fabsf(y[j])));
      }
#pragma unroll
      for (int o = TPH / 2; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
      if (on && !is_q && page >= 0) {
        const float scale = am > 0.f ? am / 448.f : 1.f;
        const size_t vec = ((static_cast<size_t>(page) * 2 + (is_v ? 1 : 0)) * p.hkv + h) * 16 + pos % 16;
        uint32_t a[2], b[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          a[j] = e4m3x2_encode(x[4 * j] / scale, x[4 * j + 1] / scale) |
                 (static_cast<uint32_t>(e4m3x2_encode(x[4 * j + 2] / scale, x[4 * j + 3] / scale)) << 16);
          b[j] = e4m3x2_encode(y[4 * j] / scale, y[4 * j + 1] / scale) |
                 (static_cast<uint32_t>(e4m3x2_encode(y[4 * j + 2] / scale, y[4 * j + 3] / scale)) << 16);
        }
        *reinterpret_cast<uint2*>(p.pool8 + vec * D + c0) = make_uint2(a[0], a[1]);
        *reinterpret_cast<uint2*>(p.pool8 + vec * D + c1) = make_uint2(b[0], b[1]);
        if (sub == 0) p.scales8[vec] = scale;
      }
    } else if (on && !is_q && page >= 0) {
      const int planes = 2 * p.kv_terms;
      uint16_t* o = p.pool + (((static_cast<size_t>(page) * planes + (is_v ? 1 : 0)) * p.hkv + h) * 16 +
                              pos % 16) * D;
      store8(o + c0, x);
      store8(o + c1, y);
      if (p.kv_terms == 2) {
        o += static_cast<size_t>(2) * p.hkv * 16 * D;
        store8_lo(o + c0, x);
        store8_lo(o + c1, y);
      }
    }
  }
}

template <int D, typename In>
cudaError_t launch_append(const RopeAppendParams& p, cudaStream_t s) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.T);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  count_launch();
  return cudaLaunchKernelEx(&cfg, rope_append_kernel<D, In>, p);
}

}  // namespace

cudaError_t rope_append_launch(const RopeAppendParams& p, int d, bool fp32, cudaStream_t s) {
  if (d == 128) return fp32 ? launch_append<128, float>(p, s) : launch_append<128, uint16_t>(p, s);
  return fp32 ? launch_append<64, float>(p, s) : launch_append<64, uint16_t>(p, s);
}

}  // namespace dflash
