// Shared by the tcgen05 kernels over the paged cache: matrix descriptors, products
// with an operand in TMEM, packed fp32 arithmetic, the ring's cursor, page loads.
#pragma once
#include "common.cuh"

namespace dflash {

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Whether one of eight bf16 is infinite or NaN: the carry out of a full exponent.
__device__ __forceinline__ bool bf16_not_finite(uint4 v) {
  auto full = [](uint32_t w) { return (w & 0x7F807F80u) + 0x00800080u; };
  return ((full(v.x) | full(v.y) | full(v.z) | full(v.w)) & 0x80008000u) != 0u;
}

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
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("mul.rn.f32x2 %0, %1, %2;"
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

// 16 columns: loaded (and waited for), stored (no wait).
__device__ __forceinline__ void tmem_ld16_raw(uint32_t taddr, uint32_t (&r)[16]) {
  float v[16];
  tmem_ld16(taddr, v);
#pragma unroll
  for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(v[i]);
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
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

// Of a V plane of 128 keys, [8-row group][column half][8 rows][128 B] (one warp): makes the keys [first, live) finite and those from live
// to the end of its page zero.  The lane's first key that was not finite, else
// 128.
template <int D>
__device__ __forceinline__ int clean_v(uint8_t* plane, int first, int live) {
  constexpr int HALVES = D / 64, PIECES = HALVES * 8;  // 16-byte pieces of a key
  auto piece = [&](int i) {
    const int key = i / PIECES, half = i / 8 % HALVES;
    return reinterpret_cast<uint4*>(plane + (key / 8) * (HALVES * 1024) + half * 1024 + (key % 8) * 128 +
                                    (((i ^ key) & 7) << 4));
  };
  const int lane = threadIdx.x % 32;
  const int i0 = max(first, 0) * PIECES + lane, i1 = min(live, 128) * PIECES;
  bool found = false;
#pragma unroll 2
  for (int i = i0; i < i1; i += 32) found |= bf16_not_finite(*piece(i));
  int bad = 128;
  if (__any_sync(0xffffffffu, found)) {
#pragma unroll 1
    for (int i = i0; i < i1; i += 32) {
      if (!bf16_not_finite(*piece(i))) continue;
      bad = min(bad, i / PIECES);
      *piece(i) = make_uint4(0u, 0u, 0u, 0u);
    }
  }
#pragma unroll 1
  for (int i = max(live, 0) * PIECES + lane; i < min((live + 15) & ~15, 128) * PIECES; i += 32)
    *piece(i) = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  __syncwarp();
  return bad;
}

}  // namespace dflash
