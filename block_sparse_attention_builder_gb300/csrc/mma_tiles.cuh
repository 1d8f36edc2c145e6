// Pieces that the dense tcgen05 kernels over 128-row tiles share: the two
// products of a block as eight MMAs each, and small helpers of the softmax.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ptx.cuh"

namespace mxsa {

// the largest of three in one instruction (NaN operands are ignored, as by fmaxf)
__device__ __forceinline__ float hmax3(float x, float y, float z) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}

template <bool kBf16>
__device__ __forceinline__ uint32_t hpack2(float a, float b) {
  if (kBf16) {
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
  }
  __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}

__device__ __forceinline__ bool hwarp_all(bool v) { return __all_sync(0xffffffffu, v); }

// eight consecutive floats to global memory (32-byte aligned)
__device__ __forceinline__ void st_global_v8(float* p, const float* v) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
               "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

// One lane of a converged warp, always the same one.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, e;\n\t}"
      : "=r"(p));
  return p != 0;
}

// Low words of the operands' shared-memory descriptors (the high word is the
// same for all: 1024 bytes between groups of 8 rows, version 1, 128-byte
// swizzle); the address field counts 16 bytes and does not overflow below.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_k_major(uint32_t saddr) { return saddr >> 4; }
__device__ __forceinline__ uint32_t desc_mn_major(uint32_t saddr) { return (saddr >> 4) | ((16384u >> 4) << 16); }
// a value that all lanes hold, in a form the compiler knows to be uniform
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }

// The eight products over 16 columns each of one block.  S = q k^T: both
// operands K-major, 64 columns to a 16 KB half, 32 bytes a step.  O (+)= P V:
// P in TMEM, 8 columns a step, V MN-major, 16 rows (2 KB) a step.
template <int kStep>
__device__ __forceinline__ void mma_qk_step(uint32_t d, uint32_t q, uint32_t k, uint32_t idesc) {
  constexpr int off = ((kStep >> 2) * 16384 + (kStep & 3) * 32) >> 4;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b32 u, v;\n\t.reg .b64 x, y;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tadd.u32 u, %1, %5;\n\tadd.u32 v, %2, %5;\n\t"
      "mov.b64 x, {u, %6};\n\tmov.b64 y, {v, %6};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
      "r"(q), "r"(k), "r"(idesc), "n"(kStep > 0), "n"(off), "r"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void mma_qk(uint32_t d, uint32_t q, uint32_t k, uint32_t idesc) {
  mma_qk_step<0>(d, q, k, idesc);
  mma_qk_step<1>(d, q, k, idesc);
  mma_qk_step<2>(d, q, k, idesc);
  mma_qk_step<3>(d, q, k, idesc);
  mma_qk_step<4>(d, q, k, idesc);
  mma_qk_step<5>(d, q, k, idesc);
  mma_qk_step<6>(d, q, k, idesc);
  mma_qk_step<7>(d, q, k, idesc);
}
template <int kStep>
__device__ __forceinline__ void mma_pv_step(uint32_t d, uint32_t tp, uint32_t v, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\t.reg .b32 x, v;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tadd.u32 x, %1, %5;\n\tadd.u32 v, %2, %6;\n\tmov.b64 y, {v, %7};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, p;\n\t}" ::"r"(d),
      "r"(tp), "r"(v), "r"(idesc), "r"(acc), "n"(kStep * 8), "n"(kStep * (2048 >> 4)), "r"(kDescHi)
      : "memory");
}
// the first and the second 64 keys
__device__ __forceinline__ void mma_pv_lo(uint32_t d, uint32_t tp, uint32_t v, uint32_t idesc, uint32_t acc) {
  mma_pv_step<0>(d, tp, v, idesc, acc);
  mma_pv_step<1>(d, tp, v, idesc, 1u);
  mma_pv_step<2>(d, tp, v, idesc, 1u);
  mma_pv_step<3>(d, tp, v, idesc, 1u);
}
__device__ __forceinline__ void mma_pv_hi(uint32_t d, uint32_t tp, uint32_t v, uint32_t idesc) {
  mma_pv_step<4>(d, tp, v, idesc, 1u);
  mma_pv_step<5>(d, tp, v, idesc, 1u);
  mma_pv_step<6>(d, tp, v, idesc, 1u);
  mma_pv_step<7>(d, tp, v, idesc, 1u);
}

// O of the thread's row times f, 16 columns at a time
__device__ __forceinline__ void scale_o(uint32_t tO, float f) {
#pragma unroll 1
  for (int cb = 0; cb < 8; ++cb) {
    uint32_t w[16];
    tmem_ld16(tO + cb * 16, w);
    tmem_ld_wait();
#pragma unroll
    for (int k = 0; k < 16; ++k) w[k] = __float_as_uint(__uint_as_float(w[k]) * f);
    tmem_st16(tO + cb * 16, w);
  }
}

// The largest of 64.
__device__ __forceinline__ float max64(const float* sv) {
  float b0 = -INFINITY, b1 = -INFINITY;
#pragma unroll
  for (int k = 0; k < 64; k += 4) {
    b0 = hmax3(b0, sv[k], sv[k + 1]);
    b1 = hmax3(b1, sv[k + 2], sv[k + 3]);
  }
  return fmaxf(b0, b1);
}

// How large the P of 64 keys may be before the reference m is raised.  Their sum,
// which is there anyway, stands for their maximum (it is within 2^6 of it).  In
// the second half of a block, where raising has to wait for a product, the limit
// is what fp16 holds: what is left so is found in the next block's first half.
constexpr float kSumLow = 1024.f, kSumHigh = 16384.f;
// How far (log2 units) the maximum may be above m where it is found anyway, and
// where such a sum asked for it: there less than the 2^4 that kSumLow says, so that
// P are made twice once and not in every block.
constexpr float kGapKnown = 8.f, kGapSum = 3.f;

// P = 2^(S * scale - m) of 64 keys of a row, packed, to TMEM; returns their sum.
template <bool kBf16>
__device__ __forceinline__ float exp_half(const float* sv, float scale_log2, float m, uint32_t tP) {
  const uint64_t scale2 = pack_f2(scale_log2, scale_log2), off2 = pack_f2(-m, -m);
  uint64_t l0 = pack_f2(0.f, 0.f), l1 = l0;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    uint32_t pk[16];
    float2 x[16];
#pragma unroll
    for (int k = 0; k < 16; ++k)
      x[k] = unpack_f2(fma_f2(pack_f2(sv[32 * q + 2 * k], sv[32 * q + 2 * k + 1]), scale2, off2));
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      x[k].x = ex2_approx(x[k].x);
      x[k].y = ex2_approx(x[k].y);
    }
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      if (k & 1) l1 = add_f2(l1, pack_f2(x[k].x, x[k].y));
      else l0 = add_f2(l0, pack_f2(x[k].x, x[k].y));
      pk[k] = hpack2<kBf16>(x[k].x, x[k].y);
    }
    tmem_st16(tP + 16 * q, pk);
  }
  const float2 ls = unpack_f2(add_f2(l0, l1));
  return ls.x + ls.y;
}

// Which of keys o .. o + 31 a row of a drafted tree sees, as bits; keys are
// numbered from the first drafted one, those before it are seen by all.  row:
// the token's mask, not read where o <= -32.
__device__ __forceinline__ uint32_t tree_bits(const uint32_t* row, int words, int o) {
  if (o <= -32) return 0xFFFFFFFFu;
  auto word = [&](int w) { return w < words ? __ldg(row + w) : 0u; };
  if (o < 0) return (word(0) << -o) | ((1u << -o) - 1);
  return __funnelshift_r(word(o >> 5), (o & 31) ? word((o >> 5) + 1) : 0u, o & 31);
}

}  // namespace mxsa
