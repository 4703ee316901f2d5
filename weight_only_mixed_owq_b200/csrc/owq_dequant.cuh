// fp16x2 arithmetic, and the bit-exact dequantisation of code pairs in registers that the gated block's
// kernels use: a pair of neighbouring codes of a row -> fp16x2 W_hat = fp16_rn(s (q - z)).
//
// The pair is lifted as (bits | 0x6400) per half, the fp16 value 1024 + q 2^o (o: the code's bit
// offset); times 2^-o plus -(1024 2^-o + z) is q - z exactly (one fma.rn.f16x2), and the product
// with s rounds once.  Selecting the bits and setting the exponent is one three-input logic
// operation; with the shared shifts a pair costs about 3.3 instructions.
#pragma once
#include "owq_format.cuh"

namespace owq {
namespace {

// fp16x2 helpers (exact integer arithmetic on small values)
__device__ __forceinline__ uint32_t h2_fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t h2_mul(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t h2_sub(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t mask, uint32_t c) {   // (a & mask) | c
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(mask), "r"(c));
  return d;
}

// Pair j of a chunk with the fp16 exponent of 1024: (bits | 0x6400) in each half, the codes at
// offset class_off(pair_class(j)).
template <int BITS>
__device__ __forceinline__ uint32_t pair_lifted(const uint32_t* w, int j) {
  constexpr uint32_t kMagic = 0x64006400u;
  if constexpr (BITS == 3) {
    constexpr uint32_t m0 = 0x00070007u, m1 = 0x00380038u, m2 = 0x01C001C0u;
    switch (j) {
      case 0: return and_or(w[0], m0, kMagic);
      case 1: return and_or(w[1], m0, kMagic);
      case 2: return and_or(w[0], m1, kMagic);
      case 3: return and_or(w[1], m1, kMagic);
      case 4: return and_or(w[0], m2, kMagic);
      case 5: return and_or(w[1], m2, kMagic);
      case 6: return and_or(w[0] >> 9, m0, kMagic);
      case 7: return and_or(w[1] >> 9, m0, kMagic);
      case 8: return and_or(w[0] >> 9, m1, kMagic);
      case 9: return and_or(w[1] >> 9, m1, kMagic);
      case 10: return and_or(w[2], m2, kMagic);
      case 11:   // the spread pair: bit e of its codes in bits 15 and 31 of word e
        return and_or(w[2] >> 7, 0x01000100u, and_or(w[1] >> 8, 0x00800080u, and_or(w[0] >> 9, 0x00400040u, kMagic)));
      case 12: return and_or(w[2], m1, kMagic);
      case 13: return and_or(w[2] >> 9, m1, kMagic);
      case 14: return and_or(w[2], m0, kMagic);
      default: return and_or(w[2] >> 9, m0, kMagic);
    }
  } else {
    const uint32_t v = w[2 * (j / 8) + (j % 2)];
    switch ((j % 8) / 2) {
      case 0: return and_or(v, 0x000F000Fu, kMagic);
      case 1: return and_or(v, 0x00F000F0u, kMagic);
      case 2: return and_or(v >> 8, 0x000F000Fu, kMagic);
      default: return and_or(v >> 8, 0x00F000F0u, kMagic);
    }
  }
}

// A row's constants: the scale splat and, per offset class c, -(1024 2^-o_c + z).
template <int BITS>
struct RowDq {
  static constexpr int kNC = BITS == 3 ? 3 : 2;
  uint32_t s2, nz[kNC];
  __device__ __forceinline__ void set(uint32_t sz) {   // scale in the low half, zero in the high
    s2 = __byte_perm(sz, sz, 0x1010);
    const uint32_t z2 = __byte_perm(sz, sz, 0x3232);
    #pragma unroll
    for (int c = 0; c < kNC; ++c)   // -2^(10 - o) as fp16, both halves
      nz[c] = h2_sub((0x8000u | ((uint32_t)(25 - class_off<BITS>(c)) << 10)) * 0x00010001u, z2);
  }
};

template <int BITS>
__device__ __forceinline__ uint32_t dequant(const uint32_t* w, int j, const RowDq<BITS>& dq) {
  const int c = pair_class<BITS>(j);
  const uint32_t scl = ((uint32_t)(15 - class_off<BITS>(c)) << 10) * 0x00010001u;   // 2^-o
  return h2_mul(h2_fma(pair_lifted<BITS>(w, j), scl, dq.nz[c]), dq.s2);
}

}  // namespace
}  // namespace owq
