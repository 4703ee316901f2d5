// What the tcgen05 products share: the tile geometry, the bit-exact fp16x2 dequantisation of a
// code pair, and the tensor maps of the packed layout.
#pragma once
#include "owq_dequant.cuh"
#include "owq_internal.cuh"
#include "owq_sm100.cuh"

namespace owq {
namespace {

constexpr int kBM = 128;               // weight rows per tile (MMA M)
constexpr int kStepCodes = 128;        // K per pipeline step
// tensor-memory columns of a CTA: the accumulator (BN) + S A stages of 64, as a power of two;
// 256 lets two CTAs share an SM
template <int BN, int S>
constexpr uint32_t tmem_cols() { return BN + 64 * S <= 256 ? 256u : 512u; }

template <int BITS, int BN>
struct Smem {
  static constexpr int kX = 2 * BN * 128;           // two 64-column swizzled activation boxes
  static constexpr int kP = kBM * 16 * BITS;        // packed tile
  static constexpr int kSZ = kBM * 4;               // (scale, zero) pairs of the step (per-group layers)
  static constexpr int kStage = ((kX + kP + kSZ) + 1023) & ~1023;
};

template <int BITS, int BN, int S>
constexpr int smem_bytes() { return S * Smem<BITS, BN>::kStage + 1024 /*barriers*/ + 1024 /*align slack*/; }

__device__ __forceinline__ uint32_t h2_splat(float v) {
  __half h = __float2half_rn(v);
  uint32_t u = __half_as_ushort(h);
  return u | (u << 16);
}

// fp16_rn(s (q - z)) of pair j of a chunk (both halves).  The pair is lifted as
// (bits | 0x6400) = 1024 + q 2^o per half, then (1024 + q 2^o) * 2^-o - (1024 2^-o + z) = q - z
// exactly (one fma.rn.f16x2), then * s rounds once: bit-exact with the definition.
template <int BITS>
__device__ __forceinline__ uint32_t dequant_pair(const uint32_t* w, int j, uint32_t s2, const uint32_t* scl,
                                                 const uint32_t* nz) {
  constexpr uint32_t kMagic = 0x64006400u;
  const int c = pair_class<BITS>(j);
  return h2_mul(h2_fma(pair_bits<BITS>(w, j) | kMagic, scl[c], nz[c]), s2);
}

// ---- tensor maps (host) ----
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled get_encoder() {
  static EncodeTiled fn = nullptr;
  if (!fn) {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiled>(f);
  }
  return fn;
}

bool encode_2d(CUtensorMap* m, CUtensorMapDataType dt, const void* base, uint64_t inner, uint64_t outer,
               uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle sw) {
  EncodeTiled enc = get_encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {inner, outer};
  const cuuint64_t strides[1] = {row_bytes};
  const cuuint32_t box[2] = {box_inner, box_outer};
  const cuuint32_t estr[2] = {1, 1};
  return enc(m, dt, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, sw,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_packed_3d(CUtensorMap* m, const void* base, int K, int N, int bits, int tiles = kBM / 16) {
  EncodeTiled enc = get_encoder();
  if (!enc) return false;
  const int Kb = K / kStepCodes;
  const uint64_t tile_blk = 16ull * 16 * bits;          // bytes of one block of a 16-row tile
  const cuuint64_t dims[3] = {tile_blk / 4, (cuuint64_t)Kb, (cuuint64_t)((N + 15) / 16)};
  const cuuint64_t strides[2] = {tile_blk, tile_blk * Kb};
  const cuuint32_t box[3] = {(cuuint32_t)(tile_blk / 4), 1, (cuuint32_t)tiles};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// (scale, zero) pairs of the 16-row tiles, tile-major [RT][G][16] 32-bit words: one box is
// the pairs of one group for `tiles` tiles
bool encode_sz_3d(CUtensorMap* m, const void* base, int G, int N, int tiles = kBM / 16) {
  EncodeTiled enc = get_encoder();
  if (!enc) return false;
  const cuuint64_t dims[3] = {16, (cuuint64_t)G, (cuuint64_t)((N + 15) / 16)};
  const cuuint64_t strides[2] = {64, 64ull * G};
  const cuuint32_t box[3] = {16, 1, (cuuint32_t)tiles};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace owq
