// What the tcgen05 products share: the tile geometry, the bit-exact fp16x2 dequantisation of a
// code pair, and the tensor maps of the packed layout.
#pragma once
#include "owq_format.cuh"
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

// ---- input gradient (W_hat^T as the A operand) ----
// Stage layout: the prefill's (dY boxes, packed block, (s, z) pairs), then what the prep warp
// derives from them.  The prep warp rewrites the packed block in place with the two rows of
// each row pair interleaved word by word ([64 pairs][4 bits words] of {row 2P, row 2P + 1}),
// rebuilds the 3-bit pair whose bits are spread over a chunk's three words as an ordinary word
// pair ([64 pairs][4 chunks], even code at bits 6-8, odd at 22-24) and writes per row pair and
// offset class {s2, -(1024 2^-o + z2)}.
template <int BITS, int BN>
struct IgSmem {
  static constexpr int kX = Smem<BITS, BN>::kX, kP = Smem<BITS, BN>::kP, kSZ = Smem<BITS, BN>::kSZ;
  static constexpr int kTma = kX + kP + kSZ;
  static constexpr int kCls = BITS == 3 ? 5 : 2;              // code offsets 0, 3, 6, 1, 4 / 0, 4
  static constexpr int kAuxD = BITS == 3 ? 64 * 4 * 8 : 0;    // [64 pairs][4 chunks] uint2
  static constexpr int kAuxS = 64 * kCls * 8;                 // [64 pairs][classes] {s2, nz2}
  static constexpr int kStage = ((kTma + kAuxD + kAuxS) + 1023) & ~1023;
};
// class of a code offset (after the byte shift): 3-bit 0, 3, 6, 1, 4 -> 0..4; 4-bit 0, 4 -> 0, 1
template <int BITS>
__host__ __device__ constexpr int ig_off_cls(int o) {
  return BITS == 3 ? (o == 0 ? 0 : o == 3 ? 1 : o == 6 ? 2 : o == 1 ? 3 : 4) : o / 4;
}
template <int BITS>
__host__ __device__ constexpr int ig_cls_off(int c) {
  return BITS == 3 ? (c == 0 ? 0 : c == 1 ? 3 : c == 2 ? 6 : c == 3 ? 1 : 4) : 4 * c;
}
template <int BITS, int BN, int S>
constexpr int ig_smem_bytes() { return S * IgSmem<BITS, BN>::kStage + 1024 /*barriers*/ + 1024 /*align slack*/; }

// The prep warp's work on one landed step (st: shared address of the stage).
template <int BITS, int BN>
__device__ __forceinline__ void ig_prep_step(uint32_t st, int lane) {
  using namespace sm100;
  using L = IgSmem<BITS, BN>;
  constexpr int W = 4 * BITS;   // words of a row's block
  #pragma unroll 1
  for (int P = lane; P < 64; P += 32) {   // one row pair per lane and pass
    uint32_t a[W], c[W];
    const uint32_t ra = st + L::kX + (2 * P) * 16 * BITS;
    #pragma unroll
    for (int v = 0; v < BITS; ++v) {
      const uint4 x = lds_u4(ra + 16 * v), y = lds_u4(ra + 16 * (BITS + v));
      a[4 * v] = x.x; a[4 * v + 1] = x.y; a[4 * v + 2] = x.z; a[4 * v + 3] = x.w;
      c[4 * v] = y.x; c[4 * v + 1] = y.y; c[4 * v + 2] = y.z; c[4 * v + 3] = y.w;
    }
    if constexpr (BITS == 3) {   // bit e of the spread pair: bit 15 / 31 of word e -> 6 + e / 22 + e
      const uint32_t aux_d = st + L::kTma + 32 * P;
      #pragma unroll
      for (int qc = 0; qc < 4; ++qc) {
        const uint32_t* x = a + 3 * qc;
        const uint32_t* y = c + 3 * qc;
        sts_u2(aux_d + 8 * qc,
               make_uint2(((x[0] >> 9) & 0x00400040u) | ((x[1] >> 8) & 0x00800080u) | ((x[2] >> 7) & 0x01000100u),
                          ((y[0] >> 9) & 0x00400040u) | ((y[1] >> 8) & 0x00800080u) | ((y[2] >> 7) & 0x01000100u)));
      }
    }
    #pragma unroll
    for (int v = 0; v < W / 2; ++v)   // the pair's own bytes, rows interleaved word by word
      sts_u4(ra + 16 * v, make_uint4(a[2 * v], c[2 * v], a[2 * v + 1], c[2 * v + 1]));
    const uint2 z = lds_u2(st + L::kX + L::kP + 8 * P);   // (s, z) of rows 2P, 2P + 1
    const uint32_t s2 = __byte_perm(z.x, z.y, 0x5410), z2 = __byte_perm(z.x, z.y, 0x7632);
    const uint32_t aux_s = st + L::kTma + L::kAuxD + 8 * L::kCls * P;
    #pragma unroll
    for (int cl = 0; cl < L::kCls; ++cl) {
      const uint32_t nego = (0x8000u | ((uint32_t)(25 - ig_cls_off<BITS>(cl)) << 10)) * 0x00010001u;   // -2^(10 - o)
      sts_u2(aux_s + 8 * cl, make_uint2(s2, h2_sub(nego, z2)));
    }
  }
}

// One column j of the block as a row of the A operand W_hat^T: where its codes sit and how a row
// pair's words become fp16_rn(s (q - z)).
template <int BITS, int BN>
struct IgColumn {
  using L = IgSmem<BITS, BN>;
  uint32_t sel, mask, sc;
  int woff, pstride, cls;
  __device__ __forceinline__ explicit IgColumn(int j) {
    const int pj = j >> 1, q = pj & 3, jj = pj >> 2, h = j & 1;
    const bool spread = BITS == 3 && jj == 11;
    // the slot of pair jj (the 3-bit table of owq_format.cuh as packed fields: word, offset / 3)
    const Slot sl = spread ? Slot{0, 6}
                  : BITS == 3 ? Slot{(int)((0xaa244444u >> (2 * jj)) & 3u), 3 * (int)((0x3041024433221100ull >> (4 * jj)) & 15u)}
                              : Slot{2 * (jj / 8) + (jj % 2), 4 * ((jj % 8) / 2)};
    const bool hi8 = !spread && sl.off >= 8;
    const int o2 = hi8 ? sl.off - 8 : sl.off;
    sel = h ? (hi8 ? 0x7733u : 0x7632u) : (hi8 ? 0x5511u : 0x5410u);
    const uint32_t m1 = ((1u << BITS) - 1u) << o2;
    mask = m1 | (m1 << 16);
    sc = ((uint32_t)(15 - o2) << 10) * 0x00010001u;                // 2^-o
    // column j's word pair (rows 2P, 2P + 1) in each row pair: the interleaved packed block, or
    // for the spread pair the prep warp's rebuilt pair (then at offset 6, the unshifted half)
    woff = spread ? L::kTma + 8 * q : L::kX + 8 * (q * BITS + sl.word);
    pstride = spread ? 32 : 32 * BITS;
    cls = ig_off_cls<BITS>(o2);
  }
  // rows 2P, 2P + 1 of row pairs P = first .. first + RP - 1
  template <int RP>
  __device__ __forceinline__ void operand(uint32_t st, int first, uint32_t (&d)[RP]) const {
    using namespace sm100;
    const uint32_t pk = st + woff + first * pstride;
    const uint32_t snp = st + L::kTma + L::kAuxD + 8 * (L::kCls * first + cls);
    #pragma unroll
    for (int pr = 0; pr < RP; ++pr) {
      const uint2 w = lds_u2(pk + pr * pstride);
      const uint32_t v = (__byte_perm(w.x, w.y, sel) & mask) | 0x64006400u;
      const uint2 sn = lds_u2(snp + 8 * L::kCls * pr);   // {s2, -(1024 2^-o + z2)} of the pair
      d[pr] = h2_mul(h2_fma(v, sc, sn.y), sn.x);   // fp16_rn(s (q - z))
    }
  }
};

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
