// Gated block for many tokens on the 5th-generation tensor cores, and its backward pass.
//
//   forward    g = x Wg^T, u = x Wu^T (W = the dequantised matrix with its weak columns in fp16),
//              h = a(g) u
//   backward   du = dh a(g), dg = dh u a'(g), with g and u recomputed from x;
//              dx = dg Wg + du Wu, both terms in one fp32 accumulator
//
// Both kernels are the prefill and input-gradient pipelines (TMA ring, A operand dequantised
// into tensor memory, tcgen05.mma with an fp32 accumulator), fed from two layers.  Every
// projection is kept in fp32 until the activation; h, dg and du are rounded to fp16 once (the
// type that activations and gradients have at every layer boundary of this library), dx once.
//
// Bound: the tensor cores from about 200 tokens (4 M N K flops forward, 8 M N K backward), the
// packed weights' bytes below.
#include <algorithm>
#include <type_traits>

#include "owq_act.cuh"
#include "owq_gemm_common.cuh"
#include "owq_mma.cuh"

namespace owq {
namespace {

using namespace sm100;

constexpr int kHalfRows = kBM / 2;     // output rows of a tile: 64 of each layer

struct GatedMaps {
  CUtensorMap x, p[2], xw[2], sz[2];   // [0] gate, [1] up
};
struct GatedGemmParams {
  const __half* scales[2];   // per-channel layers: read once per row (per-group: staged by TMA)
  const __half* zeros[2];
  const __half* w_weak[2];   // weak blocks [N][k_ld]
  int k_ld[2];               // 0: no weak columns
  const __half* dh;          // NULL: forward
  __half* out[2];            // forward: h; backward: dg, du
  float* ws;                 // split partials [split][gate, up][token - ws_t0][N]
  size_t ws_plane;           // one plane, (M - ws_t0) N floats
  int ws_t0;
  int* status;
  int N, K, M, G, act;
  int ksteps;                           // dense steps per split (blockIdx.z)
  int tail_y0, tail_sp, tail_ksteps;    // split tail, as in the prefill product
  int nw;                               // weak steps: 64 columns of each layer's weak block
  long long wait_limit;
  int skip_arrive;
};

// outputs of one element; gs, us: both projections
__device__ __forceinline__ void gated_store(const GatedGemmParams& p, size_t o, float gs, float us) {
  if (p.dh == nullptr) {
    p.out[0][o] = __float2half_rn(act_value(p.act, gs) * us);
  } else {
    float a, da;
    act_both(p.act, gs, a, da);
    const float dh = __half2float(p.dh[o]);
    p.out[0][o] = __float2half_rn(dh * us * da);
    p.out[1][o] = __float2half_rn(dh * a);
  }
}

// The prefill kernel over interleaved rows: MMA rows 32 q .. 32 q + 15 are gate rows n0 + 16 q ..,
// rows 32 q + 16 .. 32 q + 31 the up rows of the same outputs.  Lanes l and l + 16 of a warp then
// hold both projections of one output, so the epilogue pairs them with a shuffle; half of the
// columns are finished by either lane.  Weak step w: columns 64 w .. 64 w + 63 of the gate's weak
// block against its gathered activations in the first half of the step's K, the up layer's in the
// second half, each with zeros in the other layer's rows.
template <int BITS, int BN, int S, int DW, bool TAIL>
__global__ void __launch_bounds__(32 * (2 + DW), 1)
k_gated_gemm(const __grid_constant__ GatedMaps maps, const __grid_constant__ GatedGemmParams p) {
  using L = Smem<BITS, BN>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S * L::kStage);
  uint64_t* full = bars;            // [S] TMA landed
  uint64_t* empty = bars + S;       // [S] MMAs of the stage done
  uint64_t* afull = bars + 2 * S;   // [S] A tile written to tensor memory
  uint64_t* accf = bars + 3 * S;    // accumulator complete
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 3 * S + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int ty = blockIdx.y, sp = blockIdx.z, nsp = gridDim.z, ksteps = p.ksteps;
  if constexpr (TAIL) {
    if (ty >= p.tail_y0) {
      const int u = ty - p.tail_y0;
      ty = p.tail_y0 + u / p.tail_sp;
      sp = u % p.tail_sp;
      nsp = p.tail_sp;
      ksteps = p.tail_ksteps;
    }
  }
  const int n0 = blockIdx.x * kHalfRows;   // first output row
  const int m0 = ty * BN;                  // first token
  const int kb0 = sp * ksteps;
  const int nD = max(0, min(ksteps, p.K / kStepCodes - kb0));   // dense steps of this split
  const int nK = nD + (sp == nsp - 1 ? p.nw : 0);               // + the weak steps (last split)
  const bool per_group = p.G > 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&afull[s], 32 * DW);
    }
    mbar_init(accf, 1);
    fence_mbar_init();
    prefetch_tmap(&maps.x);
    prefetch_tmap(&maps.p[0]);
    prefetch_tmap(&maps.p[1]);
  }
  if (warp == 1) tmem_alloc(tmem_slot, tmem_cols<BN, S>());
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      // ---------------- TMA producer ----------------
      const uint32_t kDense = L::kX + L::kP + (per_group ? L::kSZ : 0);
      bool ok = true;
      int issued = 0;
      for (int i = 0; i < nK && ok; ++i) {
        const int s = i % S, u = i / S;
        if (u > 0) ok = mbar_wait(&empty[s], (u - 1) & 1, p.status, p.wait_limit);
        if (!ok) break;
        unsigned char* st = smem + s * L::kStage;
        if (i < nD) {
          const int kb = kb0 + i;
          mbar_arrive_expect_tx(&full[s], kDense);
          #pragma unroll
          for (int l = 0; l < 2; ++l) {
            tma_load_3d(st + L::kX + l * (L::kP / 2), &maps.p[l], &full[s], 0, kb, n0 / 16);
            if (per_group) tma_load_3d(st + L::kX + L::kP + l * (L::kSZ / 2), &maps.sz[l], &full[s], 0, kb, n0 / 16);
          }
          tma_load_2d(st, &maps.x, &full[s], kb * kStepCodes, m0);
          tma_load_2d(st + BN * 128, &maps.x, &full[s], kb * kStepCodes + 64, m0);
        } else {
          const int c0 = (i - nD) * 64;
          mbar_arrive_expect_tx(&full[s], L::kX);
          tma_load_2d(st, &maps.xw[0], &full[s], c0, m0);
          tma_load_2d(st + BN * 128, &maps.xw[1], &full[s], c0, m0);
        }
        issued = i + 1;
      }
      // never leave with copies in flight: wait for the last issued use of every stage
      for (int i = (issued > S ? issued - S : 0); i < issued; ++i)
        mbar_wait(&full[i % S], (i / S) & 1, p.status, p.wait_limit);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // ---------------- MMA issuer ----------------
      // (one base descriptor plus per-stage and per-slice offsets; the A stage's barrier implies
      // the TMA's, see the prefill kernel)
      constexpr uint32_t idesc = idesc_f16_f32(kBM, BN);
      const uint64_t dbase = desc_sw128_kmajor(smem_u32(smem));
      bool ok = true;
      for (int i = 0; i < nK && ok; ++i) {
        const int s = i % S, u = i / S;
        ok = mbar_wait(&afull[s], u & 1, p.status, p.wait_limit);
        if (!ok) break;
        tc_fence_after();
        const uint64_t ds = dbase + (uint64_t)((s * L::kStage) >> 4);
        const uint32_t at = tmem + BN + 64 * s;
        if (i < nD) {
          mma_f16_ts(tmem, at, ds, idesc, i != 0);
          #pragma unroll
          for (int kk = 1; kk < 8; ++kk)
            mma_f16_ts(tmem, at + 8 * kk, ds + (uint64_t)((((kk >> 2) * BN * 128) + (kk & 3) * 32) >> 4), idesc, 1u);
        } else {   // only the slices that hold weak columns
          #pragma unroll 1
          for (int kk = 0; kk < 8; ++kk)
            if ((i - nD) * 64 + (kk & 3) * 16 < p.k_ld[kk >> 2])
              mma_f16_ts(tmem, at + 8 * kk, ds + (uint64_t)((((kk >> 2) * BN * 128) + (kk & 3) * 32) >> 4), idesc, 1u);
        }
        mma_commit(&empty[s]);
      }
      mma_commit(accf);
    }
  } else {
    // ---------------- A operand ----------------
    // DW warps, NSL = DW / 4 per lane quarter; thread (MMA row r, slab jh) writes codes
    // 8 U jh .. 8 U jh + 8 U - 1 of its row (U = 16 / NSL), as in the prefill kernel
    constexpr int NSL = DW / 4, U = 16 / NSL;
    const int quarter = warp & 3, jh = (warp - 2) >> 2;
    const int lay = lane >> 4, tr = 16 * quarter + (lane & 15);   // layer and row of the tile
    const int orow = n0 + tr;
    const int row = min(orow, p.N - 1);
    const uint32_t lane_base = (uint32_t)(32 * quarter) << 16;
    uint32_t s2 = 0, scl[3], nz[3];
    constexpr float kOff[3] = {1.f, BITS == 3 ? 8.f : 16.f, 64.f};
    scl[0] = h2_splat(1.f);
    scl[1] = h2_splat(1.f / kOff[1]);
    scl[2] = h2_splat(1.f / kOff[2]);
    auto set_sz = [&](__half sh, __half zh) {
      const uint32_t su = __half_as_ushort(sh);
      const float z = __half2float(zh);
      s2 = su | (su << 16);
      #pragma unroll
      for (int c = 0; c < 3; ++c) nz[c] = h2_splat(-(1024.f / kOff[c] + z));
    };
    if (!per_group) set_sz(p.scales[lay][row], p.zeros[lay][row]);
    bool ok = true;
    for (int i = 0; i < nK && ok; ++i) {
      const int s = i % S, u = i / S;
      ok = mbar_wait(&full[s], u & 1, p.status, p.wait_limit);   // (also: the stage's previous MMAs are done)
      if (!ok) break;
      tc_fence_after();
      const unsigned char* st = smem + s * L::kStage;
      const uint32_t at = tmem + lane_base + BN + 64 * s + 4 * U * jh;
      uint32_t d[U / 4][16];
      if (i < nD) {
        if (per_group) {
          const __half2 sz = *reinterpret_cast<const __half2*>(st + L::kX + L::kP + lay * (L::kSZ / 2) + tr * 4);
          set_sz(__low2half(sz), __high2half(sz));
        }
        const uint4* pw = reinterpret_cast<const uint4*>(st + L::kX + lay * (L::kP / 2) + tr * 16 * BITS);
        uint32_t w[4 * BITS];
        #pragma unroll
        for (int v = 0; v < BITS; ++v) {
          const uint4 q = pw[v];
          w[4 * v] = q.x; w[4 * v + 1] = q.y; w[4 * v + 2] = q.z; w[4 * v + 3] = q.w;
        }
        auto units = [&](auto sl_c) {
          constexpr int SL = decltype(sl_c)::value;
          #pragma unroll
          for (int ju = 0; ju < U; ++ju)
            #pragma unroll
            for (int q = 0; q < 4; ++q)
              d[ju >> 2][4 * (ju & 3) + q] = dequant_pair<BITS>(w + q * BITS, U * SL + ju, s2, scl, nz);
        };
        if constexpr (NSL == 2) {
          if (jh == 0) units(std::integral_constant<int, 0>{});
          else units(std::integral_constant<int, 1>{});
        } else {
          switch (jh) {
            case 0: units(std::integral_constant<int, 0>{}); break;
            case 1: units(std::integral_constant<int, 1>{}); break;
            case 2: units(std::integral_constant<int, 2>{}); break;
            default: units(std::integral_constant<int, 3>{}); break;
          }
        }
      } else {
        // weak step: slab jh covers columns c0 .. c0 + 8 U - 1 of layer wl's part of the step
        const int wl = (8 * U * jh) / 64, c0 = (i - nD) * 64 + (8 * U * jh) % 64;
        const uint4* src = reinterpret_cast<const uint4*>(p.w_weak[lay] + (size_t)row * p.k_ld[lay] + c0);
        #pragma unroll
        for (int v = 0; v < U; ++v) {
          const uint4 q = (lay == wl && orow < p.N && c0 + 8 * v < p.k_ld[lay]) ? src[v] : make_uint4(0, 0, 0, 0);
          d[v >> 2][4 * (v & 3)] = q.x; d[v >> 2][4 * (v & 3) + 1] = q.y;
          d[v >> 2][4 * (v & 3) + 2] = q.z; d[v >> 2][4 * (v & 3) + 3] = q.w;
        }
      }
      #pragma unroll
      for (int h = 0; h < U / 4; ++h) tmem_st16(at + 16 * h, d[h]);
      tmem_st_wait();
      tc_fence_before();
      if (!(p.skip_arrive && i == 0 && threadIdx.x == 64)) mbar_arrive(&afull[s]);
    }

    // ---------------- epilogue ----------------
    const bool acc_ok = __all_sync(0xffffffffu, mbar_wait(accf, 0, p.status, p.wait_limit) && ok);
    tc_fence_after();
    #pragma unroll 1
    for (int c0 = jh * (BN / NSL); c0 < (jh + 1) * (BN / NSL); c0 += 16) {
      uint32_t v[16];
      tmem_ld16(tmem + lane_base + (uint32_t)c0, v);
      tmem_ld_wait();
      if (!acc_ok) continue;
      if (nsp > 1) {   // this split's fp32 partials
        float* w = p.ws + ((size_t)sp * 2 + lay) * p.ws_plane;
        if (orow < p.N) {
          #pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int t = m0 + c0 + j;
            if (t < p.M) w[(size_t)(t - p.ws_t0) * p.N + orow] = __uint_as_float(v[j]);
          }
        }
      } else {
        // a gate lane finishes columns 0-7, the up lane of the same output columns 8-15
        #pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t got = __shfl_xor_sync(0xffffffffu, lay ? v[j] : v[j + 8], 16);
          const float gs = __uint_as_float(lay ? got : v[j]), us = __uint_as_float(lay ? v[j + 8] : got);
          const int t = m0 + c0 + j + 8 * lay;
          if (t < p.M && orow < p.N) gated_store(p, (size_t)t * p.N + orow, gs, us);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, tmem_cols<BN, S>());
    tmem_relinquish();
  }
}

// Weak activations of every token for both layers: xw[l][m][t] = x[m][idx_l[t]] (0 past k_l).
struct GatherArgs {
  const int32_t* idx[2];
  __half* xw[2];
  int k[2], k_ld[2];   // k_ld 0: no weak columns
};
__global__ void k_gated_gather(const __half* __restrict__ x, int M, int K, const __grid_constant__ GatherArgs a, int* status) {
  const int ld = a.k_ld[0] + a.k_ld[1];
  const size_t n = (size_t)M * ld;
  for (size_t e = (size_t)blockIdx.x * blockDim.x + threadIdx.x; e < n; e += (size_t)gridDim.x * blockDim.x) {
    const size_t m = e / ld;
    const int c = (int)(e % ld), l = c >= a.k_ld[0], t = l ? c - a.k_ld[0] : c;
    a.xw[l][m * a.k_ld[l] + t] = t < a.k[l] && in_range(a.idx[l][t], K, status) ? x[m * K + a.idx[l][t]] : __float2half_rn(0.f);
  }
}

// The split outputs: the planes' partials added in split order, then the epilogue.
__global__ void k_gated_reduce(const __grid_constant__ GatedGemmParams p, int splits) {
  const size_t n = p.ws_plane, base = (size_t)p.ws_t0 * p.N;
  for (size_t e = (size_t)blockIdx.x * blockDim.x + threadIdx.x; e < n; e += (size_t)gridDim.x * blockDim.x) {
    float gs = p.ws[e], us = p.ws[n + e];
    for (int z = 1; z < splits; ++z) {
      gs += p.ws[(size_t)(2 * z) * n + e];
      us += p.ws[(size_t)(2 * z + 1) * n + e];
    }
    gated_store(p, base + e, gs, us);
  }
}

// ---------------------------------------------------------------- input gradient of both layers
// dx = dg Wg + du Wu: the input-gradient pipeline (see k_igemm_sm100: A = W_hat^T, 128 columns x
// 128 rows a step, prepared by one warp and formed column by column) run over the gate's rows and
// then the up layer's into one accumulator.  The weak columns' codes give exactly 0; their
// products with the fp16 weak blocks are computed before (k_gated_igw) and added in fp32 in the
// epilogue of the first split, so a column that is weak in one layer and packed in the other is
// still rounded once.
struct GatedIgMaps {
  CUtensorMap dy[2], p[2], sz[2], dx;
};
struct GatedIgParams {
  float* ws;        // split partials [split][M][K] (NULL: one split, fp16 dx directly)
  int* status;
  int N, K, M, group;
  int rsteps;       // 128-row steps per split, of the 2 ceil(N / 128) steps of both layers
  long long wait_limit;
  // the weak columns' products, [split][slot][M] per layer
  const float* wk[2];
  const int32_t* idx[2];
  int k[2], wsplits;
  uint32_t blk[2][kMaxBlocks];   // per column block: first weak slot << 16 | weak-column count
};

template <int BITS, int BN, int S, int DW>
__global__ void __launch_bounds__(32 * (3 + DW), 1)
k_gated_igemm(const __grid_constant__ GatedIgMaps maps, const __grid_constant__ GatedIgParams p) {
  using L = IgSmem<BITS, BN>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S * L::kStage);
  uint64_t* full = bars;            // [S] TMA landed
  uint64_t* empty = bars + S;       // [S] MMAs of the stage done
  uint64_t* afull = bars + 2 * S;   // [S] A tile written to tensor memory
  uint64_t* accf = bars + 3 * S;    // accumulator complete
  uint64_t* pfull = bars + 3 * S + 1;   // [S] prep warp's words written
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 4 * S + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.x;             // column block (128 columns)
  const int m0 = blockIdx.y * BN;       // first token
  const int nR = (p.N + 127) / 128;     // row steps of one layer
  const int rb0 = blockIdx.z * p.rsteps;                     // first step of this split
  const int nK = max(0, min(p.rsteps, 2 * nR - rb0));
  const int grp = (b * kStepCodes) / p.group;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&afull[s], 32 * DW);
      mbar_init(&pfull[s], 32);
    }
    mbar_init(accf, 1);
    fence_mbar_init();
    #pragma unroll
    for (int l = 0; l < 2; ++l) {
      prefetch_tmap(&maps.dy[l]);
      prefetch_tmap(&maps.p[l]);
      prefetch_tmap(&maps.sz[l]);
    }
  }
  if (warp == 1) tmem_alloc(tmem_slot, tmem_cols<BN, S>());
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      // ---------------- TMA producer ----------------
      bool ok = true;
      int issued = 0;
      for (int i = 0; i < nK && ok; ++i) {
        const int s = i % S, u = i / S;
        if (u > 0) ok = mbar_wait(&empty[s], (u - 1) & 1, p.status, p.wait_limit);
        if (!ok) break;
        unsigned char* st = smem + s * L::kStage;
        const int l = rb0 + i >= nR, rb = rb0 + i - (l ? nR : 0);
        mbar_arrive_expect_tx(&full[s], L::kTma);
        tma_load_3d(st + L::kX, &maps.p[l], &full[s], 0, b, rb * 8);
        tma_load_3d(st + L::kX + L::kP, &maps.sz[l], &full[s], 0, grp, rb * 8);
        tma_load_2d(st, &maps.dy[l], &full[s], rb * 128, m0);
        tma_load_2d(st + BN * 128, &maps.dy[l], &full[s], rb * 128 + 64, m0);
        issued = i + 1;
      }
      for (int i = (issued > S ? issued - S : 0); i < issued; ++i)
        mbar_wait(&full[i % S], (i / S) & 1, p.status, p.wait_limit);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // ---------------- MMA issuer ----------------
      constexpr uint32_t idesc = idesc_f16_f32(kBM, BN);
      const uint64_t dbase = desc_sw128_kmajor(smem_u32(smem));
      bool ok = true;
      for (int i = 0; i < nK && ok; ++i) {
        const int s = i % S, u = i / S;
        ok = mbar_wait(&afull[s], u & 1, p.status, p.wait_limit);
        if (!ok) break;
        tc_fence_after();
        const uint64_t ds = dbase + (uint64_t)((s * L::kStage) >> 4);
        const uint32_t at = tmem + BN + 64 * s;
        mma_f16_ts(tmem, at, ds, idesc, i != 0);
        #pragma unroll
        for (int kk = 1; kk < 8; ++kk)
          mma_f16_ts(tmem, at + 8 * kk, ds + (uint64_t)((((kk >> 2) * BN * 128) + (kk & 3) * 32) >> 4), idesc, 1u);
        mma_commit(&empty[s]);
      }
      mma_commit(accf);
    }
  } else if (warp == 2 + DW) {
    // ---------------- prep warp ----------------
    bool ok = true;
    for (int i = 0; i < nK && ok; ++i) {
      const int s = i % S, u = i / S;
      ok = mbar_wait(&full[s], u & 1, p.status, p.wait_limit);
      if (!ok) break;
      const uint32_t st = smem_u32(smem) + s * L::kStage;   // shared address of the stage
      ig_prep_step<BITS, BN>(st, lane);
      __syncwarp();
      mbar_arrive(&pfull[s]);
    }
  } else {
    // ---------------- A operand: W_hat^T ----------------
    constexpr int NSL = DW / 4, RP = 64 / NSL;
    const int quarter = warp & 3, jh = (warp - 2) >> 2;
    const int j = 32 * quarter + lane;             // column of the block
    const IgColumn<BITS, BN> cj(j);
    const uint32_t lane_base = (uint32_t)(32 * quarter) << 16;
    bool ok = true;
    for (int i = 0; i < nK && ok; ++i) {
      const int s = i % S, u = i / S;
      ok = mbar_wait(&pfull[s], u & 1, p.status, p.wait_limit);   // (implies the TMA landed)
      if (!ok) break;
      tc_fence_after();
      const uint32_t st = smem_u32(smem) + s * L::kStage;   // shared address of the stage
      uint32_t d[RP];
      cj.operand<RP>(st, RP * jh, d);
      const uint32_t at = tmem + lane_base + BN + 64 * s + RP * jh;
      #pragma unroll
      for (int c = 0; c < RP / 16; ++c)
        tmem_st16(at + 16 * c, *reinterpret_cast<const uint32_t(*)[16]>(d + 16 * c));
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&afull[s]);
    }

    // ---------------- epilogue ----------------
    // this column's weak slot in each layer (-1: packed there); added by the first split
    const int col = b * kStepCodes + j;
    int slot[2] = {-1, -1};
    if (blockIdx.z == 0) {
      #pragma unroll
      for (int l = 0; l < 2; ++l) {
        if (p.k[l] == 0) continue;
        const int first = (int)(p.blk[l][b] >> 16), cnt = (int)(p.blk[l][b] & 0xFFFFu);
        for (int t = first; t < first + cnt; ++t)
          if (in_range(t, p.k[l], p.status) && p.idx[l][t] == col) slot[l] = t;
      }
    }
    const bool acc_ok = __all_sync(0xffffffffu, mbar_wait(accf, 0, p.status, p.wait_limit) && ok);
    tc_fence_after();
    __half* s_out = reinterpret_cast<__half*>(smem);
    #pragma unroll 1
    for (int c0 = jh * (BN / NSL); c0 < (jh + 1) * (BN / NSL); c0 += 16) {
      uint32_t v[16];
      tmem_ld16(tmem + lane_base + (uint32_t)c0, v);
      tmem_ld_wait();
      #pragma unroll
      for (int l = 0; l < 2; ++l)
        if (slot[l] >= 0)
          for (int z = 0; z < p.wsplits; ++z) {
            const float* wk = p.wk[l] + ((size_t)z * p.k[l] + slot[l]) * p.M + m0 + c0;
            #pragma unroll
            for (int t = 0; t < 16; ++t)
              if (m0 + c0 + t < p.M) v[t] = __float_as_uint(__uint_as_float(v[t]) + wk[t]);
          }
      if (p.ws) {
        if (acc_ok) {
          float* w = p.ws + (size_t)blockIdx.z * p.M * p.K;
          #pragma unroll
          for (int t = 0; t < 16; ++t)
            if (m0 + c0 + t < p.M) w[(size_t)(m0 + c0 + t) * p.K + col] = __uint_as_float(v[t]);
        }
      } else {
        #pragma unroll
        for (int t = 0; t < 16; ++t)
          sts_u16(smem_u32(s_out) + 2 * ((c0 + t) * kStepCodes + j), __half_as_ushort(__float2half_rn(__uint_as_float(v[t]))));
      }
    }
    if (!p.ws) {
      fence_proxy_async_smem();          // the tile, written by the generic proxy, to the TMA
      named_bar_sync(1, 32 * DW);        // every A thread's part of the tile is written
      if (warp == 2 && lane == 0 && acc_ok) {
        tma_store_2d(&maps.dx, s_out, b * kStepCodes, m0);
        bulk_commit();
        bulk_wait_read0();               // shared memory read out before the CTA may exit
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, tmem_cols<BN, S>());
    tmem_relinquish();
  }
}

// dx = fp16_rn(the splits' partials added in split order); n = M K outputs (a multiple of 128)
__global__ void k_gated_ig_reduce(const float* __restrict__ ws, int splits, size_t n, __half* __restrict__ dx) {
  for (size_t e = 4 * ((size_t)blockIdx.x * blockDim.x + threadIdx.x); e < n; e += 4 * (size_t)gridDim.x * blockDim.x) {
    float4 v = *reinterpret_cast<const float4*>(ws + e);
    for (int z = 1; z < splits; ++z) {
      const float4 w = *reinterpret_cast<const float4*>(ws + (size_t)z * n + e);
      v.x += w.x; v.y += w.y; v.z += w.z; v.w += w.w;
    }
    __half2* o = reinterpret_cast<__half2*>(dx + e);
    o[0] = __floats2half2_rn(v.x, v.y);
    o[1] = __floats2half2_rn(v.z, v.w);
  }
}

// The weak columns' products of both layers, wk[l][split][slot][m] = sum_i dy_l[m][i] w_weak_l[i][slot]
// over a split of the rows (mma.sync m16n8k16: rows = tokens, K = weight rows, columns = slots).
// A CTA of 4 warps computes 64 tokens x 32 slots of one layer, 32 rows at a time through a 4-stage
// cp.async ring.  (As k_igw_mma, but to fp32 and token-contiguous: the input-gradient epilogue
// reads a slot's tokens.)
constexpr int kIwTok = 64, kIwCols = 32, kIwRows = 32, kIwThreads = 128, kIwStages = 4;
constexpr int kIwDyLd = kIwRows + 8, kIwWLd = kIwCols + 8;   // padded row strides (halves)

struct GatedIgwArgs {
  const __half* dy[2];
  const __half* w[2];   // [N][k_ld]
  float* wk[2];
  int k[2], k_ld[2], ctiles0;   // slot tiles of the gate layer (blockIdx.y below it)
  int N, ldy, M, per;           // per: rows per split, a multiple of 32
};
__global__ void __launch_bounds__(kIwThreads) k_gated_igw(const __grid_constant__ GatedIgwArgs a) {
  __shared__ __align__(128) __half s_dy[kIwStages][kIwTok][kIwDyLd];
  __shared__ __align__(128) __half s_w[kIwStages][kIwRows][kIwWLd];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int l = (int)blockIdx.y >= a.ctiles0;
  const __half* __restrict__ dy = a.dy[l];
  const __half* __restrict__ w = a.w[l];
  const int k = a.k[l], k_ld = a.k_ld[l];
  const int mb = blockIdx.x * kIwTok, t0 = ((int)blockIdx.y - (l ? a.ctiles0 : 0)) * kIwCols;
  const int i_lo = blockIdx.z * a.per, i_hi = min(a.N, i_lo + a.per);
  const int nchunk = max(0, (i_hi - i_lo + kIwRows - 1) / kIwRows);
  auto load = [&](int c, int st) {   // rows i_lo + 32 c .. of this split into stage st
    const int ib = i_lo + c * kIwRows;
    #pragma unroll
    for (int u = 0; u < 2; ++u) {    // dY: 64 tokens x 4 pieces of 8 rows (rows N .. ldy - 1 hold zeros)
      const int e = tid + u * kIwThreads, m = e >> 2, pc = e & 3;
      const int mm = mb + m, row = ib + pc * 8;
      const bool ok = mm < a.M && row < i_hi;
      cp_async16(&s_dy[st][m][pc * 8], dy + (ok ? (size_t)mm * a.ldy + row : 0), ok);
    }
    {                                // weak block: 32 rows x 4 pieces of 8 slots
      const int r = tid >> 2, pc = tid & 3, row = ib + r, col = t0 + pc * 8;
      const bool ok = row < i_hi && col < k_ld;
      cp_async16(&s_w[st][r][pc * 8], w + (ok ? (size_t)row * k_ld + col : 0), ok);
    }
  };
  float d[4][4];
  #pragma unroll
  for (int n = 0; n < 4; ++n)
    #pragma unroll
    for (int i = 0; i < 4; ++i) d[n][i] = 0.f;
  #pragma unroll
  for (int st = 0; st < kIwStages - 1; ++st) {
    if (st < nchunk) load(st, st);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  const int q = lane >> 3, r8 = lane & 7;   // ldmatrix: matrix q, row r8
  for (int c = 0; c < nchunk; ++c) {
    asm volatile("cp.async.wait_group %0;" :: "n"(kIwStages - 2) : "memory");
    __syncthreads();   // chunk c landed for every thread; the stage refilled below is free
    if (c + kIwStages - 1 < nchunk) load(c + kIwStages - 1, (c + kIwStages - 1) % kIwStages);
    asm volatile("cp.async.commit_group;" ::: "memory");
    const int st = c % kIwStages;
    #pragma unroll
    for (int ks = 0; ks < kIwRows / 16; ++ks) {
      const int mk = ks * 16;
      uint32_t f[4];   // tokens 16 warp + 0..15 x rows mk..mk+15
      ldsm_x4(f, &s_dy[st][warp * 16 + (q & 1) * 8 + r8][mk + (q >> 1) * 8]);
      #pragma unroll
      for (int nh = 0; nh < 2; ++nh) {
        uint32_t bb[4];   // rows mk..mk+15 x slots 16 nh..16 nh+15, read transposed (two n8 tiles)
        ldsm_x4_t(bb, &s_w[st][mk + (q & 1) * 8 + r8][nh * 16 + (q >> 1) * 8]);
        mma_16816(d[2 * nh], f, bb[0], bb[1]);
        mma_16816(d[2 * nh + 1], f, bb[2], bb[3]);
      }
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  const int g = lane >> 2, c4 = lane & 3;
  #pragma unroll
  for (int n = 0; n < 4; ++n)
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m = mb + warp * 16 + g + 8 * (i >> 1), t = t0 + n * 8 + 2 * c4 + (i & 1);
      if (m < a.M && t < k) a.wk[l][((size_t)blockIdx.z * k + t) * a.M + m] = d[n][i];
    }
}

// Rows of N values into rows of ld >= N (N % 8 != 0: the tensor map wants 16-byte row strides),
// zeros after them; both layers' gradients in one launch.
__global__ void k_gated_pad(const __half* __restrict__ a, const __half* __restrict__ b, int N, int ld, size_t rows,
                            __half* __restrict__ oa, __half* __restrict__ ob) {
  const size_t n = rows * ld;
  for (size_t e = (size_t)blockIdx.x * blockDim.x + threadIdx.x; e < n; e += (size_t)gridDim.x * blockDim.x) {
    const size_t m = e / ld;
    const int c = (int)(e % ld);
    oa[e] = c < N ? a[m * N + c] : __float2half_rn(0.f);
    ob[e] = c < N ? b[m * N + c] : __float2half_rn(0.f);
  }
}

// ---------------------------------------------------------------- host side
constexpr size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }
unsigned blocks_for(size_t n, int threads, unsigned most) {
  return (unsigned)std::max<size_t>(1, std::min<size_t>((n + threads - 1) / threads, most));
}

// workspace of one forward / backward product: both layers' weak activations, then the split partials
struct FwdPlan {
  GemmPlan g;
  int t0, nsp;              // first token with split partials, splits there
  size_t xw[2], ws, total;  // byte offsets
};
FwdPlan fwd_plan(const Layer& gate, const Layer& up, int M) {
  FwdPlan f;
  const int RT = (gate.N + kHalfRows - 1) / kHalfRows;
  f.g = gemm_plan(RT * kBM, gate.K, M, layer_sm_count(gate.device));
  const int BN = f.g.tile_tokens, TT = (M + BN - 1) / BN;
  f.t0 = f.g.tail_sp > 1 ? (TT - f.g.tail_tt) * BN : 0;
  f.nsp = f.g.tail_sp > 1 ? f.g.tail_sp : f.g.splits;
  size_t at = 0;
  const Layer* L[2] = {&gate, &up};
  for (int l = 0; l < 2; ++l) {
    f.xw[l] = at;
    if (L[l]->k > 0) at += up256((size_t)M * L[l]->k_ld * sizeof(__half));
  }
  f.ws = at;
  if (f.nsp > 1) at += up256((size_t)f.nsp * 2 * (M - f.t0) * gate.N * sizeof(float));
  f.total = at;
  return f;
}

template <int BITS, int BN, int S, int DW>
owq_status_t run_gemm(const Layer& gate, const Layer& up, int act, const __half* x, const __half* dh, __half* out0, __half* out1,
                      int M, const FwdPlan& f, unsigned char* ws, long long wait_limit, bool skip_arrive, cudaStream_t s) {
  const Layer* L[2] = {&gate, &up};
  GatedMaps maps;
  GatedGemmParams prm;
  GatherArgs ga;
  if (!encode_2d(&maps.x, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, x, (uint64_t)gate.K, (uint64_t)M, (uint64_t)gate.K * 2, 64, BN,
                 CU_TENSOR_MAP_SWIZZLE_128B))
    return OWQ_ERR_CUDA;
  for (int l = 0; l < 2; ++l) {
    prm.scales[l] = L[l]->scales;
    prm.zeros[l] = L[l]->zeros;
    prm.w_weak[l] = L[l]->w_weak;
    prm.k_ld[l] = L[l]->k > 0 ? L[l]->k_ld : 0;
    ga.idx[l] = L[l]->idx;
    ga.xw[l] = reinterpret_cast<__half*>(ws + f.xw[l]);
    ga.k[l] = L[l]->k;
    ga.k_ld[l] = prm.k_ld[l];
    maps.xw[l] = maps.x;   // (a layer without weak columns: loaded, never multiplied)
    if (!encode_packed_3d(&maps.p[l], L[l]->packed, L[l]->K, L[l]->N, BITS, kHalfRows / 16) ||
        !encode_sz_3d(&maps.sz[l], L[l]->sz_t, L[l]->G, L[l]->N, kHalfRows / 16) ||
        (L[l]->k > 0 && !encode_2d(&maps.xw[l], CU_TENSOR_MAP_DATA_TYPE_FLOAT16, ga.xw[l], (uint64_t)L[l]->k_ld, (uint64_t)M,
                                   (uint64_t)L[l]->k_ld * 2, 64, BN, CU_TENSOR_MAP_SWIZZLE_128B)))
      return OWQ_ERR_CUDA;
  }
  prm.dh = dh;
  prm.out[0] = out0;
  prm.out[1] = out1;
  prm.status = device_status_ptr();
  if (!prm.status) return OWQ_ERR_CUDA;
  prm.N = gate.N; prm.K = gate.K; prm.M = M; prm.G = gate.G; prm.act = act;
  prm.wait_limit = wait_limit; prm.skip_arrive = skip_arrive ? 1 : 0;
  prm.nw = (std::max(prm.k_ld[0], prm.k_ld[1]) + 63) / 64;
  const int RT = (gate.N + kHalfRows - 1) / kHalfRows, TT = (M + BN - 1) / BN;
  prm.ksteps = f.g.ksteps;
  prm.tail_y0 = TT - f.g.tail_tt;
  prm.tail_sp = f.g.tail_sp;
  prm.tail_ksteps = f.g.tail_ksteps;
  prm.ws = reinterpret_cast<float*>(ws + f.ws);
  prm.ws_t0 = f.t0;
  prm.ws_plane = (size_t)(M - f.t0) * gate.N;
  auto kern = k_gated_gemm<BITS, BN, S, DW, false>;
  if (f.g.tail_sp > 1) {
    if constexpr (BN > 64) kern = k_gated_gemm<BITS, BN, S, DW, true>;
    else return OWQ_ERR_CUDA;   // never planned: a tail needs two token tiles
  }
  constexpr int smem = smem_bytes<BITS, BN, S>();
  static_assert(smem <= 232448, "shared memory budget");
  static_assert(BN + 64 * S <= (int)tmem_cols<BN, S>(), "tensor memory: accumulator + A stages");
  static_assert((232448 / smem) * tmem_cols<BN, S>() <= 512, "tensor memory per SM");
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
    cudaGetLastError();
    return OWQ_ERR_CUDA;
  }
  const int ld = ga.k_ld[0] + ga.k_ld[1];
  if (ld > 0) {
    k_gated_gather<<<blocks_for((size_t)M * ld, 256, 2048), 256, 0, s>>>(x, M, gate.K, ga, prm.status);
    if (cudaGetLastError() != cudaSuccess) return OWQ_ERR_CUDA;
  }
  const dim3 grid(RT, prm.tail_y0 + f.g.tail_tt * f.g.tail_sp, f.g.splits);
  kern<<<grid, 32 * (2 + DW), smem, s>>>(maps, prm);
  if (cudaGetLastError() != cudaSuccess) return OWQ_ERR_CUDA;
  if (f.nsp > 1) {
    k_gated_reduce<<<blocks_for(prm.ws_plane, 256, 4096), 256, 0, s>>>(prm, f.nsp);
    if (cudaGetLastError() != cudaSuccess) return OWQ_ERR_CUDA;
  }
  return OWQ_OK;
}

template <int BITS>
owq_status_t dispatch_gemm(const Layer& gate, const Layer& up, int act, const __half* x, const __half* dh, __half* out0,
                           __half* out1, int M, const FwdPlan& f, unsigned char* ws, long long wl, bool skip, cudaStream_t s) {
  switch (f.g.tile_tokens) {
    case 64: return run_gemm<BITS, 64, 6, 8>(gate, up, act, x, dh, out0, out1, M, f, ws, wl, skip, s);
    case 128: return run_gemm<BITS, 128, 4, 8>(gate, up, act, x, dh, out0, out1, M, f, ws, wl, skip, s);
    default: return run_gemm<BITS, 256, 3, 16>(gate, up, act, x, dh, out0, out1, M, f, ws, wl, skip, s);
  }
}

// workspace of one input gradient: padded gradients (N % 8 != 0), the weak products, the split partials
struct IgPlan {
  int BN, splits, rsteps;   // row splits over both layers' 128-row steps
  int ldy, wsplits, wper;
  size_t pad[2], wk[2], ws, total;
};
IgPlan ig_plan(const Layer& gate, const Layer& up, int M) {
  IgPlan f;
  const int sms = layer_sm_count(gate.device);
  const int Kb = gate.K / kStepCodes, nR = 2 * ((gate.N + 127) / 128);
  f.BN = gemm_tile_tokens(M);
  const long long tiles = (long long)Kb * ((M + f.BN - 1) / f.BN);
  // fewer tiles than SMs: the rows split over CTAs, at least 4 steps each
  f.splits = tiles < sms ? (int)std::max<long long>(1, std::min<long long>(sms / tiles, nR / 4)) : 1;
  f.rsteps = (nR + f.splits - 1) / f.splits;
  f.splits = (nR + f.rsteps - 1) / f.rsteps;
  f.ldy = (gate.N + 7) & ~7;
  size_t at = 0;
  for (int l = 0; l < 2; ++l) {
    f.pad[l] = at;
    if (gate.N % 8) at += up256((size_t)M * f.ldy * sizeof(__half));
  }
  // weak products: about two CTAs per SM, at least 4 chunks of 32 rows each
  const int R = (M + kIwTok - 1) / kIwTok, C = (gate.k + kIwCols - 1) / kIwCols + (up.k + kIwCols - 1) / kIwCols;
  const int nch = (gate.N + kIwRows - 1) / kIwRows;
  f.wsplits = C > 0 ? std::max(1, std::min((2 * sms + R * C - 1) / (R * C), nch / 4)) : 1;
  f.wper = (nch + f.wsplits - 1) / f.wsplits;
  f.wsplits = (nch + f.wper - 1) / f.wper;
  f.wper *= kIwRows;
  f.wk[0] = at;
  at += up256((size_t)f.wsplits * gate.k * M * sizeof(float));
  f.wk[1] = at;
  at += up256((size_t)f.wsplits * up.k * M * sizeof(float));
  f.ws = at;
  if (f.splits > 1) at += up256((size_t)f.splits * M * gate.K * sizeof(float));
  f.total = at;
  return f;
}

template <int BITS, int BN, int S, int DW>
owq_status_t run_ig(const Layer& gate, const Layer& up, const __half* dg, const __half* du, __half* dx, int M, const IgPlan& f,
                    unsigned char* ws, long long wait_limit, cudaStream_t s) {
  const Layer* L[2] = {&gate, &up};
  const __half* dy[2] = {dg, du};
  if (gate.N % 8) {
    __half* pad[2] = {reinterpret_cast<__half*>(ws + f.pad[0]), reinterpret_cast<__half*>(ws + f.pad[1])};
    k_gated_pad<<<blocks_for((size_t)M * f.ldy, 256, 4096), 256, 0, s>>>(dg, du, gate.N, f.ldy, (size_t)M, pad[0], pad[1]);
    if (cudaGetLastError() != cudaSuccess) return OWQ_ERR_CUDA;
    dy[0] = pad[0];
    dy[1] = pad[1];
  }
  GatedIgMaps maps;
  GatedIgParams prm;
  GatedIgwArgs wa;
  const int Kb = gate.K / kStepCodes;
  for (int l = 0; l < 2; ++l) {
    if (!encode_2d(&maps.dy[l], CU_TENSOR_MAP_DATA_TYPE_FLOAT16, dy[l], (uint64_t)gate.N, (uint64_t)M, (uint64_t)f.ldy * 2, 64, BN,
                   CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_packed_3d(&maps.p[l], L[l]->packed, L[l]->K, L[l]->N, BITS) ||
        !encode_sz_3d(&maps.sz[l], L[l]->sz_t, L[l]->G, L[l]->N))
      return OWQ_ERR_CUDA;
    prm.wk[l] = wa.wk[l] = reinterpret_cast<float*>(ws + f.wk[l]);
    prm.idx[l] = L[l]->idx;
    prm.k[l] = wa.k[l] = L[l]->k;
    for (int b = 0; b < Kb; ++b) prm.blk[l][b] = L[l]->blk_weak[b];
    wa.dy[l] = dy[l];
    wa.w[l] = L[l]->w_weak;
    wa.k_ld[l] = L[l]->k_ld;
  }
  if (!encode_2d(&maps.dx, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, dx, (uint64_t)gate.K, (uint64_t)M, (uint64_t)gate.K * 2, kStepCodes, BN,
                 CU_TENSOR_MAP_SWIZZLE_NONE))
    return OWQ_ERR_CUDA;
  prm.status = device_status_ptr();
  if (!prm.status) return OWQ_ERR_CUDA;
  prm.N = gate.N; prm.K = gate.K; prm.M = M; prm.group = gate.group;
  prm.rsteps = f.rsteps;
  prm.wait_limit = wait_limit;
  prm.wsplits = f.wsplits;
  prm.ws = f.splits > 1 ? reinterpret_cast<float*>(ws + f.ws) : nullptr;
  wa.ctiles0 = (gate.k + kIwCols - 1) / kIwCols;
  wa.N = gate.N; wa.ldy = f.ldy; wa.M = M; wa.per = f.wper;
  const int C = wa.ctiles0 + (up.k + kIwCols - 1) / kIwCols;
  if (C > 0) {
    k_gated_igw<<<dim3((M + kIwTok - 1) / kIwTok, C, f.wsplits), kIwThreads, 0, s>>>(wa);
    if (cudaGetLastError() != cudaSuccess) return OWQ_ERR_CUDA;
  }
  auto kern = k_gated_igemm<BITS, BN, S, DW>;
  constexpr int smem = ig_smem_bytes<BITS, BN, S>();
  static_assert(smem <= 232448, "shared memory budget");
  static_assert((232448 / smem) * tmem_cols<BN, S>() <= 512, "tensor memory per SM");
  static_assert(BN * kStepCodes * 2 <= IgSmem<BITS, BN>::kStage, "output tile in the first stage");
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
    cudaGetLastError();
    return OWQ_ERR_CUDA;
  }
  kern<<<dim3(Kb, (M + BN - 1) / BN, f.splits), 32 * (3 + DW), smem, s>>>(maps, prm);
  if (cudaGetLastError() != cudaSuccess) return OWQ_ERR_CUDA;
  if (f.splits > 1) {
    const size_t n = (size_t)M * gate.K;
    k_gated_ig_reduce<<<blocks_for(n / 4, 256, 4096), 256, 0, s>>>(prm.ws, f.splits, n, dx);
    if (cudaGetLastError() != cudaSuccess) return OWQ_ERR_CUDA;
  }
  return OWQ_OK;
}

template <int BITS>
owq_status_t dispatch_ig(const Layer& gate, const Layer& up, const __half* dg, const __half* du, __half* dx, int M, const IgPlan& f,
                         unsigned char* ws, long long wl, cudaStream_t s) {
  switch (f.BN) {
    case 64: return run_ig<BITS, 64, 6, 8>(gate, up, dg, du, dx, M, f, ws, wl, s);
    case 128: return run_ig<BITS, 128, 4, 8>(gate, up, dg, du, dx, M, f, ws, wl, s);
    default: return run_ig<BITS, 256, 3, 16>(gate, up, dg, du, dx, M, f, ws, wl, s);
  }
}

}  // namespace

size_t gated_gemm_ws_bytes(const Layer& gate, const Layer& up, int M) { return fwd_plan(gate, up, M).total; }
size_t gated_input_grad_ws_bytes(const Layer& gate, const Layer& up, int M) { return ig_plan(gate, up, M).total; }

owq_status_t gated_gemm_sm100(const Layer& gate, const Layer& up, int act, const __half* x, const __half* dh, __half* out0,
                              __half* out1, int M, void* ws, size_t ws_bytes, long long wait_limit, bool skip_arrive,
                              cudaStream_t s) {
  const FwdPlan f = fwd_plan(gate, up, M);
  if (f.total > ws_bytes) return OWQ_ERR_NOMEM;
  unsigned char* w = static_cast<unsigned char*>(ws);
  return gate.bits == 3 ? dispatch_gemm<3>(gate, up, act, x, dh, out0, out1, M, f, w, wait_limit, skip_arrive, s)
                        : dispatch_gemm<4>(gate, up, act, x, dh, out0, out1, M, f, w, wait_limit, skip_arrive, s);
}

owq_status_t gated_input_grad_sm100(const Layer& gate, const Layer& up, const __half* dg, const __half* du, __half* dx, int M,
                                    void* ws, size_t ws_bytes, long long wait_limit, cudaStream_t s) {
  const IgPlan f = ig_plan(gate, up, M);
  if (f.total > ws_bytes) return OWQ_ERR_NOMEM;
  unsigned char* w = static_cast<unsigned char*>(ws);
  return gate.bits == 3 ? dispatch_ig<3>(gate, up, dg, du, dx, M, f, w, wait_limit, s)
                        : dispatch_ig<4>(gate, up, dg, du, dx, M, f, w, wait_limit, s);
}

}  // namespace owq
