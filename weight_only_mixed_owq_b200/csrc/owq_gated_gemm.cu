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
// packed weights' bytes below.  Measured (GPU time in short graphs; in brackets called back to back for a
// second, power-capped): 13824 x 5120, 3-bit, 2048 tokens forward 393 (457) us, 1.48 (1.27) PFLOP/s, backward
// 850 (1008) us; 11008 x 4096, 4-bit, 64 tokens forward 27.6 (30.6) us, 256 tokens backward 96 (111) us.  Below 256 tokens a step (128 codes of 256 MMA rows by the tile's tokens) is paced
// by forming the A operand: 0.35 / 0.39 / 0.50 us at 64 / 128 / 192 tokens (3-bit), 0.67 us at 256,
// where the MMAs alone want 0.53 us at the full clock.
#include <algorithm>
#include <type_traits>

#include "owq_act.cuh"
#include "owq_dequant.cuh"
#include "owq_gemm_common.cuh"
#include "owq_mma.cuh"

namespace owq {
namespace {

using namespace sm100;

constexpr int kHalfRows = kBM / 2;     // output rows of a tile: 64 of each layer
constexpr int kDW = 16;                // A-operand warps
constexpr int kGR = 2;                 // groups of them, on alternate steps
constexpr uint32_t kTmemCols = 512;    // the accumulator (BN columns), then the A stages of 64 columns
template <int BN>
constexpr int a_stages() { return BN == 256 ? 4 : BN == 192 ? 5 : 6; }

// One ring stage of a CTA: half of the step's tokens (two 128B-swizzled boxes of 64 columns), the
// packed block of its 128 rows and their (scale, zero) pairs.
template <int BITS, int BN>
struct Stage {
  static constexpr int kX = BN * 128;
  static constexpr int kP = kBM * 16 * BITS;
  static constexpr int kSZ = kBM * 4;
  static constexpr int kBytes = ((kX + kP + kSZ) + 1023) & ~1023;
  // stages: what fits, at most 12 (the ring covers the latency of the loads: a step takes 0.35 to
  // 0.7 us, a load from HBM through both rings to the MMA's end about 3 us)
  static constexpr int kFit = (232448 - 2048) / kBytes;
  static constexpr int kS = kFit < 12 ? kFit : 12;
};
template <int BITS, int BN>
constexpr int ring_smem_bytes() { return Stage<BITS, BN>::kS * Stage<BITS, BN>::kBytes + 1024 /*barriers*/ + 1024 /*align slack*/; }

// How the tiles of a product become CTA pairs: `whole` tiles take one pair each; each of the others
// is split `splits` ways over its steps (`steps` a split).  Pairs are dispatched in index order, so
// the split tiles run last.  The plain order would leave the last wave short: T tiles on P pairs take
// ceil(T / P) tile times, with the last T mod P of them split over the idle pairs about T / P.
struct TileSplit {
  int tiles, whole, splits, steps;
  __host__ __device__ int pairs() const { return whole + (tiles - whole) * splits; }
};
struct TileOf {   // a pair's part
  int tile, split, n_splits, first, steps;
};
__device__ __forceinline__ TileOf tile_of(const TileSplit& p, int pair, int all_steps) {
  TileOf t = {pair, 0, 1, 0, all_steps};
  if (pair >= p.whole) {
    const int u = pair - p.whole;
    t.tile = p.whole + u / p.splits;
    t.split = u % p.splits;
    t.n_splits = p.splits;
    t.first = t.split * p.steps;
    t.steps = max(0, min(p.steps, all_steps - t.first));
  }
  return t;
}
// fp32 partials of the split tiles: [split][tile - whole][CTA of the pair][token of the tile][MMA row]
__device__ __forceinline__ size_t partial_at(const TileSplit& p, int split, int tile, int rank, int BN) {
  return (((size_t)split * (p.tiles - p.whole) + (tile - p.whole)) * 2 + rank) * BN * kBM;
}

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
  __half* dy2[2];            // backward of few tokens: rows 2 t, 2 t + 1 = the gradients' halves of token t
  int ld2;                   // (gated_store), zeros in columns N .. ld2 - 1; NULL: not wanted
  float* ws;                 // split partials
  int* status;
  int N, K, M, G, act;
  int rts;                   // row tiles (128 output rows a pair); tile = token tile * rts + row tile
  TileSplit split;
  int nw;                    // weak steps: 64 columns of each layer's weak block
  long long wait_limit;
  int skip_arrive;
};

// A gradient as hi + 2^-11 lo, two fp16 values, in rows 2 t and 2 t + 1: hi its rounding, lo what that
// left times 2^11, exact in fp32 and at most |v|, so that it neither overflows nor (unscaled, it would from
// |v| < 2^-3 on) falls below fp16's normal range.  Off by at most 2^-22 |v|, or 2^-36.
constexpr float kLoScale = 2048.f;
__device__ __forceinline__ void store_halves(const GatedGemmParams& p, int l, int t, int row, float v) {
  const __half hi = __float2half_rn(v);
  const float lo = v - __half2float(hi);
  __half* d = p.dy2[l] + (size_t)(2 * t) * p.ld2 + row;
  d[0] = hi;
  d[p.ld2] = __float2half_rn(__hisinf(hi) ? 0.f : lo * kLoScale);
}

// outputs of one element (token t, row); gs, us: both projections; dhv: its gradient (BWD)
template <int ACT, bool BWD>
__device__ __forceinline__ void gated_store(const GatedGemmParams& p, size_t o, int t, int row, float gs, float us, __half dhv) {
  float a, da;
  act_eval<ACT>(gs, a, da);
  if constexpr (BWD) {
    const float dh = __half2float(dhv);
    const float dg = dh * us * da, du = dh * a;
    p.out[0][o] = __float2half_rn(dg);
    p.out[1][o] = __float2half_rn(du);
    if (p.dy2[0]) {
      store_halves(p, 0, t, row, dg);
      store_halves(p, 1, t, row, du);
    }
  } else {
    p.out[0][o] = __float2half_rn(a * us);
  }
}

// Epilogue of a whole tile: lanes l (gate row) and l + 16 (the up row of the same output) exchange
// halves; a gate lane finishes columns (tokens) 0-7 of every 16, the up lane 8-15.  `acc`: this
// warp's first column in tensor memory, `first`: its token for this lane, `o`: that output.  The
// backward pass fetches 8 gradients ahead, the first before the accumulator is waited for.
template <int ACT, bool BWD, int COLS, class Wait>
__device__ __forceinline__ void gated_epilogue(const GatedGemmParams& p, uint32_t acc, int first, int orow, int lay, Wait&& wait) {
  const bool row_ok = orow < p.N;
  size_t o = (size_t)first * p.N + orow;
  __half next[8];
  auto fetch = [&](int c) {
    #pragma unroll
    for (int j = 0; j < 8; ++j)
      next[j] = BWD && row_ok && first + c + j < p.M ? p.dh[o + (size_t)(c + j) * p.N] : __float2half_rn(0.f);
  };
  fetch(0);
  if (!wait()) return;
  #pragma unroll 1
  for (int c = 0; c < COLS; c += 16) {
    uint32_t v[16];
    tmem_ld16(acc + (uint32_t)c, v);
    __half dhv[8];
    #pragma unroll
    for (int j = 0; j < 8; ++j) dhv[j] = next[j];
    if (BWD && c + 16 < COLS) fetch(c + 16);
    tmem_ld_wait();
    #pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t got = __shfl_xor_sync(0xffffffffu, lay ? v[j] : v[j + 8], 16);
      const float gs = __uint_as_float(lay ? got : v[j]), us = __uint_as_float(lay ? v[j + 8] : got);
      const int t = first + c + j;
      if (row_ok && t < p.M) gated_store<ACT, BWD>(p, o + (size_t)(c + j) * p.N, t, orow, gs, us, dhv[j]);
      else if (BWD && p.dy2[0] && orow < p.ld2 && t < p.M) { store_halves(p, 0, t, orow, 0.f); store_halves(p, 1, t, orow, 0.f); }
    }
  }
}

// The prefill kernel over interleaved rows and SM pairs.  MMA rows 32 q .. 32 q + 15 of a CTA are
// gate rows n0 + 16 q .., rows 32 q + 16 .. 32 q + 31 the up rows of the same outputs.  Lanes l and
// l + 16 of a warp then hold both projections of one output, so the epilogue pairs them with a
// shuffle; half of the columns are finished by either lane.  Weak step w: columns 64 w .. 64 w + 63
// of the gate's weak block against its gathered activations in the first half of the step's K, the
// up layer's in the second half, each with zeros in the other layer's rows.
// A cluster of two CTAs computes 256 MMA rows x BN tokens with cta_group::2: each CTA unpacks its
// own 128 rows and holds half of the tokens, which halves the activations' traffic from L2 (at 256
// tokens a lone CTA would want 64 KB a step, 17 TB/s over the GPU) and their room in the ring.
// Persistent: a pair takes the parts pair, pair + P, ... (P pairs in the grid), its rings running on
// across them.  The loads of the next part, and its first kS2 steps of A operand, are under way while
// the last products of this one run and its epilogue drains the accumulator.
//   warp 0      TMA producer of the CTA's ring (freed by the MMAs' commit in both CTAs)
//   warp 1      tensor memory; in the even CTA the MMA-issuing thread
//   warps 2-17  A operand, in kGR groups on alternate steps: wait for the stage's loads, unpack, store
//               to one of kS2 tensor-memory stages, one arrival per warp on the even CTA's barrier
//               (after the wait for the loads, so the barrier covers those too); then the epilogue
template <int BITS, int BN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(32 * (2 + kDW), 1)
k_gated_gemm(const __grid_constant__ GatedMaps maps, const __grid_constant__ GatedGemmParams p) {
  using L = Stage<BITS, BN>;
  constexpr int S = L::kS, kS2 = a_stages<BN>();
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S * L::kBytes);
  uint64_t* full = bars;              // [S] TMA landed
  uint64_t* empty = bars + S;         // [S] MMAs of the stage done
  uint64_t* afull = bars + 2 * S;     // [kS2] A stage written in both CTAs (the even CTA's is used)
  uint64_t* accf = bars + 2 * S + kS2;       // accumulator complete
  uint64_t* acce = bars + 2 * S + kS2 + 1;   // accumulator read out by both CTAs (the even CTA's is used)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * S + kS2 + 2);

  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // (warp: uniform)
  const int rank = (int)cluster_ctarank();
  const int first_part = blockIdx.x >> 1, P = gridDim.x >> 1, parts = p.split.pairs();
  const int all_steps = p.K / kStepCodes;
  auto steps_of = [&](const TileOf& t) { return t.steps + (t.split == t.n_splits - 1 ? p.nw : 0); };   // + the weak steps (last split)
  auto row0_of = [&](const TileOf& t) { return ((t.tile % p.rts) * 2 + rank) * kHalfRows; };   // first output row of this CTA
  auto token0_of = [&](const TileOf& t) { return t.tile / p.rts * BN; };
  const bool per_group = p.G > 1;
  TileOf to = tile_of(p.split, first_part, all_steps);   // the part at hand
  int nK = steps_of(to), n0 = row0_of(to), m0 = token0_of(to);
  auto next = [&](int part) {
    to = tile_of(p.split, part, all_steps);
    nK = steps_of(to); n0 = row0_of(to); m0 = token0_of(to);
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < kS2; ++s) mbar_init(&afull[s], 2 * kDW / kGR);   // a lane of each warp, both CTAs
    mbar_init(accf, 1);
    mbar_init(acce, 2 * kDW);
    fence_mbar_init();
    prefetch_tmap(&maps.x);
    prefetch_tmap(&maps.p[0]);
    prefetch_tmap(&maps.p[1]);
  }
  if (warp == 1) tmem_alloc_pair(tmem_slot, kTmemCols);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // both CTAs' barriers and tensor memory are ready
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);

  if (warp == 0) {
    // ---------------- TMA producer ----------------
    // The whole warp runs the loop and one lane issues, so that the copies' operands stay in uniform
    // registers (values that a lone lane carries from part to part do not: 0.55 instead of 0.46 us a
    // step at 64 tokens).
    const uint32_t kDense = L::kX + L::kP + (per_group ? L::kSZ : 0);
    bool ok = true, waited = false;
    int s = 0, ph = 1, g = 0;   // ring stage, phase of its `empty`, steps issued
    for (int part = first_part; ok;) {
      const int n16 = __shfl_sync(0xffffffffu, n0 / 16, 0), mt = __shfl_sync(0xffffffffu, m0, 0) + rank * (BN / 2);   // mt: this CTA's tokens
      const int steps = __shfl_sync(0xffffffffu, nK, 0), nD = __shfl_sync(0xffffffffu, to.steps, 0), kb0 = __shfl_sync(0xffffffffu, to.first, 0);
      for (int i = 0; i < steps; ++i) {
        if (g >= S) ok = __all_sync(0xffffffffu, mbar_wait(&empty[s], ph, p.status, p.wait_limit));
        if (!ok) break;
        unsigned char* st = smem + s * L::kBytes;
        if (i >= nD && !waited) {
          asm volatile("griddepcontrol.wait;" ::: "memory");   // the gathered activations
          waited = true;
        }
        if (elect_one()) {
          if (i < nD) {
            const int kb = kb0 + i;
            mbar_arrive_expect_tx(&full[s], kDense);
            #pragma unroll
            for (int l = 0; l < 2; ++l) {
              tma_load_3d(st + L::kX + l * (L::kP / 2), &maps.p[l], &full[s], 0, kb, n16);
              if (per_group) tma_load_3d(st + L::kX + L::kP + l * (L::kSZ / 2), &maps.sz[l], &full[s], 0, kb, n16);
            }
            tma_load_2d(st, &maps.x, &full[s], kb * kStepCodes, mt);
            tma_load_2d(st + BN * 64, &maps.x, &full[s], kb * kStepCodes + 64, mt);
          } else {
            const int c0 = (i - nD) * 64;
            mbar_arrive_expect_tx(&full[s], L::kX);
            tma_load_2d(st, &maps.xw[0], &full[s], c0, mt);
            tma_load_2d(st + BN * 64, &maps.xw[1], &full[s], c0, mt);
          }
        }
        __syncwarp();
        ++g;
        if (++s == S) { s = 0; ph ^= 1; }
      }
      if ((part += P) >= parts) break;
      next(part);
    }
    // never leave with copies in flight: wait for the last issued use of every stage
    for (int i = (g > S ? g - S : 0); i < g; ++i)
      mbar_wait(&full[i % S], (i / S) & 1, p.status, p.wait_limit);
  } else if (warp == 1) {
    if (rank == 0) {   // the whole warp runs the loop, so that its values stay in uniform registers
      // ---------------- MMA issuer ----------------
      // (one base descriptor plus per-stage and per-slice offsets, see the prefill kernel)
      constexpr uint32_t idesc = idesc_f16_f32(2 * kBM, BN);
      const uint64_t dbase = desc_sw128_kmajor(smem_u32(smem));
      bool ok = true;
      int s = 0, a = 0, aph = 0;   // ring stage, A stage and its phase
      for (int part = first_part, it = 0;; ++it) {
        const int steps = __shfl_sync(0xffffffffu, nK, 0), nD = __shfl_sync(0xffffffffu, to.steps, 0);
        if (it > 0) ok = __all_sync(0xffffffffu, mbar_wait(acce, (it - 1) & 1, p.status, p.wait_limit));
        for (int i = 0; i < steps && ok; ++i) {
          ok = mbar_wait(&afull[a], aph, p.status, p.wait_limit);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t ds = dbase + (uint64_t)((s * L::kBytes) >> 4);
            const uint32_t at = tmem + BN + 64 * a;
            if (i < nD) {
              mma_f16_ts_pair(tmem, at, ds, idesc, i != 0);
              #pragma unroll
              for (int kk = 1; kk < 8; ++kk)
                mma_f16_ts_pair(tmem, at + 8 * kk, ds + (uint64_t)((((kk >> 2) * BN * 64) + (kk & 3) * 32) >> 4), idesc, 1u);
            } else {   // only the slices that hold weak columns
              #pragma unroll 1
              for (int kk = 0; kk < 8; ++kk)
                if ((i - nD) * 64 + (kk & 3) * 16 < p.k_ld[kk >> 2])
                  mma_f16_ts_pair(tmem, at + 8 * kk, ds + (uint64_t)((((kk >> 2) * BN * 64) + (kk & 3) * 32) >> 4), idesc, 1u);
            }
            mma_commit_pair(&empty[s]);
          }
          __syncwarp();
          if (++s == S) s = 0;
          if (++a == kS2) { a = 0; aph ^= 1; }
        }
        if (elect_one()) mma_commit_pair(accf);
        __syncwarp();
        if (!ok || (part += P) >= parts) break;
        next(part);
      }
    }
  } else {
    // ---------------- A operand ----------------
    // kDW / kGR warps of a group, NSL = kDW / kGR / 4 per lane quarter; thread (MMA row r, slab jh)
    // writes codes 8 U jh .. 8 U jh + 8 U - 1 of its row (U = 16 / NSL), as in the prefill kernel
    constexpr int NSL = kDW / kGR / 4, U = 16 / NSL;
    const int quarter = warp & 3, aw = warp - 2, grp = aw / (kDW / kGR), jh = (aw % (kDW / kGR)) >> 2;
    const int lay = lane >> 4, tr = 16 * quarter + (lane & 15);   // layer and row of the tile
    const uint32_t lane_base = (uint32_t)(32 * quarter) << 16;
    constexpr int kCols = BN / (kDW / 4);   // accumulator columns of this warp in the epilogue
    const int col0 = (aw >> 2) * kCols;
    const uint32_t acc = tmem + lane_base + (uint32_t)col0;
    RowDq<BITS> dq;
    int orow = n0 + tr, row = min(orow, p.N - 1);
    auto channel = [&]() {
      dq.set((uint32_t)__half_as_ushort(p.scales[lay][row]) | (uint32_t)__half_as_ushort(p.zeros[lay][row]) << 16);
    };
    if (!per_group) channel();
    TileOf ep = to;            // the part before, and this thread's output row in it
    int erow = orow, em0 = m0;
    int part = first_part, g0 = 0, i = grp, it = 0;   // g0: the part's first step, over all parts; it: parts before it
    int stop = nK;             // with an epilogue pending: after the steps that run ahead of it
    bool ok = true, pending = false;
    const uint32_t ring = smem_u32(smem);
    auto ready = [&](int g) {   // step g's loads have landed and its A stage's last MMAs are done
      bool r = mbar_wait(&full[g % S], (g / S) & 1, p.status, p.wait_limit);
      if (g >= kS2) r = mbar_wait(&empty[(g - kS2) % S], ((g - kS2) / S) & 1, p.status, p.wait_limit) && r;
      r = __all_sync(0xffffffffu, r);
      tc_fence_after();
      return r;
    };
    auto put = [&](int g, const uint32_t (&d)[U / 4][16]) {
      const uint32_t at = tmem + lane_base + BN + 64 * (g % kS2) + 4 * U * jh;
      #pragma unroll
      for (int h = 0; h < U / 4; ++h) tmem_st16(at + 16 * h, d[h]);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0 && !(p.skip_arrive && g == 0 && threadIdx.x == 64)) mbar_arrive_remote(&afull[g % kS2], 0);
    };
    while (true) {
      const int nD = to.steps, dense = min(stop, nD);
      for (; i < dense && ok; i += kGR) {
        const int g = g0 + i;
        if (!(ok = ready(g))) break;
        const uint32_t st = ring + (g % S) * L::kBytes;
        if (per_group) dq.set(lds_u1(st + L::kX + L::kP + lay * (L::kSZ / 2) + tr * 4));
        uint32_t w[4 * BITS], d[U / 4][16];
        #pragma unroll
        for (int v = 0; v < BITS; ++v) {
          const uint4 q = lds_u4(st + L::kX + lay * (L::kP / 2) + tr * 16 * BITS + 16 * v);
          w[4 * v] = q.x; w[4 * v + 1] = q.y; w[4 * v + 2] = q.z; w[4 * v + 3] = q.w;
        }
        auto units = [&](auto sl_c) {
          constexpr int SL = decltype(sl_c)::value;
          #pragma unroll
          for (int ju = 0; ju < U; ++ju)
            #pragma unroll
            for (int q = 0; q < 4; ++q)
              d[ju >> 2][4 * (ju & 3) + q] = dequant<BITS>(w + q * BITS, U * SL + ju, dq);
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
        put(g, d);
      }
      #pragma unroll 1
      for (; i < stop && ok; i += kGR) {
        // weak step: slab jh covers columns c0 .. c0 + 8 U - 1 of layer wl's part of the step
        const int g = g0 + i, wl = (8 * U * jh) / 64, c0 = (i - nD) * 64 + (8 * U * jh) % 64;
        const uint4* src = reinterpret_cast<const uint4*>(p.w_weak[lay] + (size_t)row * p.k_ld[lay] + c0);
        uint32_t d[U / 4][16];
        #pragma unroll
        for (int v = 0; v < U; ++v) {
          const uint4 q = (lay == wl && orow < p.N && c0 + 8 * v < p.k_ld[lay]) ? src[v] : make_uint4(0, 0, 0, 0);
          d[v >> 2][4 * (v & 3)] = q.x; d[v >> 2][4 * (v & 3) + 1] = q.y;
          d[v >> 2][4 * (v & 3) + 2] = q.z; d[v >> 2][4 * (v & 3) + 3] = q.w;
        }
        if (!(ok = ready(g))) break;   // (the weak block is static: its loads are under way meanwhile)
        put(g, d);
      }
      if (!ok) break;
      if (pending) {
        // ---------------- epilogue of the part before ----------------
        auto wait = [&]() {
          const bool acc_ok = __all_sync(0xffffffffu, mbar_wait(accf, (it - 1) & 1, p.status, p.wait_limit));
          tc_fence_after();
          return acc_ok;
        };
        if (ep.n_splits > 1) {   // this split's fp32 partials
          const bool acc_ok = wait();
          float* w = p.ws + partial_at(p.split, ep.split, ep.tile, rank, BN) + (size_t)col0 * kBM + 32 * quarter + lane;
          #pragma unroll 1
          for (int c = 0; c < kCols && acc_ok; c += 16) {
            uint32_t v[16];
            tmem_ld16(acc + (uint32_t)c, v);
            tmem_ld_wait();
            #pragma unroll
            for (int j = 0; j < 16; ++j) w[(size_t)(c + j) * kBM] = __uint_as_float(v[j]);
          }
        } else {
          with_act(p.act, [&](auto act) {
            constexpr int A = decltype(act)::value;
            const int first = em0 + col0 + 8 * lay;
            if (p.dh) gated_epilogue<A, true, kCols>(p, acc, first, erow, lay, wait);
            else gated_epilogue<A, false, kCols>(p, acc, first, erow, lay, wait);
          });
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(acce, 0);
        if (part >= parts) break;
        pending = false;
        stop = nK;
      } else {   // the next part
        pending = true;
        g0 += nK;
        i -= nK;
        ++it;
        part += P;
        ep = to;
        erow = orow;
        em0 = m0;
        stop = i;
        if (part < parts) {
          next(part);
          orow = n0 + tr;
          row = min(orow, p.N - 1);
          if (!per_group) channel();
          stop = min(kS2, nK);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();   // neither CTA leaves, or frees tensor memory, while the pair's MMAs may use it
  if (warp == 1) {
    tc_fence_after();
    tmem_free_pair(tmem, kTmemCols);
  }
}

// Weak activations of every token for both layers: xw[l][m][t] = x[m][idx_l[t]] (0 past k_l).
struct GatherArgs {
  const int32_t* idx[2];
  __half* xw[2];
  int k[2], k_ld[2];   // k_ld 0: no weak columns
};
__global__ void k_gated_gather(const __half* __restrict__ x, int M, int K, const __grid_constant__ GatherArgs a, int* status) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the product's dense steps need none of this
  const int ld = a.k_ld[0] + a.k_ld[1];
  const size_t n = (size_t)M * ld;
  for (size_t e = (size_t)blockIdx.x * blockDim.x + threadIdx.x; e < n; e += (size_t)gridDim.x * blockDim.x) {
    const size_t m = e / ld;
    const int c = (int)(e % ld), l = c >= a.k_ld[0], t = l ? c - a.k_ld[0] : c;
    a.xw[l][m * a.k_ld[l] + t] = t < a.k[l] && in_range(a.idx[l][t], K, status) ? x[m * K + a.idx[l][t]] : __float2half_rn(0.f);
  }
}

// The split tiles: their partials added in split order, then the epilogue.  A warp takes one token
// of a tile and 32 of its 64 outputs (two runs of 16 MMA rows of either layer).
__global__ void k_gated_reduce(const __grid_constant__ GatedGemmParams p, int BN) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int n_tiles = p.split.tiles - p.split.whole;
  const size_t n = (size_t)n_tiles * 2 * BN * kHalfRows, stride = (size_t)n_tiles * 2 * BN * kBM;
  for (size_t e = (size_t)blockIdx.x * blockDim.x + threadIdx.x; e < n; e += (size_t)gridDim.x * blockDim.x) {
    const int r = (int)(e % kHalfRows), t0 = (int)(e / kHalfRows % BN), u = (int)(e / kHalfRows / BN);
    const int tile = p.split.whole + u / 2, rank = u % 2;
    const int row = ((tile % p.rts) * 2 + rank) * kHalfRows + r, t = (tile / p.rts) * BN + t0;
    if (row >= p.N || t >= p.M) {
      if (p.dy2[0] && row < p.ld2 && t < p.M) { store_halves(p, 0, t, row, 0.f); store_halves(p, 1, t, row, 0.f); }
      continue;
    }
    const float* w = p.ws + partial_at(p.split, 0, tile, rank, BN) + (size_t)t0 * kBM + 32 * (r / 16) + r % 16;
    float gs = 0.f, us = 0.f;
    for (int z0 = 0; z0 < p.split.splits; z0 += 8) {   // eight splits' loads in flight
      float gz[8], uz[8];
      #pragma unroll
      for (int z = 0; z < 8; ++z) {
        const bool ok = z0 + z < p.split.splits;
        gz[z] = ok ? w[(z0 + z) * stride] : 0.f;
        uz[z] = ok ? w[(z0 + z) * stride + 16] : 0.f;
      }
      #pragma unroll
      for (int z = 0; z < 8; ++z) {
        gs += gz[z];
        us += uz[z];
      }
    }
    const size_t o = (size_t)t * p.N + row;
    with_act(p.act, [&](auto act) {
      constexpr int A = decltype(act)::value;
      if (p.dh) gated_store<A, true>(p, o, t, row, gs, us, p.dh[o]);
      else gated_store<A, false>(p, o, t, row, gs, us, __float2half_rn(0.f));
    });
  }
}

// ---------------------------------------------------------------- input gradient of both layers
// dx = dg Wg + du Wu as dx^T tiles of 128 columns (MMA M, one packed block) x BN tokens (MMA N),
// the contraction running over the gate's rows and then the up layer's, 128 rows a step, into one
// accumulator.  The A operand is W_hat^T.  A warp forms it as the decode product forms its
// fragments: lane (g, t) reads chunk t of row g of an 8-row group, so that each dequantised pair
// register is an 8 x 8 block of the matrix (rows x columns); movmatrix transposes the block in
// registers and tcgen05.st 16x128b puts two of them (16 columns) into 16 tensor-memory lanes, two
// rows packed per 32-bit column.  That is four instructions a pair beside the unpack, and shared
// memory is read only for the packed words (forming the operand column by column took two 64-bit
// shared loads and six instructions per pair of rows: 131 KB of shared reads a step, as long as
// the MMAs).  A step takes 0.45 / 0.53 / 0.64 / 0.80 us at 64 / 128 / 192 / 256 tokens.
// The weak columns' codes give exactly 0; their products with the fp16 weak blocks come from
// k_gated_igw, running beside this kernel, and are added in fp32 in the epilogue of a tile's first
// split, so that a column that is weak in one layer and packed in the other is rounded once.
struct GatedIgMaps {
  CUtensorMap dy[2], p[2], sz[2], dx;
};
struct GatedIgParams {
  float* ws;        // split partials
  int* status;
  int N, K, M, group;
  TileSplit split;  // tile = token tile * ceil(K / 256) + pair of column blocks; steps: 128 rows, the gate's first
  long long wait_limit;
  int skip_arrive;
  int halves;           // tokens 2 t, 2 t + 1 are hi and lo of token t's gradients: dx's row t is hi's + 2^-11 lo's
  const float* wk[2];   // the weak columns' products, [row split][slot][M]
  const int32_t* idx[2];
  int k[2], wsplits;
  uint32_t blk[2][kMaxBlocks];   // per column block: first weak slot << 16 | weak-column count
};

__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
// 16 lanes x 16 columns: register 2 i + h of lane 4 r + c holds lane r + 8 h, column 4 i + c
__device__ __forceinline__ void tmem_st_16x128b_x4(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
               :: "r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// The words of a chunk that its pairs 4 Q .. 4 Q + 3 (columns 32 Q .. 32 Q + 31 of the block) use
template <int BITS, int Q>
__device__ __forceinline__ void ig_load_words(uint32_t a, uint32_t (&w)[BITS]) {
  if constexpr (BITS == 4) {
    const uint2 v = lds_u2(a + 8 * (Q / 2));
    w[2 * (Q / 2)] = v.x;
    w[2 * (Q / 2) + 1] = v.y;
  } else {
    if (Q != 3) { w[0] = lds_u1(a); w[1] = lds_u1(a + 4); }
    if (Q >= 2) w[2] = lds_u1(a + 8);
  }
}

// One warp's share of a step: columns 32 Q .. 32 Q + 31, RG 8-row groups from shared address `pk`
// (packed rows) and `sz` ((scale, zero) pairs), to tensor memory at `at` (lane quarter Q).
template <int BITS, int Q, int RG>
__device__ __forceinline__ void ig_form(uint32_t pk, uint32_t sz, uint32_t at) {
  #pragma unroll
  for (int b = 0; b < RG / 4; ++b) {
    uint32_t v[2][8];   // [16-column half][16x128b registers of four row groups]
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int rg = 4 * b + i;
      uint32_t w[BITS];
      ig_load_words<BITS, Q>(pk + rg * 8 * 16 * BITS, w);
      RowDq<BITS> dq;
      dq.set(lds_u1(sz + rg * 32));
      #pragma unroll
      for (int p = 0; p < 4; ++p)
        v[p >> 1][2 * i + (p & 1)] = movmatrix(dequant<BITS>(w, 4 * Q + p, dq));
    }
    #pragma unroll
    for (int h = 0; h < 2; ++h) tmem_st_16x128b_x4(at + ((uint32_t)(16 * h) << 16) + 16 * b, v[h]);
  }
}

template <int BITS, int BN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(32 * (2 + kDW), 1)
k_gated_igemm(const __grid_constant__ GatedIgMaps maps, const __grid_constant__ GatedIgParams p) {
  using L = Stage<BITS, BN>;
  constexpr int S = L::kS, kS2 = a_stages<BN>();
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S * L::kBytes);
  uint64_t* full = bars;              // [S] TMA landed
  uint64_t* empty = bars + S;         // [S] MMAs of the stage done
  uint64_t* afull = bars + 2 * S;     // [kS2] A stage written in both CTAs (the even CTA's is used)
  uint64_t* accf = bars + 2 * S + kS2;   // accumulator complete
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * S + kS2 + 1);

  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // (warp: uniform)
  const int rank = (int)cluster_ctarank();
  const int Kb = p.K / kStepCodes, Kp = (Kb + 1) / 2;   // column blocks, and pairs of them
  const int nR = (p.N + 127) / 128;     // row steps of one layer
  const TileOf to = tile_of(p.split, blockIdx.x >> 1, 2 * nR);
  const int b = (to.tile % Kp) * 2 + rank;   // this CTA's column block (Kb odd: the last has none; it loads zeros, stores nothing)
  const int m0 = (to.tile / Kp) * BN;        // first token
  const int nK = to.steps;
  const int grp = (b * kStepCodes) / p.group;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < kS2; ++s) mbar_init(&afull[s], 2 * kDW / kGR);   // a lane of each warp, both CTAs
    mbar_init(accf, 1);
    fence_mbar_init();
    #pragma unroll
    for (int l = 0; l < 2; ++l) {
      prefetch_tmap(&maps.dy[l]);
      prefetch_tmap(&maps.p[l]);
      prefetch_tmap(&maps.sz[l]);
    }
  }
  if (warp == 1) tmem_alloc_pair(tmem_slot, kTmemCols);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // both CTAs' barriers and tensor memory are ready
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);

  if (warp == 0) {
    // ---------------- TMA producer (the whole warp, as in the forward product) ----------------
    const int mt = m0 + rank * (BN / 2);   // this CTA's tokens
    bool ok = true;
    int s = 0, ph = 1, i = 0;   // ring stage, phase of its `empty`, steps issued
    for (; i < nK; ++i) {
      if (i >= S) ok = __all_sync(0xffffffffu, mbar_wait(&empty[s], ph, p.status, p.wait_limit));
      if (!ok) break;
      unsigned char* st = smem + s * L::kBytes;
      const int l = to.first + i >= nR, rb = to.first + i - (l ? nR : 0);
      if (elect_one()) {
        mbar_arrive_expect_tx(&full[s], L::kX + L::kP + L::kSZ);
        tma_load_3d(st + L::kX, &maps.p[l], &full[s], 0, b, rb * 8);
        tma_load_3d(st + L::kX + L::kP, &maps.sz[l], &full[s], 0, grp, rb * 8);
        tma_load_2d(st, &maps.dy[l], &full[s], rb * 128, mt);
        tma_load_2d(st + BN * 64, &maps.dy[l], &full[s], rb * 128 + 64, mt);
      }
      __syncwarp();
      if (++s == S) { s = 0; ph ^= 1; }
    }
    // never leave with copies in flight: wait for the last issued use of every stage
    for (int j = (i > S ? i - S : 0); j < i; ++j)
      mbar_wait(&full[j % S], (j / S) & 1, p.status, p.wait_limit);
  } else if (warp == 1) {
    if (rank == 0) {   // the whole warp runs the loop, so that its values stay in uniform registers
      // ---------------- MMA issuer ----------------
      // (one base descriptor plus per-stage and per-slice offsets, see the prefill kernel)
      constexpr uint32_t idesc = idesc_f16_f32(2 * kBM, BN);
      const uint64_t dbase = desc_sw128_kmajor(smem_u32(smem));
      bool ok = true;
      int s = 0;
      for (int i = 0; i < nK && ok; ++i) {
        ok = mbar_wait(&afull[i % kS2], (i / kS2) & 1, p.status, p.wait_limit);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t ds = dbase + (uint64_t)((s * L::kBytes) >> 4);
          const uint32_t at = tmem + BN + 64 * (i % kS2);
          mma_f16_ts_pair(tmem, at, ds, idesc, i != 0);
          #pragma unroll
          for (int kk = 1; kk < 8; ++kk)
            mma_f16_ts_pair(tmem, at + 8 * kk, ds + (uint64_t)((((kk >> 2) * BN * 64) + (kk & 3) * 32) >> 4), idesc, 1u);
          mma_commit_pair(&empty[s]);
        }
        __syncwarp();
        if (++s == S) s = 0;
      }
      if (elect_one()) mma_commit_pair(accf);
    }
  } else {
    // ---------------- A operand: W_hat^T ----------------
    // group grp of the steps; within it lane quarter = warp % 4 (32 columns) and row slab jh
    constexpr int NSL = kDW / kGR / 4, RG = 16 / NSL;   // 8-row groups of a warp's slab
    const int quarter = warp & 3, aw = warp - 2, gr = aw / (kDW / kGR), jh = (aw % (kDW / kGR)) >> 2;
    const int g = lane >> 2, t = lane & 3;
    const uint32_t lane_base = (uint32_t)(32 * quarter) << 16;
    const uint32_t sm = smem_u32(smem);
    bool ok = true;
    for (int i = gr; i < nK && ok; i += kGR) {
      const int s = i % S, u = i / S;
      ok = mbar_wait(&full[s], u & 1, p.status, p.wait_limit);
      if (i >= kS2) ok = mbar_wait(&empty[(i - kS2) % S], ((i - kS2) / S) & 1, p.status, p.wait_limit) && ok;   // the A stage's MMAs
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const uint32_t st = sm + s * L::kBytes;
      const uint32_t pk = st + L::kX + (8 * RG * jh + g) * 16 * BITS + t * 4 * BITS;
      const uint32_t sz = st + L::kX + L::kP + (8 * RG * jh + g) * 4;
      const uint32_t at = tmem + lane_base + BN + 64 * (i % kS2) + 4 * RG * jh;
      switch (quarter) {
        case 0: ig_form<BITS, 0, RG>(pk, sz, at); break;
        case 1: ig_form<BITS, 1, RG>(pk, sz, at); break;
        case 2: ig_form<BITS, 2, RG>(pk, sz, at); break;
        default: ig_form<BITS, 3, RG>(pk, sz, at); break;
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0 && !(p.skip_arrive && i == 0 && threadIdx.x == 64)) mbar_arrive_remote(&afull[i % kS2], 0);
    }

    // ---------------- epilogue ----------------
    // One split: the fp16 tile goes through shared memory ([BN tokens][128 columns], the stages are
    // idle once the accumulator is complete) and out with one TMA store; several: fp32 partials.
    bool acc_ok = __all_sync(0xffffffffu, mbar_wait(accf, 0, p.status, p.wait_limit)) && ok;
    tc_fence_after();
    const int j = 32 * quarter + lane, col = b * kStepCodes + j;   // this thread's column
    __half* s_out = reinterpret_cast<__half*>(smem);
    // the weak columns of this block in either layer: their products' row splits added in order
    // into shared memory (behind the output tile; those that do not fit are added from global)
    constexpr int kWkCap = (S * L::kBytes - BN * kStepCodes * 2) / (BN * 4);
    int slot[2] = {-1, -1}, at_wk[2] = {0, 0}, n_weak = 0;   // this column's weak slot, and its place
    float* s_wk = reinterpret_cast<float*>(smem + BN * kStepCodes * 2);   // [weak column][BN]
    if (to.split == 0 && b < Kb) {
      #pragma unroll
      for (int l = 0; l < 2; ++l) {
        const int first = p.k[l] > 0 ? (int)(p.blk[l][b] >> 16) : 0, cnt = p.k[l] > 0 ? (int)(p.blk[l][b] & 0xFFFFu) : 0;
        if (n_weak == 0 && cnt > 0) asm volatile("griddepcontrol.wait;" ::: "memory");   // k_gated_igw's results
        for (int c = 0; c < cnt; ++c)
          if (in_range(first + c, p.k[l], p.status) && p.idx[l][first + c] == col) { slot[l] = first + c; at_wk[l] = n_weak + c; }
        const size_t plane = (size_t)p.k[l] * p.M;
        for (int e = (int)threadIdx.x - 64; e < min(cnt, kWkCap - n_weak) * BN && acc_ok; e += 32 * kDW) {
          const int c = e / BN, tk = e - c * BN;
          float v = 0.f;
          if (m0 + tk < p.M) {
            const float* wk = p.wk[l] + (size_t)(first + c) * p.M + m0 + tk;
            for (int z0 = 0; z0 < p.wsplits; z0 += 8) {   // eight splits' loads in flight
              float w[8];
              #pragma unroll
              for (int z = 0; z < 8; ++z) w[z] = z0 + z < p.wsplits ? __ldcg(wk + (z0 + z) * plane) : 0.f;
              #pragma unroll
              for (int z = 0; z < 8; ++z) v += w[z];
            }
          }
          s_wk[(n_weak + c) * BN + tk] = v;
        }
        n_weak += cnt;
      }
      named_bar_sync(1, 32 * kDW);
    }
    constexpr int kCols = BN / (kDW / 4);   // accumulator columns (tokens) of this warp
    const int col0 = (aw >> 2) * kCols;
    #pragma unroll 1
    for (int c0 = col0; c0 < col0 + kCols; c0 += 16) {
      uint32_t v[16];
      tmem_ld16(tmem + lane_base + (uint32_t)c0, v);
      tmem_ld_wait();
      #pragma unroll
      for (int l = 0; l < 2; ++l)
        if (slot[l] >= 0) {
          if (at_wk[l] < kWkCap) {
            #pragma unroll
            for (int tk = 0; tk < 16; ++tk) v[tk] = __float_as_uint(__uint_as_float(v[tk]) + s_wk[at_wk[l] * BN + c0 + tk]);
          } else {
            #pragma unroll
            for (int tk = 0; tk < 16; ++tk) {
              float w = 0.f;
              for (int z = 0; z < p.wsplits && m0 + c0 + tk < p.M; ++z)
                w += __ldcg(p.wk[l] + ((size_t)z * p.k[l] + slot[l]) * p.M + m0 + c0 + tk);
              v[tk] = __float_as_uint(__uint_as_float(v[tk]) + w);
            }
          }
        }
      if (to.n_splits > 1) {
        if (acc_ok) {
          float* w = p.ws + partial_at(p.split, to.split, to.tile, rank, BN) + (size_t)c0 * kBM + j;
          #pragma unroll
          for (int tk = 0; tk < 16; ++tk) w[tk * kBM] = __uint_as_float(v[tk]);
        }
      } else {
        if (p.halves) {
          #pragma unroll
          for (int tk = 0; tk < 16; tk += 2)
            sts_u16(smem_u32(s_out) + 2 * ((c0 + tk) / 2 * kStepCodes + j),
                    __half_as_ushort(__float2half_rn(fmaf(__uint_as_float(v[tk + 1]), 1.f / kLoScale, __uint_as_float(v[tk])))));
        } else {
          #pragma unroll
          for (int tk = 0; tk < 16; ++tk)
            sts_u16(smem_u32(s_out) + 2 * ((c0 + tk) * kStepCodes + j), __half_as_ushort(__float2half_rn(__uint_as_float(v[tk]))));
        }
      }
    }
    if (to.n_splits == 1) {
      fence_proxy_async_smem();          // the tile, written by the generic proxy, to the TMA
      named_bar_sync(1, 32 * kDW);       // every A thread's part of the tile is written
      if (warp == 2 && lane == 0 && acc_ok && b < Kb) {
        tma_store_2d(&maps.dx, s_out, b * kStepCodes, m0);
        bulk_commit();
        bulk_wait_read0();               // shared memory read out before the CTA may exit
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();   // neither CTA leaves, or frees tensor memory, while the pair's MMAs may use it
  if (warp == 1) {
    tc_fence_after();
    tmem_free_pair(tmem, kTmemCols);
  }
}

// dx of the split tiles = fp16_rn(their partials added in split order)
__global__ void k_gated_ig_reduce(const __grid_constant__ GatedIgParams p, int BN, __half* __restrict__ dx) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int n_tiles = p.split.tiles - p.split.whole, Kb = p.K / kStepCodes, Kp = (Kb + 1) / 2;
  const size_t n = (size_t)n_tiles * 2 * BN * kBM;
  for (size_t e = 4 * ((size_t)blockIdx.x * blockDim.x + threadIdx.x); e < n; e += 4 * (size_t)gridDim.x * blockDim.x) {
    const int c = (int)(e % kBM), t0 = (int)(e / kBM % BN), u = (int)(e / kBM / BN), tile = p.split.whole + u / 2;
    const int b = (tile % Kp) * 2 + u % 2, t = (tile / Kp) * BN + t0;
    if (t >= p.M || b >= Kb || (p.halves && (t & 1))) continue;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int h = p.halves; h >= 0; --h) {   // lo's products first
      for (int z0 = 0; z0 < p.split.splits; z0 += 8) {   // eight splits' loads in flight
        float4 w[8];
        #pragma unroll
        for (int z = 0; z < 8; ++z)
          w[z] = z0 + z < p.split.splits ? *reinterpret_cast<const float4*>(p.ws + (size_t)(z0 + z) * n + e + h * kBM)
                                         : make_float4(0.f, 0.f, 0.f, 0.f);
        #pragma unroll
        for (int z = 0; z < 8; ++z) { v.x += w[z].x; v.y += w[z].y; v.z += w[z].z; v.w += w[z].w; }
      }
      if (h) { v.x *= 1.f / kLoScale; v.y *= 1.f / kLoScale; v.z *= 1.f / kLoScale; v.w *= 1.f / kLoScale; }
    }
    __half2* o = reinterpret_cast<__half2*>(dx + (size_t)(t >> p.halves) * p.K + b * kStepCodes + c);
    o[0] = __floats2half2_rn(v.x, v.y);
    o[1] = __floats2half2_rn(v.z, v.w);
  }
}

// The weak columns' products of both layers, wk[l][row split][slot][m] = sum_i dy_l[m][i]
// w_weak_l[i][slot] (mma.sync m16n8k16: rows = tokens, K = weight rows, columns = slots).  A CTA of
// 4 warps computes 64 tokens x CT slots of one layer over one split of the rows, 64 rows at a time
// through a 4-stage cp.async ring.  Bound by reading the gradients, once per CT slots: 13824 rows,
// 2048 tokens, 40 slots of each layer 36.8 us (113 MB, 3.1 TB/s; 46 us with 64-byte pieces and five
// splits), 11008 rows, 256 tokens 7.1 us.  (Weak columns put into the A operand instead, loaded over
// their dequantised registers, made every step longer: 866 -> 937 us at 2048 tokens.)
constexpr int kIwTok = 64, kIwRows = 64, kIwThreads = 128, kIwStages = 4, kIwMaxSplits = 16;
constexpr int kIwDyLd = kIwRows + 8;   // padded row stride (halves)

struct GatedIgwArgs {
  const __half* dy[2];
  const __half* w[2];   // [N][k_ld]
  float* wk[2];
  int k[2], k_ld[2], ctiles0;   // slot tiles of the gate layer (blockIdx.y below it)
  int N, ldy, M, per;           // per: rows per split, a multiple of kIwRows
};
template <int CT>
constexpr int igw_smem_bytes() { return kIwStages * (kIwTok * kIwDyLd + kIwRows * (CT + 8)) * (int)sizeof(__half); }
template <int CT>
__global__ void __launch_bounds__(kIwThreads) k_gated_igw(const __grid_constant__ GatedIgwArgs a) {
  extern __shared__ __align__(1024) unsigned char smem[];
  auto s_dy = reinterpret_cast<__half (*)[kIwTok][kIwDyLd]>(smem);
  auto s_w = reinterpret_cast<__half (*)[kIwRows][CT + 8]>(s_dy + kIwStages);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the packed product runs beside this
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int l = (int)blockIdx.y >= a.ctiles0;
  const __half* __restrict__ dy = a.dy[l];
  const __half* __restrict__ w = a.w[l];
  const int k = a.k[l], k_ld = a.k_ld[l];
  const int mb = blockIdx.x * kIwTok, t0 = ((int)blockIdx.y - (l ? a.ctiles0 : 0)) * CT;
  const int i_lo = blockIdx.z * a.per, i_hi = min(a.N, i_lo + a.per);
  const int nchunk = max(0, (i_hi - i_lo + kIwRows - 1) / kIwRows);
  auto load = [&](int c, int st) {   // rows i_lo + 64 c .. of this split into stage st
    const int ib = i_lo + c * kIwRows;
    #pragma unroll
    for (int u = 0; u < kIwTok * kIwRows / 8 / kIwThreads; ++u) {   // dY: 8-row pieces (rows N .. ldy - 1 hold zeros)
      const int e = tid + u * kIwThreads, m = e / (kIwRows / 8), pc = e % (kIwRows / 8);
      const int mm = mb + m, row = ib + pc * 8;
      const bool ok = mm < a.M && row < i_hi;
      cp_async16(&s_dy[st][m][pc * 8], dy + (ok ? (size_t)mm * a.ldy + row : 0), ok);
    }
    #pragma unroll
    for (int u = 0; u < kIwRows * CT / 8 / kIwThreads; ++u) {       // weak block: CT / 8 pieces of 8 slots a row
      const int e = tid + u * kIwThreads, r = e / (CT / 8), pc = e % (CT / 8), row = ib + r, col = t0 + pc * 8;
      const bool ok = row < i_hi && col < k_ld;
      cp_async16(&s_w[st][r][pc * 8], w + (ok ? (size_t)row * k_ld + col : 0), ok);
    }
  };
  float d[CT / 8][4];
  #pragma unroll
  for (int n = 0; n < CT / 8; ++n)
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
      for (int nh = 0; nh < CT / 16; ++nh) {
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
  for (int n = 0; n < CT / 8; ++n)
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

// Measured times (us): a step of 128 codes, and of a tile what its neighbours do not hide (the
// accumulator's way out).  Steps below 256 tokens are paced by forming the A operand, which the
// tokens share; from there on by the MMAs.
struct TileCost {
  double step, tile;
};
TileCost fwd_cost(int BN) { return {BN == 64 ? 0.37 : BN == 128 ? 0.41 : BN == 192 ? 0.51 : 0.68, 0.016 * BN}; }
TileCost ig_cost(int BN) { return {BN == 64 ? 0.44 : BN == 128 ? 0.54 : BN == 192 ? 0.65 : 0.81, 0.010 * BN}; }

// The split of T tiles of `steps` steps over the SM pairs (see TileSplit): at least 4 steps a split, and
// only where the saved steps exceed the partials' way through L2 and the reduction's launch (about
// 4 us).  `us`: the estimate of the whole product.
TileSplit plan_split(long long T, int steps, int BN, TileCost c, int sms, double& us) {
  const int P = std::max(1, sms / 2);
  TileSplit s = {(int)T, (int)T, 1, steps};
  us = (double)((T + P - 1) / P) * (steps * c.step + c.tile);
  const int rem = (int)(T % P);
  if (rem == 0) return s;
  int n = std::min(P / rem, steps / 4);
  if (n < 2) return s;
  const int per = (steps + n - 1) / n;
  n = (steps + per - 1) / per;
  const double cost_us = 4.0 + 4.0 * n * rem * BN * kBM * sizeof(float) / 5e6;
  if ((steps - per) * c.step <= cost_us) return s;
  us -= (steps - per) * c.step - cost_us;
  s.whole = (int)(T - rem);
  s.splits = n;
  s.steps = per;
  return s;
}

// Tokens of a tile, for `rows` tiles across the other dimension: the width with the least estimate, a
// narrower one only for 5% and 1 us less.  Wide tiles form an A operand for more tokens; narrower ones
// leave fewer columns beyond M and fill the last wave better.  Measured, forward: 5461 x 2048 at 333
// tokens, tiles of 128 / 192 / 256: 24.4 / 26.7 / 33.0 us; 11008 x 4096 at 256 tokens: 50.5 / 56.8 /
// 44.0 us.  Over 120 products (six shapes, 64 to 1024 tokens, both directions) the choice is within
// 0.4% of the best width on average and 11% at most.
int pick_tile(int M, long long rows, int steps, int sms, TileCost (*cost)(int), TileSplit& split) {
  int best = 0;
  double best_us = 0;
  for (int BN = 256; BN >= 64; BN -= 64) {
    if (BN > 64 && M <= BN - 64) continue;   // (a narrower one holds them all)
    double us;
    const TileSplit s = plan_split(rows * ((M + BN - 1) / BN), steps, BN, cost(BN), sms, us);
    if (!best || us < 0.95 * best_us - 1.0) {
      best = BN;
      best_us = us;
      split = s;
    }
  }
  return best;
}
// the tiles of the forward product (128 output rows a pair) and of the input gradient (256 columns a pair)
int fwd_tiles(int N, int K, int M, int sms, TileSplit& split) {
  return pick_tile(M, (N + 2 * kHalfRows - 1) / (2 * kHalfRows), K / kStepCodes, sms, fwd_cost, split);
}
int ig_tiles(int N, int K, int M, int sms, TileSplit& split) {
  return pick_tile(M, (K / kStepCodes + 1) / 2, 2 * ((N + 127) / 128), sms, ig_cost, split);
}
size_t partial_bytes(const TileSplit& s, int BN) {
  return s.splits > 1 ? up256((size_t)s.splits * (s.tiles - s.whole) * 2 * BN * kBM * sizeof(float)) : 0;
}

cudaError_t launch_pdl(void* kern, dim3 grid, int threads, size_t smem, bool pdl, cudaStream_t s, void** args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelExC(&cfg, kern, args);
}

// workspace of one forward / backward product: both layers' weak activations, then the split partials
struct FwdPlan {
  int BN, rts;
  TileSplit split;
  size_t xw[2], ws, total;  // byte offsets
  __half* dy2[2] = {nullptr, nullptr};   // see GatedGemmParams
  int ld2 = 0;
};
FwdPlan fwd_plan(const Layer& gate, const Layer& up, int M) {
  FwdPlan f;
  f.rts = (gate.N + 2 * kHalfRows - 1) / (2 * kHalfRows);
  f.BN = fwd_tiles(gate.N, gate.K, M, layer_sm_count(gate.device), f.split);
  size_t at = 0;
  const Layer* L[2] = {&gate, &up};
  for (int l = 0; l < 2; ++l) {
    f.xw[l] = at;
    if (L[l]->k > 0) at += up256((size_t)M * L[l]->k_ld * sizeof(__half));
  }
  f.ws = at;
  f.total = at + partial_bytes(f.split, f.BN);
  return f;
}

template <int BITS, int BN>
owq_status_t run_gemm(const Layer& gate, const Layer& up, int act, const __half* x, const __half* dh, __half* out0, __half* out1,
                      int M, const FwdPlan& f, unsigned char* ws, long long wait_limit, bool skip_arrive, cudaStream_t s) {
  const Layer* L[2] = {&gate, &up};
  GatedMaps maps;
  GatedGemmParams prm;
  GatherArgs ga;
  if (!encode_2d(&maps.x, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, x, (uint64_t)gate.K, (uint64_t)M, (uint64_t)gate.K * 2, 64, BN / 2,
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
    maps.p[l] = L[l]->gated_p[0];
    maps.sz[l] = L[l]->gated_sz[0];
    maps.xw[l] = maps.x;   // (a layer without weak columns: x itself, loaded and never multiplied)
    if (L[l]->k > 0 &&
        !encode_2d(&maps.xw[l], CU_TENSOR_MAP_DATA_TYPE_FLOAT16, ga.xw[l], (uint64_t)L[l]->k_ld, (uint64_t)M, (uint64_t)L[l]->k_ld * 2,
                   64, BN / 2, CU_TENSOR_MAP_SWIZZLE_128B))
      return OWQ_ERR_CUDA;
  }
  prm.dh = dh;
  prm.out[0] = out0;
  prm.out[1] = out1;
  prm.dy2[0] = f.dy2[0];
  prm.dy2[1] = f.dy2[1];
  prm.ld2 = f.ld2;
  prm.status = gate.status;
  prm.N = gate.N; prm.K = gate.K; prm.M = M; prm.G = gate.G; prm.act = act;
  prm.wait_limit = wait_limit; prm.skip_arrive = skip_arrive ? 1 : 0;
  prm.nw = (std::max(prm.k_ld[0], prm.k_ld[1]) + 63) / 64;
  prm.rts = f.rts;
  prm.split = f.split;
  prm.ws = reinterpret_cast<float*>(ws + f.ws);
  auto kern = k_gated_gemm<BITS, BN>;
  constexpr int smem = ring_smem_bytes<BITS, BN>();
  static_assert(smem <= 232448 && 2 * smem > 232448, "one CTA per SM: the tensor memory of one");
  static_assert(BN + 64 * a_stages<BN>() <= (int)kTmemCols, "tensor memory: accumulator + A stages");
  static_assert(Stage<BITS, BN>::kS >= a_stages<BN>(), "an A stage's MMAs are waited for on the ring's barriers");
  static std::atomic<unsigned long long> allowed{0};
  if (allow_smem((const void*)kern, smem, gate.device, allowed) != cudaSuccess) {
    cudaGetLastError();
    return OWQ_ERR_CUDA;
  }
  const int ld = ga.k_ld[0] + ga.k_ld[1];
  if (ld > 0) {
    k_gated_gather<<<blocks_for((size_t)M * ld, 256, 2048), 256, 0, s>>>(x, M, gate.K, ga, prm.status);
    if (cudaGetLastError() != cudaSuccess) return OWQ_ERR_CUDA;
  }
  // beside the gather: only the weak steps wait for it
  void* args[] = {&maps, &prm};
  if (launch_pdl((void*)kern, dim3(2 * std::min(f.split.pairs(), layer_sm_count(gate.device) / 2)), 32 * (2 + kDW), smem, ld > 0, s, args) != cudaSuccess) {
    cudaGetLastError();
    allowed = 0;
    return OWQ_ERR_CUDA;
  }
  if (f.split.splits > 1) {
    int bn = BN;
    void* rargs[] = {&prm, &bn};
    const size_t n = (size_t)(f.split.tiles - f.split.whole) * 2 * BN * kHalfRows;
    if (launch_pdl((void*)k_gated_reduce, dim3(blocks_for(n, 256, 4096)), 256, 0, true, s, rargs) != cudaSuccess) {
      cudaGetLastError();
      return OWQ_ERR_CUDA;
    }
  }
  return OWQ_OK;
}

template <int BITS>
owq_status_t dispatch_gemm(const Layer& gate, const Layer& up, int act, const __half* x, const __half* dh, __half* out0,
                           __half* out1, int M, const FwdPlan& f, unsigned char* ws, long long wl, bool skip, cudaStream_t s) {
  switch (f.BN) {
    case 64: return run_gemm<BITS, 64>(gate, up, act, x, dh, out0, out1, M, f, ws, wl, skip, s);
    case 192: return run_gemm<BITS, 192>(gate, up, act, x, dh, out0, out1, M, f, ws, wl, skip, s);
    case 128: return run_gemm<BITS, 128>(gate, up, act, x, dh, out0, out1, M, f, ws, wl, skip, s);
    default: return run_gemm<BITS, 256>(gate, up, act, x, dh, out0, out1, M, f, ws, wl, skip, s);
  }
}

// workspace of one input gradient: padded gradients (N % 8 != 0), the weak products, the split partials
struct IgPlan {
  int BN;
  TileSplit split;
  int ldy, ct, wsplits, wper;   // weak products: slots of a tile, row splits, rows of a split
  size_t pad[2], wk[2], ws, total;
  bool halves;   // of each token's gradients two rows, already padded
};
IgPlan ig_plan(const Layer& gate, const Layer& up, int tokens, bool halves = false) {
  IgPlan f;
  const int M = halves ? 2 * tokens : tokens;
  f.halves = halves;
  const int sms = layer_sm_count(gate.device);
  f.BN = ig_tiles(gate.N, gate.K, M, sms, f.split);
  f.ldy = (gate.N + 7) & ~7;
  size_t at = 0;
  for (int l = 0; l < 2; ++l) {
    f.pad[l] = at;
    if (gate.N % 8 && !halves) at += up256((size_t)M * f.ldy * sizeof(__half));
  }
  // weak products: up to three CTAs per SM; at least 4 chunks of rows and at most kIwMaxSplits splits
  // (the input gradient's epilogue adds them)
  f.ct = std::max(gate.k, up.k) > 32 ? 64 : 32;
  const int R = (M + kIwTok - 1) / kIwTok, C = (gate.k + f.ct - 1) / f.ct + (up.k + f.ct - 1) / f.ct;
  const int nch = (gate.N + kIwRows - 1) / kIwRows;
  f.wsplits = C > 0 ? std::max(1, std::min({3 * sms / (R * C), nch / 4, kIwMaxSplits})) : 1;
  f.wper = (nch + f.wsplits - 1) / f.wsplits;
  f.wsplits = (nch + f.wper - 1) / f.wper;
  f.wper *= kIwRows;
  f.wk[0] = at;
  at += up256((size_t)f.wsplits * gate.k * M * sizeof(float));
  f.wk[1] = at;
  at += up256((size_t)f.wsplits * up.k * M * sizeof(float));
  f.ws = at;
  f.total = at + partial_bytes(f.split, f.BN);
  return f;
}

template <int CT>
cudaError_t launch_igw(const GatedIgwArgs& a, dim3 grid, int device, cudaStream_t s) {
  static std::atomic<unsigned long long> allowed{0};
  constexpr int smem = igw_smem_bytes<CT>();
  const cudaError_t e = allow_smem((const void*)k_gated_igw<CT>, smem, device, allowed);
  if (e != cudaSuccess) return e;
  k_gated_igw<CT><<<grid, kIwThreads, smem, s>>>(a);
  return cudaGetLastError();
}

template <int BITS, int BN>
owq_status_t run_ig(const Layer& gate, const Layer& up, const __half* dg, const __half* du, __half* dx, int tokens, const IgPlan& f,
                    unsigned char* ws, long long wait_limit, bool skip_arrive, cudaStream_t s) {
  const int M = f.halves ? 2 * tokens : tokens;
  const Layer* L[2] = {&gate, &up};
  const __half* dy[2] = {dg, du};
  if (gate.N % 8 && !f.halves) {
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
    if (!encode_2d(&maps.dy[l], CU_TENSOR_MAP_DATA_TYPE_FLOAT16, dy[l], (uint64_t)gate.N, (uint64_t)M, (uint64_t)f.ldy * 2, 64, BN / 2,
                   CU_TENSOR_MAP_SWIZZLE_128B))
      return OWQ_ERR_CUDA;
    maps.p[l] = L[l]->gated_p[1];
    maps.sz[l] = L[l]->gated_sz[1];
    prm.wk[l] = wa.wk[l] = reinterpret_cast<float*>(ws + f.wk[l]);
    prm.idx[l] = L[l]->idx;
    prm.k[l] = wa.k[l] = L[l]->k;
    for (int b = 0; b < Kb; ++b) prm.blk[l][b] = L[l]->blk_weak[b];
    wa.dy[l] = dy[l];
    wa.w[l] = L[l]->w_weak;
    wa.k_ld[l] = L[l]->k_ld;
  }
  if (!encode_2d(&maps.dx, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, dx, (uint64_t)gate.K, (uint64_t)tokens, (uint64_t)gate.K * 2, kStepCodes, BN,
                 CU_TENSOR_MAP_SWIZZLE_NONE))
    return OWQ_ERR_CUDA;
  prm.status = gate.status;
  prm.N = gate.N; prm.K = gate.K; prm.M = M; prm.group = gate.group;
  prm.split = f.split;
  prm.wait_limit = wait_limit; prm.skip_arrive = skip_arrive ? 1 : 0;
  prm.wsplits = f.wsplits;
  prm.halves = f.halves ? 1 : 0;
  prm.ws = reinterpret_cast<float*>(ws + f.ws);
  wa.ctiles0 = (gate.k + f.ct - 1) / f.ct;
  wa.N = gate.N; wa.ldy = f.ldy; wa.M = M; wa.per = f.wper;
  const int C = wa.ctiles0 + (up.k + f.ct - 1) / f.ct;
  auto kern = k_gated_igemm<BITS, BN>;
  constexpr int smem = ring_smem_bytes<BITS, BN>();
  static_assert(BN * kStepCodes * 2 <= Stage<BITS, BN>::kS * Stage<BITS, BN>::kBytes, "output tile in the stages");
  static std::atomic<unsigned long long> allowed{0};
  if (allow_smem((const void*)kern, smem, gate.device, allowed) != cudaSuccess) {
    cudaGetLastError();
    return OWQ_ERR_CUDA;
  }
  if (C > 0) {
    const dim3 grid((M + kIwTok - 1) / kIwTok, C, f.wsplits);
    const cudaError_t e = f.ct == 64 ? launch_igw<64>(wa, grid, gate.device, s) : launch_igw<32>(wa, grid, gate.device, s);
    if (e != cudaSuccess) {
      cudaGetLastError();
      return OWQ_ERR_CUDA;
    }
  }
  // beside the weak products: only the epilogues of blocks with weak columns wait for them
  void* args[] = {&maps, &prm};
  if (launch_pdl((void*)kern, dim3(2 * f.split.pairs()), 32 * (2 + kDW), smem, C > 0, s, args) != cudaSuccess) {
    cudaGetLastError();
    allowed = 0;
    return OWQ_ERR_CUDA;
  }
  if (f.split.splits > 1) {
    int bn = BN;
    void* rargs[] = {&prm, &bn, &dx};
    const size_t n = (size_t)(f.split.tiles - f.split.whole) * 2 * BN * kBM;
    if (launch_pdl((void*)k_gated_ig_reduce, dim3(blocks_for(n / 4, 256, 4096)), 256, 0, true, s, rargs) != cudaSuccess) {
      cudaGetLastError();
      return OWQ_ERR_CUDA;
    }
  }
  return OWQ_OK;
}

template <int BITS>
owq_status_t dispatch_ig(const Layer& gate, const Layer& up, const __half* dg, const __half* du, __half* dx, int M, const IgPlan& f,
                         unsigned char* ws, long long wl, bool skip, cudaStream_t s) {
  switch (f.BN) {
    case 64: return run_ig<BITS, 64>(gate, up, dg, du, dx, M, f, ws, wl, skip, s);
    case 192: return run_ig<BITS, 192>(gate, up, dg, du, dx, M, f, ws, wl, skip, s);
    case 128: return run_ig<BITS, 128>(gate, up, dg, du, dx, M, f, ws, wl, skip, s);
    default: return run_ig<BITS, 256>(gate, up, dg, du, dx, M, f, ws, wl, skip, s);
  }
}

}  // namespace

bool encode_gated_maps(Layer& L) {
  for (int i = 0; i < 2; ++i) {
    const int tiles = (i + 1) * kHalfRows / 16;
    if (!encode_packed_3d(&L.gated_p[i], L.packed, L.K, L.N, L.bits, tiles) || !encode_sz_3d(&L.gated_sz[i], L.sz_t, L.G, L.N, tiles))
      return false;
  }
  return true;
}

// The whole backward pass.  Up to kHalvesM tokens dx is formed from both halves of dgate and dup, twice
// as many tokens in a tile that has room for them: its error is then that of its own rounding, where
// the rounding of dgate and dup adds as much again (2.1e-4 and 2.9e-4 relative over many tokens, but
// up to 1.6 times the former over one).  Beyond that it takes them as they are returned.
namespace {
constexpr int kHalvesM = 32;
struct BwdPlan {
  FwdPlan f;
  IgPlan g;
  size_t dy2[2], total;
};
BwdPlan bwd_plan(const Layer& gate, const Layer& up, int M) {
  const bool halves = M <= kHalvesM;
  BwdPlan b = {fwd_plan(gate, up, M), ig_plan(gate, up, M, halves), {0, 0}, 0};
  b.total = std::max(b.f.total, b.g.total);
  for (int l = 0; l < 2 && halves; ++l) {
    b.dy2[l] = b.total;
    b.total += up256((size_t)2 * M * b.g.ldy * sizeof(__half));
  }
  return b;
}
}  // namespace
GatedPlan gated_plan(int N, int K, int M, int sms, int product) {
  TileSplit s;
  const int BN = product == OWQ_GATED_FORWARD
                     ? fwd_tiles(N, K, M, sms, s)
                     : ig_tiles(N, K, product == OWQ_GATED_BACKWARD && M <= kHalvesM ? 2 * M : M, sms, s);
  return {BN, s.tiles, s.whole, s.splits, s.steps};
}
size_t gated_backward_ws_bytes(const Layer& gate, const Layer& up, int M) { return bwd_plan(gate, up, M).total; }
owq_status_t gated_backward_sm100(const Layer& gate, const Layer& up, int act, const __half* x, const __half* dh, __half* dg,
                                  __half* du, __half* dx, int M, void* ws, size_t ws_bytes, long long wait_limit,
                                  bool skip_arrive, cudaStream_t s) {
  BwdPlan b = bwd_plan(gate, up, M);
  if (b.total > ws_bytes) return OWQ_ERR_NOMEM;
  unsigned char* w = static_cast<unsigned char*>(ws);
  const __half* dy[2] = {dg, du};
  if (b.g.halves) {
    b.f.ld2 = b.g.ldy;
    for (int l = 0; l < 2; ++l) dy[l] = b.f.dy2[l] = reinterpret_cast<__half*>(w + b.dy2[l]);
  }
  const owq_status_t st = gate.bits == 3 ? dispatch_gemm<3>(gate, up, act, x, dh, dg, du, M, b.f, w, wait_limit, skip_arrive, s)
                                         : dispatch_gemm<4>(gate, up, act, x, dh, dg, du, M, b.f, w, wait_limit, skip_arrive, s);
  if (st) return st;
  return gate.bits == 3 ? dispatch_ig<3>(gate, up, dy[0], dy[1], dx, M, b.g, w, wait_limit, skip_arrive, s)
                        : dispatch_ig<4>(gate, up, dy[0], dy[1], dx, M, b.g, w, wait_limit, skip_arrive, s);
}

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
                                    void* ws, size_t ws_bytes, long long wait_limit, bool skip_arrive, cudaStream_t s) {
  const IgPlan f = ig_plan(gate, up, M);
  if (f.total > ws_bytes) return OWQ_ERR_NOMEM;
  unsigned char* w = static_cast<unsigned char*>(ws);
  return gate.bits == 3 ? dispatch_ig<3>(gate, up, dg, du, dx, M, f, w, wait_limit, skip_arrive, s)
                        : dispatch_ig<4>(gate, up, dg, du, dx, M, f, w, wait_limit, skip_arrive, s);
}

}  // namespace owq
