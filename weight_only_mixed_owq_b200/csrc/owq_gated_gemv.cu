// Gated block for 1 <= M <= 16 tokens in one launch: h = act(x Wg^T) * (x Wu^T) for two packed
// layers of one shape.
//
// Mathematics: each projection is W_hat x + W_weak x[idx] with W_hat = fp16_rn(s (q - z)), the
// dequantised weight itself for every M (each code pair costs two fp16x2 operations; the cheaper
// form that scales the integer sums differs from W_hat by up to half an fp16 spacing per weight,
// and the product of two projections doubles that).  Sums, activation and product are fp32; h
// is rounded once.
//
// Bound: reading the packed weights once (HBM), closely followed by the issue of the unpack
// (about 130 warp instructions per 16 x 128 codes).
//
// Split.  The unit is a pair tile (16 gate rows and the same 16 up rows) x one 128-code block.
// A tensor-core fragment (m16n8k16) takes 8 gate rows as its rows 0-7 and the 8 up rows of the
// same outputs as its rows 8-15: one activation fragment serves both layers, and a lane ends up
// holding both projections of the same output.  A CTA owns whole pair tiles and its 16 warps
// take equal contiguous runs of the CTA's (tile, block) units, so no partial sum leaves the CTA:
// no workspace, no counters between CTAs, nothing to order between calls.  A tile's weak columns
// are extra units at the end of its run, so that the warps share them evenly too.
//
// Each warp streams its run through a private ring of bulk copies (evict-first: the weights are
// read once), the first items issued before the wait for the previous kernel.  The activations
// come in by one bulk copy per token into padded rows and reach the fragments by ldmatrix; when
// they do not fit beside the ring they are read from global memory instead.  Segments of a tile
// held by several warps meet in shared memory after one barrier and are added in unit order, so
// repeated calls give identical bits.
#include "owq_act.cuh"
#include "owq_dequant.cuh"
#include "owq_internal.cuh"
#include "owq_mma.cuh"
#include "owq_sm100.cuh"

namespace owq {
namespace {

using namespace sm100;

constexpr int kWarps = 16;
constexpr int kMaxSmem = 232448;

struct GatedGemvArgs {
  const uint32_t* packed[2];    // [0] gate, [1] up
  const __half2* sz_t[2];       // (scale, zero) pairs, tile-major
  const __half* w_weak_t[2];    // weak block, tile-major [tile][slice][16 rows][16]
  const int32_t* idx[2];
  int k[2], nsl[2];             // weak columns and their 16-wide slices
  const __half* x;
  __half* h;
  int N, K, M, act;
  int tiles;                    // pair tiles, ceil(N / 16)
  int wunits;                   // weak units of a tile (after its K / 128 dense units)
  int sub, stages;              // units per ring item, ring stages
  int tcap;                     // most tiles of one CTA
  int* status;
  long long wait_limit;
};

template <int BITS>
struct Unit {
  static constexpr int kBlk = 16 * BITS;              // bytes of one block of one row
  static constexpr int kTileBlk = 16 * kBlk;          // of a 16-row tile, one layer
  static constexpr int kSlices = kTileBlk / 512;      // weak slices per unit and layer
};
template <int BITS>
constexpr int stage_bytes(int sub, bool pg) { return sub * 2 * (Unit<BITS>::kTileBlk + (pg ? 64 : 0)); }

// shared memory: ring | barriers (16 stages + 1, then a 16-byte pad) | early segments
// [tcap][2][16][MT] fp32 | per-channel (scale, zero) pairs [tcap][2][16] | weak indices |
// activations [M][K + 8]
struct SmemPlan {
  int bars, early, sz, idx, x, total;
};
__host__ __device__ inline SmemPlan smem_plan(int stage, int stages, int MT, int tcap, bool pg, int kg, int ku, int M, int K,
                                              bool xsmem) {
  SmemPlan p;
  p.bars = kWarps * stages * stage;
  p.early = p.bars + ((kWarps * stages + 1) * 8 + 15) / 16 * 16;
  p.sz = p.early + tcap * 32 * MT * 4;
  p.idx = p.sz + (pg ? 0 : tcap * 32 * 4);
  p.x = p.idx + ((kg + 3) / 4 + (ku + 3) / 4) * 16;
  p.total = p.x + (xsmem ? M * (K + 8) * 2 : 0);
  return p;
}

__device__ __forceinline__ uint32_t lds_u1(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
template <int BITS, int NT, bool PG, bool XSMEM>
__global__ void __launch_bounds__(kWarps * 32, 1)
k_gated_gemv(const __grid_constant__ GatedGemvArgs a) {
  using U_ = Unit<BITS>;
  constexpr int MT = 8 * NT;
  extern __shared__ __align__(128) unsigned char smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, tig = lane & 3;
  const int K = a.K, Kb = K / kBlockCodes, M = a.M, S = a.stages, sub = a.sub;
  const int stage = stage_bytes<BITS>(sub, PG);
  const SmemPlan sp = smem_plan(stage, S, MT, a.tcap, PG, a.k[0], a.k[1], M, K, XSMEM);
  const uint32_t sbase = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + sp.bars) + warp * S;
  uint64_t* xbar = reinterpret_cast<uint64_t*>(smem + sp.bars) + kWarps * S;
  float* early = reinterpret_cast<float*>(smem + sp.early);
  uint32_t* s_sz = reinterpret_cast<uint32_t*>(smem + sp.sz);
  int32_t* s_idx = reinterpret_cast<int32_t*>(smem + sp.idx);   // gate's, then up's
  const int idx_up = (a.k[0] + 3) / 4 * 4;

  // this CTA's pair tiles and this warp's run of their units
  const int t0 = (int)((long long)blockIdx.x * a.tiles / gridDim.x);
  const int T = (int)((long long)(blockIdx.x + 1) * a.tiles / gridDim.x) - t0;
  const int U = Kb + a.wunits;                         // units of a tile
  const int share = (T * U + kWarps - 1) / kWarps;
  const int lo = min(warp * share, T * U), hi = min(lo + share, T * U);

  // producer (lane 0): the next item of the run into the next stage
  uint64_t pol;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(pol));
  int issued = 0, p_lt = lo / U, p_u = lo - p_lt * U, p_left = hi - lo;
  auto issue = [&]() -> bool {
    if (p_left <= 0) return false;
    const int cnt = min(min(sub, p_left), (p_u < Kb ? Kb : U) - p_u);
    const int st = issued % S;
    unsigned char* dst = smem + (size_t)(warp * S + st) * stage;
    const size_t tile = (size_t)(t0 + p_lt);
    if (p_u < Kb) {
      const uint32_t bytes = (uint32_t)(cnt * U_::kTileBlk);
      mbar_arrive_expect_tx(&bars[st], 2 * (bytes + (PG ? (uint32_t)cnt * 64 : 0u)));
      #pragma unroll
      for (int l = 0; l < 2; ++l) {
        bulk_load_hint(dst + l * sub * U_::kTileBlk, reinterpret_cast<const unsigned char*>(a.packed[l]) + (tile * Kb + p_u) * U_::kTileBlk,
                       bytes, &bars[st], pol);
        if constexpr (PG)
          bulk_load_hint(dst + 2 * sub * U_::kTileBlk + l * sub * 64, a.sz_t[l] + (tile * Kb + p_u) * 16, (uint32_t)cnt * 64,
                         &bars[st], pol);
      }
    } else {
      const int s0 = (p_u - Kb) * U_::kSlices, s1 = s0 + cnt * U_::kSlices;
      int n[2];
      #pragma unroll
      for (int l = 0; l < 2; ++l) n[l] = max(0, min(a.nsl[l], s1) - s0);
      mbar_arrive_expect_tx(&bars[st], (uint32_t)(n[0] + n[1]) * 512);
      #pragma unroll
      for (int l = 0; l < 2; ++l)
        if (n[l] > 0)
          bulk_load_hint(dst + l * sub * U_::kTileBlk,
                         reinterpret_cast<const unsigned char*>(a.w_weak_t[l]) + (tile * a.nsl[l] + s0) * 512, (uint32_t)n[l] * 512,
                         &bars[st], pol);
    }
    ++issued;
    p_left -= cnt;
    p_u += cnt;
    if (p_u == U) { p_u = 0; ++p_lt; }
    return true;
  };

  if (lane == 0) {
    for (int st = 0; st < S; ++st) mbar_init(&bars[st], 1);
    if (warp == 0) mbar_init(xbar, 1);
    fence_mbar_init();
    for (int st = 0; st < S; ++st)   // the weights do not depend on the previous kernel
      if (!issue()) break;
  }
  for (int e = threadIdx.x; e < a.k[0] + a.k[1]; e += kWarps * 32) {
    const int up = e >= a.k[0];
    s_idx[up ? idx_up + e - a.k[0] : e] = a.idx[up][up ? e - a.k[0] : e];
  }
  if constexpr (!PG)
    for (int e = threadIdx.x; e < T * 32; e += kWarps * 32)   // [tile][layer][row]
      s_sz[e] = reinterpret_cast<const uint32_t*>(a.sz_t[(e >> 4) & 1])[(size_t)(t0 + (e >> 5)) * 16 + (e & 15)];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");   // x and h belong to the previous kernel
  __syncthreads();                                     // xbar, s_idx, s_sz
  if constexpr (XSMEM) {
    if (threadIdx.x == 0) {
      mbar_arrive_expect_tx(xbar, (uint32_t)(M * K * 2));
      for (int m = 0; m < M; ++m)
        bulk_load(smem + sp.x + (size_t)m * (K + 8) * 2, a.x + (size_t)m * K, (uint32_t)K * 2, xbar);
    }
  }
  bool ok = true;   // uniform per warp
  if constexpr (XSMEM) ok = __all_sync(0xffffffffu, mbar_wait(xbar, 0, a.status, a.wait_limit));

  // this lane's activation rows: ldmatrix row (lane & 7) of token tile nt, matrix lane >> 3 (8
  // columns each); tokens past M repeat the last one (their sums are not stored)
  int xo[NT];
  const __half* xg[NT];
  const __half* xs = reinterpret_cast<const __half*>(smem + sp.x);
  #pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    xo[nt] = min(8 * nt + (lane & 7), M - 1) * (K + 8) + 8 * (lane >> 3);
    xg[nt] = a.x + (size_t)min(8 * nt + g, M - 1) * K + 2 * tig;
  }

  float D[2][NT][4];   // [row half][token tile]: rows 8 half + g, (gate, gate, up, up) x tokens
  #pragma unroll
  for (int h = 0; h < 2; ++h)
    #pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      #pragma unroll
      for (int i = 0; i < 4; ++i) D[h][nt][i] = 0.f;
  // a segment's sums: [gate, up][16 rows][MT]
  auto put = [&](float* dst) {
    #pragma unroll
    for (int h = 0; h < 2; ++h)
      #pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        #pragma unroll
        for (int l = 0; l < 2; ++l) {
          *reinterpret_cast<float2*>(dst + (l * 16 + 8 * h + g) * MT + 8 * nt + 2 * tig) =
              make_float2(D[h][nt][2 * l], D[h][nt][2 * l + 1]);
          D[h][nt][2 * l] = 0.f;
          D[h][nt][2 * l + 1] = 0.f;
        }
  };

  RowDq<BITS> dq[2][2];   // [layer][row half]
  int lt = lo / U, u = lo - lt * U, left = hi - lo, st = 0, consumed = 0, sz_lt = -1;
  uint32_t phase = 0;
  #pragma unroll 1
  while (left > 0 && ok) {
    const int cnt = min(min(sub, left), (u < Kb ? Kb : U) - u);
    ok = __all_sync(0xffffffffu, mbar_wait(&bars[st], phase, a.status, a.wait_limit));
    if (!ok) break;
    const uint32_t sa = sbase + (uint32_t)((warp * S + st) * stage);
    if (u < Kb) {
      if constexpr (!PG) {
        if (lt != sz_lt) {
          sz_lt = lt;
          #pragma unroll
          for (int l = 0; l < 2; ++l)
            #pragma unroll
            for (int h = 0; h < 2; ++h) dq[l][h].set(s_sz[lt * 32 + l * 16 + 8 * h + g]);
        }
      }
      #pragma unroll 1
      for (int c = 0; c < cnt; ++c) {
        uint32_t w[2][2][BITS];   // [layer][row half]: this lane's chunk
        #pragma unroll
        for (int l = 0; l < 2; ++l)
          #pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t wa = sa + (l * sub + c) * U_::kTileBlk + (8 * h + g) * U_::kBlk + tig * 4 * BITS;
            if constexpr (BITS == 4) {
              const uint4 q = lds_u4(wa);
              w[l][h][0] = q.x; w[l][h][1] = q.y; w[l][h][2] = q.z; w[l][h][3] = q.w;
            } else {
              #pragma unroll
              for (int j = 0; j < BITS; ++j) w[l][h][j] = lds_u1(wa + 4 * j);
            }
            if constexpr (PG) dq[l][h].set(lds_u1(sa + 2 * sub * U_::kTileBlk + (l * sub + c) * 64 + (8 * h + g) * 4));
          }
        const int kc = (u + c) * kBlockCodes;   // first column of the block
        #pragma unroll
        for (int s2 = 0; s2 < 4; ++s2) {        // 32 columns: two k slices
          uint32_t xb[NT][4];
          #pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if constexpr (XSMEM) {
              ldsm_x4(xb[nt], xs + xo[nt] + kc + 32 * s2);
            } else {
              #pragma unroll
              for (int v = 0; v < 4; ++v) xb[nt][v] = __ldg(reinterpret_cast<const unsigned int*>(xg[nt] + kc + 32 * s2 + 8 * v));
            }
          }
          #pragma unroll
          for (int s = 0; s < 2; ++s) {
            const int j = 4 * s2 + 2 * s;
            #pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t f[4] = {dequant<BITS>(w[0][h], j, dq[0][h]), dequant<BITS>(w[1][h], j, dq[1][h]),
                                     dequant<BITS>(w[0][h], j + 1, dq[0][h]), dequant<BITS>(w[1][h], j + 1, dq[1][h])};
              #pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma_16816(D[h][nt], f, xb[nt][2 * s], xb[nt][2 * s + 1]);
            }
          }
        }
      }
    } else {
      // weak slices: the layers gather different activations, so each has its own product, with
      // zeros in the other layer's rows
      const int s0 = (u - Kb) * U_::kSlices, s1 = s0 + cnt * U_::kSlices;
      #pragma unroll 1
      for (int l = 0; l < 2; ++l)
        #pragma unroll 1
        for (int sl = s0; sl < min(s1, a.nsl[l]); ++sl) {
          const uint32_t wa = sa + l * sub * U_::kTileBlk + (sl - s0) * 512;
          uint32_t b[NT][2];
          #pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            #pragma unroll
            for (int v = 0; v < 2; ++v) {   // slots 16 sl + 8 v + 2 tig, + 1 of token 8 nt + g
              uint32_t p = 0;
              #pragma unroll
              for (int q = 0; q < 2; ++q) {
                const int t = 16 * sl + 8 * v + 2 * tig + q, tok = min(8 * nt + g, M - 1);
                const int col = t < a.k[l] ? s_idx[l * idx_up + t] : -1;   // padding: 0
                if (col >= 0 && in_range(col, K, a.status)) {
                  const __half xv = XSMEM ? xs[(size_t)tok * (K + 8) + col] : a.x[(size_t)tok * K + col];
                  p |= (uint32_t)__half_as_ushort(xv) << (16 * q);
                }
              }
              b[nt][v] = p;
            }
          #pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t w0 = lds_u1(wa + (8 * h + g) * 32 + tig * 4), w1 = lds_u1(wa + (8 * h + g) * 32 + 16 + tig * 4);
            const uint32_t f[4] = {l ? 0u : w0, l ? w0 : 0u, l ? 0u : w1, l ? w1 : 0u};
            #pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_16816(D[h][nt], f, b[nt][0], b[nt][1]);
          }
        }
    }
    __syncwarp();   // every lane has read the stage
    ++consumed;
    if (lane == 0) {
      fence_proxy_async_smem();
      issue();
    }
    if (++st == S) { st = 0; phase ^= 1u; }
    left -= cnt;
    u += cnt;
    if (u == U) {
      u = 0;
      if (left > 0) put(early + (size_t)lt * 32 * MT);   // this run goes on into the next tile
      ++lt;
    }
  }
  if (!ok) {   // after a timeout: never exit with copies still on their way into this CTA's memory
    if (XSMEM && threadIdx.x == 0) mbar_wait(xbar, 0, a.status, a.wait_limit);
    if (lane == 0)
      for (int j = consumed; j < issued; ++j) mbar_wait(&bars[j % S], (uint32_t)((j / S) & 1), a.status, a.wait_limit);
  } else if (hi > lo) {
    __syncwarp();
    put(reinterpret_cast<float*>(smem + (size_t)warp * S * stage));   // the run's last segment: its ring is idle
  }
  ok = __syncthreads_and(ok);
  if (!ok) return;

  // outputs: the segments of each tile in unit order
  for (int e = threadIdx.x; e < T * 16 * M; e += kWarps * 32) {
    const int row = e & 15, tm = e >> 4, t = tm / M, m = tm - t * M;
    const int n = (t0 + t) * 16 + row;
    if (n >= a.N) continue;
    const int w0 = t * U / share, w1 = ((t + 1) * U - 1) / share;
    float gs = 0.f, us = 0.f;
    for (int w = w0; w <= w1; ++w) {
      // warp w's last segment is on this tile unless its run goes on beyond it
      const float* src = min((w + 1) * share, T * U) <= (t + 1) * U
                             ? reinterpret_cast<const float*>(smem + (size_t)w * S * stage) : early + (size_t)t * 32 * MT;
      gs += src[row * MT + m];
      us += src[(16 + row) * MT + m];
    }
    with_act(a.act, [&](auto act) {
      float v, dv;
      act_eval<decltype(act)::value>(gs, v, dv);
      a.h[(size_t)m * a.N + n] = __float2half_rn(v * us);
    });
  }
}

template <int BITS, int NT, bool PG>
cudaError_t launch_p(GatedGemvArgs& a, int grid, int dev, cudaStream_t s) {
  a.wunits = (std::max(a.nsl[0], a.nsl[1]) + Unit<BITS>::kSlices - 1) / Unit<BITS>::kSlices;
  a.tcap = (a.tiles + grid - 1) / grid;
  // the largest items and deepest rings that fit beside the activations; a ring of at least two
  // stages comes before keeping the activations in shared memory
  static constexpr int kShapes[][2] = {{4, 3}, {4, 2}, {2, 3}, {2, 2}, {1, 3}, {1, 2}};
  static std::atomic<unsigned long long> allowed[2];   // [activations in shared memory]
  void (*kern)(GatedGemvArgs) = nullptr;
  int smem = 0, in_smem = 0;
  for (int xs = 1; xs >= 0 && !kern; --xs)
    for (const auto& sh : kShapes) {
      const int total = smem_plan(stage_bytes<BITS>(sh[0], PG), sh[1], 8 * NT, a.tcap, PG, a.k[0], a.k[1], a.M, a.K, xs).total;
      if (total > kMaxSmem) continue;
      a.sub = sh[0];
      a.stages = sh[1];
      smem = total;
      in_smem = xs;
      kern = xs ? k_gated_gemv<BITS, NT, PG, true> : k_gated_gemv<BITS, NT, PG, false>;
      break;
    }
  if (!kern) return cudaErrorInvalidValue;
  cudaError_t e = allow_smem((const void*)kern, kMaxSmem, dev, allowed[in_smem]);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, a);
  if (e != cudaSuccess) allowed[in_smem] = 0;
  return e;
}

template <int BITS>
cudaError_t launch_b(GatedGemvArgs& a, bool pg, int grid, int dev, cudaStream_t s) {
  if (a.M <= 8) return pg ? launch_p<BITS, 1, true>(a, grid, dev, s) : launch_p<BITS, 1, false>(a, grid, dev, s);
  return pg ? launch_p<BITS, 2, true>(a, grid, dev, s) : launch_p<BITS, 2, false>(a, grid, dev, s);
}

}  // namespace

cudaError_t launch_gated_gemv(const Layer& gate, const Layer& up, int act, const __half* x, __half* h, int M,
                              long long wait_limit, cudaStream_t s) {
  GatedGemvArgs a{};
  const Layer* L[2] = {&gate, &up};
  for (int l = 0; l < 2; ++l) {
    a.packed[l] = L[l]->packed;
    a.sz_t[l] = L[l]->sz_t;
    a.w_weak_t[l] = L[l]->w_weak_t;
    a.idx[l] = L[l]->idx;
    a.k[l] = L[l]->k;
    a.nsl[l] = L[l]->k > 0 ? L[l]->k_ld / 16 : 0;
  }
  a.x = x;
  a.h = h;
  a.N = gate.N;
  a.K = gate.K;
  a.M = M;
  a.act = act;
  a.tiles = (gate.N + 15) / 16;
  a.status = gate.status;
  a.wait_limit = wait_limit;
  const int grid = std::min(a.tiles, layer_sm_count(gate.device));
  return gate.bits == 3 ? launch_b<3>(a, gate.G > 1, grid, gate.device, s) : launch_b<4>(a, gate.G > 1, grid, gate.device, s);
}

}  // namespace owq
