// Gated block for 1 <= M <= 16 tokens in one launch: h = act(x Wg^T) * (x Wu^T) for two packed
// layers of one shape.
//
// Mathematics: each projection is W_hat x + W_weak x[idx] with W_hat = fp16_rn(s (q - z)), the
// dequantised weight itself for every M (each code pair costs two fp16x2 operations; the cheaper
// form that scales the integer sums differs from W_hat by up to half an fp16 spacing per weight,
// and the product of two projections doubles that).  Sums, activation and product are fp32; h
// is rounded once.
//
// Bound: reading the packed weights once (HBM), closely followed by the unpack (about 130 warp
// instructions per 16 x 128 codes, four warps a scheduler).
//
// Split.  The unit is a pair tile (16 gate rows and the same 16 up rows) x one 128-code block.
// A tensor-core fragment (m16n8k16) takes 8 gate rows as its rows 0-7 and the 8 up rows of the
// same outputs as its rows 8-15: one activation fragment serves both layers, and a lane ends up
// holding both projections of the same output.  A cluster of CTAs owns whole pair tiles; its CTAs
// split K, and the 16 consumer warps of a CTA take equal contiguous runs of the CTA's (tile, block)
// units.  So no partial sum leaves the cluster: no workspace, no counters in memory, nothing to
// order between calls.  The weak columns are a phase of their own before the packed units, a warp
// taking one layer of one tile: as units of the runs they made most runs one unit longer (a unit
// takes a warp about 1 us, and the runs of 11008 x 4096 are 10 units).  Clusters have one CTA unless the activations of all of K would
// leave too little shared memory for the weight rings (16 tokens of 5120 columns: 164 KB).
//
// Each warp streams its run through a private ring of bulk copies (evict-first: the weights are
// read once), refilled as stages are read; the first items are issued before the wait for the
// previous kernel.  (A copy's operands want uniform registers: the whole warp keeps count and an
// elected lane issues; issued by lane 0 from its own registers 16 tokens took 29.8 instead of
// 28.5 us.)  (One producer warp for all rings was slower: its lanes take turns, and
// 500 cycles an item in one warp are 2 us a tile.)  The activations come in by one bulk copy
// per token into padded rows and reach the fragments by ldmatrix; when they fit in no cluster they
// are read from global memory.  Segments of a tile held by several warps meet in shared memory
// after one barrier and are added in unit order, then the CTAs' sums in rank order through
// distributed shared memory: repeated calls give identical bits.
//
// Measured (a graph of calls over three copies of the weights, GPU time per call): 11008 x 4096,
// 4-bit, one token 14.0 us (49.4 MB, 3.5 TB/s; a further tile of 16 x 4096 per CTA costs 1.95 us,
// 5.4 TB/s, the rest about 5.7 us a launch); 13824 x 5120, 3-bit, 16 tokens 28.5 us (two token tiles
// through the products: 2.2 of 4 warp instructions a cycle per SM, tensor pipe 26%, DRAM 23%, so probably the
// latency of unpack, fma, mul and MMA with four warps a scheduler).
#include "owq_act.cuh"
#include "owq_dequant.cuh"
#include "owq_internal.cuh"
#include "owq_mma.cuh"
#include "owq_sm100.cuh"

namespace owq {
namespace {

using namespace sm100;

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxSmem = 232448;
constexpr int kParamIdx = 128;

struct GatedGemvArgs {
  const uint32_t* packed[2];    // [0] gate, [1] up
  const __half2* sz_t[2];       // (scale, zero) pairs, tile-major
  const __half* w_weak_t[2];    // weak block, tile-major [tile][slice][16 rows][16]
  const int32_t* idx[2];
  int k[2], nsl[2];             // weak columns and their 16-wide slices
  const __half* x;
  __half* h;
  int N, K, M, act;
  int tile0;                    // this launch's first pair tile, of ceil(N / 16)
  int base, extra;              // tiles of a cluster: base, and one more in the first `extra`
  int cl, log_cl;               // CTAs of a cluster (a power of two)
  int sub, stages;              // units per ring item, ring stages
  int tcap;                     // most tiles of a cluster
  int bcap;                     // most 128-column blocks of a CTA
  int o_bars, o_early, o_sz, o_idx, o_x;   // shared memory offsets
  int* status;
  long long wait_limit;
  int skip;                     // test-injected: an arrival for the activations is held back in every CTA
  uint16_t idx16[2][kParamIdx]; // the first weak indices (a load would cost the prologue its latency)
};

template <int BITS>
struct Unit {
  static constexpr int kBlk = 16 * BITS;              // bytes of one block of one row
  static constexpr int kTileBlk = 16 * kBlk;          // of a 16-row tile, one layer
};
template <int BITS>
constexpr int stage_bytes(int sub, bool pg) { return sub * 2 * (Unit<BITS>::kTileBlk + (pg ? 64 : 0)); }

// shared memory: ring | barriers (a stage's copies, x, weak sums) | per tile, the weak columns' sums
// and the segment that ends the tile, when its warp goes on [tcap][2][16][MT] fp32 | per-channel
// (scale, zero) pairs [tcap][2][16] | weak indices [2][16 nsl] | activations [M][128 bcap + 8] (later
// the CTA's sums [tcap][2][16][MT])
inline int smem_plan(GatedGemvArgs& a, int stage, int MT, bool pg, bool xsmem) {   // its size
  a.o_bars = kWarps * a.stages * stage;
  a.o_early = a.o_bars + ((kWarps * a.stages + 2) * 8 + 15) / 16 * 16;
  a.o_sz = a.o_early + a.tcap * 32 * MT * 4;
  a.o_idx = a.o_sz + (pg ? 0 : a.tcap * 32 * 4);
  a.o_x = a.o_idx + (a.nsl[0] + a.nsl[1]) * 16 * 4;
  const int rows = xsmem ? a.M * (a.bcap * kBlockCodes + 8) * 2 : 0, sums = a.cl > 1 ? a.tcap * 32 * MT * 4 : 0;
  return a.o_x + std::max(rows, sums);
}

template <int BITS, int NT, bool PG, bool XSMEM>
__global__ void __launch_bounds__(kThreads, 1)
k_gated_gemv(const __grid_constant__ GatedGemvArgs a) {
  using U_ = Unit<BITS>;
  constexpr int MT = 8 * NT;
  extern __shared__ __align__(128) unsigned char smem[];
  const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0);
  const int K = a.K, Kb = K / kBlockCodes, M = a.M, S = a.stages, sub = a.sub, CL = a.cl;
  const int stage = stage_bytes<BITS>(sub, PG);
  const uint32_t sbase = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + a.o_bars) + warp * S;   // this warp's stages
  uint64_t* xbar = reinterpret_cast<uint64_t*>(smem + a.o_bars) + kWarps * S;
  uint64_t* wbar = xbar + 1;
  float* early = reinterpret_cast<float*>(smem + a.o_early);
  uint32_t* s_sz = reinterpret_cast<uint32_t*>(smem + a.o_sz);
  int32_t* s_idx = reinterpret_cast<int32_t*>(smem + a.o_idx);   // the gate's, then the up layer's; -1: padding

  // this cluster's pair tiles, this CTA's blocks of each, a warp's run of them
  // (no division before the first copies: the prologue is not hidden behind anything)
  const int rank = CL > 1 ? (int)cluster_ctarank() : 0, cluster = (int)blockIdx.x >> a.log_cl;
  const int t0 = a.tile0 + cluster * a.base + min(cluster, a.extra), T = a.base + (cluster < a.extra);
  const int b0 = (rank * Kb) >> a.log_cl, nb = (((rank + 1) * Kb) >> a.log_cl) - b0;
  const int U = nb;                                    // units of a tile in this CTA
  const bool weak = a.nsl[0] + a.nsl[1] > 0;
  const int share = (T * U + kWarps - 1) / kWarps;   // (T and U are at least 1)

  const int lo = min(warp * share, T * U), hi = min(lo + share, T * U);

  // the next item of the run into the next stage (the whole warp keeps count, one lane issues).  A
  // CTA's blocks of a tile are contiguous.
  uint64_t pol;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(pol));
  int p_lt = lo / U, p_u = lo - p_lt * U, p_left = hi - lo, p_st = 0, in_flight = 0;
  const unsigned char *p_src[2], *p_sz[2];   // block p_u of tile p_lt
  auto point = [&]() {
    #pragma unroll
    for (int l = 0; l < 2; ++l) {
      const size_t blk = (size_t)(t0 + p_lt) * Kb + b0 + p_u;
      p_src[l] = reinterpret_cast<const unsigned char*>(a.packed[l]) + blk * U_::kTileBlk;
      p_sz[l] = reinterpret_cast<const unsigned char*>(a.sz_t[l]) + blk * 64;
    }
  };
  auto issue = [&]() {
    if (p_left <= 0) return;
    unsigned char* dst = smem + (size_t)(warp * S + p_st) * stage;
    uint64_t* bar = bars + p_st;
    const int cnt = min(min(sub, p_left), U - p_u);
    const uint32_t bytes = (uint32_t)(cnt * U_::kTileBlk), zb = (uint32_t)(cnt * 64);
    if (elect_one()) {
      mbar_arrive_expect_tx(bar, 2 * (bytes + (PG ? zb : 0u)));
      #pragma unroll
      for (int l = 0; l < 2; ++l) {
        bulk_load_hint(dst + l * sub * U_::kTileBlk, p_src[l], bytes, bar, pol);
        if constexpr (PG) bulk_load_hint(dst + 2 * sub * U_::kTileBlk + l * sub * 64, p_sz[l], zb, bar, pol);
      }
    }
    __syncwarp();
    #pragma unroll
    for (int l = 0; l < 2; ++l) {
      p_src[l] += bytes;
      p_sz[l] += zb;
    }
    ++in_flight;
    if (++p_st == S) p_st = 0;
    p_left -= cnt;
    p_u += cnt;
    if (p_u == U) {
      p_u = 0;
      ++p_lt;
      if (CL > 1) point();   // (a lone CTA's tiles are contiguous too)
    }
  };

  if (lane == 0) {
    for (int i = 0; i < S; ++i) mbar_init(&bars[i], 1);
    if (warp == 0) {
      mbar_init(xbar, 1 + a.skip);
      mbar_init(wbar, kWarps);
    }
    fence_mbar_init();
  }
  __syncwarp();
  point();
  for (int i = 0; i < S; ++i) issue();   // the weights do not depend on the previous kernel
  // static too: the weak indices and the per-channel pairs
  for (int e = threadIdx.x; e < (a.nsl[0] + a.nsl[1]) * 16; e += kThreads) {
    const int l = e >= a.nsl[0] * 16, t = l ? e - a.nsl[0] * 16 : e;
    s_idx[e] = t >= a.k[l] ? -1 : t < kParamIdx ? (int)a.idx16[l][t] : a.idx[l][t];
  }
  if constexpr (!PG)
    for (int e = threadIdx.x; e < T * 32; e += kThreads)   // [tile][layer][row]
      s_sz[e] = reinterpret_cast<const uint32_t*>(a.sz_t[(e >> 4) & 1])[(size_t)(t0 + (e >> 5)) * 16 + (e & 15)];
  // weak items: layer i & 1 of tile i / 2 for i = warp, warp + 16, ...; the first four 16-column
  // slices of the next one are fetched ahead (the weak block is static).  A CTA takes the weak columns
  // of its own blocks, a run of slots since the indices ascend.
  uint32_t wf[4][4];
  int sl_lo[2] = {0, 0}, sl_hi[2] = {a.nsl[0], a.nsl[1]};
  auto weak_frag = [&](int item, int sl, uint32_t (&f)[4]) {
    const int l = item & 1;
    if (item < 2 * T && sl < (l ? sl_hi[1] : sl_hi[0])) {
      const uint32_t* p = reinterpret_cast<const uint32_t*>(a.w_weak_t[l]) + ((size_t)(t0 + item / 2) * a.nsl[l] + sl) * 128 +
                          (lane >> 2) * 8 + (lane & 3);
      f[0] = __ldg(p); f[1] = __ldg(p + 64); f[2] = __ldg(p + 4); f[3] = __ldg(p + 68);
    }
  };
  auto weak_first = [&](int item) {   // the item's first four slices
    #pragma unroll
    for (int q = 0; q < 4; ++q) weak_frag(item, ((item & 1) ? sl_lo[1] : sl_lo[0]) + q, wf[q]);
  };
  if (weak && CL == 1) weak_first(warp);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __syncthreads();   // barriers, indices, pairs
  if (weak && CL > 1) {
    #pragma unroll
    for (int l = 0; l < 2; ++l) {
      const int32_t* ix = s_idx + (l ? a.nsl[0] * 16 : 0);
      int below = 0, upto = 0;   // slots below this CTA's columns, and up to their end
      for (int t = lane; t < a.k[l]; t += 32) {
        below += ix[t] < b0 * kBlockCodes;
        upto += ix[t] < (b0 + nb) * kBlockCodes;
      }
      below = __reduce_add_sync(0xffffffffu, below);
      upto = __reduce_add_sync(0xffffffffu, upto);
      sl_lo[l] = below / 16;
      sl_hi[l] = upto > below ? (upto + 15) / 16 : below / 16;
    }
    weak_first(warp);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");   // x and h belong to the previous kernel
  if constexpr (XSMEM) {
    if (threadIdx.x == 0) {
      const uint32_t bytes = (uint32_t)(nb * kBlockCodes * 2);
      mbar_arrive_expect_tx(xbar, (uint32_t)M * bytes);
      for (int m = 0; m < M; ++m)
        bulk_load(smem + a.o_x + (size_t)m * (a.bcap * kBlockCodes + 8) * 2, a.x + (size_t)m * K + b0 * kBlockCodes, bytes, xbar);
    }
  }
  bool ok = true;    // uniform per warp
  if constexpr (XSMEM) ok = __all_sync(0xffffffffu, mbar_wait(xbar, 0, a.status, a.wait_limit));

  {
    const int g = lane >> 2, tig = lane & 3;
    // this lane's activation rows: ldmatrix row (lane & 7) of token tile nt, matrix lane >> 3 (8
    // columns each); tokens past M repeat the last one (their sums are not stored)
    uint32_t xa[NT];
    const __half* xg[NT];
    const __half* xs = reinterpret_cast<const __half*>(smem + a.o_x);
    #pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      xa[nt] = sbase + a.o_x + (min(8 * nt + (lane & 7), M - 1) * (a.bcap * kBlockCodes + 8) + 8 * (lane >> 3)) * 2;
      xg[nt] = a.x + (size_t)min(8 * nt + g, M - 1) * K + b0 * kBlockCodes + 2 * tig;
    }

    for (int item = warp; weak && item < 2 * T && ok; item += kWarps) {
      const int l = item & 1, s_lo = l ? sl_lo[1] : sl_lo[0], s_hi = l ? sl_hi[1] : sl_hi[0];
      float d[NT][4];
      #pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        #pragma unroll
        for (int i = 0; i < 4; ++i) d[nt][i] = 0.f;
      #pragma unroll 1
      for (int s0 = s_lo; s0 < s_hi; s0 += 4) {
        uint32_t xw[4][NT][2];   // the activations of slots 16 (s0 + q) + 8 v + 2 tig, + 1 of token 8 nt + g
        #pragma unroll
        for (int q = 0; q < 4; ++q)
          #pragma unroll
          for (int v = 0; v < 2; ++v) {
            if (s0 + q >= s_hi) continue;
            const int2 col = *reinterpret_cast<const int2*>(s_idx + (l ? a.nsl[0] * 16 : 0) + 16 * (s0 + q) + 8 * v + 2 * tig);
            // (padding and other CTAs' columns: 0; the padded weights are 0 and x may be infinite)
            const int c0 = col.x - b0 * kBlockCodes, c1 = col.y - b0 * kBlockCodes, nc = nb * kBlockCodes;
            const bool in0 = col.x >= 0 && c0 >= 0 && c0 < nc && in_range(col.x, K, a.status);
            const bool in1 = col.y >= 0 && c1 >= 0 && c1 < nc && in_range(col.y, K, a.status);
            #pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const int tok = min(8 * nt + g, M - 1);
              const __half* row = XSMEM ? xs + (size_t)tok * (a.bcap * kBlockCodes + 8) : a.x + (size_t)tok * K + b0 * kBlockCodes;
              const uint32_t lo16 = in0 ? __half_as_ushort(row[c0]) : 0, hi16 = in1 ? __half_as_ushort(row[c1]) : 0;
              xw[q][nt][v] = lo16 | hi16 << 16;
            }
          }
        #pragma unroll
        for (int q = 0; q < 4; ++q)
          if (s0 + q < s_hi)
            #pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_16816(d[nt], wf[q], xw[q][nt][0], xw[q][nt][1]);
        if (s0 + 4 < s_hi) {
          #pragma unroll
          for (int q = 0; q < 4; ++q) weak_frag(item, s0 + 4 + q, wf[q]);
        }
      }
      weak_first(item + kWarps);
      float* dst = early + (size_t)item * 16 * MT;
      #pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        #pragma unroll
        for (int i = 0; i < 2; ++i)
          *reinterpret_cast<float2*>(dst + (g + 8 * i) * MT + 8 * nt + 2 * tig) = make_float2(d[nt][2 * i], d[nt][2 * i + 1]);
    }
    __syncwarp();
    if (weak && lane == 0) mbar_arrive(wbar);

    float D[2][NT][4];   // [row half][token tile]: rows 8 half + g, (gate, gate, up, up) x tokens
    #pragma unroll
    for (int h = 0; h < 2; ++h)
      #pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        #pragma unroll
        for (int i = 0; i < 4; ++i) D[h][nt][i] = 0.f;
    // a segment's sums: [gate, up][16 rows][MT]; `onto` what is there
    auto put = [&](float* dst, bool onto) {
      #pragma unroll
      for (int h = 0; h < 2; ++h)
        #pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          #pragma unroll
          for (int l = 0; l < 2; ++l) {
            float2* p = reinterpret_cast<float2*>(dst + (l * 16 + 8 * h + g) * MT + 8 * nt + 2 * tig);
            float2 v = make_float2(D[h][nt][2 * l], D[h][nt][2 * l + 1]);
            if (onto) v = make_float2(p->x + v.x, p->y + v.y);
            *p = v;
            D[h][nt][2 * l] = 0.f;
            D[h][nt][2 * l + 1] = 0.f;
          }
    };

    RowDq<BITS> dq[2][2];   // [layer][row half]
    int lt = lo / U, u = lo - lt * U, left = hi - lo, st = 0, sz_lt = -1;
    uint32_t phase = 0;
    const uint32_t ring = sbase + (uint32_t)(warp * S * stage), up_off = (uint32_t)(sub * U_::kTileBlk);
    const uint32_t lane_w = (uint32_t)(g * U_::kBlk + tig * 4 * BITS);
    #pragma unroll 1
    while (left > 0 && ok) {
      const int cnt = min(min(sub, left), U - u);
      ok = __all_sync(0xffffffffu, mbar_wait(&bars[st], phase, a.status, a.wait_limit));
      if (!ok) break;
      const uint32_t sa = ring + (uint32_t)(st * stage);
      if constexpr (!PG) {
        if (lt != sz_lt) {
          sz_lt = lt;
          #pragma unroll
          for (int l = 0; l < 2; ++l)
            #pragma unroll
            for (int h = 0; h < 2; ++h) dq[l][h].set(s_sz[lt * 32 + l * 16 + 8 * h + g]);
        }
      }
      uint32_t wa = sa + lane_w, za = sa + 2 * up_off + 4 * g, xoff = (uint32_t)u * (kBlockCodes * 2);
      #pragma unroll 1
      for (int c = 0; c < cnt; ++c, wa += U_::kTileBlk, za += 64, xoff += kBlockCodes * 2) {
        uint32_t w[2][2][BITS];   // [layer][row half]: this lane's chunk
        #pragma unroll
        for (int l = 0; l < 2; ++l)
          #pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t p = wa + l * up_off + h * 8 * U_::kBlk;
            if constexpr (BITS == 4) {
              const uint4 q = lds_u4(p);
              w[l][h][0] = q.x; w[l][h][1] = q.y; w[l][h][2] = q.z; w[l][h][3] = q.w;
            } else {
              #pragma unroll
              for (int j = 0; j < BITS; ++j) w[l][h][j] = lds_u1(p + 4 * j);
            }
            if constexpr (PG) dq[l][h].set(lds_u1(za + l * (sub * 64) + h * 32));
          }
        uint32_t xf[4][NT][4];   // [32 columns: two k slices][token tile]
        #pragma unroll
        for (int s2 = 0; s2 < 4; ++s2)
          #pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if constexpr (XSMEM) {
              ldsm_x4(xf[s2][nt], xa[nt] + xoff + 64 * s2);
            } else {
              #pragma unroll
              for (int v = 0; v < 4; ++v)
                xf[s2][nt][v] = __ldg(reinterpret_cast<const unsigned int*>(xg[nt] + xoff / 2 + 32 * s2 + 8 * v));
            }
          }
        #pragma unroll
        for (int s2 = 0; s2 < 4; ++s2) {
          #pragma unroll
          for (int s = 0; s < 2; ++s) {
            const int j = 4 * s2 + 2 * s;
            #pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t f[4] = {dequant<BITS>(w[0][h], j, dq[0][h]), dequant<BITS>(w[1][h], j, dq[1][h]),
                                     dequant<BITS>(w[0][h], j + 1, dq[0][h]), dequant<BITS>(w[1][h], j + 1, dq[1][h])};
              #pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma_16816(D[h][nt], f, xf[s2][nt][2 * s], xf[s2][nt][2 * s + 1]);
            }
          }
        }
      }
      __syncwarp();   // every lane has read the stage
      --in_flight;
      fence_proxy_async_smem();
      issue();
      if (++st == S) { st = 0; phase ^= 1u; }
      left -= cnt;
      u += cnt;
      if (u == U) {
        u = 0;
        if (left > 0) {   // this run goes on into the next tile
          if (weak) ok = __all_sync(0xffffffffu, mbar_wait(wbar, 0, a.status, a.wait_limit));
          put(early + (size_t)lt * 32 * MT, weak);
        }
        ++lt;
      }
    }
    if (!ok && lane == 0) {   // after a timeout: never exit with copies on their way into this CTA's memory
      if (XSMEM && threadIdx.x == 0) {
        if (a.skip) mbar_arrive(xbar);   // (the arrival that was held back)
        mbar_wait(xbar, 0, a.status, a.wait_limit);
      }
      for (; in_flight > 0; --in_flight) {
        mbar_wait(&bars[st], phase, a.status, a.wait_limit);
        if (++st == S) { st = 0; phase ^= 1u; }
      }
    }
    if (ok && hi > lo) put(reinterpret_cast<float*>(smem + (size_t)warp * S * stage), false);   // the run's last segment: its ring is idle
  }
  ok = __syncthreads_and(ok);

  // the segments of tile t in unit order: this CTA's sums of one (row, token)
  auto segments = [&](int t, int row, int m, float& gs, float& us) {
    const int f = t * U / share, e = ((t + 1) * U - 1) / share;
    // the last warp's segment is with the weak sums if its run goes on beyond the tile, else (as the
    // other warps') in its ring
    const bool on = min((e + 1) * share, T * U) > (t + 1) * U;
    gs = us = 0.f;
    if (weak || on) {
      const float* src = early + (size_t)t * 32 * MT;
      gs = src[row * MT + m];
      us = src[(16 + row) * MT + m];
    }
    for (int w = f; w < e + !on; ++w) {
      const float* src = reinterpret_cast<const float*>(smem + (size_t)w * S * stage);
      gs += src[row * MT + m];
      us += src[(16 + row) * MT + m];
    }
  };
  auto store = [&](int t, int row, int m, float gs, float us) {
    const int n = (t0 + t) * 16 + row;
    if (n < a.N)
      with_act(a.act, [&](auto act) {
        float v, dv;
        act_eval<decltype(act)::value>(gs, v, dv);
        a.h[(size_t)m * a.N + n] = __float2half_rn(v * us);
      });
  };
  const int outs = T * 16 * M;
  if (CL == 1) {
    for (int e = threadIdx.x; e < outs && ok; e += kThreads) {
      const int row = e & 15, tm = e >> 4, t = tm / M, m = tm - t * M;
      float gs, us;
      segments(t, row, m, gs, us);
      store(t, row, m, gs, us);
    }
    return;
  }
  // several CTAs: each leaves its sums where its activations were, then finishes its share of the
  // outputs from everybody's, in rank order
  float* sums = reinterpret_cast<float*>(smem + a.o_x);   // [output][gate, up]
  for (int e = threadIdx.x; e < outs; e += kThreads) {
    const int row = e & 15, tm = e >> 4, t = tm / M, m = tm - t * M;
    float gs, us;
    segments(t, row, m, gs, us);
    sums[2 * e] = gs;
    sums[2 * e + 1] = us;
  }
  __syncwarp();
  cluster_sync();
  for (int e = rank * kThreads + threadIdx.x; e < outs && ok; e += CL * kThreads) {
    const int row = e & 15, tm = e >> 4, t = tm / M, m = tm - t * M;
    float gs = 0.f, us = 0.f;
    for (int r = 0; r < CL; ++r) {
      gs += ld_dsmem_f32(sums + 2 * e, (uint32_t)r);
      us += ld_dsmem_f32(sums + 2 * e + 1, (uint32_t)r);
    }
    store(t, row, m, gs, us);
  }
  __syncwarp();
  cluster_sync();   // no CTA leaves while its sums may still be read
}

// Clusters of `cl` CTAs that run at once, one CTA per SM (0: the driver did not say).  Fewer than SMs / cl
// from 4 CTAs on, as a cluster stays within a GPC: a grid of SMs / cl clusters would leave some for a second
// wave as long as the first (16384 x 8192, 4-bit, 12 tokens: 100 us with 37 clusters of 4).  Asked once per
// device and size.
int resident_clusters(const void* kern, int cl, int sms, int dev) {
  if (cl == 1) return sms;
  constexpr int kMaxDev = 64;
  static std::atomic<int> known[kMaxDev][4];   // [log2 cl]
  const int lg = cl == 2 ? 1 : cl == 4 ? 2 : 3;
  int n = dev < kMaxDev ? known[dev][lg].load(std::memory_order_relaxed) : 0;
  if (n > 0) return n;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(sms / cl * cl);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kMaxSmem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cl;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  if (dev < kMaxDev) known[dev][lg].store(n, std::memory_order_relaxed);
  return n;
}

// Items and rings that fit beside the activations, the largest items first (an item costs a warp
// about 70 instructions beside the 300 of each unit; one stage in flight per warp covers the
// latency of the loads from about 40 KB an SM); then the same with K split over 2, 4 and 8 CTAs;
// then, since a cluster's sums grow with its tiles, the tiles over several launches; then the
// activations from global memory.
template <int BITS, int NT, bool PG>
cudaError_t launch_p(GatedGemvArgs& a, int all, int sms, int dev, cudaStream_t s) {
  static std::atomic<unsigned long long> allowed[2];   // [activations in shared memory]
  static constexpr int kShapes[][2] = {{4, 2}, {3, 2}, {2, 2}, {1, 3}};
  int pieces = 0, smem = 0, xs = 0, per = 0, resident = 0;
  const void* clustered = (const void*)k_gated_gemv<BITS, NT, PG, true>;
  auto fits = [&](int cl, int n, int x) {
    a.cl = cl;
    per = (all + n - 1) / n;
    if (a.K / kBlockCodes < cl) return false;
    if (cl > 1 && allow_smem(clustered, kMaxSmem, dev, allowed[1]) != cudaSuccess) return false;
    if ((resident = resident_clusters(clustered, cl, sms, dev)) < 1) return false;
    const int clusters = std::max(1, std::min(per, resident));
    a.tcap = (per + clusters - 1) / clusters;
    a.bcap = (a.K / kBlockCodes + cl - 1) / cl;
    for (const auto& sh : kShapes) {
      a.sub = sh[0];
      a.stages = sh[1];
      smem = smem_plan(a, stage_bytes<BITS>(sh[0], PG), 8 * NT, PG, x);
      if (smem <= kMaxSmem) {
        pieces = n;
        xs = x;
        return true;
      }
    }
    return false;
  };
  for (int n = 1; n <= 16 && !pieces; n *= 2)
    for (int cl = 1; cl <= 8 && !pieces; cl *= 2) fits(cl, n, 1);
  for (int n = 1; n <= 1024 && !pieces; n *= 2) fits(1, n, 0);
  if (!pieces) return cudaErrorInvalidValue;
  auto kern = xs ? k_gated_gemv<BITS, NT, PG, true> : k_gated_gemv<BITS, NT, PG, false>;
  cudaError_t e = allow_smem((const void*)kern, kMaxSmem, dev, allowed[xs]);
  if (e != cudaSuccess) return e;
  for (a.log_cl = 0; 1 << a.log_cl < a.cl;) ++a.log_cl;
  for (a.tile0 = 0; a.tile0 < all; a.tile0 += per) {
    const int tiles = std::min(per, all - a.tile0), clusters = std::max(1, std::min(tiles, resident));
    a.base = tiles / clusters;
    a.extra = tiles % clusters;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(clusters * a.cl);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)a.cl;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.cl > 1 ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, kern, a);
    if (e != cudaSuccess) {
      allowed[xs] = 0;
      return e;
    }
  }
  return cudaSuccess;
}

template <int BITS>
cudaError_t launch_b(GatedGemvArgs& a, bool pg, int all, int sms, int dev, cudaStream_t s) {
  if (a.M <= 8) return pg ? launch_p<BITS, 1, true>(a, all, sms, dev, s) : launch_p<BITS, 1, false>(a, all, sms, dev, s);
  return pg ? launch_p<BITS, 2, true>(a, all, sms, dev, s) : launch_p<BITS, 2, false>(a, all, sms, dev, s);
}

}  // namespace

cudaError_t launch_gated_gemv(const Layer& gate, const Layer& up, int act, const __half* x, __half* h, int M,
                              long long wait_limit, bool skip, cudaStream_t s) {
  GatedGemvArgs a{};
  a.skip = skip ? 1 : 0;
  const Layer* L[2] = {&gate, &up};
  for (int l = 0; l < 2; ++l) {
    a.packed[l] = L[l]->packed;
    a.sz_t[l] = L[l]->sz_t;
    a.w_weak_t[l] = L[l]->w_weak_t;
    a.idx[l] = L[l]->idx;
    a.k[l] = L[l]->k;
    a.nsl[l] = L[l]->k > 0 ? L[l]->k_ld / 16 : 0;
  }
  for (int l = 0; l < 2; ++l)
    for (int t = 0; t < std::min(L[l]->k, kParamIdx); ++t) a.idx16[l][t] = L[l]->idx16[t];
  a.x = x;
  a.h = h;
  a.N = gate.N;
  a.K = gate.K;
  a.M = M;
  a.act = act;
  const int all = (gate.N + 15) / 16;   // pair tiles
  a.status = gate.status;
  a.wait_limit = wait_limit;
  const int sms = layer_sm_count(gate.device);
  return gate.bits == 3 ? launch_b<3>(a, gate.G > 1, all, sms, gate.device, s) : launch_b<4>(a, gate.G > 1, all, sms, gate.device, s);
}

}  // namespace owq
