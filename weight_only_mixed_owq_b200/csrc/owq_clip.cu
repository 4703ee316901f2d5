// Global 2-norm of many gradient tensors and their clipping, in one launch:
//   norm = sqrt(sum over all tensors of g^2),  out = g min(1, max_norm / (norm + 1e-6))
// (a norm that is not finite leaves the factor at 1: the caller sees it and skips its step).
//
// Bound: HBM.  Every value has to be read once and written once; the norm needs all of them
// before the first can be written, so what does not stay on the chip is read again.
//
// One cooperative launch of one CTA per SM.  The tensors are cut into chunks dealt round-robin to
// the CTAs.  A producer warp streams a CTA's chunks through a ring of bulk copies (up to 192 KB in
// flight, no registers behind it); 16 warps add the squares; the CTA publishes its partial sum and
// waits for the others' (bounded).  The second pass walks the chunks backwards: the last ones are
// still in the ring, the ones before them in L2, where the streaming stores leave them until they
// are read.
// Measured: 202 MB of fp32 in 224 tensors 97 us; 333 MB read, so that 71 MB of the second pass's
// input came from the ring and L2: 535 MB through memory, 5.5 TB/s.
// Squares are added in fp64, 16 bytes of values at a time (4 of fp32, 8 of fp16 or bf16): those are summed in
// fp32 (2^-24 each, averaging out) where that neither overflows nor loses small values, else one by one in fp64 (a
// conversion per value would take as long as the memory).  All sums run in a fixed order: repeated
// calls give identical bits.
#include <cuda_bf16.h>

#include "owq_internal.cuh"
#include "owq_sm100.cuh"

namespace owq {
namespace {

using namespace sm100;

constexpr int kWarps = 16, kThreads = kWarps * 32;   // and the producer warp
constexpr int kChunkBytes = 32 * 1024;               // most bytes of a chunk
constexpr int kRingBytes = 6 * kChunkBytes, kMaxSlots = 16;
// What the first pass leaves in L2 (126 MB) for the second; the rest is loaded evict-first.  202 MB
// of fp32 with 0 / 40 / 60 / 80 / 100 / 120 / 140 MB: 102.5 / 101.5 / 100.9 / 97.1 / 97.3 / 97.8 / 98.9 us,
// without any hint 101.8 (the L2's evict-last priority for what is left gave the same).
constexpr int kKeepBytes = 90 << 20;

struct ClipArgs {
  const ClipChunk* chunks;
  int n_chunks;
  int slot_bytes, slots;
  int keep;                      // a CTA's last chunks that the second pass may find in L2
  double* part;                  // [gridDim.x] partial sums
  unsigned long long* arrived;   // CTAs that have published, over all calls
  float max_norm;
  float* norm;
  int* status;
  long long wait_limit;
  int skip;                      // test-injected: CTA 0 never copies its first chunk and publishes late
};

template <int DT>
struct Vec;   // values of a 16-byte piece
template <>
struct Vec<OWQ_F32> {
  using T = float;
  static __device__ __forceinline__ float get(float v) { return v; }
  static __device__ __forceinline__ float put(float v) { return v; }
};
template <>
struct Vec<OWQ_F16> {
  using T = __half;
  static __device__ __forceinline__ float get(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half put(float v) { return __float2half_rn(v); }
};
template <>
struct Vec<OWQ_BF16> {
  using T = __nv_bfloat16;
  static __device__ __forceinline__ float get(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
};

// 16-byte pieces of a chunk: `head` values before the first aligned one, `pieces`, then a tail
template <class T>
struct Cut {
  int head, pieces;
  __device__ __forceinline__ Cut(const void* p, int n) {
    head = min(n, (int)(((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / sizeof(T)));
    pieces = (n - head) / (int)(16 / sizeof(T));
  }
};

template <int DT>
__device__ __forceinline__ double squares(const ClipChunk& c, const uint4* slot) {
  using T = typename Vec<DT>::T;
  constexpr int P = 16 / sizeof(T);
  const T* in = static_cast<const T*>(c.in);
  const Cut<T> cut(in, c.n);
  double s = 0.0;
  #pragma unroll 4
  for (int i = threadIdx.x; i < cut.pieces; i += kThreads) {
    const uint4 q = slot[i];
    const T* e = reinterpret_cast<const T*>(&q);
    float p = 0.f;
    #pragma unroll
    for (int u = 0; u < P; ++u) {
      const float v = Vec<DT>::get(e[u]);
      p = fmaf(v, v, p);
    }
    if (p >= 1e-25f && p <= 1e37f) {   // (a square lost below 1e-45 is below 2^-66 of the sum)
      s += (double)p;
    } else {
      #pragma unroll
      for (int u = 0; u < P; ++u) {
        const double v = (double)Vec<DT>::get(e[u]);
        s = fma(v, v, s);
      }
    }
  }
  const int tail = cut.head + cut.pieces * P;   // fewer than P values at either end
  const int i = (int)threadIdx.x < cut.head ? (int)threadIdx.x : tail + (int)threadIdx.x - cut.head;
  if (i < c.n && ((int)threadIdx.x < cut.head || i >= tail) && threadIdx.x < 2 * P) {
    const double v = (double)Vec<DT>::get(in[i]);
    s = fma(v, v, s);
  }
  return s;
}

template <int DT>
__device__ __forceinline__ void scale(const ClipChunk& c, const uint4* slot, float f) {
  using T = typename Vec<DT>::T;
  constexpr int P = 16 / sizeof(T);
  const T* in = static_cast<const T*>(c.in);
  T* out = static_cast<T*>(c.out);
  const Cut<T> cut(in, c.n);
  T* o = out + cut.head;
  const bool vec = (reinterpret_cast<uintptr_t>(o) & 15) == 0;
  const bool copy = f == 1.f;   // bit for bit (a product would quieten a NaN's payload)
  #pragma unroll 4
  for (int i = threadIdx.x; i < cut.pieces; i += kThreads) {
    const uint4 q = slot[i];
    const T* e = reinterpret_cast<const T*>(&q);
    uint4 r;
    T* d = reinterpret_cast<T*>(&r);
    #pragma unroll
    for (int u = 0; u < P; ++u) d[u] = copy ? e[u] : Vec<DT>::put(Vec<DT>::get(e[u]) * f);
    if (vec) {
      __stcs(reinterpret_cast<uint4*>(o) + i, r);
    } else {
      #pragma unroll
      for (int u = 0; u < P; ++u) o[(size_t)i * P + u] = d[u];
    }
  }
  const int tail = cut.head + cut.pieces * P;
  const int i = (int)threadIdx.x < cut.head ? (int)threadIdx.x : tail + (int)threadIdx.x - cut.head;
  if (i < c.n && ((int)threadIdx.x < cut.head || i >= tail) && threadIdx.x < 2 * P)
    out[i] = copy ? in[i] : Vec<DT>::put(Vec<DT>::get(in[i]) * f);
}

// sum over the consumer warps in a fixed order; the result in every one of their threads
__device__ __forceinline__ double block_sum(double v, double* s_red) {
  #pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = v;
  named_bar_sync(1, kThreads);
  v = s_red[threadIdx.x & (kWarps - 1)];
  #pragma unroll
  for (int o = kWarps / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  named_bar_sync(1, kThreads);
  return v;
}

// A CTA's chunk i sits in ring slot i % slots, in the second pass too: the slot of the last chunk of
// residue s (index last) is used last / slots + 1 times in the first pass and then once for each
// chunk last - slots, last - 2 slots, ...  `use` is the number of a use, for the barriers' phases.
struct Uses {
  int mine, slots;
  __device__ __forceinline__ int last(int i) const { return i + (mine - 1 - i) / slots * slots; }
  __device__ __forceinline__ int second(int i) const { return last(i) / slots + (last(i) - i) / slots; }   // (of a copy; last(i): the first pass's)
};

__global__ void __launch_bounds__(kThreads + 32, 1) k_clip(const __grid_constant__ ClipArgs a) {
  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ ClipChunk s_chunk[kMaxSlots];
  __shared__ uint64_t full[kMaxSlots], empty[kMaxSlots];
  __shared__ double s_red[kWarps];
  __shared__ int s_ok, s_lost;   // the grid's barrier was passed; a warp's wait in the first pass gave up
  const int G = gridDim.x, b = blockIdx.x, S = a.slots, lane = threadIdx.x & 31;
  const int mine = b < a.n_chunks ? (a.n_chunks - 1 - b) / G + 1 : 0;   // chunks b, b + G, ...
  const Uses uses{mine, S};
  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kWarps);
    }
    fence_mbar_init();
    s_lost = 0;
  }
  __syncthreads();

  if (threadIdx.x >= kThreads) {
    // ---------------- producer ----------------
    // one lane copies; the warp fetches the table entries 32 at a time
    bool ok = true;
    int copies = 0;   // lane s: copies issued into slot s
    ClipChunk mineq = {};
    uint64_t first;   // evict first: what the second pass will not find in L2 anyway, or has read
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(first));
    auto load = [&](int i, const ClipChunk& c, bool keep) {
      const int s = i % S, size = c.dtype == OWQ_F32 ? 4 : 2;
      const int head = min(c.n, (int)((16 - (reinterpret_cast<uintptr_t>(c.in) & 15)) & 15) / size);
      const uint32_t bytes = (uint32_t)((c.n - head) * size) & ~15u;
      s_chunk[s] = c;
      mbar_arrive_expect_tx(&full[s], bytes);
      if (bytes == 0) return;
      const char* from = static_cast<const char*>(c.in) + head * size;
      if (keep) bulk_load(ring + (size_t)s * a.slot_bytes, from, bytes, &full[s]);
      else bulk_load_hint(ring + (size_t)s * a.slot_bytes, from, bytes, &full[s], first);
    };
    auto entry = [&](int at) {   // of the 32 this warp holds
      ClipChunk c;
      c.in = reinterpret_cast<const void*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mineq.in), at));
      c.out = reinterpret_cast<void*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mineq.out), at));
      c.n = __shfl_sync(0xffffffffu, mineq.n, at);
      c.dtype = __shfl_sync(0xffffffffu, mineq.dtype, at);
      return c;
    };
    for (int i = 0; i < mine && ok; ++i) {
      if (i % 32 == 0 && i + lane < mine) mineq = a.chunks[b + (size_t)(i + lane) * G];
      const ClipChunk c = entry(i % 32);
      if (i >= S) ok = __all_sync(0xffffffffu, mbar_wait(&empty[i % S], (uint32_t)(i / S - 1) & 1, a.status, a.wait_limit));
      const bool skip = a.skip && b == 0 && i == 0;
      if (ok && !skip && lane == 0) load(i, c, i >= mine - a.keep);
      if (ok && !skip && lane == i % S) ++copies;
      __syncwarp();
    }
    // Every slot's first-pass uses are consumed before the second pass waits on the slots' barriers: a
    // wait by parity must not be more than one phase ahead of its barrier.
    named_bar_sync(2, kThreads + 32);
    ok = ok && !s_lost;   // (their uses were not all consumed: there is no second pass)
    for (int k = 0, i = mine - S - 1; i >= 0 && ok; --i, ++k) {   // the second pass, after the resident chunks
      if (k % 32 == 0 && i - lane >= 0) mineq = a.chunks[b + (size_t)(i - lane) * G];
      const ClipChunk c = entry(k % 32);
      // the second pass's use of the slot by chunk i + S is over: its consumption follows the first pass's
      ok = __all_sync(0xffffffffu, mbar_wait(&empty[i % S], (uint32_t)uses.second(i) & 1, a.status, a.wait_limit));
      if (ok && lane == 0) load(i, c, false);
      if (ok && lane == i % S) ++copies;
      __syncwarp();
    }
    // never leave with copies in flight: the last one issued into every slot
    if (copies > 0) mbar_wait(&full[lane], (uint32_t)(copies - 1) & 1, a.status, a.wait_limit);
    return;
  }

  // ---------------- consumers ----------------
  bool ok = true;   // uniform per warp
  double s = 0.0;
  for (int i = 0; i < mine && ok; ++i) {
    const int sl = i % S;
    ok = __all_sync(0xffffffffu, mbar_wait(&full[sl], (uint32_t)(i / S) & 1, a.status, a.wait_limit));
    const uint4* slot = reinterpret_cast<const uint4*>(ring + (size_t)sl * a.slot_bytes);
    const ClipChunk c = s_chunk[sl];
    if (ok) {
      if (c.dtype == OWQ_F32) s += squares<OWQ_F32>(c, slot);
      else if (c.dtype == OWQ_F16) s += squares<OWQ_F16>(c, slot);
      else s += squares<OWQ_BF16>(c, slot);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[sl]);
  }
  if (!ok && lane == 0) s_lost = 1;
  named_bar_sync(2, kThreads + 32);   // the producer's second pass may start
  s = block_sum(s, s_red);

  // publish, then wait until every CTA of this call has: the counter only grows, by G a call
  if (threadIdx.x == 0) {
    if (a.skip && b == 0)
      for (const long long t0 = clock64(); clock64() - t0 < 2 * a.wait_limit;) {}
    a.part[b] = s;
    __threadfence();
    const unsigned long long old = atomicAdd(a.arrived, 1ull);
    const unsigned long long want = (old / G + 1) * G;
    int all = 1;
    const long long t0 = clock64();
    while (*reinterpret_cast<volatile unsigned long long*>(a.arrived) < want)
      if (clock64() - t0 > a.wait_limit) {
        atomicOr(a.status, kStatusTimeout);
        all = 0;
        break;
      }
    __threadfence();
    s_ok = all && !s_lost;
  }
  named_bar_sync(1, kThreads);
  ok = s_ok;   // (of all warps together)
  double t = 0.0;
  for (int i = threadIdx.x; i < G; i += kThreads) t += __ldcg(a.part + i);
  t = block_sum(t, s_red);
  const float norm = (float)sqrt(t);
  const float f = norm <= 3.402823466e38f ? fminf(a.max_norm / (norm + 1e-6f), 1.f) : 1.f;   // (false for NaN too)
  if (b == 0 && threadIdx.x == 0 && ok) *a.norm = norm;

  // (a warp whose wait gave up stops: an arrival of its own for a later use of a slot could stand in for
  // another warp's, and the slot and its table entry be replaced under that one)
  for (int i = mine - 1; i >= 0 && ok; --i) {
    const int sl = i % S;
    if (i < mine - S && !(ok = __all_sync(0xffffffffu, mbar_wait(&full[sl], (uint32_t)uses.second(i) & 1, a.status, a.wait_limit)))) break;
    const uint4* slot = reinterpret_cast<const uint4*>(ring + (size_t)sl * a.slot_bytes);
    const ClipChunk c = s_chunk[sl];
    if (!(f == 1.f && c.in == c.out)) {   // (in place and unclipped: nothing to write)
      if (c.dtype == OWQ_F32) scale<OWQ_F32>(c, slot, f);
      else if (c.dtype == OWQ_F16) scale<OWQ_F16>(c, slot, f);
      else scale<OWQ_BF16>(c, slot, f);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[sl]);
  }
}

}  // namespace

// Bytes of a chunk: the work of every CTA in about eight chunks, so that the deal is even and the
// ring has something to overlap, within 4 KB (the smallest: latency) and 32 KB.
int clip_chunk_bytes(long long total_bytes, int sms) {
  const long long want = total_bytes / (8LL * sms);
  return (int)std::max<long long>(4096, std::min<long long>(kChunkBytes, (want + 4095) / 4096 * 4096));
}

cudaError_t launch_clip(const Clip& c, float max_norm, float* norm, long long wait_limit, bool skip, cudaStream_t s) {
  ClipArgs a;
  a.skip = skip ? 1 : 0;
  a.chunks = c.chunks;
  a.n_chunks = c.n_chunks;
  a.slot_bytes = c.chunk_bytes;
  a.part = c.part;
  a.arrived = c.arrived;
  a.max_norm = max_norm;
  a.norm = norm;
  a.status = c.status;
  a.wait_limit = wait_limit;
  const int per = (c.n_chunks + c.grid - 1) / c.grid;
  a.keep = kKeepBytes / (c.chunk_bytes * c.grid);
  a.slots = std::max(1, std::min({per, kRingBytes / c.chunk_bytes, kMaxSlots}));
  const int smem = a.slots * c.chunk_bytes;
  static std::atomic<unsigned long long> allowed{0};
  cudaError_t e = allow_smem((const void*)k_clip, kRingBytes, c.device, allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(c.grid);
  cfg.blockDim = dim3(kThreads + 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;   // its CTAs wait for one another
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, k_clip, a);
  if (e != cudaSuccess) allowed = 0;
  return e;
}

}  // namespace owq
