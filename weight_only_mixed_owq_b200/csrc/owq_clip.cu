// Global 2-norm of many gradient tensors and their clipping, in one launch:
//   norm = sqrt(sum over all tensors of g^2),  out = g min(1, max_norm / (norm + 1e-6))
// (a norm that is not finite leaves the factor at 1: the caller sees it and skips its step).
//
// Bound: HBM.  Every value has to be read once and written once; the norm needs all of them
// before the first can be written, so what does not stay on the chip is read again.
//
// One cooperative launch of one CTA per SM.  The tensors are cut into chunks dealt round-robin to
// the CTAs; each CTA keeps its first chunks in shared memory (about 190 KB per SM), streams the
// others, adds the squares in fp64 (no overflow, underflow or cancellation at any length; the
// conversions stay far below the memory time), publishes its partial sum and waits for the
// others' (bounded).  The second pass walks the chunks backwards: the last ones read are still in
// L2, and the streaming stores leave them there until they are read.  All sums run in a fixed
// order: repeated calls give identical bits.
#include <cuda_bf16.h>

#include "owq_internal.cuh"

namespace owq {
namespace {

constexpr int kThreads = 1024;
constexpr int kSlotBytes = 64 * 1024;   // most bytes of a chunk
constexpr int kCacheBytes = 3 * kSlotBytes;

struct ClipArgs {
  const ClipChunk* chunks;
  int n_chunks;
  int slot_bytes;     // bytes a chunk's 16-byte pieces take in shared memory
  int cached;         // chunks of a CTA kept in shared memory
  double* part;       // [gridDim.x] partial sums
  unsigned long long* arrived;   // CTAs that have published, over all calls
  float max_norm;
  float* norm;
  int* status;
  long long wait_limit;
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
__device__ __forceinline__ double squares(const ClipChunk& c, uint4* keep) {
  using T = typename Vec<DT>::T;
  constexpr int P = 16 / sizeof(T);
  const T* in = static_cast<const T*>(c.in);
  const Cut<T> cut(in, c.n);
  const uint4* v = reinterpret_cast<const uint4*>(in + cut.head);
  double s = 0.0;
  #pragma unroll 4
  for (int i = threadIdx.x; i < cut.pieces; i += kThreads) {
    const uint4 q = __ldcg(v + i);
    if (keep) keep[i] = q;
    const T* e = reinterpret_cast<const T*>(&q);
    if constexpr (DT == OWQ_F16) {   // squares of fp16 values are exact in fp32, and never overflow
      #pragma unroll
      for (int j = 0; j < P; j += 2) {
        const float a = Vec<DT>::get(e[j]), b = Vec<DT>::get(e[j + 1]);
        s += (double)fmaf(a, a, b * b);
      }
    } else {
      #pragma unroll
      for (int j = 0; j < P; ++j) {
        const double a = (double)Vec<DT>::get(e[j]);
        s = fma(a, a, s);
      }
    }
  }
  const int tail = cut.head + cut.pieces * P;   // fewer than P values at either end
  const int i = threadIdx.x < cut.head ? (int)threadIdx.x : tail + (int)threadIdx.x - cut.head;
  if (i < c.n && (threadIdx.x < cut.head || i >= tail) && threadIdx.x < 2 * P) {
    const double a = (double)Vec<DT>::get(in[i]);
    s = fma(a, a, s);
  }
  return s;
}

template <int DT>
__device__ __forceinline__ void scale(const ClipChunk& c, const uint4* kept, float f) {
  using T = typename Vec<DT>::T;
  constexpr int P = 16 / sizeof(T);
  const T* in = static_cast<const T*>(c.in);
  T* out = static_cast<T*>(c.out);
  const Cut<T> cut(in, c.n);
  const uint4* v = reinterpret_cast<const uint4*>(in + cut.head);
  T* o = out + cut.head;
  const bool vec = (reinterpret_cast<uintptr_t>(o) & 15) == 0;
  const bool copy = f == 1.f;   // bit for bit (a product would quieten a NaN's payload)
  #pragma unroll 4
  for (int i = threadIdx.x; i < cut.pieces; i += kThreads) {
    const uint4 q = kept ? kept[i] : __ldcg(v + i);
    const T* e = reinterpret_cast<const T*>(&q);
    uint4 r;
    T* d = reinterpret_cast<T*>(&r);
    #pragma unroll
    for (int j = 0; j < P; ++j) d[j] = copy ? e[j] : Vec<DT>::put(Vec<DT>::get(e[j]) * f);
    if (vec) {
      __stcs(reinterpret_cast<uint4*>(o) + i, r);
    } else {
      #pragma unroll
      for (int j = 0; j < P; ++j) o[(size_t)i * P + j] = d[j];
    }
  }
  const int tail = cut.head + cut.pieces * P;
  const int i = threadIdx.x < cut.head ? (int)threadIdx.x : tail + (int)threadIdx.x - cut.head;
  if (i < c.n && (threadIdx.x < cut.head || i >= tail) && threadIdx.x < 2 * P) out[i] = copy ? in[i] : Vec<DT>::put(Vec<DT>::get(in[i]) * f);
}

// sum over the CTA in a fixed order; the result in every thread
__device__ __forceinline__ double block_sum(double v, double* s_red) {
  #pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = s_red[threadIdx.x & 31];
  #pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  return v;
}

__global__ void __launch_bounds__(kThreads, 1) k_clip(const __grid_constant__ ClipArgs a) {
  extern __shared__ __align__(16) unsigned char cache[];
  __shared__ double s_red[32];
  __shared__ int s_ok;
  const int G = gridDim.x, b = blockIdx.x;
  const int mine = b < a.n_chunks ? (a.n_chunks - 1 - b) / G + 1 : 0;   // chunks b, b + G, ...

  double s = 0.0;
  ClipChunk next = {};
  if (mine > 0) next = a.chunks[b];
  for (int i = 0; i < mine; ++i) {
    const ClipChunk c = next;
    if (i + 1 < mine) next = a.chunks[b + (size_t)(i + 1) * G];
    uint4* keep = i < a.cached ? reinterpret_cast<uint4*>(cache + (size_t)i * a.slot_bytes) : nullptr;
    if (c.dtype == OWQ_F32) s += squares<OWQ_F32>(c, keep);
    else if (c.dtype == OWQ_F16) s += squares<OWQ_F16>(c, keep);
    else s += squares<OWQ_BF16>(c, keep);
  }
  s = block_sum(s, s_red);

  // publish, then wait until every CTA of this call has: the counter only grows, by G a call
  if (threadIdx.x == 0) {
    a.part[b] = s;
    __threadfence();
    const unsigned long long old = atomicAdd(a.arrived, 1ull);
    const unsigned long long want = (old / G + 1) * G;
    int ok = 1;
    const long long t0 = clock64();
    while (*reinterpret_cast<volatile unsigned long long*>(a.arrived) < want)
      if (clock64() - t0 > a.wait_limit) {
        atomicOr(a.status, kStatusTimeout);
        ok = 0;
        break;
      }
    __threadfence();
    s_ok = ok;
  }
  __syncthreads();
  if (!s_ok) return;
  double t = 0.0;
  for (int i = threadIdx.x; i < G; i += kThreads) t += __ldcg(a.part + i);
  t = block_sum(t, s_red);
  const float norm = (float)sqrt(t);
  const float f = norm <= 3.402823466e38f ? fminf(a.max_norm / (norm + 1e-6f), 1.f) : 1.f;   // (false for NaN too)
  if (b == 0 && threadIdx.x == 0) *a.norm = norm;

  if (mine > 0) next = a.chunks[b + (size_t)(mine - 1) * G];
  for (int i = mine - 1; i >= 0; --i) {
    const ClipChunk c = next;
    if (i > 0) next = a.chunks[b + (size_t)(i - 1) * G];
    if (f == 1.f && c.in == c.out) continue;   // in place and unclipped
    const uint4* kept = i < a.cached ? reinterpret_cast<const uint4*>(cache + (size_t)i * a.slot_bytes) : nullptr;
    if (c.dtype == OWQ_F32) scale<OWQ_F32>(c, kept, f);
    else if (c.dtype == OWQ_F16) scale<OWQ_F16>(c, kept, f);
    else scale<OWQ_BF16>(c, kept, f);
  }
}

}  // namespace

// Bytes of a chunk: the work of every CTA in about four chunks, so that the deal is even, within
// 4 KB (a few 16-byte pieces per thread or less: latency) and 64 KB (four pieces in flight each).
int clip_chunk_bytes(long long total_bytes, int sms) {
  const long long want = total_bytes / (4LL * sms);
  return (int)std::max<long long>(4096, std::min<long long>(kSlotBytes, (want + 4095) / 4096 * 4096));
}

cudaError_t launch_clip(const Clip& c, float max_norm, float* norm, long long wait_limit, cudaStream_t s) {
  ClipArgs a;
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
  a.cached = std::min(per, kCacheBytes / c.chunk_bytes);
  const int smem = a.cached * c.chunk_bytes;
  static std::atomic<unsigned long long> allowed{0};
  cudaError_t e = allow_smem((const void*)k_clip, kCacheBytes, c.device, allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(c.grid);
  cfg.blockDim = dim3(kThreads);
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
