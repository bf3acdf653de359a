// The global norm of a list of gradients, and clipping (sm_103a):
//   norm = sqrt(sum over all tensors of g^2)   or   max |g|
//   out  = round(g * min(1, max_norm / (norm + 1e-6)))
// A value's square and a thread's sums over one chunk are fp32; everything from there on is 64-bit, in an order
// that follows from the tensors' sizes and where they lie in their 16-byte words, so the same call gives the same bits.
//
// Design: bound by memory, one read for the norm and a read and a write for the clip. The tensors'
// descriptions travel as the launch's argument (no copy to the device, nothing kept between calls), and
// every tensor is cut into chunks that the CTAs take in turn, so 300 tensors of any sizes are one
// launch. The clip goes through the chunks from the last to the first: the end of the list is what the norm's
// pass left in L2. Lists that a cluster of 8 CTAs can hold are one launch for norm and clip together: the
// CTAs exchange their sums through distributed shared memory.
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "engram_internal.cuh"
#include "train.cuh"

namespace engram {
namespace {

constexpr int kThreads = 256;
constexpr int kFew = 32;           // tensors of a launch with the short argument
constexpr int kPerLaunch = 512;    // tensors of a launch with the long one (22 KB of the 32 KB allowed)
constexpr int kMaxGrid = 152 * 8;
constexpr int kVecs = 8;           // vectors of 8 values a thread has per chunk
constexpr int64_t kChunk = (int64_t)kThreads * kVecs * 8;  // values per work item: a CTA takes it
constexpr int kCluster = 8;        // CTAs of the one-launch form
constexpr int kClusterThreads = 512;
constexpr int64_t kWarpChunk = 32 * kVecs * 8;  // values per work item there: a warp takes it, so that the many
                                                // small tensors of a small model are read all at once
constexpr uint32_t kClusterChunks = 512;  // the most work items it takes

struct Item {
  const void* data;
  void* out;
  const int64_t* rows_used;  // null: all n values count
  int64_t n;
  int32_t row_len;
  int8_t type, out_type;
  int8_t head;      // values before the first one that data and out both hold on a 16-byte boundary
  int8_t wide;      // such a value exists
};

// the tensors of one launch; first[i]: the first chunk of tensor i
template <int N>
struct Batch {
  Item item[N];
  uint32_t first[N + 1];
  int32_t n;
};

__device__ __forceinline__ int64_t values_in_use(const Item& it) {
  if (it.rows_used == nullptr) return it.n;
  const int64_t r = *it.rows_used;
  return r < 0 ? 0 : (r > it.n / it.row_len ? it.n : r * it.row_len);
}

template <int TYPE>
__device__ __forceinline__ const typename Elem<TYPE>::type* in_of(const Item& it) {
  return static_cast<const typename Elem<TYPE>::type*>(it.data);
}

// Chunk q of a tensor: whole vectors of 8 values from the first boundary on. Chunk 0 takes the values
// before it as well, and whoever has the last vector the values after it. Without a common boundary
// every value is moved by itself.
struct Span8 {
  int64_t i0;        // the first vector's first value
  int m;             // vectors
  int64_t one0, n_one;  // single values [one0, one0 + n_one)
  int before;        // and [0, before)
};
template <int64_t CHUNK>
__device__ __forceinline__ Span8 span_of(const Item& it, int64_t used, int64_t q) {
  Span8 s;
  s.before = 0;
  if (!it.wide) {
    s.i0 = 0;
    s.m = 0;
    s.one0 = q * CHUNK;
    s.n_one = max((int64_t)0, min(CHUNK, used - s.one0));
    return s;
  }
  s.i0 = q * CHUNK + it.head;
  const int64_t i1 = min(s.i0 + CHUNK, used);
  s.m = i1 > s.i0 ? (int)((i1 - s.i0) >> 3) : 0;
  s.one0 = s.i0 + (int64_t)s.m * 8;
  s.n_one = max((int64_t)0, i1 - s.one0);
  if (q == 0) s.before = (int)min((int64_t)it.head, used);
  return s;
}

// the chunk's sum of squares (or its largest magnitude) over one thread's values
template <int TYPE, int THREADS>
__device__ __forceinline__ double chunk_norm(const typename Elem<TYPE>::type* p, const Span8 c, const bool is_max,
                                             const int tid) {
  float s[8] = {};
  uint32_t top = 0;  // a magnitude's bits order like the magnitude, NaN above infinity
  auto one = [&](int64_t i) {
    const float f = Elem<TYPE>::load(p + i);
    if (is_max) top = max(top, __float_as_uint(f) & 0x7fffffffu);
    else s[0] = fmaf(f, f, s[0]);
  };
  const typename Elem<TYPE>::type* v0 = p + c.i0;
  constexpr int kFly = TYPE == ENGRAM_TYPE_F32 ? 2 : 4;  // vectors in flight
#pragma unroll 1
  for (int v = tid; v < c.m; v += kFly * THREADS) {
    Raw<TYPE, 8> raw[kFly];
#pragma unroll
    for (int j = 0; j < kFly; ++j) {
      raw[j].zero();
      if (v + j * THREADS < c.m) raw[j].load(v0 + (v + j * THREADS) * 8);
    }
#pragma unroll
    for (int j = 0; j < kFly; ++j) {
      float f[8];
      raw[j].widen(f);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (is_max) top = max(top, __float_as_uint(f[e]) & 0x7fffffffu);
        else s[e] = fmaf(f[e], f[e], s[e]);
      }
    }
  }
#pragma unroll 1
  for (int64_t i = tid; i < c.n_one; i += THREADS) one(c.one0 + i);
  if (tid < c.before) one(tid);
  if (is_max) return (double)__uint_as_float(top);
  return (double)(((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7])));
}

template <int V>
__device__ __forceinline__ void store_as(void* o, int out_type, int64_t i, const float* f) {
  if (out_type == ENGRAM_TYPE_F32) store_vals<ENGRAM_TYPE_F32, V>(static_cast<float*>(o) + i, f);
  else if (out_type == ENGRAM_TYPE_BF16) store_vals<ENGRAM_TYPE_BF16, V>(static_cast<__nv_bfloat16*>(o) + i, f);
  else store_vals<ENGRAM_TYPE_F16, V>(static_cast<__half*>(o) + i, f);
}

template <int TYPE, int THREADS>
__device__ __forceinline__ void chunk_clip(const typename Elem<TYPE>::type* p, void* o, const int out_type,
                                           const Span8 c, const float coef, const int tid) {
  constexpr int kFly = TYPE == ENGRAM_TYPE_F32 ? 2 : 4;
#pragma unroll 1
  for (int v = tid; v < c.m; v += kFly * THREADS) {
    Raw<TYPE, 8> raw[kFly];
#pragma unroll
    for (int j = 0; j < kFly; ++j)
      if (v + j * THREADS < c.m) raw[j].load(p + c.i0 + (v + j * THREADS) * 8);
#pragma unroll
    for (int j = 0; j < kFly; ++j) {
      if (v + j * THREADS < c.m) {
        float f[8];
        raw[j].widen(f);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= coef;
        store_as<8>(o, out_type, c.i0 + (v + j * THREADS) * 8, f);
      }
    }
  }
  auto one = [&](int64_t i) {
    const float f = Elem<TYPE>::load(p + i) * coef;
    store_as<1>(o, out_type, i, &f);
  };
#pragma unroll 1
  for (int64_t i = tid; i < c.n_one; i += THREADS) one(c.one0 + i);
  if (tid < c.before) one(tid);
}

// THREADS threads (a CTA or a warp), this one number `tid` of them, on chunk q of a tensor
template <int THREADS>
__device__ __forceinline__ double any_norm(const Item& it, int64_t q, bool is_max, int tid) {
  const Span8 c = span_of<(int64_t)THREADS * kVecs * 8>(it, values_in_use(it), q);
  switch (it.type) {
    case ENGRAM_TYPE_F32: return chunk_norm<ENGRAM_TYPE_F32, THREADS>(in_of<ENGRAM_TYPE_F32>(it), c, is_max, tid);
    case ENGRAM_TYPE_BF16: return chunk_norm<ENGRAM_TYPE_BF16, THREADS>(in_of<ENGRAM_TYPE_BF16>(it), c, is_max, tid);
    default: return chunk_norm<ENGRAM_TYPE_F16, THREADS>(in_of<ENGRAM_TYPE_F16>(it), c, is_max, tid);
  }
}

template <int THREADS>
__device__ __forceinline__ void any_clip(const Item& it, int64_t q, float coef, int tid) {
  if (coef == 1.0f && it.out == it.data) return;
  const Span8 c = span_of<(int64_t)THREADS * kVecs * 8>(it, values_in_use(it), q);
  const int ot = it.out_type;
  switch (it.type) {
    case ENGRAM_TYPE_F32: chunk_clip<ENGRAM_TYPE_F32, THREADS>(in_of<ENGRAM_TYPE_F32>(it), it.out, ot, c, coef, tid); break;
    case ENGRAM_TYPE_BF16:
      chunk_clip<ENGRAM_TYPE_BF16, THREADS>(in_of<ENGRAM_TYPE_BF16>(it), it.out, ot, c, coef, tid);
      break;
    default: chunk_clip<ENGRAM_TYPE_F16, THREADS>(in_of<ENGRAM_TYPE_F16>(it), it.out, ot, c, coef, tid);
  }
}

// the larger of two magnitudes, NaN if either is NaN
__device__ __forceinline__ double max_nan(double a, double b) { return a != a ? a : (b != b ? b : (a > b ? a : b)); }

__device__ __forceinline__ double join(double a, double b, bool is_max) { return is_max ? max_nan(a, b) : a + b; }

// the last tensor whose first chunk is <= chunk
template <int N>
__device__ __forceinline__ int tensor_of(const Batch<N>& b, uint32_t chunk) {
  int lo = 0, hi = b.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (b.first[mid] <= chunk) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// joined over the block in a fixed order, the same value in every thread
template <int THREADS>
__device__ __forceinline__ double block_join(double v, bool is_max, double* ws) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = join(v, __shfl_xor_sync(0xffffffffu, v, o), is_max);
  if ((threadIdx.x & 31) == 0) ws[threadIdx.x >> 5] = v;
  __syncthreads();
  double r = ws[0];
  for (int w = 1; w < THREADS / 32; ++w) r = join(r, ws[w], is_max);
  __syncthreads();
  return r;
}

__device__ __forceinline__ float norm_value(double r, bool is_max) { return (float)(is_max ? r : sqrt(r)); }

__device__ __forceinline__ float clip_factor(float norm, float max_norm) {
  const float q = max_norm / (norm + 1e-6f);
  return q > 1.0f ? 1.0f : q;  // NaN stays NaN
}

template <int N>
__global__ void __launch_bounds__(kThreads, 4) norm_partial_kernel(const __grid_constant__ Batch<N> b, const int is_max,
                                                                double* __restrict__ part) {
  pdl_wait();
  pdl_trigger();
  __shared__ double ws[kThreads / 32];
  double sum = 0.0;
  const uint32_t all = b.first[b.n];
  int j = blockIdx.x < all ? tensor_of(b, blockIdx.x) : 0;
  for (uint32_t c = blockIdx.x; c < all; c += gridDim.x) {
    while (b.first[j + 1] <= c) ++j;
    sum = join(sum, any_norm<kThreads>(b.item[j], c - b.first[j], is_max, threadIdx.x), is_max);
  }
  const double r = block_join<kThreads>(sum, is_max, ws);
  if (threadIdx.x == 0) part[blockIdx.x] = r;
}

__device__ __forceinline__ float norm_of(const double* part, int n_part, bool is_max, double* ws) {
  double v = 0.0;
  for (int i = threadIdx.x; i < n_part; i += kThreads) v = join(v, part[i], is_max);
  return norm_value(block_join<kThreads>(v, is_max, ws), is_max);
}

__global__ void __launch_bounds__(kThreads) norm_finish_kernel(const double* __restrict__ part, int n_part, int is_max,
                                                               float* __restrict__ norm) {
  pdl_wait();
  pdl_trigger();
  __shared__ double ws[kThreads / 32];
  const float r = norm_of(part, n_part, is_max, ws);
  if (threadIdx.x == 0) *norm = r;
}

template <int N>
__global__ void __launch_bounds__(kThreads, 4) clip_kernel(const __grid_constant__ Batch<N> b, const int is_max,
                                                        const double* __restrict__ part, int n_part, float max_norm,
                                                        float* __restrict__ norm) {
  pdl_wait();
  pdl_trigger();
  __shared__ double ws[kThreads / 32];
  const float total = norm_of(part, n_part, is_max, ws);
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = total;
  const float coef = clip_factor(total, max_norm);
  const uint32_t all = b.first[b.n];
  int j = blockIdx.x < all ? tensor_of(b, all - 1 - blockIdx.x) : 0;
  for (uint32_t i = blockIdx.x; i < all; i += gridDim.x) {
    const uint32_t c = all - 1 - i;
    while (b.first[j] > c) --j;
    any_clip<kThreads>(b.item[j], c - b.first[j], coef, threadIdx.x);
  }
}

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// write v into the same shared variable of CTA `rank`
__device__ __forceinline__ void store_in_cta(double* p, uint32_t rank, double v) {
  const uint32_t local = static_cast<uint32_t>(__cvta_generic_to_shared(p));
  uint32_t remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(rank));
  asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(remote), "d"(v) : "memory");
}

// one cluster: the norm and, if asked, the clip
__global__ void __launch_bounds__(kClusterThreads)
    norm_clip_cluster_kernel(const __grid_constant__ Batch<kFew> b, const int is_max, const int clip, float max_norm,
                             float* __restrict__ norm) {
  pdl_wait();
  pdl_trigger();
  __shared__ double ws[kClusterThreads / 32];
  __shared__ double sums[kCluster];
  const uint32_t rank = cluster_rank(), all = b.first[b.n];
  // warps across the CTAs first, so that few items spread over all of them
  constexpr uint32_t kAll = kCluster * kClusterThreads / 32;
  const uint32_t c0 = (threadIdx.x >> 5) * kCluster + rank;
  const int lane = threadIdx.x & 31;
  double sum = 0.0;
  int j = c0 < all ? tensor_of(b, c0) : 0;
  for (uint32_t c = c0; c < all; c += kAll) {
    while (b.first[j + 1] <= c) ++j;
    sum = join(sum, any_norm<32>(b.item[j], c - b.first[j], is_max, lane), is_max);
  }
  const double mine = block_join<kClusterThreads>(sum, is_max, ws);
  cluster_barrier();  // every CTA has started before another writes into its shared memory
  if (threadIdx.x < kCluster) store_in_cta(&sums[rank], threadIdx.x, mine);
  cluster_barrier();
  double r = sums[0];
  for (int i = 1; i < kCluster; ++i) r = join(r, sums[i], is_max);
  const float total = norm_value(r, is_max);
  if (rank == 0 && threadIdx.x == 0) *norm = total;
  if (!clip) return;
  const float coef = clip_factor(total, max_norm);
  j = c0 < all ? tensor_of(b, c0) : 0;
  for (uint32_t c = c0; c < all; c += kAll) {
    while (b.first[j + 1] <= c) ++j;
    any_clip<32>(b.item[j], c - b.first[j], coef, lane);
  }
}

// Values before the first one that lies on a 16-byte boundary in data and, for a clip, in out (-1: none)
int head_of(const engram_tensor& x, bool clip) {
  const void* out = clip && x.out != nullptr ? x.out : x.data;
  const int32_t ot = clip && x.out != nullptr ? x.out_type : x.type;
  for (int h = 0; h < 8; ++h)
    if ((reinterpret_cast<uintptr_t>(x.data) + (uintptr_t)h * type_bytes(x.type)) % 16 == 0 &&
        (reinterpret_cast<uintptr_t>(out) + (uintptr_t)h * type_bytes(ot)) % 16 == 0)
      return h;
  return -1;
}

// the batch starting at tensor t0; returns the next tensor
template <int N>
int32_t fill_batch(const engram_tensor* t, int32_t n, int32_t t0, bool clip, int64_t chunk, Batch<N>* b) {
  int32_t k = 0;
  uint64_t chunks = 0;  // at most N * 2^36 / kChunk = 2^31
  for (; t0 + k < n && k < N; ++k) {
    const engram_tensor& x = t[t0 + k];
    const bool apart = clip && x.out != nullptr;
    const int head = head_of(x, clip);
    b->item[k] = Item{x.data, apart ? x.out : const_cast<void*>(x.data), x.rows_used, x.n,
                      x.rows_used != nullptr ? x.row_len : 1, (int8_t)x.type, (int8_t)(apart ? x.out_type : x.type),
                      (int8_t)(head < 0 ? 0 : head), (int8_t)(head >= 0)};
    b->first[k] = (uint32_t)chunks;
    chunks += (uint64_t)((x.n + chunk - 1) / chunk);
  }
  b->first[k] = (uint32_t)chunks;
  b->n = k;
  return t0 + k;
}

template <int N>
unsigned grid_of(const Batch<N>& b) {
  return (unsigned)std::max<uint32_t>(1u, std::min<uint32_t>(b.first[b.n], kMaxGrid));
}

template <int N>
cudaError_t launch_lists(const engram_tensor* tensors, int32_t n_tensors, int is_max, bool clip, float max_norm,
                         float* norm, double* part, cudaStream_t s) {
  int n_part = 0;
  Batch<N> b;
  for (int32_t t = 0; t < n_tensors;) {
    t = fill_batch(tensors, n_tensors, t, clip, kChunk, &b);
    const unsigned g = grid_of(b);
    const cudaError_t e = launch_pdl(norm_partial_kernel<N>, dim3(g), dim3(kThreads), 0, s, b, is_max, part + n_part);
    if (e != cudaSuccess) return e;
    n_part += (int)g;
  }
  if (!clip)
    return launch_pdl(norm_finish_kernel, dim3(1), dim3(kThreads), 0, s, (const double*)part, n_part, is_max, norm);
  for (int32_t t = (n_tensors - 1) / N * N; t >= 0; t -= N) {
    fill_batch(tensors, n_tensors, t, clip, kChunk, &b);
    const cudaError_t e = launch_pdl(clip_kernel<N>, dim3(grid_of(b)), dim3(kThreads), 0, s, b, is_max,
                                     (const double*)part, n_part, max_norm, norm);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

uint64_t grad_norm_workspace(int32_t n_tensors) {
  const uint64_t batches = (uint64_t)(n_tensors + kPerLaunch - 1) / kPerLaunch;
  return batches * kMaxGrid * sizeof(double);
}

cudaError_t launch_grad_norm(const engram_tensor* tensors, int32_t n_tensors, int32_t norm_type, bool clip,
                             float max_norm, float* norm, void* workspace, cudaStream_t s) {
  const int is_max = norm_type == ENGRAM_NORM_MAX;
  double* part = static_cast<double*>(workspace);
  if (n_tensors > kFew) return launch_lists<kPerLaunch>(tensors, n_tensors, is_max, clip, max_norm, norm, part, s);
  uint64_t chunks = 0;
  for (int32_t i = 0; i < n_tensors; ++i) chunks += (uint64_t)((tensors[i].n + kWarpChunk - 1) / kWarpChunk);
  if (chunks > kClusterChunks)
    return launch_lists<kFew>(tensors, n_tensors, is_max, clip, max_norm, norm, part, s);
  Batch<kFew> b;
  fill_batch(tensors, n_tensors, 0, clip, kWarpChunk, &b);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = ENGRAM_PDL;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kCluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(kCluster);
  cfg.blockDim = dim3(kClusterThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, norm_clip_cluster_kernel, b, is_max, (int)clip, max_norm, norm);
}

}  // namespace engram
