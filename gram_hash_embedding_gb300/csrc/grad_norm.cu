// The global norm of a list of gradients, and clipping (sm_103a):
//   norm = sqrt(sum over all tensors of g^2)   or   max |g|
//   out  = round(g * min(1, max_norm / (norm + 1e-6)))
// Each value's square and a thread's sums are fp32; the sums of a block and the join of the blocks are
// 64-bit, in a fixed order, so the same call gives the same bits.
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "engram_internal.cuh"
#include "train.cuh"

namespace engram {
namespace {

constexpr int kThreads = 256;
constexpr int kPerLaunch = 512;   // tensors whose descriptions travel as one launch's argument
constexpr int kMaxGrid = 152 * 8;
constexpr int64_t kChunk = 16384;  // values per work item

struct Item {
  const void* data;
  void* out;
  const int64_t* rows_used;  // null: all n values count
  int64_t n;
  int32_t row_len;
  int16_t type, out_type;
};

// the tensors of one launch; first[i]: the first chunk of tensor i
struct Batch {
  Item item[kPerLaunch];
  uint32_t first[kPerLaunch + 1];
  int32_t n;
};

__device__ __forceinline__ int64_t values_in_use(const Item& it) {
  if (it.rows_used == nullptr) return it.n;
  const int64_t r = *it.rows_used;
  const int64_t v = r < 0 ? 0 : r * it.row_len;
  return r > it.n / it.row_len ? it.n : v;
}

__device__ __forceinline__ float load_any(const Item& it, int64_t i) {
  switch (it.type) {
    case ENGRAM_TYPE_F32: return static_cast<const float*>(it.data)[i];
    case ENGRAM_TYPE_BF16: return __bfloat162float(static_cast<const __nv_bfloat16*>(it.data)[i]);
    default: return __half2float(static_cast<const __half*>(it.data)[i]);
  }
}

__device__ __forceinline__ void store_any(const Item& it, int64_t i, float v) {
  switch (it.out_type) {
    case ENGRAM_TYPE_F32: static_cast<float*>(it.out)[i] = v; break;
    case ENGRAM_TYPE_BF16: static_cast<__nv_bfloat16*>(it.out)[i] = __float2bfloat16_rn(v); break;
    default: static_cast<__half*>(it.out)[i] = __float2half_rn(v);
  }
}

// the larger of two magnitudes, NaN if either is NaN
__device__ __forceinline__ double max_nan(double a, double b) { return a != a ? a : (b != b ? b : (a > b ? a : b)); }

__device__ __forceinline__ double join(double a, double b, bool is_max) { return is_max ? max_nan(a, b) : a + b; }

__device__ __forceinline__ int tensor_of(const Batch& b, uint32_t chunk) {
  int lo = 0, hi = b.n - 1;  // the last tensor whose first chunk is <= chunk
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (b.first[mid] <= chunk) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// joined over the block in a fixed order; valid in thread 0
__device__ __forceinline__ double block_join(double v, bool is_max, double* ws) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = join(v, __shfl_xor_sync(0xffffffffu, v, o), is_max);
  if ((threadIdx.x & 31) == 0) ws[threadIdx.x >> 5] = v;
  __syncthreads();
  double r = ws[0];
  for (int w = 1; w < kThreads / 32; ++w) r = join(r, ws[w], is_max);
  __syncthreads();
  return r;
}

__global__ void __launch_bounds__(kThreads) norm_partial_kernel(const __grid_constant__ Batch b, const int is_max,
                                                                double* __restrict__ part) {
  pdl_wait();
  pdl_trigger();
  __shared__ double ws[kThreads / 32];
  double sum = 0.0;
  for (uint32_t c = blockIdx.x; c < b.first[b.n]; c += gridDim.x) {
    const int j = tensor_of(b, c);
    const Item& it = b.item[j];
    const int64_t i0 = (int64_t)(c - b.first[j]) * kChunk, i1 = min(i0 + kChunk, values_in_use(it));
    float f = 0.f;
    for (int64_t i = i0 + threadIdx.x; i < i1; i += kThreads) {
      const float v = load_any(it, i);
      if (is_max) f = (fabsf(v) > f || v != v) ? fabsf(v) : f; else f = fmaf(v, v, f);
    }
    sum = join(sum, (double)f, is_max);
  }
  const double r = block_join(sum, is_max, ws);
  if (threadIdx.x == 0) part[blockIdx.x] = r;
}

__device__ __forceinline__ float norm_of(const double* part, int n_part, bool is_max, double* ws) {
  double v = 0.0;
  for (int i = threadIdx.x; i < n_part; i += kThreads) v = join(v, part[i], is_max);
  const double r = block_join(v, is_max, ws);
  return (float)(is_max ? r : sqrt(r));
}

__global__ void __launch_bounds__(kThreads) norm_finish_kernel(const double* __restrict__ part, int n_part, int is_max,
                                                               float* __restrict__ norm) {
  pdl_wait();
  pdl_trigger();
  __shared__ double ws[kThreads / 32];
  const float r = norm_of(part, n_part, is_max, ws);
  if (threadIdx.x == 0) *norm = r;
}

__global__ void __launch_bounds__(kThreads) clip_kernel(const __grid_constant__ Batch b, const int is_max,
                                                        const double* __restrict__ part, int n_part, float max_norm,
                                                        float* __restrict__ norm) {
  pdl_wait();
  pdl_trigger();
  __shared__ double ws[kThreads / 32];
  const float total = norm_of(part, n_part, is_max, ws);
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = total;
  const float q = max_norm / (total + 1e-6f);
  const float coef = q > 1.0f ? 1.0f : q;  // NaN stays NaN
  for (uint32_t c = blockIdx.x; c < b.first[b.n]; c += gridDim.x) {
    const int j = tensor_of(b, c);
    const Item& it = b.item[j];
    if (coef == 1.0f && it.out == it.data) continue;
    const int64_t i0 = (int64_t)(c - b.first[j]) * kChunk, i1 = min(i0 + kChunk, values_in_use(it));
    for (int64_t i = i0 + threadIdx.x; i < i1; i += kThreads) store_any(it, i, load_any(it, i) * coef);
  }
}

// the batch starting at tensor t0; returns the next tensor
int32_t fill_batch(const engram_tensor* t, int32_t n, int32_t t0, Batch* b) {
  int32_t k = 0;
  uint64_t chunks = 0;
  for (; t0 + k < n && k < kPerLaunch; ++k) {
    const engram_tensor& x = t[t0 + k];
    const uint64_t more = (uint64_t)((x.n + kChunk - 1) / kChunk);
    if (chunks + more > 0xffffffffu) break;
    b->item[k] = Item{x.data, x.out != nullptr ? x.out : const_cast<void*>(x.data), x.rows_used, x.n,
                      x.rows_used != nullptr ? x.row_len : 1, (int16_t)x.type,
                      (int16_t)(x.out != nullptr ? x.out_type : x.type)};
    b->first[k] = (uint32_t)chunks;
    chunks += more;
  }
  b->first[k] = (uint32_t)chunks;
  b->n = k;
  return t0 + k;
}

unsigned grid_of(const Batch& b) { return (unsigned)std::max<uint32_t>(1u, std::min<uint32_t>(b.first[b.n], kMaxGrid)); }

}  // namespace

uint64_t grad_norm_workspace(int32_t n_tensors) {
  const uint64_t batches = (uint64_t)(n_tensors + kPerLaunch - 1) / kPerLaunch;
  return batches * kMaxGrid * sizeof(double);
}

cudaError_t launch_grad_norm(const engram_tensor* tensors, int32_t n_tensors, int32_t norm_type, bool clip,
                             float max_norm, float* norm, void* workspace, cudaStream_t s) {
  const int is_max = norm_type == ENGRAM_NORM_MAX;
  double* part = static_cast<double*>(workspace);
  int n_part = 0;
  Batch b;
  for (int32_t t = 0; t < n_tensors;) {
    t = fill_batch(tensors, n_tensors, t, &b);
    const unsigned g = grid_of(b);
    cudaError_t e = launch_pdl(norm_partial_kernel, dim3(g), dim3(kThreads), 0, s, b, is_max, part + n_part);
    if (e != cudaSuccess) return e;
    n_part += (int)g;
  }
  if (!clip || n_tensors == 0)
    return launch_pdl(norm_finish_kernel, dim3(1), dim3(kThreads), 0, s, (const double*)part, n_part, is_max, norm);
  for (int32_t t = 0; t < n_tensors;) {
    t = fill_batch(tensors, n_tensors, t, &b);
    cudaError_t e = launch_pdl(clip_kernel, dim3(grid_of(b)), dim3(kThreads), 0, s, b, is_max, (const double*)part,
                               n_part, max_norm, norm);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace engram
