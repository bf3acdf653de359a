// Internal declarations of the training operators: trainable embedding rows and their gradient
// (embed.cu), the gate's gradient (gate_grad.cu), the gradient norm and clipping (grad_norm.cu).
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "../../include/engram.h"

namespace engram {

// ------------------------------------------------------------------ values of the three float types
__host__ __device__ constexpr int type_bytes(int t) { return t == ENGRAM_TYPE_F32 ? 4 : 2; }

template <int TYPE>
struct Elem;
template <>
struct Elem<ENGRAM_TYPE_F32> {
  using type = float;
  static __device__ __forceinline__ float load(const float* p) { return *p; }
  static __device__ __forceinline__ void store(float* p, float v) { *p = v; }
};
template <>
struct Elem<ENGRAM_TYPE_BF16> {
  using type = __nv_bfloat16;
  static __device__ __forceinline__ float load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
};
template <>
struct Elem<ENGRAM_TYPE_F16> {
  using type = __half;
  static __device__ __forceinline__ float load(const __half* p) { return __half2float(*p); }
  static __device__ __forceinline__ void store(__half* p, float v) { *p = __float2half_rn(v); }
};

// V consecutive values: V = 8 with one access of 16 bytes for the 16-bit types and of 32 for fp32 (two of 16 where
// the address is on no 32-byte boundary: a warp's halves of sectors cost the pass that writes 2.1 GB of clipped
// fp32 values 930 us instead of 575); V = 4 with half of that (rows of 100 values, say); V = 1 for rows whose width or
// alignment allows neither. Raw<> keeps them as loaded, so that many loads can be in flight before the first
// is widened.
template <int TYPE, int V>
struct Raw;
template <int TYPE>
struct Raw<TYPE, 8> {
  uint4 a, b;  // b: the second half of 8 fp32 values
  __device__ __forceinline__ void load(const typename Elem<TYPE>::type* p) {
    if constexpr (TYPE == ENGRAM_TYPE_F32) {
      if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {
        asm("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
            : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
            : "l"(p)
            : "memory");
      } else {
        a = reinterpret_cast<const uint4*>(p)[0];
        b = reinterpret_cast<const uint4*>(p)[1];
      }
    } else {
      a = *reinterpret_cast<const uint4*>(p);
    }
  }
  __device__ __forceinline__ void zero() {
    a = make_uint4(0u, 0u, 0u, 0u);
    if constexpr (TYPE == ENGRAM_TYPE_F32) b = make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ void widen(float* f) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
    if constexpr (TYPE == ENGRAM_TYPE_F32) {
      const uint32_t u[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[i] = __uint_as_float(w[i]);
        f[4 + i] = __uint_as_float(u[i]);
      }
    } else if constexpr (TYPE == ENGRAM_TYPE_BF16) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        f[2 * i] = v.x;
        f[2 * i + 1] = v.y;
      }
    }
  }
};
template <>
struct Raw<ENGRAM_TYPE_F32, 4> {
  float4 a;
  __device__ __forceinline__ void load(const float* p) { a = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void zero() { a = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void widen(float* f) const {
    f[0] = a.x;
    f[1] = a.y;
    f[2] = a.z;
    f[3] = a.w;
  }
};
template <int TYPE>
struct Raw<TYPE, 4> {
  uint2 a;
  __device__ __forceinline__ void load(const typename Elem<TYPE>::type* p) { a = *reinterpret_cast<const uint2*>(p); }
  __device__ __forceinline__ void zero() { a = make_uint2(0u, 0u); }
  __device__ __forceinline__ void widen(float* f) const {
    const typename Elem<TYPE>::type* e = reinterpret_cast<const typename Elem<TYPE>::type*>(&a);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = Elem<TYPE>::load(e + i);
  }
};
template <int TYPE>
struct Raw<TYPE, 1> {
  typename Elem<TYPE>::type a;
  __device__ __forceinline__ void load(const typename Elem<TYPE>::type* p) { a = *p; }
  __device__ __forceinline__ void zero() { Elem<TYPE>::store(&a, 0.f); }
  __device__ __forceinline__ void widen(float* f) const { f[0] = Elem<TYPE>::load(&a); }
};

template <int TYPE>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  static_assert(TYPE != ENGRAM_TYPE_F32, "16-bit types only");
  uint32_t r;
  if constexpr (TYPE == ENGRAM_TYPE_BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    r = *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __half2 v = __floats2half2_rn(lo, hi);
    r = *reinterpret_cast<const uint32_t*>(&v);
  }
  return r;
}

// V values rounded once (to nearest even) to the stored type. ONCE: with an evict-first policy, for what is
// written and not read again by the same call
template <int TYPE, int V, bool ONCE = false>
__device__ __forceinline__ void store_vals(typename Elem<TYPE>::type* p, const float* f) {
  if constexpr (V == 1) {
    Elem<TYPE>::store(p, f[0]);
  } else if constexpr (V == 4 && TYPE == ENGRAM_TYPE_F32) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  } else if constexpr (V == 4) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack2<TYPE>(f[0], f[1]), pack2<TYPE>(f[2], f[3]));
  } else if constexpr (TYPE == ENGRAM_TYPE_F32) {
    if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {
      if constexpr (ONCE)
        asm volatile("st.global.L2::evict_first.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(f[0]),
                     "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7])
                     : "memory");
      else
        asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(f[0]), "f"(f[1]),
                     "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7])
                     : "memory");
    } else {
      reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
      reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
  } else {
    const uint4 v =
        make_uint4(pack2<TYPE>(f[0], f[1]), pack2<TYPE>(f[2], f[3]), pack2<TYPE>(f[4], f[5]), pack2<TYPE>(f[6], f[7]));
    if constexpr (ONCE) __stcs(reinterpret_cast<uint4*>(p), v);
    else *reinterpret_cast<uint4*>(p) = v;
  }
}

// calls f(integral_constant<TYPE>) for a runtime type code
template <typename F>
cudaError_t with_type(int32_t t, F&& f) {
  switch (t) {
    case ENGRAM_TYPE_F32: return f(std::integral_constant<int, ENGRAM_TYPE_F32>{});
    case ENGRAM_TYPE_BF16: return f(std::integral_constant<int, ENGRAM_TYPE_BF16>{});
    case ENGRAM_TYPE_F16: return f(std::integral_constant<int, ENGRAM_TYPE_F16>{});
    default: return cudaErrorInvalidValue;
  }
}

// ------------------------------------------------------------------------------------ embedding rows
struct EmbedArgs {
  const int64_t* idx;  // token t's row ids at idx[t * idx_stride + c]
  int64_t idx_stride;
  int64_t T;
  int32_t n_cols;
  int64_t rows;
  int32_t dim;
  float scale;
};
cudaError_t launch_embed(const EmbedArgs& a, const void* W, int64_t row_stride, int32_t w_type, void* out,
                         int32_t out_type, cudaStream_t s);

struct EmbedGradArgs {
  EmbedArgs e;
  const void* dout;      // token t's gradients at dout + t * dout_stride + c * dim (elements)
  int64_t dout_stride;
  int32_t dout_type;
  void* grad;            // sparse: [n][dim], row u belongs to grad_rows[u]; dense: [rows] rows of grad_stride
  int64_t grad_stride;
  int32_t grad_type;
  int64_t* grad_rows;    // sparse form only (null: dense form)
  int64_t* count;        // sparse form only
  int32_t accumulate;    // dense form: add to what grad holds
};
uint64_t embed_grad_workspace(int64_t n, int64_t rows, int32_t dim);
cudaError_t launch_embed_grad(const EmbedGradArgs& a, void* workspace, cudaStream_t s);

// -------------------------------------------------------------------------------- the gate's gradient
struct GateGradArgs {
  const uint16_t *x, *kv, *qw, *kw, *dout;
  const uint8_t* mask;  // may be null
  int64_t T;
  int32_t hc, dim;
  float eps;
  uint16_t *dx, *dkv;
  float *dq, *dk;
};
uint64_t gate_grad_workspace(int64_t T, int32_t hc, int32_t dim);
// withhold >= 0: the test hook of engram_gate_grad_withhold
cudaError_t launch_gate_grad(const GateGradArgs& a, void* workspace, cudaStream_t s, int64_t withhold = -1);

// The same from checkpoints in 8 bits (gate_grad8.cu): E4M3 codes [T][hc][dim] and [T][hc + 1][dim] with a UE8M0 scale for
// each `block` columns of a row. `g`: the rest of the arguments (its x and kv unused).
struct GateGrad8Args {
  GateGradArgs g;
  const uint8_t *x, *xs, *kv, *kvs;
  int32_t block;
};
uint64_t gate_grad8_workspace(int64_t T, int32_t hc, int32_t dim);
cudaError_t launch_gate_grad8(const GateGrad8Args& a, void* workspace, cudaStream_t s, int64_t withhold = -1);

// ------------------------------------------------------------------------- gradient norm and clipping
uint64_t grad_norm_workspace(int32_t n_tensors);
// clip false: only the norm (max_norm and the tensors' out unused)
cudaError_t launch_grad_norm(const engram_tensor* tensors, int32_t n_tensors, int32_t norm_type, bool clip,
                             float max_norm, float* norm, void* workspace, cudaStream_t s);

}  // namespace engram
