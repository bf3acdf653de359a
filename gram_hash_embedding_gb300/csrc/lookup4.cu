// Rows of a 4-bit table (sm_103a): ParallelEngramEmbedding.forward of the engram-first/lookup page with E2M1 codes in
// blocks of 32 (UE8M0 scales) or 16 (E4M3 scales) instead of fp8 rows, either read back to bf16 or gathered as they
// stand into an operand of the 4-bit product. An id outside the table gives a row of +0.
//
// Bound by DRAM: a row is dim / 2 bytes of codes at a random place and dim / block bytes of scales at another.
#include <cstdint>
#include <type_traits>

#include "engram_internal.cuh"
#include "lowbit.cuh"
#include "train.cuh"

namespace engram {
namespace {

constexpr int kThreads = 256;
constexpr int kFly = 4;  // units in flight a thread

__device__ __forceinline__ float scale4(uint32_t b, bool nv) {
  return nv ? widen_scale<ENGRAM_SCALE_E4M3>(b) : widen_scale<ENGRAM_SCALE_E8M0>(b);
}

// where the id of entry e (token e / n_cols, column e % n_cols) lies
template <typename N>
__device__ __forceinline__ int64_t id_at(const Lookup4Args& a, N e) {
  if (a.idx_stride == a.n_cols) return (int64_t)e;
  const N t = e / (uint32_t)a.n_cols;
  return (int64_t)t * a.idx_stride + (int64_t)(e - t * (uint32_t)a.n_cols);
}

// 16 bf16 values, 32 bytes at once where the address allows; evicted first, so that rows that ids repeat stay in L2 longer
__device__ __forceinline__ void st_row32(uint16_t* to, const float* v) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = bf16x2_rn(v[2 * i], v[2 * i + 1]);
  if ((reinterpret_cast<uintptr_t>(to) & 31) == 0) {
    asm volatile("st.global.L2::evict_first.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(w[0]), "r"(w[1]),
                 "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    __stcs(reinterpret_cast<uint4*>(to), make_uint4(w[0], w[1], w[2], w[3]));
    __stcs(reinterpret_cast<uint4*>(to) + 1, make_uint4(w[4], w[5], w[6], w[7]));
  }
}

// A unit is 16 values: 8 bytes of codes, 32 of output. N: the type that numbers units (32 bits where they fit).
template <bool NV, typename N>
__global__ void __launch_bounds__(kThreads) lookup4_kernel(const Lookup4Args a, uint16_t* __restrict__ out, const N units) {
  pdl_wait();
  pdl_trigger();
  const uint32_t per_row = a.dim / 16;
  const int64_t spr = a.dim / a.block;
  const N u0 = (N)blockIdx.x * (kThreads * kFly) + threadIdx.x;
  int64_t r[kFly];
  uint32_t k[kFly];
#pragma unroll
  for (int i = 0; i < kFly; ++i) {
    const N u = u0 + i * kThreads;
    r[i] = -1;
    k[i] = 0;
    if (u < units) {
      const N e = u / per_row;
      k[i] = (uint32_t)(u - e * per_row);
      r[i] = a.idx[id_at<N>(a, e)];
    }
  }
  uint2 w[kFly];
  uint32_t b[kFly];
#pragma unroll
  for (int i = 0; i < kFly; ++i) {
    w[i] = make_uint2(0u, 0u);
    b[i] = 0u;
    if (r[i] >= 0 && r[i] < a.table_rows) {
      w[i] = __ldg(reinterpret_cast<const uint2*>(a.Q + r[i] * (a.dim >> 1)) + k[i]);
      b[i] = __ldg(a.S + r[i] * spr + (NV ? k[i] : k[i] >> 1));
    }
  }
#pragma unroll
  for (int i = 0; i < kFly; ++i) {
    const N u = u0 + i * kThreads;
    if (u >= units) continue;
    float v[16];
    const float s = scale4(b[i], NV);
    widen_e2m1x8(w[i].x, s, v);
    widen_e2m1x8(w[i].y, s, v + 8);
    if (a.scale != 1.0f) {
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] *= a.scale;
    }
    st_row32(out + (int64_t)u * 16, v);
  }
}

// A unit is a piece of 32 values where dim allows (BYTES = 16), else of 16 (BYTES = 8), with its scales.
template <bool NV, int BYTES, typename N>
__global__ void __launch_bounds__(kThreads)
    lookup4_operand_kernel(const Lookup4Args a, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales, const N units) {
  pdl_wait();
  pdl_trigger();
  using V = std::conditional_t<BYTES == 16, uint4, uint2>;
  constexpr int kScales = NV ? BYTES / 8 : 1;  // scales of a unit
  const uint32_t per_row = a.dim / (2 * BYTES);
  const int64_t spr = a.dim / a.block;
  const int64_t groups = scale_groups((int64_t)a.n_cols * a.dim, a.block);
  const int64_t all = spr * a.n_cols;  // scales of a token
  const N u0 = (N)blockIdx.x * (kThreads * kFly) + threadIdx.x;
#pragma unroll
  for (int i = 0; i < kFly; ++i) {
    const N u = u0 + i * kThreads;
    if (u >= units) continue;
    const N e = u / per_row;
    const uint32_t k = (uint32_t)(u - e * per_row);
    const int64_t r = a.idx[id_at<N>(a, e)];
    const bool ok = r >= 0 && r < a.table_rows;
    V w = {};
    if (ok) w = __ldg(reinterpret_cast<const V*>(a.Q + r * (a.dim >> 1)) + k);
    *reinterpret_cast<V*>(codes + (int64_t)u * BYTES) = w;
    const int64_t t = (int64_t)(e / (uint32_t)a.n_cols);
    const int64_t c = (int64_t)e - t * a.n_cols;
#pragma unroll
    for (int j = 0; j < kScales; ++j) {
      const int64_t at = c * spr + (int64_t)k * kScales + j;
      scales[tiled_scale_at(t, at, groups)] = ok ? __ldg(a.S + r * spr + (int64_t)k * kScales + j) : 0;
      if (at == all - 1)  // the token's last scale: the rest of its group of four is 0
        for (int64_t p = at + 1; p & 3; ++p) scales[tiled_scale_at(t, p, groups)] = 0;
    }
  }
}

template <typename F>
cudaError_t with_units(int64_t units, F&& f) {
  const int64_t ctas = (units + kThreads * kFly - 1) / (kThreads * kFly);
  if (ctas > 0x7fffffffll) return cudaErrorInvalidValue;
  // a CTA's last unit must be numbered as well
  if (ctas * (kThreads * kFly) <= 0xffffffffll) return f((uint32_t)units, (unsigned)ctas);
  return f((uint64_t)units, (unsigned)ctas);
}

}  // namespace

cudaError_t launch_lookup4(const Lookup4Args& a, uint16_t* out, cudaStream_t s) {
  return with_units(a.T * a.n_cols * (a.dim / 16), [&](auto units, unsigned ctas) {
    using N = decltype(units);
    auto kern = a.block == 16 ? lookup4_kernel<true, N> : lookup4_kernel<false, N>;
    return launch_pdl(kern, dim3(ctas), dim3(kThreads), 0, s, a, out, units);
  });
}

cudaError_t launch_lookup4_operand(const Lookup4Args& a, uint8_t* codes, uint8_t* scales, cudaStream_t s) {
  const int bytes = a.dim % 32 == 0 ? 16 : 8;
  return with_units(a.T * a.n_cols * (a.dim / (2 * bytes)), [&](auto units, unsigned ctas) {
    using N = decltype(units);
    auto kern = lookup4_operand_kernel<false, 16, N>;
    if (a.block == 16) kern = bytes == 16 ? lookup4_operand_kernel<true, 16, N> : lookup4_operand_kernel<true, 8, N>;
    return launch_pdl(kern, dim3(ctas), dim3(kThreads), 0, s, a, codes, scales, units);
  });
}

}  // namespace engram
