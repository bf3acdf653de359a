// What the kernels of the gate's gradient share (gate_grad.cu on bf16 inputs, gate_grad8.cu on 8-bit checkpoints): a
// copy's scalars from its sums, vectors of 8 columns, sums over a warp, the exchange within a cluster. The formulas are in
// gate_grad.cu.
#pragma once

#include <cstdint>

#include "engram_internal.cuh"
#include "tc_ptx.cuh"
#include "train.cuh"

namespace engram {
namespace gate {

constexpr int kSms = 152;
constexpr int kMaxSmem = 226 << 10;
constexpr uint64_t kSettleNs = 100000;  // after a wait has run out: far longer than a store to another SM takes

struct CopyGrad {
  float gate, c, ea, eb, m;  // gate, c, e / A, e / B, |dot|
};

// The scalars of one residual copy from its four sums
__device__ __forceinline__ CopyGrad copy_grad(float sh, float sk, float sd, float su, float rd, float eps,
                                              float inv_sqrt_dim) {
  const float ra = rsqrtf(sh * rd + eps), rb = rsqrtf(sk * rd + eps);
  const float r = ra * rb * inv_sqrt_dim;
  const float dot = sd * r;
  // a NaN dot stays one and makes the gate and all of the copy's gradients NaN (fmaxf would take the bound for it)
  const float m = fabsf(dot), bounded = m < 1e-6f ? 1e-6f : m, ri = rsqrtf(bounded);  // 1 / |z|
  CopyGrad g;
  g.m = m;
  // from exp(-|z|), so that neither the gate nor 1 - gate cancels: gate (1 - gate) = x / (1 + x)^2
  const float x = expf(-bounded * ri), y = __frcp_rn(1.0f + x);
  g.gate = dot < 0.f ? x * y : y;
  const float ddot = m < 1e-6f ? 0.f : su * (x * y * y) * (0.5f * ri);
  const float e = ddot * dot * rd;
  g.c = ddot * r;
  g.ea = e * ra * ra;
  g.eb = e * rb * rb;
  return g;
}

// 8 bf16 values as 4 pairs: the arithmetic runs two values an instruction (the packed fp32 forms), which
// round like the single ones
struct Vec8 {
  float2 p[4];
};

__device__ __forceinline__ Vec8 widen8(const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  Vec8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.p[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
  return r;
}

__device__ __forceinline__ void st8(uint16_t* p, const Vec8& v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pack2<ENGRAM_TYPE_BF16>(v.p[i].x, v.p[i].y);
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 minus(float2 v) { return make_float2(-v.x, -v.y); }

// one row's part of a token into shared memory, counted in bytes on `bar`
__device__ __forceinline__ void copy_row(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void copy_row(void* dst, const void* src, uint32_t bytes, uint32_t bar) {
  copy_row(tc::smem_u32(dst), src, bytes, bar);
}

// Sums of N values over the warp, N a power of two <= 32: lane l ends with the total of value
// l / (32 / N), in N - 1 + log2(32 / N) shuffles instead of 5 N.
template <int N>
__device__ __forceinline__ float warp_reduce_scatter(float (&s)[N], int lane) {
#pragma unroll
  for (int w = N / 2, off = 16; w >= 1; w /= 2, off /= 2) {
    const bool up = lane & off;
#pragma unroll
    for (int j = 0; j < w; ++j) {
      const float give = up ? s[j] : s[j + w];
      const float keep = up ? s[j + w] : s[j];
      s[j] = keep + __shfl_xor_sync(0xffffffffu, give, off);
    }
  }
  float r = s[0];
#pragma unroll
  for (int off = 16 / N; off >= 1; off /= 2) r += __shfl_xor_sync(0xffffffffu, r, off);
  return r;
}

// A sum and what its roundings lost, so far: twice the precision of fp32. Where sum(h w key) cancels to almost
// nothing, the gate's slope (1 / sqrt of it) magnifies its error, and a few such tokens set the error of the weights'
// gradients: up to 1e-3 of them at widths of some hundred columns. So a token with a copy of |dot| < kSmallDot has
// that sum formed once more in this way (for every token it cost 687 instead of 538 us at 16,384 tokens of
// 4 x 5,120).
constexpr float kSmallDot = 0.03125f;
struct Sum2 {
  float hi, lo;
};

__device__ __forceinline__ Sum2 add2(const Sum2& a, const Sum2& b) {
  Sum2 r;
  r.hi = __fadd_rn(a.hi, b.hi);
  const float z = __fsub_rn(r.hi, a.hi);
  r.lo = __fadd_rn(__fadd_rn(a.lo, b.lo), __fadd_rn(__fsub_rn(a.hi, __fsub_rn(r.hi, z)), __fsub_rn(b.hi, z)));
  return r;
}

// one thread's part of sum(h w key): h * key and q_weight * k_weight are exact (bf16 factors), their product comes in
// two parts, and both are summed
__device__ __forceinline__ Sum2 dot_part(const Vec8& h, const Vec8& k, const Vec8& w) {
  float2 hi = {}, lo = {};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 hk = __fmul2_rn(h.p[e], k.p[e]), term = __fmul2_rn(hk, w.p[e]);
    const float2 sum = __fadd2_rn(hi, term), z = __fadd2_rn(sum, minus(hi));
    lo = __fadd2_rn(lo, __ffma2_rn(hk, w.p[e], minus(term)));
    lo = __fadd2_rn(lo, __fadd2_rn(__fadd2_rn(hi, minus(__fadd2_rn(sum, minus(z)))), __fadd2_rn(term, minus(z))));
    hi = sum;
  }
  return add2(Sum2{hi.x, lo.x}, Sum2{hi.y, lo.y});
}

// warp_reduce_scatter for N sums of that kind
template <int N>
__device__ __forceinline__ Sum2 warp_reduce_scatter2(Sum2 (&s)[N], int lane) {
#pragma unroll
  for (int w = N / 2, off = 16; w >= 1; w /= 2, off /= 2) {
    const bool up = lane & off;
#pragma unroll
    for (int j = 0; j < w; ++j) {
      const Sum2 give = up ? s[j] : s[j + w];
      const Sum2 keep = up ? s[j + w] : s[j];
      s[j] = add2(keep, Sum2{__shfl_xor_sync(0xffffffffu, give.hi, off), __shfl_xor_sync(0xffffffffu, give.lo, off)});
    }
  }
  Sum2 r = s[0];
#pragma unroll
  for (int off = 16 / N; off >= 1; off /= 2)
    r = add2(r, Sum2{__shfl_xor_sync(0xffffffffu, r.hi, off), __shfl_xor_sync(0xffffffffu, r.lo, off)});
  return r;
}

// Write v to the same shared variable of CTA `rank` and count its 4 bytes on that CTA's mbarrier. Unlike a
// cluster barrier's release this waits for none of the thread's global stores.
__device__ __forceinline__ void send(float* p, uint32_t bar, uint32_t rank, float v) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.f32 [%0], %1, [%2];" ::"r"(
                   tc::map_to_rank(tc::smem_u32(p), rank)),
               "f"(v), "r"(tc::map_to_rank(bar, rank))
               : "memory");
}

inline uint64_t round256(uint64_t b) { return (b + 255) & ~(uint64_t)255; }

}  // namespace gate

// the weights' gradients from `parts` rows of hc * dim partial sums (gate_grad.cu)
cudaError_t launch_gate_weight_finish(const GateGradArgs& a, const float* part, int parts, cudaStream_t s);

}  // namespace engram
