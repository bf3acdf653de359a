// The gradient of the Engram gate (sm_103a): engram_gate's out_i = h_i + gate_i * value for a token's
// residual copies i, differentiated. With u = the gradient of out_i, w = q_weight_i * k_weight_i,
//   A = mean(h^2) + eps, B = mean(key^2) + eps, r = (A * B * dim)^-1/2, dot = r * sum(h * w * key)
//   m = |dot|, gate = sigmoid(copysign(sqrt(max(m, 1e-6)), dot)), dg = sum(u * value)
//   ddot = dg * gate * (1 - gate) * (m >= 1e-6 ? 1 / (2 sqrt(m)) : 0),  c = ddot * r, e = ddot * dot / dim
//   dh     = u + c * w * key - (e / A) * h
//   dkey   = c * w * h - (e / B) * key
//   dvalue = sum_i gate_i * u_i
//   dq     = k_weight * sum_t c * h * key,  dk = q_weight * the same sum
// in fp32, everything recomputed from the forward's inputs. A masked token's gate is the constant 0:
// dh = u, dkey = dvalue = 0 and no part in dq and dk, whatever its key and value hold.
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "engram_internal.cuh"
#include "train.cuh"

namespace engram {
namespace {

constexpr int kThreads = 256;
constexpr int kSplits = 64;  // parts of the token axis in the weights' sums

struct CopyGrad {
  float gate, c, ea, eb;  // gate, c, e / A, e / B
};

// The scalars of one residual copy from its four sums
__device__ __forceinline__ CopyGrad copy_grad(float sh, float sk, float sd, float su, float rd, float eps,
                                              float inv_sqrt_dim) {
  const float A = sh * rd + eps, B = sk * rd + eps;
  const float r = (1.0f / sqrtf(A)) * (1.0f / sqrtf(B)) * inv_sqrt_dim;
  const float dot = sd * r;
  const float m = fabsf(dot), root = sqrtf(fmaxf(m, 1e-6f));
  CopyGrad g;
  // from exp(-|z|), so that neither the gate nor 1 - gate cancels: gate (1 - gate) = x / (1 + x)^2
  const float x = expf(-root), y = 1.0f / (1.0f + x);
  g.gate = dot < 0.f ? x * y : y;
  const float ddot = m >= 1e-6f ? su * (x * y * y) * (0.5f / root) : 0.f;
  const float e = ddot * dot * rd;
  g.c = ddot * r;
  g.ea = e / A;
  g.eb = e / B;
  return g;
}

__device__ __forceinline__ void bf16x8(const uint16_t* p, float* f) {
  Raw<ENGRAM_TYPE_BF16, 8> r;
  r.load(reinterpret_cast<const __nv_bfloat16*>(p));
  r.widen(f);
}

__device__ __forceinline__ void st8(uint16_t* p, const float* f) {
  store_vals<ENGRAM_TYPE_BF16, 8>(reinterpret_cast<__nv_bfloat16*>(p), f);
}

// one CTA per token; cs[t][i] = c for the weights' sums
template <int HC>
__global__ void __launch_bounds__(kThreads) gate_grad_kernel(const GateGradArgs a, const float rd,
                                                             const float inv_sqrt_dim, float* __restrict__ cs) {
  pdl_wait();
  pdl_trigger();
  __shared__ float red[4 * HC][kThreads / 32];
  __shared__ CopyGrad gs[HC];
  const int64_t t = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nvec = a.dim >> 3;
  const uint16_t* xt = a.x + t * HC * a.dim;
  const uint16_t* ut = a.dout + t * HC * a.dim;
  const uint16_t* kt = a.kv + t * (HC + 1) * a.dim;
  const uint16_t* vt = kt + (int64_t)HC * a.dim;
  uint16_t* dxt = a.dx + t * HC * a.dim;
  uint16_t* dkt = a.dkv + t * (HC + 1) * a.dim;
  const bool open = a.mask == nullptr || a.mask[t] != 0;
  if (!open) {
    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
    for (int v = tid; v < nvec * HC; v += kThreads)
      reinterpret_cast<uint4*>(dxt)[v] = reinterpret_cast<const uint4*>(ut)[v];
    for (int v = tid; v < nvec * (HC + 1); v += kThreads) reinterpret_cast<uint4*>(dkt)[v] = z;
    if (tid < HC) cs[t * HC + tid] = 0.f;
    return;
  }
  float s[HC][4] = {};
  for (int v = tid; v < nvec; v += kThreads) {
    float val[8];
    bf16x8(vt + 8 * v, val);
#pragma unroll
    for (int i = 0; i < HC; ++i) {
      const int64_t o = (int64_t)i * a.dim + 8 * v;
      float h[8], k[8], u[8], q[8], w[8];
      bf16x8(xt + o, h);
      bf16x8(kt + o, k);
      bf16x8(ut + o, u);
      bf16x8(a.qw + o, q);
      bf16x8(a.kw + o, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        s[i][0] = fmaf(h[e], h[e], s[i][0]);
        s[i][1] = fmaf(k[e], k[e], s[i][1]);
        s[i][2] = fmaf(h[e] * (q[e] * w[e]), k[e], s[i][2]);
        s[i][3] = fmaf(u[e], val[e], s[i][3]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < HC; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s[i][q] += __shfl_xor_sync(0xffffffffu, s[i][q], o);
      if (lane == 0) red[4 * i + q][warp] = s[i][q];
    }
  __syncthreads();
  if (tid < HC) {
    float f[4];
    for (int q = 0; q < 4; ++q) {
      f[q] = 0.f;
      for (int w = 0; w < kThreads / 32; ++w) f[q] += red[4 * tid + q][w];
    }
    gs[tid] = copy_grad(f[0], f[1], f[2], f[3], rd, a.eps, inv_sqrt_dim);
    cs[t * HC + tid] = gs[tid].c;
  }
  __syncthreads();
  for (int v = tid; v < nvec; v += kThreads) {
    float dv[8] = {};
#pragma unroll
    for (int i = 0; i < HC; ++i) {
      const int64_t o = (int64_t)i * a.dim + 8 * v;
      const CopyGrad g = gs[i];
      float h[8], k[8], u[8], q[8], w[8], dh[8], dk[8];
      bf16x8(xt + o, h);
      bf16x8(kt + o, k);
      bf16x8(ut + o, u);
      bf16x8(a.qw + o, q);
      bf16x8(a.kw + o, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float cw = g.c * (q[e] * w[e]);
        dh[e] = u[e] + (cw * k[e] - g.ea * h[e]);
        dk[e] = cw * h[e] - g.eb * k[e];
        dv[e] = fmaf(g.gate, u[e], dv[e]);
      }
      st8(dxt + o, dh);
      st8(dkt + o, dk);
    }
    st8(dkt + (int64_t)HC * a.dim + 8 * v, dv);
  }
}

// part[split][i][col] = sum over the split's tokens of c * h * key
__global__ void __launch_bounds__(kThreads) gate_weight_sums_kernel(const GateGradArgs a, const float* __restrict__ cs,
                                                                    float* __restrict__ part) {
  pdl_wait();
  pdl_trigger();
  const int col = blockIdx.x * kThreads + threadIdx.x, i = blockIdx.y;
  if (col >= a.dim) return;
  const int64_t t0 = a.T * blockIdx.z / gridDim.z, t1 = a.T * (blockIdx.z + 1) / gridDim.z;
  float acc = 0.f;
  for (int64_t t = t0; t < t1; ++t) {
    if (a.mask != nullptr && a.mask[t] == 0) continue;
    const float h = __uint_as_float((uint32_t)a.x[(t * a.hc + i) * a.dim + col] << 16);
    const float k = __uint_as_float((uint32_t)a.kv[(t * (a.hc + 1) + i) * a.dim + col] << 16);
    acc = fmaf(cs[t * a.hc + i] * h, k, acc);
  }
  part[((int64_t)blockIdx.z * a.hc + i) * a.dim + col] = acc;
}

__global__ void __launch_bounds__(kThreads) gate_weight_finish_kernel(const GateGradArgs a, const float* __restrict__ part,
                                                                      int splits) {
  pdl_wait();
  pdl_trigger();
  const int n = a.hc * a.dim, j = blockIdx.x * kThreads + threadIdx.x;
  if (j >= n) return;
  float acc = 0.f;
  for (int z = 0; z < splits; ++z) acc += part[(int64_t)z * n + j];
  a.dq[j] = acc * __uint_as_float((uint32_t)a.kw[j] << 16);
  a.dk[j] = acc * __uint_as_float((uint32_t)a.qw[j] << 16);
}

inline uint64_t round256(uint64_t b) { return (b + 255) & ~(uint64_t)255; }

}  // namespace

uint64_t gate_grad_workspace(int64_t T, int32_t hc, int32_t dim) {
  return round256((uint64_t)T * hc * 4) + round256((uint64_t)kSplits * hc * dim * 4);
}

cudaError_t launch_gate_grad(const GateGradArgs& a, void* workspace, cudaStream_t s) {
  float* cs = static_cast<float*>(workspace);
  float* part = cs + round256((uint64_t)a.T * a.hc * 4) / 4;
  const float rd = 1.0f / (float)a.dim, isd = (float)(1.0 / sqrt((double)a.dim));
  const int splits = (int)std::min<int64_t>(a.T, kSplits);
  cudaError_t e = cudaSuccess;
  if (a.T > 0) {
    auto go = [&](auto hc) {
      return launch_pdl(gate_grad_kernel<hc()>, dim3((unsigned)a.T), dim3(kThreads), 0, s, a, rd, isd, cs);
    };
    switch (a.hc) {
      case 1: e = go(std::integral_constant<int, 1>{}); break;
      case 2: e = go(std::integral_constant<int, 2>{}); break;
      case 4: e = go(std::integral_constant<int, 4>{}); break;
      case 8: e = go(std::integral_constant<int, 8>{}); break;
      default: return cudaErrorInvalidValue;
    }
    if (e != cudaSuccess) return e;
    e = launch_pdl(gate_weight_sums_kernel, dim3((a.dim + kThreads - 1) / kThreads, a.hc, splits), dim3(kThreads), 0,
                   s, a, (const float*)cs, part);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(gate_weight_finish_kernel, dim3((a.hc * a.dim + kThreads - 1) / kThreads), dim3(kThreads), 0, s, a,
                    (const float*)part, splits);
}

}  // namespace engram
