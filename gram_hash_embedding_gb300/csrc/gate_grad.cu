// The gradient of the Engram gate (sm_103a): engram_gate's out_i = h_i + gate_i * value for a token's
// residual copies i, differentiated. With u = the gradient of out_i, w = q_weight_i * k_weight_i,
//   A = mean(h^2) + eps, B = mean(key^2) + eps, r = (A * B * dim)^-1/2, dot = r * sum(h * w * key)
//   m = |dot|, gate = sigmoid(copysign(sqrt(max(m, 1e-6)), dot)), dg = sum(u * value)
//   ddot = dg * gate * (1 - gate) * (m >= 1e-6 ? 1 / (2 sqrt(m)) : 0),  c = ddot * r, e = ddot * dot / dim
//   dh     = u + c * w * key - (e / A) * h
//   dkey   = c * w * h - (e / B) * key
//   dvalue = sum_i gate_i * u_i
//   dq     = k_weight * sum_t c * h * key,  dk = q_weight * the same sum
// in fp32 (sum(h * w * key) in twice that where it is almost 0), everything recomputed from the forward's inputs. A
// masked token's gate is the constant 0: dh = u, dkey = dvalue = 0 and no part in dq and dk, whatever its key and value
// hold.
//
// Design: bound by memory (a token reads (3 hc + 1) dim and writes (2 hc + 1) dim bf16 values, once), but
// every output needs sums over the whole row first, and the weights' gradients are sums over all tokens
// in hc * dim accumulators. So a cluster of CTAs takes whole tokens, in turn with the other clusters: bulk
// copies bring a token's rows into shared memory two tokens ahead, and a thread owns the same 8 columns of
// every copy from the first token to the last, with its part of the weights' sums in registers. Per token
// there is one exchange, of the 4 hc sums: a reduce-scatter in each warp, then every warp sends its sums into
// the shared memory of each CTA of the cluster (asynchronous stores that count their bytes on an mbarrier; a
// cluster barrier would wait for the thread's global stores of the token before), and one warp of each CTA
// forms the token's scalars. That chain is what limits the rate, so it is kept short: approximate reciprocal
// roots, no integer division. The cluster is as small as registers and shared memory allow (2 CTAs at dim
// 5120 and 4 copies: one cluster on each pair of SMs).
// 16,384 tokens, dim 5120, 4 copies, a tenth of the tokens masked (they read only dout): 542 to 547 us, 3.55 GB at
// 6.5 TB/s (0.97 of the copy bandwidth). Tried: copies
// of 16 bytes by each thread into its own slots instead of bulk copies 735 us; a cluster barrier and IEEE
// roots and divisions in every warp 796 us; two groups of threads with two copies each 683 us (with 8 copies two
// groups of four are kept: 4,096 tokens of 8 x 5,120 take 374 us instead of 700, floor 263); clusters
// of 4, two to an SM, 690 us where all of them fit and 1,217 us where 2 of 76 had to wait.
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "engram_internal.cuh"
#include "proj.cuh"
#include "tc_ptx.cuh"
#include "train.cuh"

namespace engram {
namespace {

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
__device__ __forceinline__ void copy_row(uint4* dst, const uint16_t* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   tc::smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
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

// the most threads of a CTA: what the registers allow
constexpr int max_threads(int hc, int cg) { return hc <= 2 ? 640 : (cg == 1 ? 320 : 384); }

// HC copies, S stages. CG groups of threads take HC / CG copies each of the same columns: 8 copies in one thread leave too
// few threads on an SM (the stages' shared memory is per column) and no registers for the weights.
// WHOLE: a CTA has whole rows. It brings each tensor's rows of a token, which lie together, by one copy: three for
// 3 HC + 1 (9,557 tokens of 8 x 464: 80 -> 68 us), and has no cluster's code. One kernel for both kinds took 8,192 tokens
// of 4 x 2,048 136 us instead of 122 and, two CTAs a token, 16,384 of 4 x 5,120 556 instead of 545.
// withhold: the token whose sums the cluster's first CTA does not send (the test hook; -1: none)
template <int HC, int CG, int S, bool WHOLE>
__global__ void __launch_bounds__(max_threads(HC, CG))
    gate_grad_kernel(const GateGradArgs a, const float rd, const float inv_sqrt_dim, const int nv, const int ctas,
                     float* __restrict__ part, unsigned int* __restrict__ status, const int64_t withhold) {
  pdl_wait();
  pdl_trigger();
  constexpr int kArrays = 3 * HC + 1;   // rows of a token: h and dout of the copies, their keys, the value
  const int cs = WHOLE ? 1 : ctas;      // CTAs of the cluster
  constexpr int kU = WHOLE ? HC : 2 * HC, kK = WHOLE ? 2 * HC : HC;  // a stage's rows of dout and of the keys
  constexpr int N = 4 * HC;             // sums of a token
  constexpr int HPT = HC / CG;          // copies of a thread
  constexpr int M = 4 * HPT;            // sums of a warp
  constexpr bool kKeepW = HPT <= 4;     // the weights stay in registers; 8 copies read them again (L1, L2)
  extern __shared__ uint4 smem[];
  __shared__ float4 scal[2][HC];
  __shared__ int again[2];
  __shared__ volatile int dead;  // a wait has run out: nothing more is fetched or sent, the results are not to be used
  __shared__ __align__(8) uint64_t bars[2 + S];  // of red's two halves: the bytes of a token's sums; of the stages
  const int tid = threadIdx.x, nthr = blockDim.x, lane = tid & 31, warp = tid >> 5, nw = nthr >> 5;
  const int cluster = blockIdx.x / cs, nc = gridDim.x / cs;
  const uint32_t rank = blockIdx.x % cs;
  const int per_group = nthr / CG, group = CG == 1 ? 0 : tid / per_group, gt = tid - group * per_group;
  const int g0 = group * HPT, wg = nw / CG;  // its first copy, and the warps of a group
  float4* dvp = reinterpret_cast<float4*>(smem + (size_t)S * kArrays * nv);  // [CG - 1][2][per_group]
  float* red = reinterpret_cast<float*>(dvp + (CG - 1) * 2 * per_group);     // [2][CG][cs][wg][M]
  const int cnt = min(nv, (a.dim >> 3) - (int)rank * nv);  // this CTA's vectors of a row
  const bool on = gt < cnt;
  const int me = min(gt, cnt - 1);  // threads past the row read its last vector and use nothing of it
  const int64_t row0 = 8 * (int64_t)rank * nv;   // its first column
  const int64_t col = row0 + 8 * gt;
  const int64_t gcol = (int64_t)g0 * a.dim + col;  // the thread's place in its first copy
  const uint32_t bar0 = tc::smem_u32(bars);
  auto slot = [&](int st, int j) -> const uint4& { return smem[(st * kArrays + j) * nv + me]; };
  // one thread starts a token's copies
  uint32_t last = ~0u;  // (that thread's) bit st: the parity of the stage's last copies
  auto fetch = [&](int64_t t, int st, bool open) {
    if (t >= a.T || dead) return;
    last ^= 1u << st;
    const uint32_t bytes = 16 * cnt, bar = bar0 + 16 + 8 * st;
    uint4* to = smem + (size_t)st * kArrays * nv;
    tc::mbar_arrive_expect_tx(bar, bytes * (open ? kArrays : HC));
    const uint16_t* u = a.dout + t * HC * a.dim + row0;
    const uint16_t* h = a.x + t * HC * a.dim + row0;
    const uint16_t* k = a.kv + t * (HC + 1) * a.dim + row0;
    if (WHOLE) {
      copy_row(to + kU * nv, u, bytes * HC, bar);
      if (open) {
        copy_row(to, h, bytes * HC, bar);
        copy_row(to + kK * nv, k, bytes * (HC + 1), bar);
      }
      return;
    }
    for (int i = 0; i < HC; ++i) copy_row(to + (kU + i) * nv, u + (int64_t)i * a.dim, bytes, bar);
    if (open) {
      for (int i = 0; i < HC; ++i) {
        copy_row(to + i * nv, h + (int64_t)i * a.dim, bytes, bar);
        copy_row(to + (kK + i) * nv, k + (int64_t)i * a.dim, bytes, bar);
      }
      copy_row(to + 3 * HC * nv, k + (int64_t)HC * a.dim, bytes, bar);
    }
  };
  auto open_at = [&](int64_t t) { return t < a.T && (a.mask == nullptr || a.mask[t] != 0) ? 1u : 0u; };

  auto load_weights = [&](int i) {
    Vec8 w = {};
    if (on) {
      const Vec8 q = widen8(__ldg(reinterpret_cast<const uint4*>(a.qw + gcol + (int64_t)i * a.dim)));
      const Vec8 k = widen8(__ldg(reinterpret_cast<const uint4*>(a.kw + gcol + (int64_t)i * a.dim)));
#pragma unroll
      for (int e = 0; e < 4; ++e) w.p[e] = __fmul2_rn(q.p[e], k.p[e]);
    }
    return w;
  };
  Vec8 w_kept[kKeepW ? HPT : 1];
  if constexpr (kKeepW) {
#pragma unroll
    for (int i = 0; i < HPT; ++i) w_kept[i] = load_weights(i);
  }
  auto weights = [&](int i) {
    if constexpr (kKeepW) return w_kept[i];
    else return load_weights(i);
  };
  Vec8 dw[HPT] = {};
  if (tid == 0) {
    dead = 0;
    for (int i = 0; i < 2 + S; ++i) tc::mbar_init(bar0 + 8 * i, 1);
    tc::fence_barrier_init();
  }
  if (cs > 1) tc::cluster_sync();  // every CTA's barriers exist before another CTA sends to them
  else __syncthreads();
  // bit j of `open`: the mask of the cluster's token j places on
  uint32_t open = 0;
#pragma unroll
  for (int j = 0; j < S; ++j) open |= open_at(cluster + (int64_t)j * nc) << j;
  if (tid == 0)
    for (int j = 0; j < S - 1; ++j) fetch(cluster + (int64_t)j * nc, j, (open >> j) & 1);
  int st = 0, buf = 0;
  uint32_t phase = 0;   // bit b: the parity of bars[b]'s current phase
  auto wait = [&](int b) {
    if (!dead && !tc::mbar_wait(bar0 + 8 * b, (phase >> b) & 1, const_cast<const volatile int*>(&dead))) {
      dead = 1;
      atomicOr(status, ENGRAM_STATUS_TIMEOUT);
    }
    phase ^= 1u << b;
  };
  for (int64_t t = cluster; t < a.T; t += nc) {
    const uint32_t next = open_at(t + (int64_t)S * nc);
    wait(2 + st);
    // the stage of the token before is free once every thread has passed this token's first barrier
    auto refill = [&]() {
      if (tid == 0) fetch(t + (int64_t)(S - 1) * nc, st == 0 ? S - 1 : st - 1, (open >> (S - 1)) & 1);
    };
    uint16_t* dxt = a.dx + t * HC * a.dim + gcol;
    uint16_t* dkt = a.dkv + t * (HC + 1) * a.dim + gcol;
    if (open & 1) {
      float s[M];
      {
        const Vec8 v = widen8(slot(st, 3 * HC));
#pragma unroll
        for (int i = 0; i < HPT; ++i) {
          const Vec8 h = widen8(slot(st, g0 + i)), k = widen8(slot(st, kK + g0 + i)), u = widen8(slot(st, kU + g0 + i));
          const Vec8 w = weights(i);
          float2 q[4] = {};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            q[0] = __ffma2_rn(h.p[e], h.p[e], q[0]);
            q[1] = __ffma2_rn(k.p[e], k.p[e], q[1]);
            q[2] = __ffma2_rn(__fmul2_rn(h.p[e], k.p[e]), w.p[e], q[2]);
            q[3] = __ffma2_rn(u.p[e], v.p[e], q[3]);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) s[4 * i + e] = on ? q[e].x + q[e].y : 0.f;  // past the row: another vector's
        }
      }
      const float mine = warp_reduce_scatter<M>(s, lane);
      float* to = red + (((buf * CG + group) * cs + rank) * wg + (warp - group * wg)) * M + lane / (32 / M);
      if (lane % (32 / M) == 0) {
        if (cs == 1) *to = mine;
        else if (!dead && (t != withhold || rank != 0))
          for (int r = 0; r < cs; ++r) send(to, bar0 + 8 * buf, r, mine);
      }
      if (cs == 1) __syncthreads();
      // red[buf] is written again two exchanges on: whoever does has the sums of the exchange between from every
      // CTA, each sent past the barrier below that follows the reads here
      float f[4];  // (the scalar warp's) the sums of copy lane % HC
      if (warp == nw - 1) {
        if (cs > 1) {
          // once dead, the barrier's phase may be open still: another arrival would be one too many
          if (lane == 0 && !dead) tc::mbar_arrive_expect_tx(bar0 + 8 * buf, (uint32_t)(cs * nw * M * 4));
          wait(buf);
        }
        // lane l: every (32 / N)-th part of sum l % N by the warps of its copy's group, which lie together (a division
        // per part here held the other warps up: the call took 696 us instead of 537)
        const int parts_of_group = cs * wg;
        const float* from = red + (buf * CG + lane % N / M) * parts_of_group * M + lane % M;
        float sum = 0.f;
#pragma unroll 5
        for (int j = lane / N; j < parts_of_group; j += 32 / N) sum += from[j * M];
#pragma unroll
        for (int off = N; off < 32; off *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, off);
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = __shfl_sync(0xffffffffu, sum, 4 * (lane % HC) + e);
        const CopyGrad g = copy_grad(f[0], f[1], f[2], f[3], rd, a.eps, inv_sqrt_dim);
        if (lane < HC) scal[buf][lane] = make_float4(g.gate, g.c, -g.ea, -g.eb);
        // the same sums in the same order in every CTA of the cluster, so the same answer
        const bool any = __any_sync(0xffffffffu, g.m < kSmallDot);
        if (lane == 0) again[buf] = any;
      }
      __syncthreads();
      refill();
      if (again[buf]) {  // sum(h w key) once more, in twice the precision
        buf ^= 1;
        Sum2 d[HPT];
#pragma unroll
        for (int i = 0; i < HPT; ++i) {
          const Vec8 h = widen8(slot(st, g0 + i)), k = widen8(slot(st, kK + g0 + i)), w = weights(i);
          d[i] = Sum2{0.f, 0.f};
          if (on) d[i] = dot_part(h, k, w);
        }
        const Sum2 mine2 = warp_reduce_scatter2<HPT>(d, lane);
        float* to2 = red + (((buf * CG + group) * cs + rank) * wg + (warp - group * wg)) * M + 2 * (lane / (32 / HPT));
        if (lane % (32 / HPT) == 0) {
          if (cs == 1) {
            to2[0] = mine2.hi;
            to2[1] = mine2.lo;
          } else if (!dead) {
            for (int r = 0; r < cs; ++r) {
              send(to2, bar0 + 8 * buf, r, mine2.hi);
              send(to2 + 1, bar0 + 8 * buf, r, mine2.lo);
            }
          }
        }
        if (cs == 1) __syncthreads();
        if (warp == nw - 1) {
          if (cs > 1) {
            if (lane == 0 && !dead) tc::mbar_arrive_expect_tx(bar0 + 8 * buf, (uint32_t)(cs * nw * 2 * HPT * 4));
            wait(buf);
          }
          const int parts_of_group = cs * wg;
          const float* from = red + (buf * CG + lane % HC / HPT) * parts_of_group * M + 2 * (lane % HPT);
          Sum2 sum = {0.f, 0.f};
          for (int j = lane / HC; j < parts_of_group; j += 32 / HC) sum = add2(sum, Sum2{from[j * M], from[j * M + 1]});
#pragma unroll
          for (int off = HC; off < 32; off *= 2)
            sum = add2(sum, Sum2{__shfl_xor_sync(0xffffffffu, sum.hi, off), __shfl_xor_sync(0xffffffffu, sum.lo, off)});
          const CopyGrad g = copy_grad(f[0], f[1], sum.hi + sum.lo, f[3], rd, a.eps, inv_sqrt_dim);
          if (lane < HC) scal[buf][lane] = make_float4(g.gate, g.c, -g.ea, -g.eb);
        }
        __syncthreads();
      }
      Vec8 dv = {};
      if (on) {
#pragma unroll
        for (int i = 0; i < HPT; ++i) {
          const float4 g = scal[buf][g0 + i];  // gate, c, -e / A, -e / B
          const Vec8 h = widen8(slot(st, g0 + i)), k = widen8(slot(st, kK + g0 + i)), u = widen8(slot(st, kU + g0 + i));
          const Vec8 w = weights(i);
          Vec8 dh, dk;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 cw = __fmul2_rn(both(g.y), w.p[e]);
            dh.p[e] = __ffma2_rn(cw, k.p[e], __ffma2_rn(both(g.z), h.p[e], u.p[e]));
            dk.p[e] = __ffma2_rn(cw, h.p[e], __fmul2_rn(both(g.w), k.p[e]));
            dv.p[e] = __ffma2_rn(both(g.x), u.p[e], dv.p[e]);
            dw[i].p[e] = __ffma2_rn(both(g.y), __fmul2_rn(h.p[e], k.p[e]), dw[i].p[e]);
          }
          st8(dxt + i * a.dim, dh);
          st8(dkt + i * a.dim, dk);
        }
        if (group > 0) {
          dvp[(2 * group - 2) * per_group + gt] = make_float4(dv.p[0].x, dv.p[0].y, dv.p[1].x, dv.p[1].y);
          dvp[(2 * group - 1) * per_group + gt] = make_float4(dv.p[2].x, dv.p[2].y, dv.p[3].x, dv.p[3].y);
        }
      }
      if constexpr (CG > 1) {  // the other groups go on; group 0 waits for their parts of the value's gradient, which the
                               // barrier of the next token's sums keeps until it has read them
        if (group > 0) asm volatile("bar.arrive 1, %0;" ::"r"(nthr) : "memory");
        else asm volatile("bar.sync 1, %0;" ::"r"(nthr) : "memory");
      }
      if (group == 0 && on) {
#pragma unroll
        for (int g = 0; g < CG - 1; ++g) {
          const float4 lo = dvp[2 * g * per_group + gt], hi = dvp[(2 * g + 1) * per_group + gt];
          dv.p[0] = __fadd2_rn(dv.p[0], make_float2(lo.x, lo.y));
          dv.p[1] = __fadd2_rn(dv.p[1], make_float2(lo.z, lo.w));
          dv.p[2] = __fadd2_rn(dv.p[2], make_float2(hi.x, hi.y));
          dv.p[3] = __fadd2_rn(dv.p[3], make_float2(hi.z, hi.w));
        }
        st8(a.dkv + (t * (HC + 1) + HC) * a.dim + col, dv);
      }
      buf ^= 1;
    } else {  // the whole cluster skips the sums
      __syncthreads();
      refill();
      if (on) {
        const uint4 z = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int i = 0; i < HPT; ++i) {
          *reinterpret_cast<uint4*>(dxt + i * a.dim) = slot(st, kU + g0 + i);
          *reinterpret_cast<uint4*>(dkt + i * a.dim) = z;
        }
        if (group == 0) *reinterpret_cast<uint4*>(a.dkv + (t * (HC + 1) + HC) * a.dim + col) = z;
      }
    }
    open = open >> 1 | next << (S - 1);
    st = st == S - 1 ? 0 : st + 1;
  }
  if (on) {
#pragma unroll
    for (int i = 0; i < HPT; ++i) {
      float* to = part + (int64_t)cluster * HC * a.dim + gcol + (int64_t)i * a.dim;
      const float2* d = dw[i].p;
      *reinterpret_cast<float4*>(to) = make_float4(d[0].x, d[0].y, d[1].x, d[1].y);
      *reinterpret_cast<float4*>(to + 4) = make_float4(d[2].x, d[2].y, d[3].x, d[3].y);
    }
  }
  if (dead) {  // copies may still be on their way into this CTA's memory, and sums into another's
    if (tid == 0)
      for (int st = 0; st < S; ++st)
        if (cluster + (int64_t)st * nc < a.T) tc::mbar_wait(bar0 + 16 + 8 * st, (last >> st) & 1, nullptr);
    const uint64_t t0 = tc::global_timer_ns();
    while (tc::global_timer_ns() - t0 < kSettleNs) {}
  }
  if (cs > 1) tc::cluster_sync();  // no CTA leaves while another may send to it
}

// The weights' gradients from the clusters' parts: LANES lanes take 4 columns each, the CTA's THREADS / LANES groups of
// them take every so many-th part, and the groups' sums are added in order. Few parts (the large widths): 128
// columns a CTA, 8 groups. Many (narrow rows, whose CTAs are small and many): 32 columns, 128 groups; with 8
// groups 3,040 parts took 33 us.
template <int LANES, int THREADS>
__global__ void __launch_bounds__(THREADS) gate_weight_finish_kernel(const GateGradArgs a,
                                                                     const float* __restrict__ part, int parts) {
  pdl_wait();
  pdl_trigger();
  constexpr int kGroups = THREADS / LANES;
  __shared__ float4 sum_s[kGroups][LANES];
  const int n = a.hc * a.dim, lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
  const int j = (blockIdx.x * LANES + lane) * 4;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](const float4 v) {
    s.x += v.x;
    s.y += v.y;
    s.z += v.z;
    s.w += v.w;
  };
  if (j < n) {
#pragma unroll 8
    for (int z = group; z < parts; z += kGroups) add(*reinterpret_cast<const float4*>(part + (int64_t)z * n + j));
  }
  sum_s[group][lane] = s;
  __syncthreads();
  // 8 groups at a time, twice where there are many
#pragma unroll
  for (int left = kGroups; left > 1;) {
    const int next = left > 8 ? left / 8 : 1, each = left / next;
    if (group < next) {
      s = sum_s[group * each][lane];
      for (int g = 1; g < each; ++g) add(sum_s[group * each + g][lane]);
    }
    __syncthreads();
    if (group < next) sum_s[group][lane] = s;
    __syncthreads();
    left = next;
  }
  if (group != 0 || j >= n) return;
  const uint2 q = *reinterpret_cast<const uint2*>(a.qw + j), k = *reinterpret_cast<const uint2*>(a.kw + j);
  auto lo = [](uint32_t v) { return __uint_as_float(v << 16); };
  auto hi = [](uint32_t v) { return __uint_as_float(v & 0xffff0000u); };
  *reinterpret_cast<float4*>(a.dq + j) = make_float4(s.x * lo(k.x), s.y * hi(k.x), s.z * lo(k.y), s.w * hi(k.y));
  *reinterpret_cast<float4*>(a.dk + j) = make_float4(s.x * lo(q.x), s.y * hi(q.x), s.z * lo(q.y), s.w * hi(q.y));
}

inline uint64_t round256(uint64_t b) { return (b + 255) & ~(uint64_t)255; }

// the threads that an SM's registers hold
constexpr int resident_threads(int hc) { return hc == 1 ? 896 : hc == 2 ? 736 : 384; }

struct Shape {
  int cs, cg, nv, threads, stages;  // CTAs per cluster, groups of copies, vectors and threads per CTA
  int64_t smem, clusters;
};

// The smallest cluster (with one exception below) whose CTAs hold their columns in registers and three stages of
// shared memory (8 copies: in two groups of threads; of more than 12,000 columns or so: in one, and two stages); more
// CTAs a token when there are too few tokens for every SM. Few clusters rather than many when every cluster would see
// few tokens: each leaves hc * dim partial sums behind.
Shape shape_of(int64_t T, int32_t hc, int32_t dim) {
  Shape s;
  const int nvec = dim / 8;
  auto set = [&](int cs, int cg, int stages) {
    s.cs = cs;
    s.cg = cg;
    s.stages = stages;
    s.nv = (nvec + cs - 1) / cs;
    const int per_group = (s.nv + 31) / 32 * 32;
    s.threads = per_group * cg;
    s.smem = (int64_t)stages * (3 * hc + 1) * s.nv * 16 + (cg - 1) * per_group * 32ll +
             2ll * cs * (s.threads / 32) * 4 * (hc / cg) * 4;
    return s.threads <= max_threads(hc, cg) && s.smem <= kMaxSmem;
  };
  const int cg = hc == 8 ? 2 : 1;
  int cs = 1;
  while (cs < 8 && !set(cs, cg, 3)) cs *= 2;
  while (cs < 8 && T * cs * 2 <= kSms && nvec / (cs * 2) >= 64) cs *= 2;
  // CTAs resident on an SM, by shared memory and registers
  auto resident = [&]() {
    return std::max<int64_t>(1, std::min<int64_t>((kMaxSmem + 1024) / (s.smem + 1024), resident_threads(hc) / s.threads));
  };
  if (!set(cs, cg, 3)) {
    set(cs, 1, 2);
  } else if (cs < 8) {
    // one more halving where it brings half as many columns again onto an SM: more tokens' chains at a time (8,192 of
    // 4 x 3,616: 251 -> 215 us; 20,000 of 1 x 3,800: 248 -> 194). Where it brings as many as before it costs up to a
    // quarter (8,192 of 8 x 1,024: 139 -> 165).
    const int64_t columns = s.nv * resident();
    set(cs * 2, cg, 3);
    if (s.nv * resident() * 5 < columns * 7) set(cs, cg, 3);
  }
  s.clusters = std::min({T, std::max<int64_t>(1, kSms * resident() / s.cs), std::max<int64_t>(kSms / s.cs, (T + 3) / 4)});
  return s;
}

template <int HC, int CG, int S, bool WHOLE>
cudaError_t launch_shape(const GateGradArgs& a, const Shape& sh, float* part, int* parts, int64_t withhold,
                         cudaStream_t s) {
  auto kern = gate_grad_kernel<HC, CG, S, WHOLE>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sh.smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = ENGRAM_PDL;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = sh.cs;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.blockDim = dim3(sh.threads);
  cfg.dynamicSmemBytes = sh.smem;
  cfg.stream = s;
  cfg.attrs = attr;
  // CTAs that hold whole rows launch without the attribute: as clusters of one, 8 at most were resident on an SM
  cfg.numAttrs = sh.cs > 1 ? 2 : 1;
  // no more clusters than can be resident: one that had to wait would run its share of the tokens alone
  cfg.gridDim = dim3((unsigned)(sh.clusters * sh.cs));
  int64_t clusters = sh.clusters;
  if (sh.cs > 1 && clusters > 1) {
    int resident = 0;
    e = cudaOccupancyMaxActiveClusters(&resident, kern, &cfg);
    if (e != cudaSuccess) return e;
    clusters = std::max<int64_t>(1, std::min<int64_t>(clusters, resident));
  } else if (clusters > kSms) {
    int resident = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&resident, kern, sh.threads, sh.smem);
    if (e != cudaSuccess) return e;
    clusters = std::min<int64_t>(clusters, std::max<int64_t>(1, resident) * kSms);
  }
  unsigned int* status = nullptr;
  e = device_status_word(&status);
  if (e != cudaSuccess) return e;
  *parts = (int)clusters;
  cfg.gridDim = dim3((unsigned)(clusters * sh.cs));
  return cudaLaunchKernelEx(&cfg, kern, a, 1.0f / (float)a.dim, (float)(1.0 / sqrt((double)a.dim)), sh.nv, sh.cs, part,
                            status, withhold);
}

}  // namespace

uint64_t gate_grad_workspace(int64_t T, int32_t hc, int32_t dim) {
  return round256((uint64_t)shape_of(T, hc, dim).clusters * hc * dim * 4);
}

cudaError_t launch_gate_grad(const GateGradArgs& a, void* workspace, cudaStream_t s, int64_t withhold) {
  float* part = static_cast<float*>(workspace);
  int parts = 0;
  if (a.T > 0) {
    const Shape sh = shape_of(a.T, a.hc, a.dim);
    cudaError_t e = cudaErrorInvalidValue;
    auto launch = [&](auto hc, auto cg, auto stages) {
      constexpr int HC = decltype(hc)::value, CG = decltype(cg)::value, S = decltype(stages)::value;
      if constexpr (S == 3)  // with two stages rows are too wide for one CTA
        if (sh.cs == 1) return launch_shape<HC, CG, S, true>(a, sh, part, &parts, withhold, s);
      return launch_shape<HC, CG, S, false>(a, sh, part, &parts, withhold, s);
    };
    using std::integral_constant;
    const integral_constant<int, 1> one;
    const integral_constant<int, 2> two;
    const integral_constant<int, 3> three;
    switch (a.hc) {
      case 1: e = launch(one, one, three); break;
      case 2: e = launch(two, one, three); break;
      case 4: e = launch(integral_constant<int, 4>{}, one, three); break;
      case 8:
        e = sh.cg == 2 ? launch(integral_constant<int, 8>{}, two, three) : launch(integral_constant<int, 8>{}, one, two);
        break;
    }
    if (e != cudaSuccess) return e;
  }
  const int n = a.hc * a.dim;
  if (parts > 256)
    return launch_pdl(gate_weight_finish_kernel<8, 1024>, dim3((n + 31) / 32), dim3(1024), 0, s, a, (const float*)part,
                      parts);
  return launch_pdl(gate_weight_finish_kernel<32, 256>, dim3((n + 127) / 128), dim3(256), 0, s, a, (const float*)part,
                    parts);
}

}  // namespace engram
