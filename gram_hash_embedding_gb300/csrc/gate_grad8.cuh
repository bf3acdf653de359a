// What the kernels of the gate's gradient from 8-bit checkpoints share: gate_grad8.cu (a cluster holds a row) and
// gate_grad8_rows.cu (lanes of a warp do).
#pragma once

#include <cstdint>

#include "dequant.cuh"
#include "gate_grad.cuh"
#include "train.cuh"

namespace engram {
namespace gate {

// 8 E4M3 codes, without their block's scale
__device__ __forceinline__ Vec8 widen_codes(const uint2& v) {
  const uint32_t w[4] = {v.x, v.x >> 16, v.y, v.y >> 16};
  Vec8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) f16x2_to_f32(e4m3x2_to_f16x2(w[i] & 0xffffu), r.p[i].x, r.p[i].y);
  return r;
}

// A checkpoint's scale 2^(b - 127). A NaN (255) comes out as infinity: the codes of such a block are 0, and 0 times it is a
// NaN again.
__device__ __forceinline__ float pow2(uint32_t b) { return __uint_as_float(max(b << 23, 0x00400000u)); }

}  // namespace gate

// narrow rows: CTAs that leave a part of the weights' gradients each (0: the rows are too wide), and their launch
int gate_grad8_rows_parts(int64_t T, int32_t hc, int32_t dim);
cudaError_t launch_gate_grad8_rows(const GateGrad8Args& a, float* part, int parts, cudaStream_t s);

}  // namespace engram
