// Trainable embedding rows (sm_103a): the lookup with a scale, and its gradient by sorted row ids.
//
//   out[t][c]  = round(scale * W[idx[t][c]])                    (+0 where idx is outside [0, rows))
//   G[r]       = scale * sum over (t, c) with idx[t][c] == r of dout[t][c]
//
// The gradient's sums run in fp32 in an order that depends on the ids alone (ascending position), so
// the same call gives the same bits. The ids are sorted (a stable radix sort of (row id, position)
// pairs), equal ids become one segment, and every segment is summed and written once.
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "engram_internal.cuh"
#include "train.cuh"

namespace engram {
namespace {

constexpr int kThreads = 256;

// ------------------------------------------------------------------------------------------- lookup
template <int WT, int OT, int V>
__global__ void __launch_bounds__(kThreads)
    embed_kernel(const EmbedArgs a, const typename Elem<WT>::type* __restrict__ W, const int64_t row_stride,
                 typename Elem<OT>::type* __restrict__ out) {
  pdl_wait();
  pdl_trigger();
  const int per_row = a.dim / V;
  const int64_t units = a.T * a.n_cols * per_row;
  for (int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x; u < units; u += (int64_t)gridDim.x * kThreads) {
    const int64_t e = u / per_row;
    const int k = (int)(u - e * per_row) * V;
    const int64_t t = e / a.n_cols;
    const int64_t r = a.idx[t * a.idx_stride + (e - t * a.n_cols)];
    Raw<WT, V> raw;
    raw.zero();
    if (r >= 0 && r < a.rows) raw.load(W + r * row_stride + k);
    float f[V];
    raw.widen(f);
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = (r >= 0 && r < a.rows) ? f[i] * a.scale : 0.f;
    store_vals<OT, V>(out + e * a.dim + k, f);
  }
}

// -------------------------------------------------------------------------------------- radix sort
// Least significant digit first, up to kMaxBits bits a pass; per pass a count of every digit per
// tile, a scan over the tiles of each digit, and a stable scatter. Keys are row ids as 32-bit values,
// with `rows` itself standing for every id outside the table, so those sort to the end.
constexpr int kMaxBits = 8;
constexpr int kMaxBins = 1 << kMaxBits;
constexpr int kPerThread = 16;
constexpr int kTile = kThreads * kPerThread;  // pairs per tile (one CTA)

struct SortPass {
  const uint32_t* key_in;  // null in the first pass: keys come from the ids, positions are implicit
  const uint32_t* pos_in;
  uint32_t* key_out;
  uint32_t* pos_out;
  uint32_t* counts;  // [bins][tiles]
  uint32_t* totals;  // [bins]
  int64_t n;
  int32_t tiles, shift, bins;
};

__device__ __forceinline__ uint32_t key_at(const EmbedArgs& e, const SortPass& p, int64_t i) {
  if (p.key_in != nullptr) return p.key_in[i];
  const int64_t t = i / e.n_cols;
  const int64_t r = e.idx[t * e.idx_stride + (i - t * e.n_cols)];
  return r >= 0 && r < e.rows ? (uint32_t)r : (uint32_t)e.rows;
}

__global__ void __launch_bounds__(kThreads) sort_count_kernel(const EmbedArgs e, const SortPass p) {
  pdl_wait();
  pdl_trigger();
  __shared__ uint32_t hist[kMaxBins];
  for (int b = threadIdx.x; b < p.bins; b += kThreads) hist[b] = 0;
  __syncthreads();
  const int64_t base = (int64_t)blockIdx.x * kTile;
#pragma unroll 4
  for (int j = 0; j < kPerThread; ++j) {
    const int64_t i = base + j * kThreads + threadIdx.x;
    if (i < p.n) atomicAdd(&hist[(key_at(e, p, i) >> p.shift) & (p.bins - 1)], 1u);
  }
  __syncthreads();
  for (int b = threadIdx.x; b < p.bins; b += kThreads) p.counts[(int64_t)b * p.tiles + blockIdx.x] = hist[b];
}

// one warp per digit: counts[b][tile] becomes the pairs of digit b in the tiles before
__global__ void __launch_bounds__(kThreads) sort_scan_kernel(const SortPass p) {
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (b >= p.bins) return;
  uint32_t* c = p.counts + (int64_t)b * p.tiles;
  uint32_t run = 0;
  for (int t0 = 0; t0 < p.tiles; t0 += 32) {
    const int t = t0 + lane;
    const uint32_t v = t < p.tiles ? c[t] : 0u;
    uint32_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (t < p.tiles) c[t] = run + x - v;
    run += __shfl_sync(0xffffffffu, x, 31);
  }
  if (lane == 0) p.totals[b] = run;
}

// exclusive scan over the block of one value per thread
__device__ __forceinline__ uint32_t block_exclusive(uint32_t v, uint32_t* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  uint32_t before = 0;
  for (int w = 0; w < warp; ++w) before += warp_sums[w];
  __syncthreads();
  return before + x - v;
}

__global__ void __launch_bounds__(kThreads) sort_scatter_kernel(const EmbedArgs e, const SortPass p) {
  pdl_wait();
  pdl_trigger();
  constexpr int kWarps = kThreads / 32;
  __shared__ uint32_t wh[kWarps][kMaxBins];  // pairs of each digit in each warp, then where they start
  __shared__ uint32_t start[kMaxBins];       // a digit's first place in the sorted tile
  __shared__ uint32_t gbase[kMaxBins];       // its first place in the output, less start
  __shared__ uint32_t warp_sums[kWarps];
  __shared__ uint32_t sk[kTile], sp[kTile];  // the tile in digit order
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int b = tid; b < kWarps * kMaxBins; b += kThreads) (&wh[0][0])[b] = 0;
  __syncthreads();
  // a warp takes 32 * kPerThread consecutive pairs, 32 at a time, so (step, lane) is position order
  const int64_t base = (int64_t)blockIdx.x * kTile + (int64_t)warp * 32 * kPerThread;
  uint32_t key[kPerThread], pos[kPerThread], rank[kPerThread];
#pragma unroll
  for (int j = 0; j < kPerThread; ++j) {
    const int64_t i = base + j * 32 + lane;
    if (i < p.n) {
      key[j] = key_at(e, p, i);
      pos[j] = p.key_in != nullptr ? p.pos_in[i] : (uint32_t)i;
    }
  }
#pragma unroll
  for (int j = 0; j < kPerThread; ++j) {
    const int64_t i = base + j * 32 + lane;
    const bool in = i < p.n;
    const uint32_t d = in ? (key[j] >> p.shift) & (p.bins - 1) : 0xffffffffu;
    const unsigned same = __match_any_sync(0xffffffffu, d);
    const int before = __popc(same & ((1u << lane) - 1u));
    uint32_t have = 0;
    if (in) have = wh[warp][d];
    __syncwarp();
    if (in && before == 0) wh[warp][d] = have + __popc(same);
    __syncwarp();
    rank[j] = have + before;
  }
  __syncthreads();
  // per digit: the warps' starts, the tile's total
  uint32_t total = 0;
  if (tid < p.bins) {
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const uint32_t c = wh[w][tid];
      wh[w][tid] = total;
      total += c;
    }
  }
  const uint32_t first = block_exclusive(tid < p.bins ? total : 0u, warp_sums);
  const uint32_t all = block_exclusive(tid < p.bins ? p.totals[tid] : 0u, warp_sums);
  if (tid < p.bins) {
    start[tid] = first;
    gbase[tid] = all + p.counts[(int64_t)tid * p.tiles + blockIdx.x] - first;
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kPerThread; ++j) {
    const int64_t i = base + j * 32 + lane;
    if (i < p.n) {
      const uint32_t d = (key[j] >> p.shift) & (p.bins - 1);
      const uint32_t at = start[d] + wh[warp][d] + rank[j];
      sk[at] = key[j];
      sp[at] = pos[j];
    }
  }
  __syncthreads();
  const int64_t left = p.n - (int64_t)blockIdx.x * kTile;
  const int m = left < kTile ? (int)left : kTile;
  for (int i = tid; i < m; i += kThreads) {
    const uint32_t k = sk[i];
    const uint32_t g = gbase[(k >> p.shift) & (p.bins - 1)] + i;
    p.key_out[g] = k;
    p.pos_out[g] = sp[i];
  }
}

// -------------------------------------------------------------------------------------- segments
// A segment is the run of one row id in the sorted keys; its number among the segments is `slot`.
constexpr int kSegTile = 2048;

__device__ __forceinline__ bool is_head(const uint32_t* key, int64_t i, uint32_t rows) {
  const uint32_t k = key[i];
  return k < rows && (i == 0 || key[i - 1] != k);
}

__global__ void __launch_bounds__(kThreads) head_count_kernel(const uint32_t* __restrict__ key, int64_t n,
                                                              uint32_t rows, uint32_t* __restrict__ heads) {
  pdl_wait();
  pdl_trigger();
  int c = 0;
  for (int j = threadIdx.x; j < kSegTile; j += kThreads) {
    const int64_t i = (int64_t)blockIdx.x * kSegTile + j;
    c += __syncthreads_count(i < n && is_head(key, i, rows));
  }
  if (threadIdx.x == 0) heads[blockIdx.x] = (uint32_t)c;
}

// seg_start[u] = first sorted pair of segment u (seg_start[count] = the pairs inside the table);
// the sparse form's grad_rows (-1 past the count) and count
__global__ void __launch_bounds__(kThreads)
    segments_kernel(const uint32_t* __restrict__ key, int64_t n, uint32_t rows, const uint32_t* __restrict__ heads,
                    int32_t tiles, uint32_t* __restrict__ seg_start, uint32_t* __restrict__ n_seg,
                    int64_t* __restrict__ grad_rows, int64_t* __restrict__ count) {
  pdl_wait();
  pdl_trigger();
  __shared__ uint32_t sum_s[2];
  __shared__ uint32_t warp_sums[kThreads / 32];
  if (threadIdx.x < 2) sum_s[threadIdx.x] = 0;
  __syncthreads();
  uint32_t before = 0, all = 0;
  for (int t = threadIdx.x; t < tiles; t += kThreads) {
    const uint32_t h = heads[t];
    all += h;
    if (t < (int)blockIdx.x) before += h;
  }
  atomicAdd(&sum_s[0], before);
  atomicAdd(&sum_s[1], all);
  __syncthreads();
  uint32_t u = sum_s[0];
  const uint32_t total = sum_s[1];
  for (int j = threadIdx.x; j < kSegTile; j += kThreads) {
    const int64_t i = (int64_t)blockIdx.x * kSegTile + j;
    const bool h = i < n && is_head(key, i, rows);
    const uint32_t off = block_exclusive(h ? 1u : 0u, warp_sums);
    if (h) {
      seg_start[u + off] = (uint32_t)i;
      if (grad_rows != nullptr) grad_rows[u + off] = key[i];
    }
    if (i < n && key[i] >= rows && (i == 0 || key[i - 1] < rows)) seg_start[total] = (uint32_t)i;
    if (i == n - 1 && key[i] < rows) seg_start[total] = (uint32_t)n;
    if (grad_rows != nullptr && i < n && i >= (int64_t)total) grad_rows[i] = -1;
    u += __syncthreads_count(h);
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *n_seg = total;
    if (count != nullptr) *count = total;
  }
}

__global__ void __launch_bounds__(32) no_segments_kernel(int64_t* count) {
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x == 0) *count = 0;
}

// ------------------------------------------------------------------------------------ segment sums
// one warp per (segment, 32 * V columns)
template <int DT, int GT, int V>
__global__ void __launch_bounds__(kThreads)
    segment_sum_kernel(const EmbedGradArgs a, const uint32_t* __restrict__ key, const uint32_t* __restrict__ pos,
                       const uint32_t* __restrict__ seg_start, const uint32_t* __restrict__ n_seg) {
  pdl_wait();
  pdl_trigger();
  using D = typename Elem<DT>::type;
  using G = typename Elem<GT>::type;
  const int lane = threadIdx.x & 31;
  const int k = ((int)blockIdx.y * 32 + lane) * V;
  const uint32_t total = *n_seg;
  for (int64_t u = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); u < total;
       u += (int64_t)gridDim.x * (kThreads / 32)) {
    const uint32_t i0 = seg_start[u], i1 = seg_start[u + 1];
    float acc[V] = {};
    for (uint32_t i = i0; i < i1; ++i) {
      const uint32_t p = pos[i], t = p / (uint32_t)a.e.n_cols;
      if (k < a.e.dim) {
        Raw<DT, V> raw;
        raw.load((const D*)a.dout + t * a.dout_stride + (int64_t)(p - t * a.e.n_cols) * a.e.dim + k);
        float f[V];
        raw.widen(f);
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] += f[j];
      }
    }
    if (k < a.e.dim) {
      const int64_t row = a.grad_rows != nullptr ? u : (int64_t)key[i0];
      G* g = (G*)a.grad + row * a.grad_stride + k;
#pragma unroll
      for (int j = 0; j < V; ++j) acc[j] *= a.e.scale;
      if (a.accumulate) {
        Raw<GT, V> raw;
        raw.load(g);
        float f[V];
        raw.widen(f);
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] = f[j] + acc[j];
      }
      store_vals<GT, V>(g, acc);
    }
  }
}

template <int GT>
__global__ void __launch_bounds__(kThreads)
    zero_rows_kernel(typename Elem<GT>::type* grad, int64_t rows, int32_t dim, int64_t stride) {
  pdl_wait();
  pdl_trigger();
  const int64_t units = rows * dim;
  for (int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x; u < units; u += (int64_t)gridDim.x * kThreads) {
    const int64_t r = u / dim;
    Elem<GT>::store(grad + r * stride + (u - r * dim), 0.f);
  }
}

inline uint64_t round256(uint64_t b) { return (b + 255) & ~(uint64_t)255; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct Layout {  // byte offsets into the workspace
  uint64_t key[2], pos[2], counts, totals, heads, seg_start, n_seg, end;
};
Layout layout_of(int64_t n) {
  Layout l;
  uint64_t at = 0;
  auto take = [&](uint64_t bytes) {
    const uint64_t p = at;
    at += round256(bytes);
    return p;
  };
  for (int i = 0; i < 2; ++i) {
    l.key[i] = take((uint64_t)n * 4);
    l.pos[i] = take((uint64_t)n * 4);
  }
  l.counts = take((uint64_t)ceil_div(n, kTile) * kMaxBins * 4);
  l.totals = take(kMaxBins * 4);
  l.heads = take((uint64_t)ceil_div(n, kSegTile) * 4);
  l.seg_start = take((uint64_t)(n + 1) * 4);
  l.n_seg = take(4);
  l.end = at;
  return l;
}

inline bool wide(const void* p, int64_t stride, int32_t dim, int32_t type) {
  const int per = 16 / type_bytes(type);
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride % per == 0 && dim % 8 == 0;
}

}  // namespace

cudaError_t launch_embed(const EmbedArgs& a, const void* W, int64_t row_stride, int32_t w_type, void* out,
                         int32_t out_type, cudaStream_t s) {
  const bool v8 = wide(W, row_stride, a.dim, w_type) && wide(out, a.dim, a.dim, out_type);
  const int64_t units = a.T * a.n_cols * (a.dim / (v8 ? 8 : 1));
  const int64_t grid = std::min<int64_t>(ceil_div(units, kThreads), 152 * 64);
  return with_type(w_type, [&](auto wt) {
    return with_type(out_type, [&](auto ot) {
      using WE = typename Elem<wt()>::type;
      using OE = typename Elem<ot()>::type;
      if (v8)
        return launch_pdl(embed_kernel<wt(), ot(), 8>, dim3((unsigned)grid), dim3(kThreads), 0, s, a, (const WE*)W,
                          row_stride, (OE*)out);
      return launch_pdl(embed_kernel<wt(), ot(), 1>, dim3((unsigned)grid), dim3(kThreads), 0, s, a, (const WE*)W,
                        row_stride, (OE*)out);
    });
  });
}

uint64_t embed_grad_workspace(int64_t n, int64_t, int32_t) { return n > 0 ? layout_of(n).end : 0; }

cudaError_t launch_embed_grad(const EmbedGradArgs& a, void* workspace, cudaStream_t s) {
  const int64_t n = a.e.T * a.e.n_cols;
  const bool sparse = a.grad_rows != nullptr || a.count != nullptr;
  cudaError_t e = cudaSuccess;
  if (!sparse && !a.accumulate && a.e.rows > 0) {
    e = with_type(a.grad_type, [&](auto gt) {
      using G = typename Elem<gt()>::type;
      const int64_t grid = std::min<int64_t>(ceil_div(a.e.rows * a.e.dim, kThreads), 152 * 16);
      return launch_pdl(zero_rows_kernel<gt()>, dim3((unsigned)grid), dim3(kThreads), 0, s, (G*)a.grad, a.e.rows,
                        a.e.dim, a.grad_stride);
    });
    if (e != cudaSuccess) return e;
  }
  if (n == 0) {
    if (!sparse) return cudaSuccess;
    return launch_pdl(no_segments_kernel, dim3(1), dim3(32), 0, s, a.count);
  }
  const Layout l = layout_of(n);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  auto u32 = [&](uint64_t off) { return reinterpret_cast<uint32_t*>(ws + off); };
  int bits = 1;
  while (bits < 32 && ((uint64_t)a.e.rows >> bits) != 0) ++bits;  // `rows` itself is a key
  const int passes = (bits + kMaxBits - 1) / kMaxBits, width = (bits + passes - 1) / passes;
  const int tiles = (int)ceil_div(n, kTile);
  for (int q = 0; q < passes; ++q) {
    SortPass p;
    p.key_in = q == 0 ? nullptr : u32(l.key[q & 1]);
    p.pos_in = q == 0 ? nullptr : u32(l.pos[q & 1]);
    p.key_out = u32(l.key[(q + 1) & 1]);
    p.pos_out = u32(l.pos[(q + 1) & 1]);
    p.counts = u32(l.counts);
    p.totals = u32(l.totals);
    p.n = n;
    p.tiles = tiles;
    p.shift = q * width;
    p.bins = 1 << std::min(width, 32 - q * width);
    e = launch_pdl(sort_count_kernel, dim3(tiles), dim3(kThreads), 0, s, a.e, p);
    if (e != cudaSuccess) return e;
    e = launch_pdl(sort_scan_kernel, dim3((unsigned)ceil_div(p.bins, kThreads / 32)), dim3(kThreads), 0, s, p);
    if (e != cudaSuccess) return e;
    e = launch_pdl(sort_scatter_kernel, dim3(tiles), dim3(kThreads), 0, s, a.e, p);
    if (e != cudaSuccess) return e;
  }
  const uint32_t *key = u32(l.key[passes & 1]), *pos = u32(l.pos[passes & 1]);
  const int seg_tiles = (int)ceil_div(n, kSegTile);
  e = launch_pdl(head_count_kernel, dim3(seg_tiles), dim3(kThreads), 0, s, key, n, (uint32_t)a.e.rows, u32(l.heads));
  if (e != cudaSuccess) return e;
  e = launch_pdl(segments_kernel, dim3(seg_tiles), dim3(kThreads), 0, s, key, n, (uint32_t)a.e.rows,
                 (const uint32_t*)u32(l.heads), seg_tiles, u32(l.seg_start), u32(l.n_seg), a.grad_rows, a.count);
  if (e != cudaSuccess) return e;
  const bool v8 = wide(a.dout, a.dout_stride, a.e.dim, a.dout_type) && wide(a.grad, a.grad_stride, a.e.dim, a.grad_type);
  const unsigned chunks = (unsigned)ceil_div(a.e.dim, 32 * (v8 ? 8 : 1));
  const unsigned gx = (unsigned)std::min<int64_t>(ceil_div(n, kThreads / 32), 152 * 8);
  return with_type(a.dout_type, [&](auto dt) {
    return with_type(a.grad_type, [&](auto gt) {
      if (v8)
        return launch_pdl(segment_sum_kernel<dt(), gt(), 8>, dim3(gx, chunks), dim3(kThreads), 0, s, a, key, pos,
                          (const uint32_t*)u32(l.seg_start), (const uint32_t*)u32(l.n_seg));
      return launch_pdl(segment_sum_kernel<dt(), gt(), 1>, dim3(gx, chunks), dim3(kThreads), 0, s, a, key, pos,
                        (const uint32_t*)u32(l.seg_start), (const uint32_t*)u32(l.n_seg));
    });
  });
}

}  // namespace engram
