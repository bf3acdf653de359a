// Trainable embedding rows (sm_103a): the lookup with a scale, and its gradient by sorted row ids.
//
//   out[t][c]  = round(scale * W[idx[t][c]])                    (+0 where idx is outside [0, rows))
//   G[r]       = scale * sum over (t, c) with idx[t][c] == r of dout[t][c]
//
// The gradient's sums run in fp32 in an order that depends on the ids, their number and dim alone, so the same ids and
// gradients give the same bits, also at other addresses and strides. The ids are sorted (a stable radix sort of (row id, position)
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
// A CTA writes kThreads * kFly consecutive vectors of the output, kFly of them a thread and all of their rows in
// flight at once. N: the type that numbers vectors (32 bits where they fit: 64-bit divisions cost more than
// the copy). The output goes out with an evict-first policy: rows that ids repeat stay in L2 longer.
// 65,536 x 24 bf16 rows of 128 values (half of the ids repeat): 92 us, 0.94 of the copy bandwidth counting each
// distinct row once; 1, 2 and 8 vectors a thread 143, 106 and 129 us; with 64-bit divisions and one vector 123 us.
constexpr int kFly = 4;

template <int WT, int OT, int V, typename N>
__global__ void __launch_bounds__(kThreads)
    embed_kernel(const EmbedArgs a, const typename Elem<WT>::type* __restrict__ W, const int64_t row_stride,
                 typename Elem<OT>::type* __restrict__ out, const N units) {
  pdl_wait();
  pdl_trigger();
  const uint32_t per_row = a.dim / V;
  const N u0 = (N)blockIdx.x * (kThreads * kFly) + threadIdx.x;
  int64_t r[kFly];
  uint32_t k[kFly];
#pragma unroll
  for (int j = 0; j < kFly; ++j) {
    const N u = u0 + j * kThreads;
    r[j] = -1;
    if (u < units) {
      const N e = u / per_row;
      k[j] = (uint32_t)(u - e * per_row) * V;
      int64_t at = (int64_t)e;
      if (a.idx_stride != a.n_cols) {
        const N t = e / (uint32_t)a.n_cols;
        at = (int64_t)t * a.idx_stride + (int64_t)(e - t * (uint32_t)a.n_cols);
      }
      r[j] = a.idx[at];
    }
  }
  Raw<WT, V> raw[kFly];
#pragma unroll
  for (int j = 0; j < kFly; ++j) {
    raw[j].zero();
    if (r[j] >= 0 && r[j] < a.rows) raw[j].load(W + r[j] * row_stride + k[j]);
  }
#pragma unroll
  for (int j = 0; j < kFly; ++j) {
    const N u = u0 + j * kThreads;
    if (u < units) {
      const bool ok = r[j] >= 0 && r[j] < a.rows;
      float f[V];
      raw[j].widen(f);
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = ok ? f[i] * a.scale : 0.f;
      store_vals<OT, V, true>(out + (int64_t)u * V, f);
    }
  }
}

// -------------------------------------------------------------------------------------- radix sort
// Least significant digit first, up to kMaxBits bits a pass; per pass a count of every digit per
// tile, a scan over the tiles of each digit, and a stable scatter. Keys are row ids as 32-bit values,
// with `rows` itself standing for every id outside the table, so those sort to the end. The first count
// also writes the keys, so that the ids are read once.
// 1.57 million ids of a table of 384 million rows (29 bits, 3 passes): 75 us of the call's 208. A pass is 4 us of
// counting (7 in the first), 4 of scanning and 14 of scattering, which no memory bounds (25 MB out of L2): the ranks'
// ballots and the exchange do. Tiles of 512 threads x 12 pairs measured best (whole call: 8 pairs 231, 16 pairs 254,
// 256 threads x 16 pairs 248 us), of 4 pairs while that makes two tiles an SM at most (20,000 ids: 31 us on the GPU
// instead of 43; 600,000: 69 us a call instead of 71; but 700,000: 76 instead of 74); 8-bit passes with
// __match_any_sync instead of ballots 15 us more.
constexpr int kMaxBits = 10;
constexpr int kMaxBins = 1 << kMaxBits;
constexpr int kSortThreads = 512;
// Pairs a thread has of a tile (one CTA's pairs): 12, and 4 for calls of few ids
constexpr int kPairs = 12, kPairsFew = 4;
constexpr int64_t kFewIds = 2 * 152 * kSortThreads * kPairsFew;
constexpr int pairs_of(int64_t n) { return n <= kFewIds ? kPairsFew : kPairs; }

// With few counts a pass has no scan of its own: every CTA of the scatter adds up the tiles' counts itself, which costs
// less than a launch (348,000 ids of a table of 2,520 rows, 170 tiles of 64 counts: 49 us instead of 52; but 581,000 of
// 2.7 million rows, 95 tiles of 256 counts, 93 us for 75: all CTAs ask L2 for the same lines)
constexpr int kFewTiles = 32;
constexpr int64_t kFewCounts = 12 << 10;
__host__ __device__ inline bool few_counts(int tiles, int bits) {
  return tiles <= kFewTiles || ((int64_t)tiles << bits) <= kFewCounts;
}

struct SortPass {
  uint32_t* key_in;        // written by the first pass's count
  const uint32_t* pos_in;  // null in the first pass: the positions are 0, 1, 2, ...
  uint32_t* key_out;
  uint32_t* pos_out;
  uint32_t* counts;  // [tiles][bins]
  uint32_t* totals;  // [bins]
  int64_t n;
  int32_t tiles, shift, bits;
};

__device__ __forceinline__ uint32_t key_of_id(const EmbedArgs& e, uint32_t i) {
  int64_t at = i;
  if (e.idx_stride != e.n_cols) {
    const uint32_t t = i / (uint32_t)e.n_cols;
    at = (int64_t)t * e.idx_stride + (i - t * (uint32_t)e.n_cols);
  }
  const int64_t r = e.idx[at];
  return r >= 0 && r < e.rows ? (uint32_t)r : (uint32_t)e.rows;
}

template <bool FIRST, int kPerThread>
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const EmbedArgs e, const SortPass p) {
  pdl_wait();
  pdl_trigger();
  __shared__ uint32_t hist[kMaxBins];
  const int bins = 1 << p.bits;
  for (int b = threadIdx.x; b < bins; b += kSortThreads) hist[b] = 0;
  __syncthreads();
  const uint32_t base = blockIdx.x * (uint32_t)(kSortThreads * kPerThread), n = (uint32_t)p.n;
  // a thread has runs of 4 pairs
  static_assert(kPerThread % 4 == 0, "a tile is whole runs");
  uint32_t key[kPerThread] = {};
#pragma unroll
  for (int j = 0; j < kPerThread; j += 4) {
    const uint32_t i = base + (j / 4 * kSortThreads + threadIdx.x) * 4;
    if (FIRST) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (i + q < n) key[j + q] = key_of_id(e, i + q);
    } else if (i < n) {  // the arrays reach past n
      const uint4 v = *reinterpret_cast<const uint4*>(p.key_in + i);
      key[j] = v.x;
      key[j + 1] = v.y;
      key[j + 2] = v.z;
      key[j + 3] = v.w;
    }
  }
#pragma unroll
  for (int j = 0; j < kPerThread; j += 4) {
    const uint32_t i = base + (j / 4 * kSortThreads + threadIdx.x) * 4;
    if (FIRST && i < n) *reinterpret_cast<uint4*>(p.key_in + i) = make_uint4(key[j], key[j + 1], key[j + 2], key[j + 3]);
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (i + q < n) atomicAdd(&hist[(key[j + q] >> p.shift) & (bins - 1)], 1u);
  }
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += kSortThreads) p.counts[((int64_t)blockIdx.x << p.bits) + b] = hist[b];
}

// counts[tile][digit] becomes the pairs of the digit in the tiles before. A CTA takes 32 digits, a lane each, and
// a warp a 32nd of the tiles.
constexpr int kScanThreads = 1024;
__global__ void __launch_bounds__(kScanThreads) sort_scan_kernel(const SortPass p) {
  pdl_wait();
  pdl_trigger();
  __shared__ uint32_t part[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, bins = 1 << p.bits;
  const int d = blockIdx.x * 32 + lane, per = (p.tiles + 31) / 32;
  const int t0 = warp * per, t1 = min(p.tiles, t0 + per);
  uint32_t* c = p.counts + d;
  uint32_t sum = 0;
  if (d < bins) {
#pragma unroll 8
    for (int t = t0; t < t1; ++t) sum += c[(int64_t)t << p.bits];
  }
  part[warp][lane] = sum;
  __syncthreads();
  // warp w scans digit w's parts
  const uint32_t v = part[lane][warp];
  uint32_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  part[lane][warp] = x - v;
  if (lane == 31 && blockIdx.x * 32 + warp < bins) p.totals[blockIdx.x * 32 + warp] = x;
  __syncthreads();
  if (d >= bins) return;
  uint32_t run = part[warp][lane];
#pragma unroll 8
  for (int t = t0; t < t1; ++t) {
    const uint32_t n = c[(int64_t)t << p.bits];
    c[(int64_t)t << p.bits] = run;
    run += n;
  }
}

// exclusive scan over the block of one value per thread; warp_sums: 32 words
template <int THREADS>
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
  // every warp sums the warps before it
  uint32_t s = lane < warp && lane < THREADS / 32 ? warp_sums[lane] : 0u;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  __syncthreads();
  return s + x - v;
}

constexpr int kSortWarps = kSortThreads / 32;
constexpr int kDigits = kMaxBins / kSortThreads;  // digits of a thread: two, which share a word of the warps' counts
static_assert(kDigits == 2 && kSortThreads * kPairs < 65536, "the counts of two digits are one word of two 16-bit halves");
constexpr int scatter_smem(int pairs) {
  return kSortThreads * pairs * 8 + kSortWarps * kMaxBins * 2 + kMaxBins * 4 + 32 * 4;
}

// The stable scatter of a tile: places inside the sorted tile first (the pairs' order is (warp, step, lane), a warp
// taking 32 * kPerThread consecutive pairs 32 at a time), an exchange through shared memory, then runs of equal digits
// go out together. The warps' counts are 16-bit, all digits of all warps, whatever the pass's width.
template <bool FIRST, int kPerThread>
__global__ void __launch_bounds__(kSortThreads, 2) sort_scatter_kernel(const SortPass p) {
  constexpr int kTile = kSortThreads * kPerThread;
  pdl_wait();
  pdl_trigger();
  extern __shared__ uint32_t smem[];
  uint32_t* sk = smem;                    // [kTile] the tile in digit order
  uint32_t* sp = sk + kTile;              // [kTile]
  uint32_t* wh = sp + kTile;              // [kSortWarps][kMaxBins / 2] two 16-bit counts a word, then places
  uint32_t* go = wh + kSortWarps * kMaxBins / 2;  // [kMaxBins] a digit's first place in the output less that in the tile
  uint32_t* warp_sums = go + kMaxBins;            // [32]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, bins = 1 << p.bits;
  const int64_t tile0 = (int64_t)blockIdx.x * kTile;
  const int left = (int)min((int64_t)kTile, p.n - tile0);
  uint32_t key[kPerThread], pos[kPerThread];
  const int base = warp * 32 * kPerThread + lane;
#pragma unroll
  for (int j = 0; j < kPerThread; ++j) {
    key[j] = 0;
    pos[j] = (uint32_t)(tile0 + base + j * 32);
    if (base + j * 32 < left) {
      key[j] = p.key_in[tile0 + base + j * 32];
      if (!FIRST) pos[j] = p.pos_in[tile0 + base + j * 32];
    }
  }
  for (int b = tid; b < kSortWarps * kMaxBins / 8; b += kSortThreads)
    reinterpret_cast<uint4*>(wh)[b] = make_uint4(0u, 0u, 0u, 0u);
  // where each of the thread's digits goes: the digits before it, the same digit in the tiles before
  uint32_t tot[kDigits], there[kDigits];
#pragma unroll
  for (int q = 0; q < kDigits; ++q) tot[q] = there[q] = 0;
  const int row = bins / kDigits;  // a tile's counts, in words of two digits
  const uint2* c2 = reinterpret_cast<const uint2*>(p.counts);
  if (few_counts(p.tiles, p.bits)) {
    // the digits of word tid % row, of every groups-th tile; the parts meet in shared memory, in the tile's place
    const int group = tid / row, groups = min(16, kSortThreads / row);
    const uint2* c = c2 + (tid - group * row);
#pragma unroll 8
    for (int t = group < groups ? group : p.tiles; t < p.tiles; t += groups) {
      const uint2 v = c[t * row];
      tot[0] += v.x;
      tot[1] += v.y;
      if (t < (int)blockIdx.x) {
        there[0] += v.x;
        there[1] += v.y;
      }
    }
    if (groups > 1) {
      uint4* parts = reinterpret_cast<uint4*>(smem);
      parts[tid] = make_uint4(tot[0], tot[1], there[0], there[1]);
      __syncthreads();
      tot[0] = tot[1] = there[0] = there[1] = 0;
      if (tid < row) {
        for (int g = 0; g < groups; ++g) {
          const uint4 v = parts[g * row + tid];
          tot[0] += v.x;
          tot[1] += v.y;
          there[0] += v.z;
          there[1] += v.w;
        }
      }
    }
  } else if (tid < row) {
    const uint2 n = reinterpret_cast<const uint2*>(p.totals)[tid], v = c2[(int64_t)blockIdx.x * row + tid];
    tot[0] = n.x;
    tot[1] = n.y;
    there[0] = v.x;
    there[1] = v.y;
  }
  const uint32_t all = block_exclusive<kSortThreads>(tot[0] + tot[1], warp_sums);
  there[0] += all;
  there[1] += all + tot[0];
  // lanes of the warp with the same digit: a ballot per bit (of 6 at least), all steps together
  unsigned same[kPerThread];
#pragma unroll
  for (int j = 0; j < kPerThread; ++j) same[j] = __ballot_sync(0xffffffffu, base + j * 32 < left);
#pragma unroll
  for (int b = 0; b < kMaxBits; ++b) {
    if (b >= 6 && b >= p.bits) break;
    const uint32_t bit = b < p.bits ? 1u << (p.shift + b) : 0u;
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) {
      const bool set = key[j] & bit;
      const unsigned v = __ballot_sync(0xffffffffu, set);
      same[j] &= set ? v : ~v;
    }
  }
  uint16_t* mine = reinterpret_cast<uint16_t*>(wh + warp * kMaxBins / 2);
  uint32_t rank[kPerThread / 2];  // two 16-bit ranks a word
#pragma unroll
  for (int j = 0; j < kPerThread; ++j) {
    const bool in = base + j * 32 < left;
    const uint32_t d = (key[j] >> p.shift) & (bins - 1);
    const int before = __popc(same[j] & ((1u << lane) - 1u));
    uint32_t have = 0;
    if (in) have = mine[d];
    __syncwarp();
    if (in && before == 0) mine[d] = (uint16_t)(have + __popc(same[j]));
    __syncwarp();
    if (j % 2 == 0) rank[j / 2] = have + before;
    else rank[j / 2] |= (have + before) << 16;
  }
  __syncthreads();
  // the warps' counts of the thread's two digits become places: digits before, warps before
  uint32_t c[kSortWarps], sum = 0;
#pragma unroll
  for (int w = 0; w < kSortWarps; ++w) {
    c[w] = wh[w * kMaxBins / 2 + tid];
    sum += c[w];  // no carry: a half is at most kTile
  }
  const uint32_t n0 = sum & 0xffffu, n1 = sum >> 16;
  const uint32_t at = block_exclusive<kSortThreads>(n0 + n1, warp_sums);
  uint32_t run = at | (at + n0) << 16;
#pragma unroll
  for (int w = 0; w < kSortWarps; ++w) {
    wh[w * kMaxBins / 2 + tid] = run;
    run += c[w];
  }
  go[tid * kDigits] = there[0] - at;
  go[tid * kDigits + 1] = there[1] - (at + n0);
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kPerThread; ++j) {
    if (base + j * 32 < left) {
      const uint32_t d = (key[j] >> p.shift) & (bins - 1);
      const uint32_t place = mine[d] + (rank[j / 2] >> (16 * (j % 2)) & 0xffffu);
      sk[place] = key[j];
      sp[place] = pos[j];
    }
  }
  __syncthreads();
#pragma unroll 4
  for (int i = tid; i < left; i += kSortThreads) {
    const uint32_t k = sk[i];
    const uint32_t g = go[(k >> p.shift) & (bins - 1)] + i;
    p.key_out[g] = k;
    p.pos_out[g] = sp[i];
  }
}

// -------------------------------------------------------------------------------------- segments
// A segment is the run of one row id in the sorted keys. The sparse form numbers the segments: ids[i] is
// the number of the segment that sorted pair i belongs to (kNone outside the table). The dense form
// needs no numbers: there the keys themselves serve as ids.
constexpr int kSegTile = 2048;
constexpr uint32_t kNone = 0xffffffffu;

constexpr int kSegPer = kSegTile / kThreads;

// bit j: pair i0 + j begins a segment. The keys are read 4 at a time; the array reaches kBatch past n.
__device__ __forceinline__ uint32_t head_bits(const uint32_t* key, int64_t i0, int64_t n, uint32_t rows,
                                              uint32_t (&k)[kSegPer]) {
  uint32_t bits = 0;
  if (i0 >= n) return 0;
#pragma unroll
  for (int j = 0; j < kSegPer; j += 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(key + i0 + j);
    k[j] = v.x;
    k[j + 1] = v.y;
    k[j + 2] = v.z;
    k[j + 3] = v.w;
  }
  uint32_t before = i0 == 0 ? ~k[0] : key[i0 - 1];
#pragma unroll
  for (int j = 0; j < kSegPer; ++j) {
    if (i0 + j < n && k[j] < rows && k[j] != before) bits |= 1u << j;
    before = k[j];
  }
  return bits;
}

__global__ void __launch_bounds__(kThreads) head_count_kernel(const uint32_t* __restrict__ key, int64_t n,
                                                              uint32_t rows, uint32_t* __restrict__ heads) {
  pdl_wait();
  pdl_trigger();
  __shared__ uint32_t sum;
  if (threadIdx.x == 0) sum = 0;
  __syncthreads();
  uint32_t k[kSegPer];
  const int c = __popc(head_bits(key, ((int64_t)blockIdx.x * kThreads + threadIdx.x) * kSegPer, n, rows, k));
  const int w = __reduce_add_sync(0xffffffffu, c);
  if ((threadIdx.x & 31) == 0) atomicAdd(&sum, (uint32_t)w);
  __syncthreads();
  if (threadIdx.x == 0) heads[blockIdx.x] = sum;
}

// ids, and the sparse form's grad_rows (-1 past the count) and count. Calls of up to kNumbered ids need neither of these
// two kernels: there every CTA of the sums counts the heads of all ids itself, which costs less than two launches
// (9,000 ids: 38 us a call instead of 40; 32,000: 45 instead of 48; but 65,000: 67 instead of 55).
constexpr int64_t kNumbered = 32768;
__global__ void __launch_bounds__(kThreads)
    segments_kernel(const uint32_t* __restrict__ key, int64_t n, uint32_t rows, const uint32_t* __restrict__ heads,
                    int32_t tiles, uint32_t* __restrict__ ids, int64_t* __restrict__ grad_rows,
                    int64_t* __restrict__ count) {
  pdl_wait();
  pdl_trigger();
  __shared__ uint32_t sum_s[2], n_rows;
  __shared__ uint32_t warp_sums[32];
  __shared__ uint32_t rows_s[kSegTile];  // the rows that begin here, for whole-line stores
  if (threadIdx.x < 2) sum_s[threadIdx.x] = 0;
  __syncthreads();
  const int64_t i0 = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * kSegPer;
  uint32_t k[kSegPer];
  const uint32_t bits = head_bits(key, i0, n, rows, k);
  uint32_t before = 0, all = 0;
  for (int t = threadIdx.x; t < tiles; t += kThreads) {
    const uint32_t h = heads[t];
    all += h;
    if (t < (int)blockIdx.x) before += h;
  }
  before = __reduce_add_sync(0xffffffffu, before);
  all = __reduce_add_sync(0xffffffffu, all);
  if ((threadIdx.x & 31) == 0) {
    atomicAdd(&sum_s[0], before);
    atomicAdd(&sum_s[1], all);
  }
  uint32_t off = block_exclusive<kThreads>(__popc(bits), warp_sums);
  const uint32_t u0 = sum_s[0], total = sum_s[1];
  uint32_t id[kSegPer];
#pragma unroll
  for (int j = 0; j < kSegPer; ++j) {
    if (bits >> j & 1) rows_s[off++] = k[j];
    id[j] = i0 < n && k[j] < rows ? u0 + off - 1 : kNone;
  }
  if (threadIdx.x == kThreads - 1) n_rows = off;
  if (i0 < n) {
#pragma unroll
    for (int j = 0; j < kSegPer; j += 4)
      *reinterpret_cast<uint4*>(ids + i0 + j) = make_uint4(id[j], id[j + 1], id[j + 2], id[j + 3]);
  }
  __syncthreads();
  for (int j = threadIdx.x; j < (int)n_rows; j += kThreads) grad_rows[u0 + j] = rows_s[j];
  for (int j = threadIdx.x; j < kSegTile; j += kThreads) {
    const int64_t i = (int64_t)blockIdx.x * kSegTile + j;
    if (i < n && i >= (int64_t)total) grad_rows[i] = -1;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) *count = total;
}

__global__ void __launch_bounds__(32) no_segments_kernel(int64_t* count) {
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x == 0) *count = 0;
}

// Calls of up to kSmall ids: a pair's place is counted, not sorted for. It is the number of smaller keys plus the
// number of equal ones before it, n^2 comparisons that all SMs share: 6,144 pairs take 38 million, a few
// microseconds (15 from a cold start), where a radix sort in one CTA took 40 to 50. At 8,192 the whole call takes 25 us,
// through the radix passes 37 to 40; at 16,384 counting would take 57 us against 37 to 41. A CTA places 32 pairs, a
// lane each; its 8 warps take an eighth of the keys each.
constexpr int kSmall = 8192;
constexpr int kPlaced = 32;  // pairs placed by a CTA

__global__ void __launch_bounds__(kThreads) place_small_kernel(const EmbedArgs e, const int n,
                                                               uint32_t* __restrict__ key_out,
                                                               uint32_t* __restrict__ pos_out) {
  pdl_wait();
  pdl_trigger();
  constexpr int kWarps = kThreads / 32;
  __shared__ __align__(16) uint32_t sk[kSmall];
  __shared__ int part[kWarps][32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int vecs = (n + 3) / 4;  // the last one is filled up with a key above every other
#pragma unroll 8
  for (int i = tid; i < vecs * 4; i += kThreads) sk[i] = i < n ? key_of_id(e, i) : 0xffffffffu;
  __syncthreads();
  const int i0 = blockIdx.x * kPlaced, i = i0 + lane;
  const uint32_t mine = sk[min(i, n - 1)];
  const uint4* sv = reinterpret_cast<const uint4*>(sk);
  int c = 0;
  // keys below `limit` in vectors [v0, v1)
  auto count = [&](int v0, int v1, uint32_t limit) {
#pragma unroll 4
    for (int v = v0; v < v1; ++v) {
      const uint4 k = sv[v];
      c += (k.x < limit) + (k.y < limit) + (k.z < limit) + (k.w < limit);
    }
  };
  const int a = vecs * warp / kWarps, b = vecs * (warp + 1) / kWarps;
  const int m0 = i0 / 4, m1 = m0 + kPlaced / 4;  // the vectors of the CTA's own pairs
  count(a, min(b, m0), mine + 1);                // before them equal keys count too (keys are at most 2^32 - 2)
  for (int j = max(a, m0) * 4; j < min(b, m1) * 4; ++j) c += sk[j] < mine || (sk[j] == mine && j < i);
  count(max(a, m1), b, mine);
  part[warp][lane] = c;
  __syncthreads();
  if (warp != 0 || i >= n) return;
  for (int w = 1; w < kWarps; ++w) c += part[w][lane];
  key_out[c] = mine;
  pos_out[c] = (uint32_t)i;
}

// ------------------------------------------------------------------------------------ segment sums
// Bound by memory: every gradient row is read once, every distinct row written once. 1.57 million bf16 rows of 128 values,
// 0.82 million distinct, fp32 sums: 133 us, 0.82 GB at 6.2 TB/s (0.92 of the copy bandwidth). The sums before this form, a
// warp per distinct row, took the call 1,658 us: the row that ids name most often was one warp's work.
// The sorted pairs are cut into units of `per_unit` consecutive ones, whatever segments they belong to,
// so a row named a million times and a million rows named once cost the same. A group of 2^glog lanes
// takes one unit and V columns a lane, with kBatch rows of dout in flight; it writes the segments that
// lie inside its unit. What is left are runs that cross a unit's ends: the CTA joins its units' parts in
// shared memory, in order, and leaves at most two parts for the kernel that joins the CTAs' (segments
// that span CTAs). Every sum's order follows from the sorted ids alone.
constexpr int kBatch = 8;

struct SumArgs {
  const uint32_t* ids;
  const uint32_t* pos;
  uint32_t limit;  // ids from here on are no rows
  int32_t number;  // sparse form of up to kNumbered ids: ids are keys, and this kernel numbers the segments and writes
                   // grad_rows and count
  int64_t n;
  int32_t glog, per_unit, chunks;
  int64_t tiles;
  float* lead;   // [tiles][dim4]: the part of a segment that began in an earlier tile
  float* trail;  // [tiles][dim4]: the part of a segment that goes on in the next tile
  int32_t dim4;  // dim rounded up to 4
  uint8_t* flags;  // [tiles] kOpen, kCloses, kThrough
  uint32_t* open_row;  // [tiles] with kOpen: the row of grad that the segment belongs to
  // dense form without accumulation: CTAs from tiles * chunks on write the rows that no id names
  int32_t zero_rows;  // rows per such CTA
};
constexpr int kOpen = 1;     // a segment that begins here goes on in the next unit (tile)
constexpr int kCloses = 2;   // the segment that began earlier ends here
constexpr int kThrough = 4;  // it neither begins nor ends here

template <int GT, int V>
__device__ __forceinline__ void finish_row(const EmbedGradArgs& a, uint32_t row, int k, float* acc) {
  typename Elem<GT>::type* g = static_cast<typename Elem<GT>::type*>(a.grad) + (int64_t)row * a.grad_stride + k;
#pragma unroll
  for (int j = 0; j < V; ++j) acc[j] *= a.e.scale;
  if (a.accumulate) {
    Raw<GT, V> raw;
    raw.load(g);
    float f[V];
    raw.widen(f);
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] += f[j];
  }
  store_vals<GT, V>(g, acc);
}

// Rows [r0, r0 + m) that no id names, in words of the widest type that their addresses and width allow
template <typename Word>
__device__ __forceinline__ void zero_words(uint8_t* row0, int64_t stride, int m, int per_row, const uint8_t* named) {
  for (int i = threadIdx.x; i < m * per_row; i += kThreads) {
    const int r = i / per_row;
    if (!named[r]) reinterpret_cast<Word*>(row0 + r * stride)[i - r * per_row] = Word{};
  }
}

template <int GT>
__device__ __forceinline__ void zero_rows(const EmbedGradArgs& a, const SumArgs& s, int64_t block) {
  // row r has an id exactly if the first sorted id >= r is r
  __shared__ uint8_t named[kThreads];
  const int64_t r0 = block * s.zero_rows;
  const int m = (int)min((int64_t)s.zero_rows, a.e.rows - r0);
  if ((int)threadIdx.x < m) {
    const uint32_t r = (uint32_t)(r0 + threadIdx.x);
    int64_t lo = 0, hi = s.n;
    while (lo < hi) {
      const int64_t mid = (lo + hi) >> 1;
      if (s.ids[mid] < r) lo = mid + 1; else hi = mid;
    }
    named[threadIdx.x] = lo < s.n && s.ids[lo] == r;
  }
  __syncthreads();
  constexpr int kSize = sizeof(typename Elem<GT>::type);
  const int64_t stride = a.grad_stride * kSize;
  uint8_t* row0 = static_cast<uint8_t*>(a.grad) + r0 * stride;
  const int bytes = a.e.dim * kSize;
  const uint64_t any = reinterpret_cast<uintptr_t>(row0) | (uint64_t)stride | (uint64_t)bytes;
  if (any % 16 == 0) zero_words<uint4>(row0, stride, m, bytes / 16, named);
  else if (any % 8 == 0) zero_words<uint2>(row0, stride, m, bytes / 8, named);
  else if (any % 4 == 0) zero_words<uint32_t>(row0, stride, m, bytes / 4, named);
  else zero_words<uint16_t>(row0, stride, m, bytes / 2, named);
}

template <int DT, int GT, int V>
__global__ void __launch_bounds__(kThreads) segment_sum_kernel(const EmbedGradArgs a, const SumArgs s) {
  pdl_wait();
  pdl_trigger();
  using D = typename Elem<DT>::type;
  __shared__ float lead_s[kThreads * V];  // [unit][column of the chunk]
  __shared__ uint8_t flag_s[kThreads];
  const int64_t work = s.tiles * s.chunks;
  if ((int64_t)blockIdx.x >= work) {
    zero_rows<GT>(a, s, (int64_t)blockIdx.x - work);
    return;
  }
  const int64_t tile = blockIdx.x / s.chunks;
  const int chunk = (int)(blockIdx.x - tile * s.chunks);
  const int G = 1 << s.glog, units = kThreads >> s.glog;
  const int unit = threadIdx.x >> s.glog, gl = threadIdx.x & (G - 1);
  const int k = (chunk * G + gl) * V;
  const bool on = k < a.e.dim;
  const int64_t i0 = min(s.n, (tile * units + unit) * s.per_unit), i1 = min(s.n, i0 + s.per_unit);
  const D* dout = static_cast<const D*>(a.dout) + k;
  const bool packed = a.dout_stride == (int64_t)a.e.n_cols * a.e.dim;

  float acc[V];
  uint32_t cur = kNone;  // the running segment's id
  uint32_t slot = 0;     // number: its number, or that of the one before the unit's first head
  bool leading = i0 > 0 && i0 < i1 && s.ids[i0 - 1] == s.ids[i0];
  if (s.number) {
    __shared__ uint32_t sums[2], warp_sums[32];
    if (threadIdx.x < 2) sums[threadIdx.x] = 0;
    __syncthreads();
    const int64_t tile0 = tile * units * s.per_unit;
    uint32_t before = 0, all = 0, k8[kSegPer];
    for (int64_t i = threadIdx.x * kSegPer; i < s.n; i += kThreads * kSegPer) {
      const uint32_t bits = head_bits(s.ids, i, s.n, s.limit, k8);
      all += __popc(bits);
      if (i < tile0) before += __popc(bits);  // tile0 is a multiple of kSegPer
    }
    before = __reduce_add_sync(0xffffffffu, before);
    all = __reduce_add_sync(0xffffffffu, all);
    if ((threadIdx.x & 31) == 0) {
      atomicAdd(&sums[0], before);
      atomicAdd(&sums[1], all);
    }
    uint32_t own = 0;
    if (gl == 0)
      for (int64_t i = i0; i < i1; i += kSegPer) own += __popc(head_bits(s.ids, i, s.n, s.limit, k8));
    const uint32_t off = block_exclusive<kThreads>(own, warp_sums);
    slot = sums[0] + __shfl_sync(0xffffffffu, off, threadIdx.x & 31 & ~(G - 1)) - 1;
    if (chunk == 0) {
      for (int j = threadIdx.x; j < units * s.per_unit; j += kThreads)
        if (tile0 + j < s.n && tile0 + j >= sums[1]) a.grad_rows[tile0 + j] = -1;
      if (blockIdx.x == 0 && threadIdx.x == 0) *a.count = sums[1];
    }
  }
  int flag = 0;
  auto put_lead = [&]() {
#pragma unroll
    for (int j = 0; j < V; ++j) lead_s[threadIdx.x * V + j] = acc[j];
  };
  auto close = [&]() {  // the running segment ends inside this unit
    if (leading) {
      put_lead();
      flag |= kCloses;
      leading = false;
    } else if (on) {
      finish_row<GT, V>(a, s.number ? slot : cur, k, acc);
    }
  };
  for (int64_t i = i0; i < i1; i += kBatch) {
    uint32_t id[kBatch];
    Raw<DT, V> raw[kBatch];
    // per_unit is a multiple of kBatch, so these are aligned; the arrays reach a batch past n
    const uint4 a0 = *reinterpret_cast<const uint4*>(s.ids + i), a1 = *reinterpret_cast<const uint4*>(s.ids + i + 4);
    const uint4 p0 = *reinterpret_cast<const uint4*>(s.pos + i), p1 = *reinterpret_cast<const uint4*>(s.pos + i + 4);
    const uint32_t ia[kBatch] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
    const uint32_t pa[kBatch] = {p0.x, p0.y, p0.z, p0.w, p1.x, p1.y, p1.z, p1.w};
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      id[j] = i + j < i1 && ia[j] < s.limit ? ia[j] : kNone;
      raw[j].zero();
      if (id[j] != kNone && on) {
        int64_t at = (int64_t)pa[j] * a.e.dim;
        if (!packed) {
          const uint32_t t = pa[j] / (uint32_t)a.e.n_cols;
          at = (int64_t)t * a.dout_stride + (int64_t)(pa[j] - t * a.e.n_cols) * a.e.dim;
        }
        raw[j].load(dout + at);
      }
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      float f[V];
      raw[j].widen(f);
      if (id[j] != cur) {
        if (cur != kNone) close();
        // a new segment; a leading run began in an earlier unit
        if (s.number && id[j] != kNone && !(leading && cur == kNone)) {
          ++slot;
          if (chunk == 0 && gl == 0) a.grad_rows[slot] = id[j];
        }
        cur = id[j];
#pragma unroll
        for (int q = 0; q < V; ++q) acc[q] = f[q];
      } else {
#pragma unroll
        for (int q = 0; q < V; ++q) acc[q] += f[q];
      }
    }
    if (id[kBatch - 1] == kNone) break;
  }
  if (cur != kNone) {
    if (i1 < s.n && s.ids[i1] == cur) {
      if (leading) put_lead();
      flag |= leading ? kThrough : kOpen;
    } else {
      close();
    }
  }
  if (gl == 0) flag_s[unit] = (uint8_t)flag;
  __syncthreads();

  auto lead_of = [&](int u) { return lead_s + ((u << s.glog) + gl) * V; };
  auto part = [&](float* to) {
    if (!on) return;
#pragma unroll
    for (int j = 0; j < V; ++j) to[tile * s.dim4 + k + j] = acc[j];
  };
  if (flag & kOpen) {  // acc holds the trailing part
    int v = unit + 1;
    for (; v < units; ++v) {
      const float* l = lead_of(v);
#pragma unroll
      for (int j = 0; j < V; ++j) acc[j] += l[j];
      if (flag_s[v] & kCloses) break;
    }
    if (v == units) {
      part(s.trail);
      if (chunk == 0 && gl == 0) s.open_row[tile] = s.number ? slot : cur;
    } else if (on) {
      finish_row<GT, V>(a, s.number ? slot : cur, k, acc);
    }
  }
  if (unit == 0 && (flag & (kCloses | kThrough))) {
    const float* l0 = lead_of(0);
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] = l0[j];
    for (int v = 1; v < units && !(flag_s[v - 1] & kCloses); ++v) {
      const float* l = lead_of(v);
#pragma unroll
      for (int j = 0; j < V; ++j) acc[j] += l[j];
    }
    part(s.lead);
  }
  if (threadIdx.x == 0 && chunk == 0) {
    int f = 0, v = 0;
    while (v < units && (flag_s[v] & kThrough)) ++v;
    if (v == units) f = kThrough;
    else if (flag_s[v] & kCloses) f = kCloses;
    for (v = units - 1; v > 0 && (flag_s[v] & kThrough); --v) {}
    if (flag_s[v] & kOpen) f |= kOpen;
    s.flags[tile] = (uint8_t)f;
  }
}

// Segments that span tiles: the CTA of the tile where one begins adds the parts of the tiles it crosses.
// 8 warps take consecutive eighths of the parts, and the eighths are added in order.
constexpr int kJoinCols = 128;
template <int GT>
__global__ void __launch_bounds__(kThreads) segment_join_kernel(const EmbedGradArgs a, const SumArgs s) {
  pdl_wait();
  pdl_trigger();
  constexpr int kWarps = kThreads / 32;
  __shared__ float4 part[kWarps][32];
  __shared__ int last_s;
  const int64_t b = blockIdx.x;
  if (!(s.flags[b] & kOpen)) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // the tile where the segment ends: the first one after b that it does not go through
  int64_t last = b + 1;
  for (;; last += kThreads) {
    if (threadIdx.x == 0) last_s = kThreads;
    __syncthreads();
    const int64_t t = last + threadIdx.x;
    if (t >= s.tiles || !(s.flags[t] & kThrough)) atomicMin(&last_s, (int)threadIdx.x);
    __syncthreads();
    const int at = last_s;
    __syncthreads();
    if (at < kThreads) {
      last += at;
      break;
    }
  }
  const int64_t m = last - b;  // parts after the first
  const int k = blockIdx.y * kJoinCols + lane * 4;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
  if (k < a.e.dim) {
    const int64_t j0 = m * warp / kWarps, j1 = m * (warp + 1) / kWarps;
    if (warp == 0) sum = *reinterpret_cast<const float4*>(s.trail + b * s.dim4 + k);
#pragma unroll 8
    for (int64_t j = j0; j < j1; ++j) {
      const float4 v = *reinterpret_cast<const float4*>(s.lead + (b + 1 + j) * s.dim4 + k);
      sum.x += v.x;
      sum.y += v.y;
      sum.z += v.z;
      sum.w += v.w;
    }
  }
  part[warp][lane] = sum;
  __syncthreads();
  if (warp != 0 || k >= a.e.dim) return;
  for (int w = 1; w < kWarps; ++w) {
    const float4 v = part[w][lane];
    sum.x += v.x;
    sum.y += v.y;
    sum.z += v.z;
    sum.w += v.w;
  }
  const uint32_t row = s.open_row[b];
  const float f[4] = {sum.x, sum.y, sum.z, sum.w};
  for (int j = 0; j < 4 && k + j < a.e.dim; ++j) {
    float v = f[j];
    finish_row<GT, 1>(a, row, k + j, &v);
  }
}

template <int GT>
__global__ void __launch_bounds__(kThreads)
    all_zero_kernel(typename Elem<GT>::type* grad, int64_t rows, int32_t dim, int64_t stride) {
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

// How the sums are cut up: 2^glog lanes a unit, per_unit pairs a unit, chunks of columns, tiles of units. Which pairs meet
// in a unit and in a tile decides the order of the sums, so it follows from n and dim alone: from the widest access that
// rows of dim values allow, whatever access a call's types, addresses and strides allow (v values; a narrower one takes
// more chunks of as many lanes: 1.57 million bf16 rows of 128 at odd addresses 388 us a call, 374 with a cut of their own,
// 199 where they are aligned).
struct Cut {
  int glog, per_unit, chunks;
  int64_t tiles;
};
constexpr int widest(int32_t dim) { return dim % 8 == 0 ? 8 : dim % 4 == 0 ? 4 : 1; }
// One CTA on each of the 152 SMs: longer units leave fewer parts to join and wait for ids less often (1.1 million ids of
// 1,342 rows of 64 bf16: 98 us of the call with 8 CTAs an SM wanted, 90 with 1, 2, 3 or 4; 498,000 fp32 rows: 82, 71).
// Units of 64 and 16 pairs at most for 1.57 million ids of 128: 215 and 224 us, of 32: 210.
constexpr int64_t kWantCtas = 152;
constexpr int64_t kZeroCtas = 1216;  // of zeros: 8 on each SM
Cut cut_of(int64_t n, int32_t dim, int v) {
  Cut c;
  const int lanes = (int)ceil_div(dim, widest(dim));
  c.glog = 0;
  while (c.glog < 5 && (1 << c.glog) < lanes) ++c.glog;
  const int units = kThreads >> c.glog, chunks = (int)ceil_div(lanes, 1 << c.glog);
  // the longest units that still give every SM work; a unit of one batch where there is too little
  c.per_unit = 32;
  while (c.per_unit > kBatch && ceil_div(n, (int64_t)units * c.per_unit) * chunks < kWantCtas) c.per_unit >>= 1;
  c.tiles = ceil_div(n, (int64_t)units * c.per_unit);
  c.chunks = (int)ceil_div(ceil_div(dim, v), 1 << c.glog);
  return c;
}

// The most tiles of any call of up to n ids, for a workspace that serves them all: units shorter than 32 pairs were chosen
// because units twice as long would leave fewer than kWantCtas CTAs.
int64_t most_tiles(int64_t n, int32_t dim) {
  const Cut c = cut_of(n, dim, widest(dim));
  const int64_t shortest = ceil_div(n, (int64_t)(kThreads >> c.glog) * kBatch);
  return std::max(c.tiles, std::min(shortest, 2 * (ceil_div(kWantCtas, c.chunks) - 1)));
}

struct Layout {  // byte offsets into the workspace; no offset and no size falls as n grows
  uint64_t key[2], pos[2], ids, counts, totals, heads, lead, trail, flags, open_row, end;
};
Layout layout_of(int64_t n, int32_t dim) {
  Layout l;
  uint64_t at = 0;
  auto take = [&](uint64_t bytes) {
    const uint64_t p = at;
    at += round256(bytes);
    return p;
  };
  for (int i = 0; i < 2; ++i) {
    l.key[i] = take((uint64_t)(n + kBatch) * 4);
    l.pos[i] = take((uint64_t)(n + kBatch) * 4);
  }
  l.ids = take((uint64_t)(n + kBatch) * 4);
  const int64_t sort_tiles = std::max(ceil_div(std::min(n, kFewIds), kSortThreads * kPairsFew),
                                      n > kFewIds ? ceil_div(n, kSortThreads * kPairs) : 0);
  l.counts = take((uint64_t)sort_tiles * kMaxBins * 4);
  l.totals = take(kMaxBins * 4);
  l.heads = take((uint64_t)ceil_div(n, kSegTile) * 4);
  const uint64_t tiles = (uint64_t)most_tiles(n, dim);
  const uint64_t dim4 = (uint64_t)ceil_div(dim, 4) * 4;
  l.lead = take(tiles * dim4 * 4);
  l.trail = take(tiles * dim4 * 4);
  l.flags = take(tiles);
  l.open_row = take(tiles * 4);
  l.end = at;
  return l;
}

// values that one access of a row may take: 8, 4 or 1
inline int vec_of(const void* p, int64_t stride, int32_t dim, int32_t type) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(p);
  const int size = type_bytes(type);
  if (at % 16 == 0 && stride * size % 16 == 0 && dim % 8 == 0) return 8;
  return at % (4 * size) == 0 && stride % 4 == 0 && dim % 4 == 0 ? 4 : 1;
}

// calls f(integral_constant<V>)
template <typename F>
cudaError_t with_vec(int v, F&& f) {
  if (v == 8) return f(std::integral_constant<int, 8>{});
  if (v == 4) return f(std::integral_constant<int, 4>{});
  return f(std::integral_constant<int, 1>{});
}

}  // namespace

cudaError_t launch_embed(const EmbedArgs& a, const void* W, int64_t row_stride, int32_t w_type, void* out,
                         int32_t out_type, cudaStream_t s) {
  const int vec = std::min(vec_of(W, row_stride, a.dim, w_type), vec_of(out, a.dim, a.dim, out_type));
  const int64_t units = a.T * a.n_cols * (a.dim / vec);
  const int64_t grid = ceil_div(units, kThreads * kFly);
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  const bool few = units < (int64_t)UINT32_MAX - kThreads * kFly;
  return with_type(w_type, [&](auto wt) {
    return with_type(out_type, [&](auto ot) {
      return with_vec(vec, [&](auto v) {
        using WE = typename Elem<wt()>::type;
        using OE = typename Elem<ot()>::type;
        auto go = [&](auto kern, auto n) {
          return launch_pdl(kern, dim3((unsigned)grid), dim3(kThreads), 0, s, a, (const WE*)W, row_stride, (OE*)out, n);
        };
        return few ? go(embed_kernel<wt(), ot(), v(), uint32_t>, (uint32_t)units)
                   : go(embed_kernel<wt(), ot(), v(), uint64_t>, (uint64_t)units);
      });
    });
  });
}

uint64_t embed_grad_workspace(int64_t n, int64_t, int32_t dim) { return n > 0 ? layout_of(n, dim).end : 0; }

cudaError_t launch_embed_grad(const EmbedGradArgs& a, void* workspace, cudaStream_t s) {
  const int64_t n = a.e.T * a.e.n_cols;
  const bool sparse = a.grad_rows != nullptr || a.count != nullptr;
  const bool zero = !sparse && !a.accumulate;
  if (n == 0) {
    if (sparse) return launch_pdl(no_segments_kernel, dim3(1), dim3(32), 0, s, a.count);
    return with_type(a.grad_type, [&](auto gt) {
      using G = typename Elem<gt()>::type;
      const int64_t grid = std::min<int64_t>(ceil_div(a.e.rows * a.e.dim, kThreads), 152 * 16);
      return launch_pdl(all_zero_kernel<gt()>, dim3((unsigned)grid), dim3(kThreads), 0, s, (G*)a.grad, a.e.rows,
                        a.e.dim, a.grad_stride);
    });
  }
  const Layout l = layout_of(n, a.e.dim);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  auto u32 = [&](uint64_t off) { return reinterpret_cast<uint32_t*>(ws + off); };
  cudaError_t e = cudaSuccess;
  int bits = 1;
  while (bits < 32 && ((uint64_t)a.e.rows >> bits) != 0) ++bits;  // `rows` itself is a key
  const int passes = (bits + kMaxBits - 1) / kMaxBits, width = (bits + passes - 1) / passes;
  const uint32_t *key, *pos, *ids;
  if (n <= kSmall) {
    e = launch_pdl(place_small_kernel, dim3((unsigned)ceil_div(n, kPlaced)), dim3(kThreads), 0, s, a.e, (int)n,
                   u32(l.key[0]), u32(l.pos[0]));
    if (e != cudaSuccess) return e;
    key = u32(l.key[0]);
    pos = u32(l.pos[0]);
  } else {
    const int pairs = pairs_of(n), tiles = (int)ceil_div(n, kSortThreads * pairs);
    const bool few = pairs == kPairsFew;
    for (int q = 0; q < passes; ++q) {
      SortPass p;
      p.key_in = u32(l.key[q & 1]);
      p.pos_in = q == 0 ? nullptr : u32(l.pos[q & 1]);
      p.key_out = u32(l.key[(q + 1) & 1]);
      p.pos_out = u32(l.pos[(q + 1) & 1]);
      p.counts = u32(l.counts);
      p.totals = u32(l.totals);
      p.n = n;
      p.tiles = tiles;
      p.shift = q * width;
      p.bits = std::min(width, 32 - q * width);
      auto count = few ? (q == 0 ? sort_count_kernel<true, kPairsFew> : sort_count_kernel<false, kPairsFew>)
                       : (q == 0 ? sort_count_kernel<true, kPairs> : sort_count_kernel<false, kPairs>);
      e = launch_pdl(count, dim3(tiles), dim3(kSortThreads), 0, s, a.e, p);
      if (e != cudaSuccess) return e;
      if (!few_counts(tiles, p.bits))
        e = launch_pdl(sort_scan_kernel, dim3((unsigned)ceil_div((int64_t)1 << p.bits, 32)), dim3(kScanThreads), 0, s, p);
      if (e != cudaSuccess) return e;
      auto scatter = few ? (q == 0 ? sort_scatter_kernel<true, kPairsFew> : sort_scatter_kernel<false, kPairsFew>)
                         : (q == 0 ? sort_scatter_kernel<true, kPairs> : sort_scatter_kernel<false, kPairs>);
      e = cudaFuncSetAttribute(scatter, cudaFuncAttributeMaxDynamicSharedMemorySize, scatter_smem(pairs));
      if (e != cudaSuccess) return e;
      e = launch_pdl(scatter, dim3(tiles), dim3(kSortThreads), scatter_smem(pairs), s, p);
      if (e != cudaSuccess) return e;
    }
    key = u32(l.key[passes & 1]);
    pos = u32(l.pos[passes & 1]);
    if (sparse && n > kNumbered) {
      const int seg_tiles = (int)ceil_div(n, kSegTile);
      uint32_t* heads = u32(l.heads);
      e = launch_pdl(head_count_kernel, dim3(seg_tiles), dim3(kThreads), 0, s, key, n, (uint32_t)a.e.rows, heads);
      if (e != cudaSuccess) return e;
      e = launch_pdl(segments_kernel, dim3(seg_tiles), dim3(kThreads), 0, s, key, n, (uint32_t)a.e.rows,
                     (const uint32_t*)heads, seg_tiles, u32(l.ids), a.grad_rows, a.count);
      if (e != cudaSuccess) return e;
    }
  }
  const bool number = sparse && n <= kNumbered;
  ids = sparse && !number ? u32(l.ids) : key;
  const int vec = std::min(vec_of(a.dout, a.dout_stride, a.e.dim, a.dout_type),
                           vec_of(a.grad, a.grad_stride, a.e.dim, a.grad_type));
  const Cut c = cut_of(n, a.e.dim, vec);
  SumArgs m;
  m.ids = ids;
  m.pos = pos;
  m.limit = sparse && !number ? kNone : (uint32_t)a.e.rows;
  m.number = number;
  m.n = n;
  m.glog = c.glog;
  m.per_unit = c.per_unit;
  m.chunks = c.chunks;
  m.tiles = c.tiles;
  m.lead = reinterpret_cast<float*>(ws + l.lead);
  m.trail = reinterpret_cast<float*>(ws + l.trail);
  m.dim4 = (int32_t)ceil_div(a.e.dim, 4) * 4;
  m.flags = ws + l.flags;
  m.open_row = u32(l.open_row);
  const int64_t row_bytes = (int64_t)a.e.dim * type_bytes(a.grad_type);
  // 128 KB a CTA, less where that would leave SMs without one
  const int64_t zero_bytes = std::max<int64_t>(4 << 10, std::min<int64_t>(128 << 10, a.e.rows * row_bytes / kZeroCtas));
  m.zero_rows = (int)std::max<int64_t>(1, std::min<int64_t>(kThreads, zero_bytes / row_bytes));
  const int64_t grid = c.tiles * c.chunks + (zero ? ceil_div(a.e.rows, m.zero_rows) : 0);
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  return with_type(a.grad_type, [&](auto gt) {
    cudaError_t r = with_type(a.dout_type, [&](auto dt) {
      return with_vec(vec, [&](auto v) {
        return launch_pdl(segment_sum_kernel<dt(), gt(), v()>, dim3((unsigned)grid), dim3(kThreads), 0, s, a, m);
      });
    });
    if (r != cudaSuccess || c.tiles == 1) return r;
    return launch_pdl(segment_join_kernel<gt()>, dim3((unsigned)c.tiles, (unsigned)ceil_div(a.e.dim, kJoinCols)),
                      dim3(kThreads), 0, s, a, m);
  });
}

}  // namespace engram
