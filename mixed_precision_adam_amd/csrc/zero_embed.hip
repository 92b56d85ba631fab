// zero_embed.hip -- token embedding and its table's gradient
// (include/zero_shard.h, "the ends of a model"), for CDNA4 (gfx950).
//
// Both stream HBM.  A lane works on units of 8 neighbouring elements:
// one 16-byte access in the 16-bit formats, two in fp32.  The addresses need
// no more alignment than their elements have (global accesses of 16 bytes may
// start anywhere), so ragged rows take the same path; only the last
// cols mod 8 elements of a row go one by one.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "zero_common.h"
#include "zero_units.h"

// Sums of products may fuse: nothing here is specified operation by operation.
#pragma clang fp contract(fast)

namespace {

using namespace zero_detail;

// ------------------------------------------------------------------ embedding, forward

constexpr int64_t kMaxGroups = int64_t(1) << 20;  // workgroups of one launch; they stride over what is left

// One workgroup copies `per` tokens' rows at a time, up to four units a thread,
// one after the other: what keeps loads in flight is the workgroups, not the
// thread.  Bound by HBM: 16384 rows of 4096 bf16 in 50.4 us a call (5.3 TB/s of a
// row read and one written a token; a copy between two buffers makes 4.7, here
// frequent words' rows come from the caches), 8 rows of 1600 in 6.8, which is the
// call's host time.
template <int TD, int OD>
__global__ __launch_bounds__(kBlock) void embed_forward_kernel(Rows table, int64_t first, const void* __restrict__ ids,
                                                               int id_bytes, float scale, Rows out, uint32_t per,
                                                               uint32_t units) {
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * per; t0 < out.rows; t0 += static_cast<int64_t>(gridDim.x) * per) {
    const uint32_t here = static_cast<uint32_t>(out.rows - t0 < per ? out.rows - t0 : per);
    for (uint32_t k = threadIdx.x; k < here * units; k += kBlock) {
      const uint32_t t = k / units, u = k - t * units;
      const uint32_t row = local_row(ids, id_bytes, t0 + t, first, table.rows);
      const int n = unit_size(out.cols, u);
      Unit<TD> w;
      w.clear();
      if (row != kNoRow) w.load(table.at<TD>(row, u * 8), n);
      Unit<OD> y;
#pragma unroll
      for (int i = 0; i < 8; ++i) y.set(i, w.get(i) * scale);
      y.store(out.at<OD>(t0 + t, u * 8), n);
    }
  }
}

// ------------------------------------------------------------------ embedding, the table's gradient
//
// dW[v] = scale · sum of dy[t] over the tokens of v.  Rows of dy are read once
// and rows of dW written once; everything else is small.  A row of dW belongs
// to one wavefront (one column tile of 512 at a time), which adds its tokens'
// rows in the order of the text: no atomics on sums, so no order of arrival.
// Measured, calls behind one another: 301 tokens added to 50257x1600 bf16 7.9 us
// (one launch), 8192 tokens and every row written 81 us (2.3 TB/s of rows),
// 32769 tokens of 5120 fp16 added to an fp32 half table 143 us (3.5 TB/s).

constexpr int kTileCols = 512;  // 64 lanes of one unit
constexpr int kFillRows = 64;   // rows of dW that one workgroup looks over for rows without tokens

// A finished sum of one row's unit into dW.
template <int GD>
__device__ __forceinline__ void put_row(const Rows& dw, uint32_t row, int64_t col, int n, const float* acc, float scale,
                                        bool accumulate) {
  void* at = dw.at<GD>(row, col);
  Unit<GD> old, sum;
  old.clear();
  if (accumulate) old.load(at, n);
#pragma unroll
  for (int i = 0; i < 8; ++i) sum.set(i, old.get(i) + acc[i] * scale);
  sum.store(at, n);
}

// Zeros for the rows of [row0, row0 + kFillRows) whose bit in `met` is not set.
template <int GD>
__device__ __forceinline__ void fill_rows(const Rows& dw, int64_t row0, uint64_t met) {
  Unit<GD> zero;
  zero.clear();
  const int units = static_cast<int>((dw.cols + 7) / 8);
  for (int r = threadIdx.x >> 6; r < kFillRows; r += kBlock / 64) {
    if (row0 + r >= dw.rows || ((met >> r) & 1u)) continue;
    for (int u = threadIdx.x & 63; u < units; u += 64)
      zero.store(dw.at<GD>(row0 + r, static_cast<int64_t>(u) * 8), unit_size(dw.cols, u));
  }
}

// Up to kFew tokens: no sort, one launch where the sorted form has four to seven
// (its counts, a pass for every 9 bits of the row, the sums, the join).  Both
// forms measured at the same sizes, this one before the sorted one: 512 tokens
// added to 50257x1600 bf16 7.4 and 37.8 us, with every row written 35.3 and 58.0;
// 512 onto 32000x4096 8.2 and 38.4; 512 onto 1000x256 7.4 and 33.2; at 65 tokens
// 7.5 and 35.5.  The border lies on the safe side of where they meet: at 1024
// tokens this form takes 9.6 and 17.3 us (1600 and 4096 columns) against 39.1 and
// 44.2, growing with tokens times columns.  A workgroup belongs to one token and column
// tile; unless an earlier token has the same row it finds the others by
// comparing, its four wavefronts add a quarter of them each, and the quarters
// are joined in order.  Workgroups from `sums` on fill the rows without tokens.
constexpr int kFew = 512;

template <int YD, int GD>
__global__ __launch_bounds__(kBlock) void embed_grad_few_kernel(const void* __restrict__ ids, int id_bytes,
                                                                int64_t first, Rows dy, float scale, Rows dw,
                                                                int accumulate, uint32_t tiles, uint32_t sums) {
  __shared__ uint32_t key[kFew];
  __shared__ uint16_t list[kFew];
  __shared__ float part[3][kTileCols];
  __shared__ uint32_t met[2];
  __shared__ uint32_t count;
  const int tokens = static_cast<int>(dy.rows);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (blockIdx.x >= sums) {
    const int64_t row0 = static_cast<int64_t>(blockIdx.x - sums) * kFillRows;
    if (threadIdx.x < 2) met[threadIdx.x] = 0;
    __syncthreads();
    for (int t = threadIdx.x; t < tokens; t += kBlock) {
      const uint32_t row = local_row(ids, id_bytes, t, first, dw.rows);
      if (row != kNoRow && row >= row0 && row < row0 + kFillRows) {
        const uint32_t r = static_cast<uint32_t>(row - row0);
        atomicOr(&met[r >> 5], 1u << (r & 31));
      }
    }
    __syncthreads();
    fill_rows<GD>(dw, row0, met[0] | static_cast<uint64_t>(met[1]) << 32);
    return;
  }
  const int me = static_cast<int>(blockIdx.x / tiles);
  const int64_t col = static_cast<int64_t>(blockIdx.x % tiles) * kTileCols + lane * 8;
  const uint32_t mine = local_row(ids, id_bytes, me, first, dw.rows);
  if (mine == kNoRow) return;
  int earlier = 0;
  for (int t = threadIdx.x; t < tokens; t += kBlock) {
    key[t] = local_row(ids, id_bytes, t, first, dw.rows);
    earlier |= t < me && key[t] == mine;
  }
  if (__syncthreads_or(earlier)) return;
  if (wave == 0) {
    uint32_t n = 0;
    for (int t0 = me & ~63; t0 < tokens; t0 += 64) {
      const bool same = t0 + lane < tokens && t0 + lane >= me && key[t0 + lane] == mine;
      const uint64_t hits = __ballot(same);
      if (same) list[n + __popcll(hits & ((1ull << lane) - 1))] = static_cast<uint16_t>(t0 + lane);
      n += __popcll(hits);
    }
    if (lane == 0) count = n;
  }
  __syncthreads();
  const int n = unit_size(dy.cols, col / 8);
  const int per = static_cast<int>((count + 3) / 4);
  const int lo = wave * per, hi = min(lo + per, static_cast<int>(count));
  float acc[8] = {};
  if (n > 0) {
    for (int k = lo; k < hi; k += 4) {
      Unit<YD> y[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        y[j].clear();
        if (k + j < hi) y[j].load(dy.at<YD>(list[k + j], col), n);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += k + j < hi ? y[j].get(i) : 0.0f;
    }
  }
  if (wave > 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) part[wave - 1][i * 64 + lane] = acc[i];
  }
  __syncthreads();
  if (wave == 0 && n > 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = ((acc[i] + part[0][i * 64 + lane]) + part[1][i * 64 + lane]) + part[2][i * 64 + lane];
    put_row<GD>(dw, mine, col, n, acc, scale, accumulate != 0);
  }
}

// More tokens: a stable radix sort of (row, token) by row, 9 bits or fewer a
// pass, least digit first.  The tokens are split into at most kSortBlocks
// equal parts of four wavefronts each; a pass ranks a wavefront's tokens by
// comparing digits with ballots.  counts[pass][part][digit] comes from the
// pass before (the first one's from sort_count_kernel), with integer atomics,
// whose order does not show.
constexpr int kSortBlocks = 64, kMaxDigits = 512;

struct Sort {
  uint32_t tokens, per_block, per_wave;  // per_block = 4·per_wave
  int blocks, passes, digit_bits;
};

inline Sort sort_shape(int64_t tokens, int64_t rows) {
  Sort s{};
  s.tokens = static_cast<uint32_t>(tokens);
  s.per_wave = static_cast<uint32_t>(ceil_div(ceil_div(tokens, kSortBlocks * 4), 64) * 64);
  s.per_block = 4 * s.per_wave;
  s.blocks = static_cast<int>(ceil_div(tokens, s.per_block));
  int bits = 1;
  while ((rows >> bits) != 0) ++bits;  // rows itself stands for "no row" and sorts last
  s.passes = (bits + 8) / 9;
  s.digit_bits = (bits + s.passes - 1) / s.passes;
  return s;
}

__global__ __launch_bounds__(kBlock) void sort_count_kernel(const void* __restrict__ ids, int id_bytes, int64_t first,
                                                            int64_t rows, Sort s, uint32_t* __restrict__ counts,
                                                            uint32_t* __restrict__ met, int64_t met_words) {
  __shared__ uint32_t hist[kMaxDigits];
  const uint32_t digits = 1u << s.digit_bits;
  for (uint32_t d = threadIdx.x; d < digits; d += kBlock) hist[d] = 0;
  __syncthreads();
  const uint32_t lo = blockIdx.x * s.per_block;
  const uint32_t hi = s.tokens - lo < s.per_block ? s.tokens : lo + s.per_block;
  for (uint32_t t = lo + threadIdx.x; t < hi; t += kBlock) {
    const uint32_t row = local_row(ids, id_bytes, t, first, rows);
    atomicAdd(&hist[(row == kNoRow ? static_cast<uint32_t>(rows) : row) & (digits - 1)], 1u);
  }
  __syncthreads();
  for (uint32_t d = threadIdx.x; d < digits; d += kBlock) {
    counts[static_cast<size_t>(blockIdx.x) * kMaxDigits + d] = hist[d];
    for (int p = 1; p < s.passes; ++p) counts[(static_cast<size_t>(p) * kSortBlocks + blockIdx.x) * kMaxDigits + d] = 0;
  }
  for (int64_t w = static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x; w < met_words; w += static_cast<int64_t>(gridDim.x) * kBlock)
    met[w] = 0;
}

// One pass.  The first takes the rows from the ids and marks them in `met`.
__global__ __launch_bounds__(kBlock) void sort_pass_kernel(const void* __restrict__ ids, int id_bytes, int64_t first,
                                                           int64_t rows, Sort s, int pass,
                                                           const uint2* __restrict__ from, uint2* __restrict__ to,
                                                           uint32_t* __restrict__ counts, uint32_t* __restrict__ met) {
  __shared__ uint32_t at[4][kMaxDigits];  // a wavefront's digits first counted, then where its next one goes
  __shared__ uint32_t wave_sum[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t digits = 1u << s.digit_bits;
  const int shift = pass * s.digit_bits;
  const uint32_t lo = min(blockIdx.x * s.per_block + wave * s.per_wave, s.tokens);
  const uint32_t hi = s.tokens - lo < s.per_wave ? s.tokens : lo + s.per_wave;
  auto item = [&](uint32_t t) {
    if (pass > 0) return from[t];
    const uint32_t row = local_row(ids, id_bytes, t, first, rows);
    return make_uint2(row == kNoRow ? static_cast<uint32_t>(rows) : row, t);
  };
  for (uint32_t k = threadIdx.x; k < 4 * kMaxDigits; k += kBlock) at[k / kMaxDigits][k % kMaxDigits] = 0;
  __syncthreads();
  for (uint32_t t = lo + lane; t < hi; t += 64) atomicAdd(&at[wave][(item(t).x >> shift) & (digits - 1)], 1u);
  __syncthreads();
  // Two neighbouring digits a thread: their counts in the parts before this one and in all parts.
  const uint32_t* mine = counts + static_cast<size_t>(pass) * kSortBlocks * kMaxDigits;
  uint32_t before[2] = {0, 0}, all[2] = {0, 0};
  if (2 * threadIdx.x < digits) {
    for (int b = 0; b < s.blocks; ++b) {
      const uint2 c = *reinterpret_cast<const uint2*>(mine + static_cast<size_t>(b) * kMaxDigits + 2 * threadIdx.x);
      all[0] += c.x;
      all[1] += c.y;
      before[0] += b < static_cast<int>(blockIdx.x) ? c.x : 0u;
      before[1] += b < static_cast<int>(blockIdx.x) ? c.y : 0u;
    }
  }
  // Exclusive sum over the digits.
  uint32_t sum = all[0] + all[1];
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const uint32_t up = __shfl_up(sum, off, 64);
    sum += lane >= off ? up : 0u;
  }
  if (lane == 63) wave_sum[wave] = sum;
  __syncthreads();
  uint32_t base = sum - all[0] - all[1];
  for (int w = 0; w < wave; ++w) base += wave_sum[w];
  if (2 * threadIdx.x < digits) {
    uint32_t start[2] = {base + before[0], base + all[0] + before[1]};
    for (int w = 0; w < 4; ++w) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t c = at[w][2 * threadIdx.x + k];
        at[w][2 * threadIdx.x + k] = start[k];
        start[k] += c;
      }
    }
  }
  __syncthreads();
  uint32_t* next = counts + static_cast<size_t>(pass + 1) * kSortBlocks * kMaxDigits;
  // Only this wavefront reads and writes its digits' places from here on, in LDS, which keeps a wavefront's accesses in
  // order: what is needed is that the compiler keeps it too, once the places are read and once they are moved on.
  const auto in_order = [] {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  };
  for (uint32_t t0 = lo; t0 < hi; t0 += 64) {
    const bool some = t0 + lane < hi;
    const uint2 kv = some ? item(t0 + lane) : make_uint2(0, 0);
    const uint32_t digit = (kv.x >> shift) & (digits - 1);
    uint64_t same = __ballot(some);
    for (int b = 0; b < s.digit_bits; ++b) {
      const uint64_t ones = __ballot((digit >> b) & 1u);
      same &= (digit >> b) & 1u ? ones : ~ones;
    }
    const uint32_t rank = __popcll(same & ((1ull << lane) - 1)), many = __popcll(same);
    const uint32_t start = some ? at[wave][digit] : 0u;
    in_order();
    if (some) {
      if (rank == 0) at[wave][digit] = start + many;
      const uint32_t p = start + rank;
      to[p] = kv;
      if (pass == 0 && kv.x < rows && !((met[kv.x >> 5] >> (kv.x & 31)) & 1u)) atomicOr(&met[kv.x >> 5], 1u << (kv.x & 31));
      if (pass + 1 < s.passes)
        atomicAdd(&next[static_cast<size_t>(p / s.per_block) * kMaxDigits + ((kv.x >> (shift + s.digit_bits)) & (digits - 1))], 1u);
    }
    in_order();
  }
}

// The sums.  A wavefront takes `per` sorted tokens (a chunk) and one column
// tile.  A row whose tokens all lie in the chunk is written at once; the sums
// of a row that reaches in from the chunk before go to edge 0 of the chunk,
// those of one that begins here and goes on to edge 1, and
// embed_grad_join_kernel adds them up.
struct Chunks {
  uint32_t tokens, per, chunks, tiles;
  int64_t edge_cols;  // elements of one edge
};

template <int YD, int GD>
__global__ __launch_bounds__(kBlock) void embed_grad_kernel(const uint2* __restrict__ sorted, Chunks c, Rows dy,
                                                            float scale, Rows dw, int accumulate,
                                                            float* __restrict__ edges,
                                                            const uint32_t* __restrict__ met, uint32_t sums) {
  if (blockIdx.x >= sums) {
    const int64_t row0 = static_cast<int64_t>(blockIdx.x - sums) * kFillRows;
    const uint64_t bits = met[row0 / 32] | static_cast<uint64_t>(met[row0 / 32 + 1]) << 32;
    fill_rows<GD>(dw, row0, bits);
    return;
  }
  const int lane = threadIdx.x & 63;
  const uint32_t item = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
  const uint32_t chunk = item / c.tiles;
  if (chunk >= c.chunks) return;
  const int64_t col = static_cast<int64_t>(item % c.tiles) * kTileCols + lane * 8;
  const int n = unit_size(dy.cols, col / 8);
  const uint32_t none = static_cast<uint32_t>(dw.rows);
  const uint32_t lo = chunk * c.per, hi = c.tokens - lo < c.per ? c.tokens : lo + c.per;
  const uint32_t reaches_in = lo > 0 ? sorted[lo - 1].x : none;
  const uint32_t goes_on = hi < c.tokens ? sorted[hi].x : none;
  float acc[8] = {};
  uint32_t row = sorted[lo].x;
  bool head = row == reaches_in;
  auto leave = [&](bool last) {  // the row's tokens in this chunk are all added
    if (row < none && n > 0) {
      if (head || (last && row == goes_on)) {
        float* edge = edges + (static_cast<int64_t>(chunk) * 2 + (head ? 0 : 1)) * c.edge_cols + col;
#pragma unroll
        for (int q = 0; q < 2; ++q) *reinterpret_cast<f32x4*>(edge + 4 * q) = f32x4{acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]};
      } else {
        put_row<GD>(dw, row, col, n, acc, scale, accumulate != 0);
      }
    }
  };
  constexpr int kDeep = 8;
  for (uint32_t p0 = lo; p0 < hi; p0 += 64) {
    const uint2 kv = p0 + lane < hi ? sorted[p0 + lane] : make_uint2(none, 0);
    const int here = static_cast<int>(hi - p0 < 64 ? hi - p0 : 64);
    for (int j0 = 0; j0 < here; j0 += kDeep) {
      Unit<YD> y[kDeep];
#pragma unroll
      for (int j = 0; j < kDeep; ++j) {
        y[j].clear();
        const uint32_t r = __builtin_amdgcn_readlane(kv.x, (j0 + j) & 63), t = __builtin_amdgcn_readlane(kv.y, (j0 + j) & 63);
        if (j0 + j < here && r < none && n > 0) y[j].load(dy.at<YD>(t, col), n);
      }
#pragma unroll
      for (int j = 0; j < kDeep; ++j) {
        if (j0 + j < here) {
          const uint32_t r = __builtin_amdgcn_readlane(kv.x, (j0 + j) & 63);
          if (r != row) {
            leave(false);
            row = r;
            head = false;
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[i] += y[j].get(i);
        }
      }
    }
  }
  leave(true);
}

// Rows that reach over chunks: a workgroup for each chunk and column tile, at
// work only where such a row begins in the chunk.  Its wavefronts add a
// quarter of the row's edges each.
template <int GD>
__global__ __launch_bounds__(kBlock) void embed_grad_join_kernel(const uint2* __restrict__ sorted, Chunks c,
                                                                 int64_t cols, float scale, Rows dw, int accumulate,
                                                                 const float* __restrict__ edges) {
  __shared__ float part[3][kTileCols];
  const uint32_t chunk = blockIdx.x / c.tiles;
  const uint32_t lo = chunk * c.per, hi = lo + c.per;
  if (hi >= c.tokens) return;
  const uint32_t row = sorted[hi].x;
  if (row >= dw.rows || sorted[hi - 1].x != row) return;              // no row goes on
  if (sorted[lo].x == row && lo > 0 && sorted[lo - 1].x == row) return;  // it began before
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  // The first token past the row's: 64 probes at a time.
  uint32_t from = hi + 1, to = c.tokens;
  while (from < to) {
    const uint32_t step = (to - from + 63) / 64;
    const uint64_t probe = static_cast<uint64_t>(from) + static_cast<uint64_t>(lane + 1) * step - 1;
    const bool same = probe < to && sorted[probe].x == row;
    const uint32_t k = __popcll(__ballot(same));
    from += k * step;
    to = to - from < step - 1 ? to : from + step - 1;
  }
  const uint32_t last = (from - 1) / c.per;  // the chunk of the row's last token
  const int many = static_cast<int>(last - chunk) + 1, per = (many + 3) / 4;
  const int64_t col = static_cast<int64_t>(blockIdx.x % c.tiles) * kTileCols + lane * 8;
  const int n = unit_size(cols, col / 8);
  float acc[8] = {};
  if (n > 0) {
    const int end = min(wave * per + per, many);
#pragma unroll 4
    for (int k = wave * per; k < end; ++k) {
      const float* edge = edges + (static_cast<int64_t>(chunk + k) * 2 + (k == 0 ? 1 : 0)) * c.edge_cols + col;
      const f32x4 a = *reinterpret_cast<const f32x4*>(edge), b = *reinterpret_cast<const f32x4*>(edge + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[i] += a[i];
        acc[4 + i] += b[i];
      }
    }
  }
  if (wave > 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) part[wave - 1][i * 64 + lane] = acc[i];
  }
  __syncthreads();
  if (wave == 0 && n > 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = ((acc[i] + part[0][i * 64 + lane]) + part[1][i * 64 + lane]) + part[2][i * 64 + lane];
    put_row<GD>(dw, row, col, n, acc, scale, accumulate != 0);
  }
}

constexpr int64_t kMostChunks = 8192;

struct EmbedSpace {  // parts of the workspace, as byte offsets
  size_t a, b, counts, met, edges, bytes;
  Chunks c;
};

// Words of the bits that mark the rows with tokens: two for each kFillRows.
constexpr int64_t met_words(int64_t rows) { return ceil_div(rows, kFillRows) * 2; }

inline EmbedSpace embed_space(int64_t tokens, int64_t rows, int64_t cols) {
  EmbedSpace w{};
  if (tokens <= kFew) {
    w.bytes = 256;
    return w;
  }
  w.c.tokens = static_cast<uint32_t>(tokens);
  w.c.per = 32;  // past 2^18 tokens longer chunks: the edges stay a small part of the rows
  while (ceil_div(tokens, w.c.per) > kMostChunks) w.c.per *= 2;
  w.c.chunks = static_cast<uint32_t>(ceil_div(tokens, w.c.per));
  w.c.tiles = static_cast<uint32_t>(ceil_div(cols, kTileCols));
  w.c.edge_cols = static_cast<int64_t>(w.c.tiles) * kTileCols;
  w.a = 0;
  w.b = up256(8 * static_cast<size_t>(tokens));
  w.counts = 2 * w.b;
  w.edges = w.counts + static_cast<size_t>(4) * kSortBlocks * kMaxDigits * 4;
  // As many edges as any smaller number of tokens has (longer chunks make fewer).
  const int64_t most = std::min<int64_t>(ceil_div(tokens, 32), kMostChunks);
  w.met = w.edges + up256(static_cast<size_t>(most) * 2 * w.c.edge_cols * 4);
  w.bytes = w.met + up256(static_cast<size_t>(met_words(rows)) * 4);
  return w;
}

}  // namespace

extern "C" {

int zero_embed_forward(const zero_rows* table, int64_t first_row, const void* ids_dev, int32_t id_bytes, double scale,
                       const zero_rows* out, void* stream) {
  const char* fn = "zero_embed_forward";
  int rc = rows_ok(fn, "table", table);
  if (rc == ZERO_OK) rc = rows_ok(fn, "out", out);
  if (rc == ZERO_OK) rc = ids_ok(fn, ids_dev, id_bytes, out->rows);
  if (rc != ZERO_OK) return rc;
  if (table->cols != out->cols) return fail(ZERO_ERR_INVALID, "%s: table and out differ in cols", fn);
  if (first_row < 0) return fail(ZERO_ERR_INVALID, "%s: first_row < 0", fn);
  if (!finite32(scale)) return fail(ZERO_ERR_INVALID, "%s: scale is not finite in fp32", fn);
  if (out->rows == 0) return ZERO_OK;
  const int64_t units = ceil_div(out->cols, 8);
  // Four units a thread once that leaves workgroups for every CU; before, one token a workgroup.
  const int64_t per = std::max<int64_t>(1, std::min<int64_t>(4 * kBlock / units, out->rows / 1024));
  const int64_t groups = std::min(ceil_div(out->rows, per), kMaxGroups);
  return with_dtype(table->dt, [&](auto td) {
    return with_dtype(out->dt, [&](auto od) {
      hipLaunchKernelGGL((embed_forward_kernel<td.value, od.value>), dim3(static_cast<unsigned>(groups)), dim3(kBlock),
                         0, static_cast<hipStream_t>(stream), device_rows(table), first_row, ids_dev, id_bytes,
                         static_cast<float>(scale), device_rows(out), static_cast<uint32_t>(per),
                         static_cast<uint32_t>(units));
      return launch_status(fn);
    });
  });
}

size_t zero_embed_grad_workspace_bytes(int64_t n_tokens, int64_t table_rows, int64_t cols) {
  if (!sizes_ok(n_tokens, cols) || !sizes_ok(table_rows, 1)) return 0;
  return embed_space(n_tokens, table_rows, cols).bytes;
}

int zero_embed_grad(const void* ids_dev, int32_t id_bytes, int64_t first_row, const zero_rows* out_grad, double scale,
                    const zero_rows* table_grad, int32_t accumulate, void* ws_dev, size_t ws_bytes, void* stream) {
  const char* fn = "zero_embed_grad";
  int rc = rows_ok(fn, "out_grad", out_grad);
  if (rc == ZERO_OK) rc = rows_ok(fn, "table_grad", table_grad);
  if (rc == ZERO_OK) rc = ids_ok(fn, ids_dev, id_bytes, out_grad->rows);
  if (rc != ZERO_OK) return rc;
  if (table_grad->cols != out_grad->cols) return fail(ZERO_ERR_INVALID, "%s: out_grad and table_grad differ in cols", fn);
  if (first_row < 0) return fail(ZERO_ERR_INVALID, "%s: first_row < 0", fn);
  if (!finite32(scale)) return fail(ZERO_ERR_INVALID, "%s: scale is not finite in fp32", fn);
  const int64_t tokens = out_grad->rows, rows = table_grad->rows, cols = out_grad->cols;
  const EmbedSpace w = embed_space(tokens, rows, cols);
  if (!ws_dev || !aligned16(ws_dev) || ws_bytes < w.bytes)
    return fail(ZERO_ERR_INVALID, "%s: workspace of %zu bytes, %zu needed, 16-byte aligned", fn, ws_dev ? ws_bytes : 0,
                w.bytes);
  if (rows == 0 || (tokens == 0 && accumulate)) return ZERO_OK;
  const int64_t fills = accumulate ? 0 : ceil_div(rows, kFillRows);
  const int64_t tiles = ceil_div(cols, kTileCols);
  const int64_t sums = tokens <= kFew ? tokens * tiles : ceil_div(static_cast<int64_t>(w.c.chunks) * tiles, 4);
  if (tiles * std::max<int64_t>(w.c.chunks, 1) >= kLaunchGroups || sums + fills >= kLaunchGroups)
    return fail(ZERO_ERR_INVALID, "%s: too many rows or columns for one launch", fn);
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const dim3 grid(static_cast<unsigned>(sums + fills)), block(kBlock);
  const float by = static_cast<float>(scale);
  if (tokens <= kFew) {
    return with_dtype(out_grad->dt, [&](auto yd) {
      return with_dtype(table_grad->dt, [&](auto gd) {
        hipLaunchKernelGGL((embed_grad_few_kernel<yd.value, gd.value>), grid, block, 0, st, ids_dev, id_bytes,
                           first_row, device_rows(out_grad), by, device_rows(table_grad), accumulate != 0 ? 1 : 0,
                           static_cast<uint32_t>(tiles), static_cast<uint32_t>(sums));
        return launch_status(fn);
      });
    });
  }
  char* ws = static_cast<char*>(ws_dev);
  uint2* buffers[2] = {reinterpret_cast<uint2*>(ws + w.a), reinterpret_cast<uint2*>(ws + w.b)};
  uint32_t* counts = reinterpret_cast<uint32_t*>(ws + w.counts);
  uint32_t* met = reinterpret_cast<uint32_t*>(ws + w.met);
  float* edges = reinterpret_cast<float*>(ws + w.edges);
  const Sort s = sort_shape(tokens, rows);
  hipLaunchKernelGGL(sort_count_kernel, dim3(s.blocks), block, 0, st, ids_dev, id_bytes, first_row, rows, s, counts,
                     met, met_words(rows));
  for (int p = 0; p < s.passes; ++p)
    hipLaunchKernelGGL(sort_pass_kernel, dim3(s.blocks), block, 0, st, ids_dev, id_bytes, first_row, rows, s, p,
                       buffers[(p + 1) & 1], buffers[p & 1], counts, met);
  const uint2* sorted = buffers[(s.passes + 1) & 1];
  rc = launch_status(fn);
  if (rc != ZERO_OK) return rc;
  return with_dtype(table_grad->dt, [&](auto gd) {
    with_dtype(out_grad->dt, [&](auto yd) {
      hipLaunchKernelGGL((embed_grad_kernel<yd.value, gd.value>), grid, block, 0, st, sorted, w.c, device_rows(out_grad),
                         by, device_rows(table_grad), accumulate != 0 ? 1 : 0, edges, met, static_cast<uint32_t>(sums));
      return 0;
    });
    hipLaunchKernelGGL((embed_grad_join_kernel<gd.value>), dim3(w.c.chunks * w.c.tiles), block, 0, st, sorted, w.c,
                       cols, by, device_rows(table_grad), accumulate != 0 ? 1 : 0, edges);
    return launch_status(fn);
  });
}

}  // extern "C"
