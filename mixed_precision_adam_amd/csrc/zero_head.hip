// zero_head.hip -- softmax cross entropy of a linear head over a large
// vocabulary and its gradients (include/zero_shard.h, "the ends of a model"),
// for CDNA4 (gfx950).
//
// With x of T rows and the table W of V rows, both of d columns:
//   z = x Wᵀ,  lse_t = log sum_v exp z_tv,  loss_t = lse_t - z_t,label
//   G = softmax(z) - onehot,  dx = f G W,  dW = f Gᵀ x,  f = scale·loss scale/count
// Three products of 2TVd operations each; everything else is small.  Tokens go
// through in blocks whose scores fit the last-level cache.  The first product's
// epilogue takes the maximum and the sum of exponentials of every piece of 64
// words from the fp32 scores, and keeps each score as 16 bits: how far it is
// below its piece's maximum, in 2048ths of an octave.  That is off by at most
// 2^-12 octaves (1.7e-4 of the exponential), finer than the rounding that the
// factor of the other two products needs, so the scores are computed once and
// never held in 32 bits.  softmax_kernel turns the codes into G, rounded once.
// The label's word is left out of maxima and sums: with R the logarithm of the
// sum over the others, loss_t = log(1 + exp(R - z_t,label)), which keeps its
// digits where the label is all but certain, and so does expm1(-loss_t), the
// label's factor in G.  Taken as lse_t - z_t,label both would end at the last
// digit of a score (1e-6 at a score of 20).
//
// Measured (calls behind one another): 4096 tokens x 50257 words x 1600 columns
// bf16 2.59 ms, 4096 x 32000 x 4096 fp16 3.06 to 3.17 ms; in a trace, where a
// pass takes 2.74 and 3.34, the three products are 87 and 91% of it, at 690 to 945
// and 950 to 1200 TFLOP/s.  Losses alone of 33 tokens over 50257 x 1600 take 56.6
// us; reading the table at a large copy's rate would take 34.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "zero_common.h"
#include "zero_units.h"

#pragma clang fp contract(fast)

namespace {

using namespace zero_detail;

// ------------------------------------------------------------------ the product
//
// C[m][n] = sum_k A[m][k] B[n][k], both operands with k contiguous.  A
// workgroup of 8 wavefronts (2 by 4, 128x64 each) makes a tile of 256x256 in
// steps of 64 along k.  The steps go through two buffers of 64 KiB each in LDS,
// filled by loads that write LDS directly; 16-byte chunk c of row r lies at
// place c ^ (r & 7) of its row, so eight neighbouring rows' chunks fall into
// eight different bank groups.  The operands are swapped in the matrix
// instruction (B's rows first): a lane then holds four neighbouring n of one m.

constexpr int kTileM = 256, kTileN = 256, kStep = 64, kThreads = 512;
constexpr int kBlocksM = 8, kBlocksN = 4;  // 16x16 blocks of a wavefront

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// An operand: rows of k elements, `ld` elements from one to the next.
struct Operand {
  const char* data;
  int64_t rows, ld;
};

struct Product {
  Operand a, b;
  int64_t k;        // multiple of kStep
  int32_t tiles_m, tiles_n;
  int32_t splits, steps;  // k-steps of each split but perhaps the last
};

template <int DT>
__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (DT == ZERO_BF16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  } else {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
}

// The memory of a tile's rows: loads past its end read zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t tile_rows(const Operand& o, int64_t row0, int64_t k) {
  const int64_t rows = o.rows - row0 < 256 ? o.rows - row0 : 256;
  const int64_t bytes = rows > 0 ? ((rows - 1) * o.ld + k) * 2 : 0;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(o.data + row0 * o.ld * 2), 0, static_cast<int>(bytes), 0x00020000);
}

typedef __attribute__((address_space(3))) void* lds_ptr;

// One step of one operand into LDS: 256 rows of 128 bytes.
__device__ __forceinline__ void stage(__amdgpu_buffer_rsrc_t rows, char* lds, const uint32_t (&at)[4], int step) {
  const int wave = threadIdx.x >> 6;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rows, (lds_ptr)(lds + j * 8192 + wave * 1024), 16, at[j], step * 128, 0, 0);
}

// A wavefront's loads into LDS have landed before it meets the others: staged
// data is there for all of them behind this.  The barrier alone promises that
// only as far as the compiler counts these loads among what it has to wait for.
__device__ __forceinline__ void meet() {
  __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0); the other counters are left as they are
  __syncthreads();
}

template <int DT>
struct Tile {
  f32x4 acc[kBlocksM][kBlocksN];

  // The element that acc[i][j][q] is of, within the tile.
  __device__ __forceinline__ static int m(int i) { return (threadIdx.x >> 8) * 128 + i * 16 + (threadIdx.x & 15); }
  __device__ __forceinline__ static int n(int j) { return ((threadIdx.x >> 6) & 3) * 64 + j * 16 + ((threadIdx.x >> 4) & 3) * 4; }

  __device__ __forceinline__ void add_step(const char* a, const char* b) {
    const int lane = threadIdx.x & 63;
    const uint32_t row_a = ((threadIdx.x >> 8) * 128 + (lane & 15)) * 128;
    const uint32_t row_b = (((threadIdx.x >> 6) & 3) * 64 + (lane & 15)) * 128;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t chunk = ((h * 4 + (lane >> 4)) ^ (lane & 7)) * 16;
      u32x4 fa[kBlocksM], fb[kBlocksN];
#pragma unroll
      for (int i = 0; i < kBlocksM; ++i) fa[i] = *reinterpret_cast<const u32x4*>(a + row_a + i * 2048 + chunk);
#pragma unroll
      for (int j = 0; j < kBlocksN; ++j) fb[j] = *reinterpret_cast<const u32x4*>(b + row_b + j * 2048 + chunk);
#pragma unroll
      for (int i = 0; i < kBlocksM; ++i)
#pragma unroll
        for (int j = 0; j < kBlocksN; ++j) acc[i][j] = mfma<DT>(fb[j], fa[i], acc[i][j]);
    }
  }

  __device__ __forceinline__ void compute(const Product& p, int tile_m, int tile_n, int split) {
    __shared__ __attribute__((aligned(16))) char a0[32768], a1[32768], b0[32768], b1[32768];
#pragma unroll
    for (int i = 0; i < kBlocksM; ++i)
#pragma unroll
      for (int j = 0; j < kBlocksN; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
    const __amdgpu_buffer_rsrc_t ra = tile_rows(p.a, static_cast<int64_t>(tile_m) * kTileM, p.k);
    const __amdgpu_buffer_rsrc_t rb = tile_rows(p.b, static_cast<int64_t>(tile_n) * kTileN, p.k);
    uint32_t va[4], vb[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t row = j * 64 + threadIdx.x / 8, chunk = (threadIdx.x & 7) ^ (row & 7);
      va[j] = row * static_cast<uint32_t>(p.a.ld) * 2 + chunk * 16;
      vb[j] = row * static_cast<uint32_t>(p.b.ld) * 2 + chunk * 16;
    }
    const int all = static_cast<int>(p.k / kStep);
    const int lo = split * p.steps, hi = min(lo + p.steps, all);
    if (lo >= hi) return;
    stage(ra, a0, va, lo);
    stage(rb, b0, vb, lo);
#pragma unroll 1
    for (int s = lo; s < hi; s += 2) {
      meet();  // step s has arrived, and nobody reads the other buffers any more
      if (s + 1 < hi) {
        stage(ra, a1, va, s + 1);
        stage(rb, b1, vb, s + 1);
      }
      add_step(a0, b0);
      meet();
      if (s + 1 < hi) {
        if (s + 2 < hi) {
          stage(ra, a0, va, s + 2);
          stage(rb, b0, vb, s + 2);
        }
        add_step(a1, b1);
      }
    }
  }
};

// Which tile and split workgroup b works on.  Workgroups go to the eight XCDs
// in turn: each XCD takes a run of neighbouring tiles, in columns of 8 rows of
// tiles, so that the tiles in flight on one L2 share their operands.
struct Place {
  int m, n, split;
};
__device__ __forceinline__ Place place_of(const Product& p) {
  const int tiles = p.tiles_m * p.tiles_n, n = tiles * p.splits;
  int b = blockIdx.x;
  const int whole = n / 8 * 8;
  if (b < whole) b = b % 8 * (n / 8) + b / 8;
  Place w;
  w.split = b / tiles;
  b -= w.split * tiles;
  const int group = b / (8 * p.tiles_n), first = group * 8, rows = min(p.tiles_m - first, 8);
  b -= group * 8 * p.tiles_n;
  w.m = first + b % rows;
  w.n = b / rows;
  return w;
}

// ------------------------------------------------------------------ scores

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr int kPiece = 64;             // words whose scores share a maximum
constexpr float kCodeSteps = 2048.0f;  // of an octave
constexpr uint32_t kNoCode = 65535;

struct Block {             // a block of tokens
  int64_t first;           // its first token
  int32_t tokens, padded;  // padded: rows of the codes, a multiple of 256
};

// The scores of a tile into codes (nullptr: none), and for each row and piece
// the maximum and the sum of 2^(score - maximum) over the words that are not
// the token's label; all in octaves.
template <int DT>
__global__ __launch_bounds__(kThreads) void scores_kernel(Product p, Block blk, int64_t vocab,
                                                          const void* __restrict__ labels, int label_bytes,
                                                          uint16_t* __restrict__ codes, int64_t code_stride,
                                                          float2* __restrict__ pieces, int64_t n_pieces,
                                                          float* __restrict__ label_score) {
  const Place w = place_of(p);
  Tile<DT> t;
  t.compute(p, w.m, w.n, 0);
  const int n_wave = w.n * kTileN + ((threadIdx.x >> 6) & 3) * kPiece;  // the wavefront's piece
  const int group = (threadIdx.x >> 4) & 3;
#pragma unroll
  for (int i = 0; i < kBlocksM; ++i) {
    const int m = w.m * kTileM + t.m(i);
    const uint32_t label = m < blk.tokens ? local_row(labels, label_bytes, blk.first + m, 0, vocab) : kNoRow;
    float z[kBlocksN][4], top = -INFINITY;
#pragma unroll
    for (int j = 0; j < kBlocksN; ++j) {
      const int n = w.n * kTileN + t.n(j);
#pragma unroll
      for (int q = 0; q < 4; ++q) z[j][q] = n + q < vocab ? t.acc[i][j][q] * kLog2e : -INFINITY;
      const uint32_t q_label = label - static_cast<uint32_t>(n);
      if (q_label < 4) {
        label_score[m] = q_label == 0 ? z[j][0] : q_label == 1 ? z[j][1] : q_label == 2 ? z[j][2] : z[j][3];
#pragma unroll
        for (int q = 0; q < 4; ++q) z[j][q] = q_label == q ? -INFINITY : z[j][q];
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) top = fmaxf(top, z[j][q]);
    }
    top = fmaxf(top, __shfl_xor(top, 16, 64));
    top = fmaxf(top, __shfl_xor(top, 32, 64));
    const float base = top == -INFINITY ? 0.0f : top;  // nothing but -inf: the sum is 0
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < kBlocksN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) sum += __builtin_amdgcn_exp2f(z[j][q] - base);
    sum += __shfl_xor(sum, 16, 64);
    sum += __shfl_xor(sum, 32, 64);
    if (m >= blk.tokens) continue;
    if (group == 0 && n_wave < vocab) pieces[static_cast<int64_t>(m) * n_pieces + n_wave / kPiece] = make_float2(top, sum);
    if (codes) {
#pragma unroll
      for (int j = 0; j < kBlocksN; ++j) {
        uint32_t c[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) c[q] = static_cast<uint32_t>(fminf((base - z[j][q]) * kCodeSteps + 0.5f, 65535.0f));
        *reinterpret_cast<u32x2*>(codes + m * code_stride + w.n * kTileN + t.n(j)) = u32x2{c[0] | c[1] << 16, c[2] | c[3] << 16};
      }
    }
  }
}

// A wavefront for each token: its logarithm of the sum, and its loss.
__global__ __launch_bounds__(kBlock) void lse_kernel(Block blk, int64_t vocab, const void* __restrict__ labels,
                                                     int label_bytes, const float2* __restrict__ pieces,
                                                     int64_t n_pieces, const float* __restrict__ label_score,
                                                     float* __restrict__ lse, float* __restrict__ losses) {
  const int m = blockIdx.x * (kBlock / 64) + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (m >= blk.tokens) return;
  const float2* mine = pieces + static_cast<int64_t>(m) * n_pieces;
  float top = -INFINITY, sum = 0.0f;
  for (int64_t k = lane; k < n_pieces; k += 64) {
    const float2 v = mine[k];
    const float higher = fmaxf(top, v.x), base = higher == -INFINITY ? 0.0f : higher;
    sum = sum * __builtin_amdgcn_exp2f(top - base) + v.y * __builtin_amdgcn_exp2f(v.x - base);
    top = higher;
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    const float t2 = __shfl_xor(top, off, 64), s2 = __shfl_xor(sum, off, 64);
    const float higher = fmaxf(top, t2), base = higher == -INFINITY ? 0.0f : higher;
    const float a = sum * __builtin_amdgcn_exp2f(top - base), b = s2 * __builtin_amdgcn_exp2f(t2 - base);
    sum = a + b;
    top = higher;
  }
  if (lane == 0) {
    const bool counts = local_row(labels, label_bytes, blk.first + m, 0, vocab) != kNoRow;
    float loss = 0.0f, l = 0.0f;  // l is not read for a token that does not count
    if (counts) {
      const float rest = top + __builtin_amdgcn_logf(sum), own = label_score[m], above = rest - own;
      const float more = log1pf(__builtin_amdgcn_exp2f(-fabsf(above)));  // what the smaller of the two adds to the larger
      loss = fmaxf(above, 0.0f) * kLn2 + more;
      l = fmaxf(rest, own) + more * kLog2e;
      // fmaxf passes over a NaN, and above is -inf for an own score of +inf
      if (above != above || own == INFINITY) loss = l = __builtin_nanf("");
    }
    lse[m] = l;
    losses[blk.first + m] = loss;
  }
}

// ------------------------------------------------------------------ the factor of the gradients' products

// 64 tokens by 64 words: codes -> G in place, and Gᵀ.  fp16 holds G times 2^15:
// a probability of 1/V would fall among its subnormals otherwise.
constexpr float kHalfScale = 32768.0f;

template <int DT>
__global__ __launch_bounds__(kBlock) void softmax_kernel(Block blk, int64_t vocab, const void* __restrict__ labels,
                                                         int label_bytes, uint16_t* __restrict__ codes,
                                                         int64_t code_stride, const float2* __restrict__ pieces,
                                                         int64_t n_pieces, const float* __restrict__ losses,
                                                         const float* __restrict__ lse, uint16_t* __restrict__ turned,
                                                         int64_t turned_stride) {
  __shared__ uint16_t tile[64][64 + 2];
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 64;
  const int m0 = blockIdx.y * 64;
#pragma unroll
  for (int pass = 0; pass < 2; ++pass) {
    const int r = pass * 32 + (threadIdx.x >> 3), c = (threadIdx.x & 7) * 8, m = m0 + r;
    const uint32_t label = m < blk.tokens ? local_row(labels, label_bytes, blk.first + m, 0, vocab) : kNoRow;
    uint16_t* at = codes + m * code_stride + n0 + c;
    Unit<DT> g;
    g.clear();
    if (label != kNoRow && n0 < vocab) {
      const u32x4 q = *reinterpret_cast<const u32x4*>(at);
      const float l = lse[m], base = pieces[static_cast<int64_t>(m) * n_pieces + blockIdx.x].x - l;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t code = i & 1 ? q[i / 2] >> 16 : q[i / 2] & 0xFFFFu;
        float p = code == kNoCode ? l - l : __builtin_amdgcn_exp2f(base - static_cast<float>(code) * (1.0f / kCodeSteps));
        if (n0 + c + i == label) p = expm1f(-losses[blk.first + m]);
        if (n0 + c + i >= vocab) p = 0.0f;
        g.set(i, DT == ZERO_FP16 ? p * kHalfScale : p);
      }
    }
    *reinterpret_cast<u32x4*>(at) = u32x4{g.w[0], g.w[1], g.w[2], g.w[3]};
#pragma unroll
    for (int i = 0; i < 8; ++i) tile[c + i][r] = static_cast<uint16_t>(g.w[i / 2] >> (i & 1 ? 16 : 0));
  }
  __syncthreads();
#pragma unroll
  for (int pass = 0; pass < 2; ++pass) {
    const int r = pass * 32 + (threadIdx.x >> 3), c = (threadIdx.x & 7) * 8;
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const uint32_t*>(&tile[r][c + 2 * i]);
    *reinterpret_cast<u32x4*>(turned + (n0 + r) * turned_stride + m0 + c) = v;
  }
}

// to[c][r] = from[r][c] for a tile of 64x64 a workgroup; zeros past from's
// rows, and, with labels, for tokens that do not count.
template <int DT>
__global__ __launch_bounds__(kBlock) void turn_kernel(Rows from, const void* __restrict__ labels, int label_bytes,
                                                      int64_t first, int64_t vocab, uint16_t* __restrict__ to,
                                                      int64_t to_stride) {
  __shared__ uint16_t tile[64][64 + 2];
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * 64, c0 = static_cast<int64_t>(blockIdx.y) * 64;
#pragma unroll
  for (int pass = 0; pass < 2; ++pass) {
    const int64_t r = pass * 32 + (threadIdx.x >> 3), c = (threadIdx.x & 7) * 8;
    const int n = unit_size(from.cols, (c0 + c) / 8);
    Unit<DT> v;
    v.clear();
    const bool counts = r0 + r < from.rows && (!labels || local_row(labels, label_bytes, first + r0 + r, 0, vocab) != kNoRow);
    if (counts && n > 0) v.load(from.at<DT>(r0 + r, c0 + c), n);
#pragma unroll
    for (int i = 0; i < 8; ++i) tile[c + i][r] = static_cast<uint16_t>(v.w[i / 2] >> (i & 1 ? 16 : 0));
  }
  __syncthreads();
#pragma unroll
  for (int pass = 0; pass < 2; ++pass) {
    const int64_t r = pass * 32 + (threadIdx.x >> 3), c = (threadIdx.x & 7) * 8;
    if (c0 + r >= from.cols) continue;
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const uint32_t*>(&tile[r][c + 2 * i]);
    *reinterpret_cast<u32x4*>(to + (c0 + r) * to_stride + r0 + c) = v;
  }
}

// Rows onto 16-byte lines, with zeros behind them up to to_stride.
template <int DT>
__global__ __launch_bounds__(kBlock) void align_kernel(Rows from, uint16_t* __restrict__ to, int64_t to_stride) {
  const uint32_t units = static_cast<uint32_t>(to_stride / 8);
  for (int64_t r = blockIdx.x; r < from.rows; r += gridDim.x) {
    for (uint32_t u = threadIdx.x; u < units; u += kBlock) {
      const int n = unit_size(from.cols, u);
      Unit<DT> v;
      v.clear();
      if (n > 0) v.load(from.at<DT>(r, static_cast<int64_t>(u) * 8), n);
      *reinterpret_cast<u32x4*>(to + r * to_stride + u * 8) = u32x4{v.w[0], v.w[1], v.w[2], v.w[3]};
    }
  }
}

// ------------------------------------------------------------------ the gradients

// One split of G W into fp32 partial rows.
template <int DT>
__global__ __launch_bounds__(kThreads) void x_grad_kernel(Product p, int32_t tokens, int64_t cols,
                                                          float* __restrict__ parts, int64_t part_stride,
                                                          int64_t part_size) {
  const Place w = place_of(p);
  Tile<DT> t;
  t.compute(p, w.m, w.n, w.split);
#pragma unroll
  for (int i = 0; i < kBlocksM; ++i) {
    const int64_t m = static_cast<int64_t>(w.m) * kTileM + t.m(i);
    if (m >= tokens) continue;
#pragma unroll
    for (int j = 0; j < kBlocksN; ++j) {
      const int64_t n = static_cast<int64_t>(w.n) * kTileN + t.n(j);
      if (n < cols) *reinterpret_cast<f32x4*>(parts + w.split * part_size + m * part_stride + n) = t.acc[i][j];
    }
  }
}

// The splits' sum, in order, times the factor.
template <int DT>
__global__ __launch_bounds__(kBlock) void x_grad_join_kernel(Block blk, int64_t vocab, const void* __restrict__ labels,
                                                             int label_bytes, const float* __restrict__ parts,
                                                             int64_t part_stride, int64_t part_size, int splits,
                                                             const float* __restrict__ factor, Rows dx) {
  const uint32_t units = static_cast<uint32_t>((dx.cols + 7) / 8);
  const float f = *factor * (DT == ZERO_FP16 ? 1.0f / kHalfScale : 1.0f);
  for (int m = blockIdx.x; m < blk.tokens; m += gridDim.x) {
    const bool counts = local_row(labels, label_bytes, blk.first + m, 0, vocab) != kNoRow;
    for (uint32_t u = threadIdx.x; u < units; u += kBlock) {
      float sum[8] = {};
      if (counts) {
#pragma unroll 4
        for (int s = 0; s < splits; ++s) {
          const float* at = parts + s * part_size + m * part_stride + u * 8;
          const f32x4 a = *reinterpret_cast<const f32x4*>(at), b = *reinterpret_cast<const f32x4*>(at + 4);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            sum[i] += a[i];
            sum[4 + i] += b[i];
          }
        }
      }
      Unit<DT> out;
#pragma unroll
      for (int i = 0; i < 8; ++i) out.set(i, counts ? sum[i] * f : 0.0f);
      out.store(dx.at<DT>(blk.first + m, static_cast<int64_t>(u) * 8), unit_size(dx.cols, u));
    }
  }
}

// Gᵀ x of one block of tokens, added to what the blocks before left in `sums`
// (nullptr for the first); the last block writes the gradient.
template <int DT>
__global__ __launch_bounds__(kThreads) void table_grad_kernel(Product p, float* __restrict__ sums, int64_t sum_stride,
                                                              int first, int last, const float* __restrict__ factor,
                                                              int accumulate, Rows dw) {
  const Place w = place_of(p);
  Tile<DT> t;
  t.compute(p, w.m, w.n, 0);
  const float f = *factor * (DT == ZERO_FP16 ? 1.0f / kHalfScale : 1.0f);
#pragma unroll
  for (int i = 0; i < kBlocksM; ++i) {
    const int64_t m = static_cast<int64_t>(w.m) * kTileM + t.m(i);
    if (m >= dw.rows) continue;
#pragma unroll
    for (int j = 0; j < kBlocksN; ++j) {
      const int64_t n = static_cast<int64_t>(w.n) * kTileN + t.n(j);
      if (n >= dw.cols) continue;
      f32x4 v = t.acc[i][j];
      f32x4* at = reinterpret_cast<f32x4*>(sums + m * sum_stride + n);
      if (!first) v += *at;
      if (!last) {
        *at = v;
        continue;
      }
      uint16_t* out = static_cast<uint16_t*>(dw.at<DT>(m, n));
      const int some = dw.cols - n < 4 ? static_cast<int>(dw.cols - n) : 4;
      uint32_t h[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float old = accumulate && q < some ? widen<DT>(out[q]) : 0.0f;
        h[q] = narrow<DT>(old + v[q] * f);
      }
      typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
      if (some == 4) {
        *reinterpret_cast<u32x2_any*>(out) = u32x2_any{h[0] | h[1] << 16, h[2] | h[3] << 16};
      } else {
#pragma unroll
        for (int q = 0; q < 3; ++q)
          if (q < some) out[q] = static_cast<uint16_t>(h[q]);
      }
    }
  }
}

// ------------------------------------------------------------------ counts and the mean

constexpr int kOneGroup = 1024;

// How many tokens count, and the gradients' factor.
__global__ __launch_bounds__(kOneGroup) void count_kernel(const void* __restrict__ labels, int label_bytes,
                                                          int64_t tokens, int64_t vocab, double scale,
                                                          const zero_step_state* __restrict__ state,
                                                          int64_t* __restrict__ count, float* __restrict__ factor) {
  double many = 0.0;  // exact up to 2^53
  uint32_t none = 0;
  for (int64_t t = threadIdx.x; t < tokens; t += kOneGroup) many += local_row(labels, label_bytes, t, 0, vocab) != kNoRow ? 1.0 : 0.0;
  block_reduce<kOneGroup>(many, none);
  if (threadIdx.x == 0) {
    *count = static_cast<int64_t>(many);
    *factor = static_cast<float>(scale * (state ? state->loss_scale : 1.0) / (many > 0.0 ? many : 1.0));
  }
}

__global__ __launch_bounds__(kOneGroup) void mean_kernel(const float* __restrict__ losses, int64_t tokens,
                                                         const int64_t* __restrict__ count, float* __restrict__ loss) {
  double sum = 0.0;
  uint32_t none = 0;
  for (int64_t t = threadIdx.x; t < tokens; t += kOneGroup) sum += static_cast<double>(losses[t]);
  block_reduce<kOneGroup>(sum, none);
  if (threadIdx.x == 0) *loss = static_cast<float>(sum / static_cast<double>(*count > 0 ? *count : 1));
}

// ------------------------------------------------------------------ sizes

constexpr int64_t kMostVocab = int64_t(1) << 22, kMostCols = int64_t(1) << 16;  // 32-bit offsets within a tile's rows
// The codes of a block of tokens: as many as fit the 256 MB last-level cache.
// Measured with 2^27, 2^28, 2^29 and 2^30 (bf16, workspaces without the table's
// copy): 4096 tokens x 50257 x 1600 2.96, 2.62, 2.41 and 2.41 ms in 0.78, 1.10,
// 1.10 and 1.10 GiB, 16384 tokens 11.1, 10.5, 10.1 and 10.4 in 0.78, 1.10, 1.62
// and 2.72; 4096 x 32000 x 4096 3.32, 3.06, 3.06 and 3.08, 8192 tokens 6.61, 6.22,
// 6.11 and 6.10.  Half costs 6 to 13%; twice gains 2 to 8% where it spares a block,
// whose sums of the table's gradient go through memory, for half as much memory
// again once there are tokens to fill it.
constexpr int64_t kCodeBytes = int64_t(1) << 28;
// What a block holds for each element of its hidden rows: copies on 16-byte
// lines and turned, 2 bytes each, and 4 of the sums before they are rounded.
// Over a small vocabulary these are what grows with a block, not the codes:
// 1 GiB for them, 26,112 tokens at 5120 columns.  Measured with 2^29, 2^30 and
// 2^31 over 500 words of 4096 columns: 65,536 tokens 3.32, 3.13 and 3.14 ms.
constexpr int64_t kRowBytes = int64_t(1) << 30;
constexpr int64_t kCus = 256, kMostParts = 512;

constexpr int64_t round_up(int64_t n, int64_t to) { return ceil_div(n, to) * to; }

struct Space {
  int64_t k, vocab_padded, n_pieces, block, part_stride;
  size_t factor, label_score, lse, pieces, x, table, codes, turned, x_turned, table_turned, parts, sums, bytes;
};

// How many parts the sum over the vocabulary is split into: the number that
// takes the fewest rounds of steps over the CUs.  A workgroup costs about 12
// steps besides its own (filling its buffers, writing its part).
int split_count(int64_t tiles, int64_t steps) {
  int best = 1;
  int64_t least = std::numeric_limits<int64_t>::max();
  for (int64_t s = 1; s <= std::min(std::max<int64_t>(kMostParts / tiles, 1), steps); ++s) {
    const int64_t cost = ceil_div(tiles * s, kCus) * (ceil_div(steps, s) + 12);
    if (cost < least) {
      least = cost;
      best = static_cast<int>(s);
    }
  }
  return best;
}

// With or without room for the table's rows on 16-byte lines, which comes last: a
// call whose table is read where it is fits a workspace made without it.
Space space_of(int64_t tokens, int64_t vocab, int64_t cols, bool gradients, bool table_copy) {
  Space s{};
  s.k = round_up(cols, kStep);
  s.vocab_padded = round_up(vocab, kTileN);
  s.n_pieces = ceil_div(vocab, kPiece);
  const int64_t fit = std::min(kCodeBytes / (2 * s.vocab_padded), kRowBytes / (8 * s.k));
  const int64_t most = std::max<int64_t>(fit / kTileM, 1) * kTileM;
  s.block = std::min(most, std::max<int64_t>(round_up(tokens, kTileM), kTileM));
  s.part_stride = round_up(cols, 8);
  size_t at = 0;
  const auto part = [&](int64_t bytes) {
    const size_t here = at;
    at += up256(static_cast<size_t>(bytes));
    return here;
  };
  s.factor = part(4);
  s.label_score = part(4 * s.block);
  s.lse = part(4 * s.block);
  s.pieces = part(8 * s.block * s.n_pieces);
  s.x = part(2 * s.block * s.k);
  if (gradients) {
    s.codes = part(2 * s.block * s.vocab_padded);
    s.turned = part(2 * s.block * s.vocab_padded);
    s.x_turned = part(2 * s.block * cols);
    s.table_turned = part(2 * s.vocab_padded * cols);
    // The most that a block of as many tokens or fewer splits into.
    int64_t rows = 0;
    for (int64_t m = kTileM; m <= s.block; m += kTileM) {
      const int splits = split_count(m / kTileM * ceil_div(cols, kTileN), s.vocab_padded / kStep);
      rows = std::max(rows, splits * std::min(m, std::max<int64_t>(tokens, 1)));
    }
    s.parts = part(4 * rows * s.part_stride);
    s.sums = part(tokens > s.block ? 4 * vocab * s.part_stride : 0);
  }
  s.table = part(table_copy ? 2 * vocab * s.k : 0);
  s.bytes = at;
  return s;
}

Product product(Operand a, Operand b, int64_t k, int splits) {
  Product p{};
  p.a = a;
  p.b = b;
  p.k = k;
  p.tiles_m = static_cast<int32_t>(ceil_div(a.rows, kTileM));
  p.tiles_n = static_cast<int32_t>(ceil_div(b.rows, kTileN));
  p.splits = splits;
  p.steps = static_cast<int32_t>(ceil_div(k / kStep, splits));
  return p;
}

// Whether the products can read rows where they are: whole steps of k on
// 16-byte lines, and offsets within a tile in 32 bits.
bool direct(const zero_rows* r) {
  return r->cols % kStep == 0 && r->stride % 8 == 0 && aligned16(r->data) && r->stride < (int64_t(1) << 22);
}

bool head_sizes_ok(int64_t tokens, int64_t vocab, int64_t cols) {
  return sizes_ok(tokens, cols) && vocab >= 1 && vocab <= kMostVocab && cols <= kMostCols &&
         round_up(vocab, kTileN) / 64 * ceil_div(cols, 64) < kLaunchGroups;
}

struct Call {
  const char* fn;
  const zero_rows *x, *table;
  const void* labels;
  int32_t label_bytes;
  float *losses, *loss;
  int64_t* count;
  void* ws;
  size_t ws_bytes;
  hipStream_t stream;
  // gradients only
  double scale;
  const zero_step_state* state;
  const zero_rows *x_grad, *table_grad;
  int32_t accumulate;
};

int check(const Call& c, bool gradients) {
  const char* fn = c.fn;
  int rc = rows_ok(fn, "x", c.x);
  if (rc == ZERO_OK) rc = rows_ok(fn, "table", c.table);
  if (rc == ZERO_OK) rc = ids_ok(fn, c.labels, c.label_bytes, c.x->rows);
  if (rc != ZERO_OK) return rc;
  if (!dtype_ok(c.x->dt) || c.table->dt != c.x->dt)
    return fail(ZERO_ERR_INVALID, "%s: x and table must have one 16-bit dtype, got %d and %d", fn, c.x->dt, c.table->dt);
  if (c.table->cols != c.x->cols) return fail(ZERO_ERR_INVALID, "%s: x and table differ in cols", fn);
  if (!head_sizes_ok(c.x->rows, c.table->rows, c.x->cols))
    return fail(ZERO_ERR_INVALID, "%s: a table of %lld rows of %lld: out of range", fn,
                static_cast<long long>(c.table->rows), static_cast<long long>(c.table->cols));
  if ((c.x->rows > 0 && !c.losses) || !c.loss || !c.count) return fail(ZERO_ERR_INVALID, "%s: NULL output", fn);
  if (unaligned(c.losses, 4) || unaligned(c.loss, 4) || unaligned(c.count, 8))
    return fail(ZERO_ERR_INVALID, "%s: misaligned output", fn);
  if (gradients) {
    for (int k = 0; k < 2; ++k) {
      const zero_rows *g = k == 0 ? c.x_grad : c.table_grad, *of = k == 0 ? c.x : c.table;
      const char* name = k == 0 ? "x_grad" : "table_grad";
      rc = rows_ok(fn, name, g);
      if (rc != ZERO_OK) return rc;
      if (g->rows != of->rows || g->cols != of->cols || g->dt != of->dt)
        return fail(ZERO_ERR_INVALID, "%s: %s has another shape or dtype than what it is of", fn, name);
    }
    if (!finite32(c.scale)) return fail(ZERO_ERR_INVALID, "%s: scale is not finite in fp32", fn);
    if (!aligned8(c.state)) return fail(ZERO_ERR_INVALID, "%s: misaligned step state", fn);
  }
  const Space s = space_of(c.x->rows, c.table->rows, c.x->cols, gradients, !direct(c.table));
  if (!c.ws || (reinterpret_cast<uintptr_t>(c.ws) & 255) != 0 || c.ws_bytes < s.bytes)
    return fail(ZERO_ERR_INVALID, "%s: workspace of %zu bytes, %zu needed, 256-byte aligned", fn, c.ws ? c.ws_bytes : 0,
                s.bytes);
  return ZERO_OK;
}

#define LAUNCH(kernel, groups, threads, ...) \
  hipLaunchKernelGGL(kernel, groups, dim3(threads), 0, c.stream, __VA_ARGS__)

template <int DT>
int run(const Call& c, bool gradients) {
  const int64_t tokens = c.x->rows, vocab = c.table->rows, cols = c.x->cols;
  const Space s = space_of(tokens, vocab, cols, gradients, !direct(c.table));
  char* ws = static_cast<char*>(c.ws);
  float* factor = reinterpret_cast<float*>(ws + s.factor);
  float* label_score = reinterpret_cast<float*>(ws + s.label_score);
  float* lse = reinterpret_cast<float*>(ws + s.lse);
  float2* pieces = reinterpret_cast<float2*>(ws + s.pieces);
  uint16_t* codes = gradients ? reinterpret_cast<uint16_t*>(ws + s.codes) : nullptr;
  uint16_t* turned = reinterpret_cast<uint16_t*>(ws + s.turned);
  uint16_t* x_turned = reinterpret_cast<uint16_t*>(ws + s.x_turned);
  uint16_t* table_turned = reinterpret_cast<uint16_t*>(ws + s.table_turned);
  float* parts = reinterpret_cast<float*>(ws + s.parts);
  float* sums = reinterpret_cast<float*>(ws + s.sums);
  const auto groups = [](int64_t n) { return dim3(static_cast<unsigned>(std::min<int64_t>(n, int64_t(1) << 20))); };

  LAUNCH(count_kernel, dim3(1), kOneGroup, c.labels, c.label_bytes, tokens, vocab, c.scale, c.state, c.count, factor);
  Operand table{static_cast<const char*>(c.table->data), vocab, c.table->stride};
  if (!direct(c.table)) {
    table = Operand{ws + s.table, vocab, s.k};
    LAUNCH((align_kernel<DT>), groups(vocab), kBlock, device_rows(c.table), reinterpret_cast<uint16_t*>(ws + s.table), s.k);
  }
  if (gradients)
    LAUNCH((turn_kernel<DT>), dim3(s.vocab_padded / 64, ceil_div(cols, 64)), kBlock, device_rows(c.table), nullptr, 4,
           int64_t(0), vocab, table_turned, s.vocab_padded);
  for (int64_t first = 0; first < std::max<int64_t>(tokens, 1); first += s.block) {
    Block blk;
    blk.first = first;
    blk.tokens = static_cast<int32_t>(std::min(s.block, tokens - first));
    blk.padded = static_cast<int32_t>(std::max<int64_t>(round_up(blk.tokens, kTileM), kTileM));
    zero_rows here = *c.x;
    here.data = here.data ? static_cast<char*>(here.data) + first * here.stride * 2 : nullptr;
    here.rows = blk.tokens;
    Operand x{static_cast<const char*>(here.data), blk.tokens, here.stride};
    if (blk.tokens > 0) {
      if (!direct(&here)) {
        x = Operand{ws + s.x, blk.tokens, s.k};
        LAUNCH((align_kernel<DT>), groups(blk.tokens), kBlock, device_rows(&here), reinterpret_cast<uint16_t*>(ws + s.x), s.k);
      }
      const Product p = product(x, table, s.k, 1);
      LAUNCH((scores_kernel<DT>), dim3(static_cast<unsigned>(p.tiles_m * p.tiles_n)), kThreads, p, blk, vocab, c.labels,
             c.label_bytes, codes, s.vocab_padded, pieces, s.n_pieces, label_score);
      LAUNCH(lse_kernel, groups(ceil_div(blk.tokens, kBlock / 64)), kBlock, blk, vocab, c.labels, c.label_bytes, pieces,
             s.n_pieces, label_score, lse, c.losses);
    }
    if (!gradients) continue;
    LAUNCH((softmax_kernel<DT>), dim3(s.vocab_padded / 64, blk.padded / 64), kBlock, blk, vocab, c.labels, c.label_bytes,
           codes, s.vocab_padded, pieces, s.n_pieces, c.losses, lse, turned, static_cast<int64_t>(blk.padded));
    LAUNCH((turn_kernel<DT>), dim3(blk.padded / 64, ceil_div(cols, 64)), kBlock, device_rows(&here), c.labels,
           c.label_bytes, first, vocab, x_turned, static_cast<int64_t>(blk.padded));
    if (blk.tokens > 0) {
      const int64_t tiles = ceil_div(blk.tokens, kTileM) * ceil_div(cols, kTileN);
      const Product p = product(Operand{reinterpret_cast<char*>(codes), blk.tokens, s.vocab_padded},
                                Operand{reinterpret_cast<char*>(table_turned), cols, s.vocab_padded}, s.vocab_padded,
                                split_count(tiles, s.vocab_padded / kStep));
      const int64_t part_size = blk.tokens * s.part_stride;
      LAUNCH((x_grad_kernel<DT>), dim3(static_cast<unsigned>(tiles * p.splits)), kThreads, p, blk.tokens, cols, parts,
             s.part_stride, part_size);
      LAUNCH((x_grad_join_kernel<DT>), groups(blk.tokens), kBlock, blk, vocab, c.labels, c.label_bytes, parts,
             s.part_stride, part_size, p.splits, factor, device_rows(c.x_grad));
    }
    const Product p = product(Operand{reinterpret_cast<char*>(turned), vocab, blk.padded},
                              Operand{reinterpret_cast<char*>(x_turned), cols, blk.padded}, blk.padded, 1);
    LAUNCH((table_grad_kernel<DT>), dim3(static_cast<unsigned>(p.tiles_m * p.tiles_n)), kThreads, p, sums, s.part_stride,
           first == 0 ? 1 : 0, first + s.block >= tokens ? 1 : 0, factor, c.accumulate, device_rows(c.table_grad));
  }
  LAUNCH(mean_kernel, dim3(1), kOneGroup, c.losses, tokens, c.count, c.loss);
  return launch_status(c.fn);
}

int head(const Call& c, bool gradients) {
  const int rc = check(c, gradients);
  if (rc != ZERO_OK) return rc;
  return c.x->dt == ZERO_BF16 ? run<ZERO_BF16>(c, gradients) : run<ZERO_FP16>(c, gradients);
}

}  // namespace

extern "C" {

size_t zero_loss_head_workspace_bytes(int64_t n_tokens, int64_t vocab, int64_t cols, int32_t gradients) {
  if (!head_sizes_ok(n_tokens, vocab, cols)) return 0;
  return space_of(n_tokens, vocab, cols, gradients != 0, true).bytes;
}

size_t zero_loss_head_workspace_bytes_for(int64_t n_tokens, const zero_rows* table, int32_t gradients) {
  if (rows_ok("zero_loss_head_workspace_bytes_for", "table", table) != ZERO_OK || !dtype_ok(table->dt) ||
      !head_sizes_ok(n_tokens, table->rows, table->cols))
    return 0;
  return space_of(n_tokens, table->rows, table->cols, gradients != 0, !direct(table)).bytes;
}

int zero_loss_head(const zero_rows* x, const zero_rows* table, const void* labels_dev, int32_t label_bytes,
                   float* losses_dev, float* loss_dev, int64_t* count_dev, void* ws_dev, size_t ws_bytes,
                   void* stream) {
  Call c{"zero_loss_head", x,      table,    labels_dev, label_bytes, losses_dev, loss_dev,
         count_dev,        ws_dev, ws_bytes, static_cast<hipStream_t>(stream), 1.0, nullptr, nullptr, nullptr, 0};
  return head(c, false);
}

int zero_loss_head_grad(const zero_rows* x, const zero_rows* table, const void* labels_dev, int32_t label_bytes,
                        double scale, const zero_step_state* state_dev, float* losses_dev, float* loss_dev,
                        int64_t* count_dev, const zero_rows* x_grad, const zero_rows* table_grad, int32_t accumulate,
                        void* ws_dev, size_t ws_bytes, void* stream) {
  Call c{"zero_loss_head_grad", x,      table,    labels_dev, label_bytes, losses_dev, loss_dev,
         count_dev,             ws_dev, ws_bytes, static_cast<hipStream_t>(stream), scale, state_dev, x_grad,
         table_grad,            accumulate != 0 ? 1 : 0};
  return head(c, true);
}

}  // extern "C"
