// zero_norm.hip -- layer norm, with or without the mean, and its backward pass
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

// ------------------------------------------------------------------ layer norm
//
// A row lives in the registers of one wavefront, or of the four of a
// workgroup where it is longer than 1024: NU units a lane.  The forward pass
// takes the mean first and then the squares of the differences, which loses
// nothing where the mean is large.  Both passes move each row once.  Measured,
// calls behind one another: forward 16384x1600 bf16 34 us (3.1 TB/s), 8 rows
// 8.5 us (host time); backward 16384x1600 bf16 78 us (2.0 TB/s), 8191x5120 fp16
// without the mean 72.6 us (3.5 TB/s).

constexpr int kWaves = kBlock / 64;
constexpr int64_t kMaxGroups = int64_t(1) << 20;  // workgroups of one launch; they stride over what is left

template <int WPR>
__device__ __forceinline__ void row_sum2(float& a, float& b, float (*lds)[2][kWaves], int& turn) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    a += __shfl_xor(a, off, 64);
    b += __shfl_xor(b, off, 64);
  }
  if constexpr (WPR > 1) {  // two slots in turn: one barrier is enough
    turn ^= 1;
    if ((threadIdx.x & 63) == 0) {
      lds[turn][0][threadIdx.x >> 6] = a;
      lds[turn][1][threadIdx.x >> 6] = b;
    }
    __syncthreads();
    a = (lds[turn][0][0] + lds[turn][0][1]) + (lds[turn][0][2] + lds[turn][0][3]);
    b = (lds[turn][1][0] + lds[turn][1][1]) + (lds[turn][1][2] + lds[turn][1][3]);
  }
}

// Unit k of a lane's: which of the row's.
template <int WPR>
__device__ __forceinline__ int lane_unit(int k) {
  return WPR > 1 ? k * kBlock + static_cast<int>(threadIdx.x) : k * 64 + static_cast<int>(threadIdx.x & 63);
}

// Units of a lane that every row of the form's range has in full: with_row_shape
// gives a row to the first form whose NU units a lane hold it, so a row is longer
// than what the next smaller form holds (NU - 1 units a lane, or 4 below 8).
template <int NU>
constexpr int kWholeUnits = NU == 8 ? 4 : NU - 1;

// Elements of a lane's unit k, which is the row's unit u.  Without TAIL the rows
// are whole units, and the code for part of one (a third of the kernels'
// registers) is left out; with it only a lane's last units carry that code (in
// all of them it sent rows of 8193 to 16384 ragged columns to scratch memory).
template <int NU, bool TAIL>
__device__ __forceinline__ int norm_unit_size(int64_t cols, int k, int u) {
  if (k < kWholeUnits<NU>) return 8;
  return TAIL ? unit_size(cols, u) : static_cast<int64_t>(u) * 8 < cols ? 8 : 0;
}

// Weights of format DT or fp32 (w32).
template <int DT>
__device__ __forceinline__ void load_weight(const void* p, bool w32, int64_t col, int n, float* out) {
  if (DT != ZERO_FP32 && w32) {
    Unit<ZERO_FP32> w;
    w.clear();
    w.load(static_cast<const float*>(p) + col, n);
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i] = w.get(i);
  } else {
    Unit<DT> w;
    w.clear();
    w.load(static_cast<const char*>(p) + col * Unit<DT>::kBytes, n);
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i] = w.get(i);
  }
}

template <int DT, int NU, int WPR, bool TAIL>
__global__ __launch_bounds__(kBlock) void layernorm_forward_kernel(Rows x, const void* __restrict__ weight,
                                                                   const void* __restrict__ bias, int w32, float eps,
                                                                   int center, Rows y, float* __restrict__ mean,
                                                                   float* __restrict__ rstd) {
  __shared__ float lds[2][2][kWaves];
  int turn = 0;
  const int64_t first = WPR > 1 ? blockIdx.x : static_cast<int64_t>(blockIdx.x) * kWaves + (threadIdx.x >> 6);
  const int64_t step = WPR > 1 ? gridDim.x : static_cast<int64_t>(gridDim.x) * kWaves;
  const float inv = 1.0f / static_cast<float>(x.cols);
  for (int64_t row = first; row < x.rows; row += step) {
    Unit<DT> v[NU];
    float sum = 0.0f, none = 0.0f;
#pragma unroll
    for (int k = 0; k < NU; ++k) {
      const int u = lane_unit<WPR>(k), n = norm_unit_size<NU, TAIL>(x.cols, k, u);
      v[k].clear();
      if (n > 0) v[k].load(x.at<DT>(row, static_cast<int64_t>(u) * 8), n);
    }
    float mu = 0.0f;
    if (center) {
#pragma unroll
      for (int k = 0; k < NU; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += v[k].get(i);
      row_sum2<WPR>(sum, none, lds, turn);
      mu = sum * inv;
    }
    float sq = 0.0f;
#pragma unroll
    for (int k = 0; k < NU; ++k) {
      const int n = norm_unit_size<NU, TAIL>(x.cols, k, lane_unit<WPR>(k));
      if (n >= 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) sq += (v[k].get(i) - mu) * (v[k].get(i) - mu);
      } else if (n > 0) {
#pragma unroll
        for (int i = 0; i < 7; ++i) sq += i < n ? (v[k].get(i) - mu) * (v[k].get(i) - mu) : 0.0f;
      }
    }
    row_sum2<WPR>(sq, none, lds, turn);
    const float r = 1.0f / sqrtf(sq * inv + eps);
#pragma unroll
    for (int k = 0; k < NU; ++k) {
      const int u = lane_unit<WPR>(k), n = norm_unit_size<NU, TAIL>(x.cols, k, u);
      if (n > 0) {
        const int64_t col = static_cast<int64_t>(u) * 8;
        float w[8], b[8];
        load_weight<DT>(weight, w32 != 0, col, n, w);
        if (bias) load_weight<DT>(bias, w32 != 0, col, n, b);
        Unit<DT> out;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float h = (v[k].get(i) - mu) * r;
          out.set(i, bias ? h * w[i] + b[i] : h * w[i]);
        }
        out.store(y.at<DT>(row, col), n);
      }
    }
    if ((WPR > 1 ? threadIdx.x : threadIdx.x & 63) == 0) {
      if (center && mean) mean[row] = mu;
      if (rstd) rstd[row] = r;
    }
  }
}

// The backward pass reads x and y_grad once.  A workgroup keeps the sums of
// its rows' weight and bias gradients in registers over all its rows and
// leaves one pair of partial rows; layernorm_join_kernel adds the pairs.
template <int DT, int NU, int WPR, bool TAIL>
__global__ __launch_bounds__(kBlock) void layernorm_grad_kernel(Rows x, Rows dy, const void* __restrict__ weight,
                                                                int w32, int center, const float* __restrict__ mean,
                                                                const float* __restrict__ rstd, Rows dx,
                                                                float* __restrict__ parts, int64_t part_cols) {
  constexpr int kParts = WPR > 1 ? 1 : kWaves;
  __shared__ float lds[2][2][kWaves];
  int turn = 0;
  const int wave = threadIdx.x >> 6;
  const int64_t first = WPR > 1 ? blockIdx.x : static_cast<int64_t>(blockIdx.x) * kWaves + wave;
  const int64_t step = WPR > 1 ? gridDim.x : static_cast<int64_t>(gridDim.x) * kWaves;
  const float inv = 1.0f / static_cast<float>(x.cols);
  float dw[NU][8] = {}, db[NU][8] = {};
  for (int64_t row = first; row < x.rows; row += step) {
    Unit<DT> a[NU], g[NU];
#pragma unroll
    for (int k = 0; k < NU; ++k) {
      const int u = lane_unit<WPR>(k), n = norm_unit_size<NU, TAIL>(x.cols, k, u);
      a[k].clear();
      g[k].clear();
      if (n > 0) {
        a[k].load(x.at<DT>(row, static_cast<int64_t>(u) * 8), n);
        g[k].load(dy.at<DT>(row, static_cast<int64_t>(u) * 8), n);
      }
    }
    const float mu = center ? mean[row] : 0.0f, r = rstd[row];
    float level = 0.0f, along = 0.0f;
#pragma unroll
    for (int k = 0; k < NU; ++k) {
      const int u = lane_unit<WPR>(k), n = norm_unit_size<NU, TAIL>(x.cols, k, u);
      float w[8] = {};
      if (n > 0 && dx.data) load_weight<DT>(weight, w32 != 0, static_cast<int64_t>(u) * 8, n, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float h = (a[k].get(i) - mu) * r, gi = g[k].get(i), d = gi * w[i];
        dw[k][i] += gi * h;  // past the row's end gi is 0, and w with it
        db[k][i] += gi;
        level += d;
        along += d * h;
      }
    }
    if (!dx.data) continue;
    row_sum2<WPR>(level, along, lds, turn);
    level = center ? level * inv : 0.0f;
    along *= inv;
#pragma unroll
    for (int k = 0; k < NU; ++k) {
      const int u = lane_unit<WPR>(k), n = norm_unit_size<NU, TAIL>(x.cols, k, u);
      if (n > 0) {
        float w[8];
        load_weight<DT>(weight, w32 != 0, static_cast<int64_t>(u) * 8, n, w);
        Unit<DT> out;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float h = (a[k].get(i) - mu) * r;
          out.set(i, r * (g[k].get(i) * w[i] - level - h * along));
        }
        out.store(dx.at<DT>(row, static_cast<int64_t>(u) * 8), n);
      }
    }
  }
  if (!parts) return;
  float* mine = parts + (static_cast<int64_t>(blockIdx.x) * kParts + (WPR > 1 ? 0 : wave)) * 2 * part_cols;
#pragma unroll
  for (int k = 0; k < NU; ++k) {
    const int64_t col = static_cast<int64_t>(lane_unit<WPR>(k)) * 8;
    if (col < x.cols) {
#pragma unroll
      for (int q = 0; q < 8; q += 4) {
        *reinterpret_cast<f32x4*>(mine + col + q) = f32x4{dw[k][q], dw[k][q + 1], dw[k][q + 2], dw[k][q + 3]};
        *reinterpret_cast<f32x4*>(mine + part_cols + col + q) = f32x4{db[k][q], db[k][q + 1], db[k][q + 2], db[k][q + 3]};
      }
    }
  }
}

// Adds the partial rows: a workgroup of 16 wavefronts for 64 columns of one of
// the two gradients, each wavefront a sixteenth of the parts in order, then
// the sixteen in order.
constexpr int kJoinWaves = 16;

template <int GD>
__global__ __launch_bounds__(kJoinWaves * 64) void layernorm_join_kernel(const float* __restrict__ parts, int n_parts,
                                                                         int64_t part_cols, int64_t cols,
                                                                         void* __restrict__ dw, void* __restrict__ db,
                                                                         int accumulate) {
  __shared__ float sums[kJoinWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 64 + lane;
  char* out = static_cast<char*>(blockIdx.y == 0 ? dw : db);
  if (!out) return;
  const int per = (n_parts + kJoinWaves - 1) / kJoinWaves;
  const int lo = wave * per, hi = min(lo + per, n_parts);
  float acc = 0.0f;
  if (col < cols) {
#pragma unroll 8
    for (int p = lo; p < hi; ++p) acc += parts[(static_cast<int64_t>(p) * 2 + blockIdx.y) * part_cols + col];
  }
  sums[wave][lane] = acc;
  __syncthreads();
  if (wave > 0 || col >= cols) return;
#pragma unroll
  for (int w = 1; w < kJoinWaves; ++w) acc += sums[w][lane];
  if constexpr (GD == ZERO_FP32) {
    float* p = reinterpret_cast<float*>(out) + col;
    *p = accumulate ? *p + acc : acc;
  } else {
    uint16_t* p = reinterpret_cast<uint16_t*>(out) + col;
    *p = static_cast<uint16_t>(narrow<GD>(accumulate ? widen<GD>(*p) + acc : acc));
  }
}

// Workgroups of the backward pass: enough to fill the chip twice over, few
// enough that their partial rows stay a small part of what is read (512 pairs of
// fp32 rows against 16384 rows of 16 bits: 4% written and 4% read).  Measured
// with 256, 512, 1024 and 2048: 16384x1600 bf16 109, 78, 50 and 49 us; 8191x5120
// fp16 without the mean 93, 72, 82 and 91; 16384x768 42, 34, 43 and 62; 2048x1600
// 17.3, 14.2, 15.3 and 20.8.  512 is the best of them but for many rows of 1025
// to 2048 columns, one unit a lane, where twice as many hide more of a row's waits.
constexpr int64_t kGradGroups = 512;
constexpr int64_t kLongRow = 1024;  // past it a workgroup shares a row

struct NormSpace {
  int64_t groups, parts, part_cols;
  size_t bytes;
};

inline NormSpace norm_space(int64_t rows, int64_t cols) {
  NormSpace w{};
  const int64_t per = cols > kLongRow ? 1 : kWaves;
  w.groups = std::min<int64_t>(std::max<int64_t>(ceil_div(rows, per), 1), kGradGroups);
  w.parts = w.groups * per;
  w.part_cols = ceil_div(cols, 8) * 8;
  w.bytes = up256(static_cast<size_t>(w.parts) * 2 * static_cast<size_t>(w.part_cols) * 4);
  return w;
}

// Units a lane, and wavefronts a row, for rows of `cols` elements.
template <typename F>
int with_row_shape(int64_t cols, F&& f) {
  using std::integral_constant;
  const int64_t units = ceil_div(cols, 8);
  const auto shape = [&](auto nu, auto wpr) {
    return cols % 8 != 0 ? f(nu, wpr, std::true_type{}) : f(nu, wpr, std::false_type{});
  };
  if (units <= 64) return shape(integral_constant<int, 1>{}, integral_constant<int, 1>{});
  if (cols <= kLongRow) return shape(integral_constant<int, 2>{}, integral_constant<int, 1>{});
  if (units <= kBlock) return shape(integral_constant<int, 1>{}, integral_constant<int, kWaves>{});
  if (units <= 2 * kBlock) return shape(integral_constant<int, 2>{}, integral_constant<int, kWaves>{});
  if (units <= 3 * kBlock) return shape(integral_constant<int, 3>{}, integral_constant<int, kWaves>{});
  if (units <= 4 * kBlock) return shape(integral_constant<int, 4>{}, integral_constant<int, kWaves>{});
  return shape(integral_constant<int, 8>{}, integral_constant<int, kWaves>{});
}

int same_shape(const char* fn, const char* name, const zero_rows* a, const zero_rows* x) {
  if (a->rows != x->rows || a->cols != x->cols || a->dt != x->dt)
    return fail(ZERO_ERR_INVALID, "%s: %s has another shape or dtype than x", fn, name);
  return ZERO_OK;
}

int weight_ok(const char* fn, const void* weight, const void* bias, zero_dtype wdt, const zero_rows* x) {
  if (wdt != x->dt && wdt != ZERO_FP32) return fail(ZERO_ERR_INVALID, "%s: weight of dtype %d", fn, wdt);
  if (!weight) return fail(ZERO_ERR_INVALID, "%s: no weight", fn);
  const uintptr_t align = static_cast<uintptr_t>(dtype_bytes(wdt));
  if (unaligned(weight, align) || unaligned(bias, align)) return fail(ZERO_ERR_INVALID, "%s: weight misaligned", fn);
  if (x->cols > ZERO_LAYERNORM_MAX_COLS)
    return fail(ZERO_ERR_INVALID, "%s: rows of %lld elements, at most %d", fn, static_cast<long long>(x->cols),
                ZERO_LAYERNORM_MAX_COLS);
  return ZERO_OK;
}

}  // namespace

extern "C" {

int zero_layernorm_forward(const zero_rows* x, const void* weight_dev, const void* bias_dev, zero_dtype wdt, double eps,
                           int32_t center, const zero_rows* y, float* mean_dev, float* rstd_dev, void* stream) {
  const char* fn = "zero_layernorm_forward";
  int rc = rows_ok(fn, "x", x);
  if (rc == ZERO_OK) rc = rows_ok(fn, "y", y);
  if (rc == ZERO_OK) rc = same_shape(fn, "y", y, x);
  if (rc == ZERO_OK) rc = weight_ok(fn, weight_dev, bias_dev, wdt, x);
  if (rc != ZERO_OK) return rc;
  if (!(eps >= 0.0) || !finite32(eps)) return fail(ZERO_ERR_INVALID, "%s: eps out of range", fn);
  if (unaligned(mean_dev, 4) || unaligned(rstd_dev, 4)) return fail(ZERO_ERR_INVALID, "%s: misaligned statistics", fn);
  if (x->rows == 0) return ZERO_OK;
  return with_dtype(x->dt, [&](auto dt) {
    return with_row_shape(x->cols, [&](auto nu, auto wpr, auto tail) {
      const int64_t groups = std::min(ceil_div(x->rows, wpr.value > 1 ? 1 : kWaves), kMaxGroups);
      hipLaunchKernelGGL((layernorm_forward_kernel<dt.value, nu.value, wpr.value, tail.value>), dim3(static_cast<unsigned>(groups)),
                         dim3(kBlock), 0, static_cast<hipStream_t>(stream), device_rows(x), weight_dev, bias_dev,
                         wdt == ZERO_FP32 ? 1 : 0, static_cast<float>(eps), center != 0 ? 1 : 0, device_rows(y),
                         mean_dev, rstd_dev);
      return launch_status(fn);
    });
  });
}

size_t zero_layernorm_grad_workspace_bytes(int64_t n_rows, int64_t cols) {
  if (!sizes_ok(n_rows, cols) || cols > ZERO_LAYERNORM_MAX_COLS) return 0;
  return norm_space(n_rows, cols).bytes;
}

int zero_layernorm_grad(const zero_rows* x, const zero_rows* y_grad, const void* weight_dev, zero_dtype wdt,
                        int32_t center, const float* mean_dev, const float* rstd_dev, const zero_rows* x_grad,
                        void* weight_grad_dev, void* bias_grad_dev, zero_dtype gdt, int32_t accumulate, void* ws_dev,
                        size_t ws_bytes, void* stream) {
  const char* fn = "zero_layernorm_grad";
  int rc = rows_ok(fn, "x", x);
  if (rc == ZERO_OK) rc = rows_ok(fn, "y_grad", y_grad);
  if (rc == ZERO_OK && x_grad) rc = rows_ok(fn, "x_grad", x_grad);
  if (rc == ZERO_OK) rc = same_shape(fn, "y_grad", y_grad, x);
  if (rc == ZERO_OK && x_grad) rc = same_shape(fn, "x_grad", x_grad, x);
  if (rc == ZERO_OK) rc = weight_ok(fn, weight_dev, nullptr, wdt, x);
  if (rc != ZERO_OK) return rc;
  if (!any_dtype_ok(gdt)) return fail(ZERO_ERR_INVALID, "%s: unknown gradient dtype %d", fn, gdt);
  const uintptr_t align = static_cast<uintptr_t>(dtype_bytes(gdt));
  if (unaligned(weight_grad_dev, align) || unaligned(bias_grad_dev, align))
    return fail(ZERO_ERR_INVALID, "%s: gradient misaligned", fn);
  if (x->rows > 0 && (!rstd_dev || (center && !mean_dev))) return fail(ZERO_ERR_INVALID, "%s: no statistics", fn);
  if (unaligned(mean_dev, 4) || unaligned(rstd_dev, 4)) return fail(ZERO_ERR_INVALID, "%s: misaligned statistics", fn);
  const NormSpace w = norm_space(x->rows, x->cols);
  if (!ws_dev || !aligned16(ws_dev) || ws_bytes < w.bytes)
    return fail(ZERO_ERR_INVALID, "%s: workspace of %zu bytes, %zu needed, 16-byte aligned", fn, ws_dev ? ws_bytes : 0,
                w.bytes);
  const bool sums = weight_grad_dev || bias_grad_dev;
  if ((!sums && !x_grad) || (x->rows == 0 && (!sums || accumulate))) return ZERO_OK;
  float* parts = sums ? static_cast<float*>(ws_dev) : nullptr;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  // Without rows one workgroup still leaves its sums, zeros.
  rc = with_dtype(x->dt, [&](auto dt) {
    return with_row_shape(x->cols, [&](auto nu, auto wpr, auto tail) {
      hipLaunchKernelGGL((layernorm_grad_kernel<dt.value, nu.value, wpr.value, tail.value>), dim3(static_cast<unsigned>(w.groups)),
                         dim3(kBlock), 0, st, device_rows(x), device_rows(y_grad), weight_dev,
                         wdt == ZERO_FP32 ? 1 : 0, center != 0 ? 1 : 0, mean_dev, rstd_dev,
                         x_grad ? device_rows(x_grad) : Rows{}, parts, w.part_cols);
      return launch_status(fn);
    });
  });
  if (rc != ZERO_OK || !sums) return rc;
  return with_dtype(gdt, [&](auto gd) {
    hipLaunchKernelGGL((layernorm_join_kernel<gd.value>), dim3(static_cast<unsigned>(ceil_div(x->cols, 64)), 2),
                       dim3(kJoinWaves * 64), 0, st, parts, static_cast<int>(w.parts), w.part_cols, x->cols,
                       weight_grad_dev, bias_grad_dev, accumulate != 0 ? 1 : 0);
    return launch_status(fn);
  });
}

}  // extern "C"
