// zero_units.h -- rows in device memory and their units of 8 elements, for the
// operators that work on rows.  Internal.
#ifndef ZERO_UNITS_H
#define ZERO_UNITS_H

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "zero_common.h"

namespace zero_detail {

// What a kernel needs of a zero_rows.
struct Rows {
  char* data;
  int64_t rows, cols, stride;
  template <int DT>
  __device__ __forceinline__ void* at(int64_t row, int64_t col) const {
    return data + (row * stride + col) * (DT == ZERO_FP32 ? 4 : 2);
  }
};

// 16 bytes that may start at any element.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32_any __attribute__((aligned(2)));

// 8 neighbouring elements of a row, as they are held in memory.
template <int DT>
struct Unit {
  static constexpr int kBytes = DT == ZERO_FP32 ? 4 : 2;
  static constexpr int kWords = 2 * kBytes;
  uint32_t w[kWords];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int k = 0; k < kWords; ++k) w[k] = 0;
  }
  // The first n elements (n > 0; 8 and more: all), the others as they were.
  __device__ __forceinline__ void load(const void* p, int n) {
    if (n >= 8) {
#pragma unroll
      for (int k = 0; k < kWords; k += 4) {
        const u32x4_any v = *reinterpret_cast<const u32x4_any*>(static_cast<const char*>(p) + 4 * k);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[k + j] = v[j];
      }
    } else {
      load_part(p, n);
    }
  }
  __device__ __forceinline__ void store(void* p, int n) const {
    if (n >= 8) {
#pragma unroll
      for (int k = 0; k < kWords; k += 4) {
        u32x4_any v;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = w[k + j];
        *reinterpret_cast<u32x4_any*>(static_cast<char*>(p) + 4 * k) = v;
      }
    } else {
      store_part(p, n);
    }
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (DT == ZERO_FP32) {
      return __uint_as_float(w[i]);
    } else if constexpr (DT == ZERO_BF16) {
      return __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    } else {
      return widen<ZERO_FP16>(w[i / 2] >> (i & 1 ? 16 : 0));
    }
  }
  // A row's last unit, 1 to 7 elements: at most one access of 4, of 2 and of 1.
  __device__ __forceinline__ void load_part(const void* p, int n) {
    if constexpr (DT == ZERO_FP32) {
      const uint32_t* q = static_cast<const uint32_t*>(p);
      if (n & 4) {
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = q[k];
      }
      if (n & 2) {
        const uint32_t a = q[n & 4], b = q[(n & 4) + 1];
        w[0] = n & 4 ? w[0] : a;
        w[1] = n & 4 ? w[1] : b;
        w[4] = n & 4 ? a : w[4];
        w[5] = n & 4 ? b : w[5];
      }
      if (n & 1) {
        const uint32_t a = q[n - 1];
        w[0] = n == 1 ? a : w[0];
        w[2] = n == 3 ? a : w[2];
        w[4] = n == 5 ? a : w[4];
        w[6] = n == 7 ? a : w[6];
      }
    } else {
      const uint16_t* q = static_cast<const uint16_t*>(p);
      if (n & 4) {
        w[0] = *reinterpret_cast<const u32_any*>(q);
        w[1] = *reinterpret_cast<const u32_any*>(q + 2);
      }
      if (n & 2) {
        const uint32_t a = *reinterpret_cast<const u32_any*>(q + (n & 4));
        w[0] = n & 4 ? w[0] : a;
        w[2] = n & 4 ? a : w[2];
      }
      if (n & 1) {
        const uint32_t a = q[n - 1];
        w[0] = n == 1 ? (w[0] & 0xFFFF0000u) | a : w[0];
        w[1] = n == 3 ? (w[1] & 0xFFFF0000u) | a : w[1];
        w[2] = n == 5 ? (w[2] & 0xFFFF0000u) | a : w[2];
        w[3] = n == 7 ? (w[3] & 0xFFFF0000u) | a : w[3];
      }
    }
  }
  // The words are copied before one is chosen: a choice between elements of w would be one between addresses, and would
  // put the unit into scratch memory, whole units' stores included.
  __device__ __forceinline__ void store_part(void* p, int n) const {
    const uint32_t w0 = w[0], w1 = w[1], w2 = w[2], w3 = w[3];
    if constexpr (DT == ZERO_FP32) {
      const uint32_t w4 = w[4], w5 = w[5], w6 = w[6];
      uint32_t* q = static_cast<uint32_t*>(p);
      if (n & 4) {
        q[0] = w0;
        q[1] = w1;
        q[2] = w2;
        q[3] = w3;
      }
      if (n & 2) {
        q[n & 4] = n & 4 ? w4 : w0;
        q[(n & 4) + 1] = n & 4 ? w5 : w1;
      }
      if (n & 1) q[n - 1] = n == 1 ? w0 : n == 3 ? w2 : n == 5 ? w4 : w6;
    } else {
      uint16_t* q = static_cast<uint16_t*>(p);
      if (n & 4) {
        *reinterpret_cast<u32_any*>(q) = w0;
        *reinterpret_cast<u32_any*>(q + 2) = w1;
      }
      if (n & 2) *reinterpret_cast<u32_any*>(q + (n & 4)) = n & 4 ? w2 : w0;
      if (n & 1) q[n - 1] = static_cast<uint16_t>(n == 1 ? w0 : n == 3 ? w1 : n == 5 ? w2 : w3);
    }
  }
  // Rounds once, to nearest.  Elements are set in order: the even one of a
  // word clears it.
  __device__ __forceinline__ void set(int i, float f) {
    if constexpr (DT == ZERO_FP32) {
      w[i] = __float_as_uint(f);
    } else {
      const uint32_t h = narrow<DT>(f);
      w[i / 2] = i & 1 ? (w[i / 2] & 0xFFFFu) | h << 16 : h;
    }
  }
};

// Elements that unit u of a row has: 8, fewer at the row's end, none or a
// negative number past it.
__device__ __forceinline__ int unit_size(int64_t cols, int64_t u) {
  const int64_t n = cols - u * 8;
  return static_cast<int>(n < 8 ? n : 8);
}

constexpr uint32_t kNoRow = 0xFFFFFFFFu;

// The row that token t names in a table of `rows` rows whose first is row
// `first` of the vocabulary, or kNoRow.
__device__ __forceinline__ uint32_t local_row(const void* ids, int id_bytes, int64_t t, int64_t first, int64_t rows) {
  const int64_t id = id_bytes == 8 ? static_cast<const int64_t*>(ids)[t] : static_cast<const int32_t*>(ids)[t];
  return id >= first && id - first < rows ? static_cast<uint32_t>(id - first) : kNoRow;
}

// Calls f with the format as a constant.
template <typename F>
int with_dtype(int dt, F&& f) {
  switch (dt) {
    case ZERO_BF16: return f(std::integral_constant<int, ZERO_BF16>{});
    case ZERO_FP16: return f(std::integral_constant<int, ZERO_FP16>{});
    default: return f(std::integral_constant<int, ZERO_FP32>{});
  }
}

// Workgroups of kBlock threads that a launch can have: its threads are counted
// in 32 bits.
constexpr int64_t kLaunchGroups = (int64_t(1) << 32) / kBlock;

inline bool any_dtype_ok(int dt) { return dtype_ok(dt) || dt == ZERO_FP32; }
inline int64_t dtype_bytes(int dt) { return dt == ZERO_FP32 ? 4 : 2; }
inline bool unaligned(const void* p, uintptr_t align) { return (reinterpret_cast<uintptr_t>(p) & (align - 1)) != 0; }
inline Rows device_rows(const zero_rows* r) { return Rows{static_cast<char*>(r->data), r->rows, r->cols, r->stride}; }

constexpr size_t up256(size_t n) { return (n + 255) / 256 * 256; }
// Sizes that a zero_rows may have.
inline bool sizes_ok(int64_t rows, int64_t cols) {
  constexpr int64_t most = std::numeric_limits<int32_t>::max();
  return rows >= 0 && rows <= most && cols >= 1 && cols <= most;
}

// Checks one zero_rows.
inline int rows_ok(const char* fn, const char* name, const zero_rows* r) {
  if (!r) return fail(ZERO_ERR_INVALID, "%s: %s is NULL", fn, name);
  if (!any_dtype_ok(r->dt)) return fail(ZERO_ERR_INVALID, "%s: %s: unknown dtype %d", fn, name, r->dt);
  constexpr int64_t most = std::numeric_limits<int32_t>::max();
  if (r->rows < 0 || r->rows > most || r->cols < 1 || r->cols > most || r->stride < r->cols ||
      r->stride > (int64_t(1) << 40) / std::max<int64_t>(r->rows, 1))
    return fail(ZERO_ERR_INVALID, "%s: %s: %lld rows of %lld, stride %lld: out of range", fn, name,
                static_cast<long long>(r->rows), static_cast<long long>(r->cols), static_cast<long long>(r->stride));
  if (r->rows > 0 && !r->data) return fail(ZERO_ERR_INVALID, "%s: %s has no data", fn, name);
  if (unaligned(r->data, static_cast<uintptr_t>(dtype_bytes(r->dt))))
    return fail(ZERO_ERR_INVALID, "%s: %s is not aligned to its elements", fn, name);
  return ZERO_OK;
}

inline int ids_ok(const char* fn, const void* ids, int32_t id_bytes, int64_t n) {
  if (id_bytes != 4 && id_bytes != 8) return fail(ZERO_ERR_INVALID, "%s: ids of %d bytes", fn, id_bytes);
  if (n > 0 && !ids) return fail(ZERO_ERR_INVALID, "%s: no ids", fn);
  if (unaligned(ids, static_cast<uintptr_t>(id_bytes))) return fail(ZERO_ERR_INVALID, "%s: ids misaligned", fn);
  return ZERO_OK;
}

// Whether a factor that kernels take in fp32 is finite there: a larger one would
// make NaN of what has to stay zero.
inline bool finite32(double f) { return std::isfinite(static_cast<float>(f)); }

}  // namespace zero_detail

#endif  // ZERO_UNITS_H
