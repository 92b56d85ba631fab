// zero_common.h -- what the library's sources share: limits, error reporting,
// the 16-bit formats, the update of one element and the streaming helpers.
// Internal; the public interface is include/zero_shard.h.
#ifndef ZERO_COMMON_H
#define ZERO_COMMON_H

#include <hip/hip_runtime.h>

#include <cstdint>
#include <limits>

#include "zero_shard.h"

#pragma clang fp contract(off)

namespace zero_detail {

// ------------------------------------------------------------------ errors

// Records the calling thread's error message and returns `code`.
__attribute__((visibility("hidden"))) int fail(int code, const char* fmt, ...);
// ZERO_OK, or the launch error the runtime holds.
__attribute__((visibility("hidden"))) int launch_status(const char* what);

constexpr int64_t kMaxPsi = ZERO_MAX_NUMEL;  // 2^58: keeps 16·Ψ and N·S in range
static_assert(kMaxPsi == std::numeric_limits<int64_t>::max() / 32, "element-count limit");

// ceil(a / b) for a >= 0, b > 0, without forming a + b - 1 (which can overflow).
constexpr int64_t ceil_div(int64_t a, int64_t b) { return a / b + (a % b != 0 ? 1 : 0); }

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kBlock = 256;  // 4 wavefronts of 64

// Streaming kernels capped at 4 wavefronts per SIMD (measurements at each
// kernel): the compiler reserves registers so that no more fit on a SIMD.
#define STREAMING_KERNEL __global__ __launch_bounds__(kBlock) __attribute__((amdgpu_waves_per_eu(1, 4)))

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }
inline bool fp32_aligned(const void* a, const void* b, const void* c, const void* d) {
  return ((reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b) | reinterpret_cast<uintptr_t>(c) |
           reinterpret_cast<uintptr_t>(d)) & 3u) == 0;
}

// ------------------------------------------------------------------ 16-bit formats

// Widen one 16-bit value (in the low half of h) to fp32; exact for both formats.
template <int DT>
__device__ __forceinline__ float widen(uint32_t h) {
  if constexpr (DT == ZERO_BF16) {
    return __uint_as_float(h << 16);
  } else {
    return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(h)));
  }
}

// fp32 -> bf16, round to nearest, ties to even; NaN stays a quiet NaN.
__device__ __forceinline__ uint32_t bf16_rne(float f) {
  const uint32_t u = __float_as_uint(f);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return (u >> 16) | 0x40u;
  return (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
}

// fp32 -> the parameter format PT (bf16 or IEEE binary16), round to nearest,
// ties to even.  The binary16 conversion is the hardware's (v_cvt_f16_f32 in
// the default round-to-nearest-even mode, binary16 denormals kept): overflow
// gives infinity, tiny values become subnormals or zero.
template <int PT>
__device__ __forceinline__ uint32_t narrow(float f) {
  if constexpr (PT == ZERO_BF16) {
    return bf16_rne(f);
  } else {
    return __builtin_bit_cast(uint16_t, static_cast<_Float16>(f));
  }
}

// ------------------------------------------------------------------ the update of one element

struct AdamScalars {
  float b1, omb1, b2, omb2, eps, decay, step_size, bc2_sqrt, gscale;
};

// One element of the update, each line one rounded fp32 operation.
__device__ __forceinline__ void adam_element(float g, float& p, float& m, float& v, const AdamScalars& s) {
  g = g * s.gscale;
  const float m_keep = s.b1 * m;
  const float m_add = s.omb1 * g;
  m = m_keep + m_add;
  const float gg = g * g;
  const float v_keep = s.b2 * v;
  const float v_add = s.omb2 * gg;
  v = v_keep + v_add;
  float d = sqrtf(v);
  d = d / s.bc2_sqrt;
  d = d + s.eps;
  float u = m / d;
  u = s.step_size * u;
  const float p_dec = p * s.decay;
  p = p_dec - u;
}

// The decision over the ranks' square-norms and flags, on one thread: updates
// the step state (all but its scalars) and returns whether the step is taken
// (then st->adam_step and st->grad_scale are its t and factor).
__device__ __forceinline__ bool take_decision(const double* __restrict__ sq, const int32_t* __restrict__ flags,
                                              int32_t n_ranks, double max_norm, zero_step_state* __restrict__ st) {
  double global = 0.0;
  bool overflow = false;
  for (int32_t r = 0; r < n_ranks; ++r) {
    global += sq[r];
    overflow = overflow || flags[r] != 0;
  }
  const double scale = st->loss_scale;
  st->iteration += 1;
  // The host decision refuses these cases with ZERO_ERR_INVALID; here the
  // step is skipped, the error recorded, and the scale, good-step count and
  // Adam t are left as they are.
  const double unscaled = global / (scale * scale);
  if (!(scale > 0.0) || !isfinite(scale) || (!overflow && !isfinite(unscaled))) {
    st->skip = 1;
    st->error = ZERO_STEP_ERR_LOSS_SCALE;
    st->grad_scale = 0.0;
    st->global_norm = __builtin_nan("");
    return false;
  }
  st->error = 0;
  if (overflow) {
    st->skip = 1;
    st->grad_scale = 0.0;
    st->global_norm = __builtin_nan("");
    st->loss_scale = scale * 0.5;
    st->good_steps = 0;
    return false;
  }
  double coef = 1.0;
  if (max_norm > 0.0) {
    const double c = max_norm / (sqrt(unscaled) + 1e-6);
    coef = c < 1.0 ? c : 1.0;
  }
  int32_t good = st->good_steps + 1;
  double new_scale = scale;
  if (good >= st->growth_interval) {
    new_scale = scale * 2.0;
    good = 0;
  }
  st->skip = 0;
  st->grad_scale = coef / scale;
  st->global_norm = sqrt(unscaled);
  st->loss_scale = new_scale;
  st->good_steps = good;
  st->adam_step += 1;
  return true;
}

// The update's nine scalars for Adam step t and factor gscale, derived in fp64
// as the host derives them (adam_scalars), each rounded once.
__device__ __forceinline__ void device_scalars(double lr, double beta1, double beta2, double eps, double wd, int64_t t,
                                               double gscale, float* __restrict__ out) {
  const double bc1 = 1.0 - pow(beta1, static_cast<double>(t));
  const double bc2 = 1.0 - pow(beta2, static_cast<double>(t));
  out[0] = static_cast<float>(beta1);
  out[1] = static_cast<float>(1.0 - beta1);
  out[2] = static_cast<float>(beta2);
  out[3] = static_cast<float>(1.0 - beta2);
  out[4] = static_cast<float>(eps);
  out[5] = static_cast<float>(1.0 - lr * wd);
  out[6] = static_cast<float>(lr / bc1);
  out[7] = static_cast<float>(sqrt(bc2));
  out[8] = static_cast<float>(gscale);
}

// Checks the hyper-parameters and derives the fp32 scalars from fp64 host
// arithmetic (each rounded once).
__attribute__((visibility("hidden"))) int adam_scalars(const char* fn, const zero_adamw_hparams* hp, AdamScalars* s);

// ------------------------------------------------------------------ streaming

// Streaming accesses: every byte the update touches is used exactly once, so
// loads and stores carry the non-temporal hint (measured on MI355X: the
// stores are worth 13% to the tiled update, the loads a few percent more).
template <typename T>
__device__ __forceinline__ T ld_stream(const T* p) {
  return __builtin_nontemporal_load(p);
}
template <typename T>
__device__ __forceinline__ void st_stream(T* p, T v) {
  __builtin_nontemporal_store(v, p);
}

constexpr int64_t kTile = ZERO_STATE_TILE;

// The dispatcher deals a launch's workgroups to the eight XCDs in turn, so
// workgroup b runs on XCD b mod 8.  Remapping workgroups to tiles so that each
// XCD takes kXcdGroup adjacent tiles at a time (the first 8·kXcdGroup
// workgroups cover 8·kXcdGroup adjacent tiles, XCD x taking the x-th run of
// kXcdGroup) is faster on MI355X: groups of 8 gained 0.5-1.2% over no
// grouping, and with the occupancy cap below, update time on the GPT-2 rank
// shard relative to groups of 8 is: 16 -0.3%, 20 -0.6%, 24 -1.9%, 28 +0.5%,
// 32 -1.2%, 40 +0.8%, 48 -1.1%, 64 +0.2%; with 24 the Llama-7B, Llama-13B
// and 1T shards gain 1.7% too.  A whole contiguous range per XCD was 2-3%
// slower than no grouping.  A bijection on [0, n): workgroups past the last
// whole span of 8·kXcdGroup keep their own index.
constexpr int64_t kXcds = 8, kXcdGroup = 24;
__device__ __forceinline__ int64_t xcd_grouped(int64_t b, int64_t n) {
  constexpr int64_t kSpan = kXcds * kXcdGroup;
  if (b >= n / kSpan * kSpan) return b;
  const int64_t x = b % kXcds, q = b / kXcds;
  return q / kXcdGroup * kSpan + x * kXcdGroup + q % kXcdGroup;
}

// The update is issued in launches of at most 2^25 elements (32768 tiles).
// Measured on MI355X (tiled state, bf16): one launch over a 3.25e9-element
// shard sustains 5.58 TB/s and over a 1.95e8-element shard 6.10 TB/s, while
// launches of 2^24 / 2^25 / 2^26 / 2^27 elements give 6.32 / 6.39 / 6.33 /
// 6.20 TB/s at every shard size.  Over a long grid the workgroups of the
// eight XCDs drift apart in the address space; a launch boundary brings
// them back together at the cost of one drain.
constexpr int64_t kUpdateElemsPerLaunch = int64_t(1) << 25;

// Sum over a workgroup of NT threads in a fixed tree: butterfly inside each
// wavefront, then the NT/64 wavefront sums in order.  Result valid in thread 0.
template <int NT = kBlock>
__device__ __forceinline__ void block_reduce(double& acc, uint32_t& bad) {
  __shared__ double wsum[NT / 64];
  __shared__ uint32_t wbad[NT / 64];
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    acc = acc + __shfl_xor(acc, off, 64);
    bad |= __shfl_xor(bad, off, 64);
  }
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (lane == 0) {
    wsum[wave] = acc;
    wbad[wave] = bad;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    acc = wsum[0];
    bad = wbad[0];
#pragma unroll
    for (int w = 1; w < NT / 64; ++w) {
      acc = acc + wsum[w];
      bad |= wbad[w];
    }
  }
}

inline bool dtype_ok(int dt) { return dt == ZERO_BF16 || dt == ZERO_FP16; }

}  // namespace zero_detail

#endif  // ZERO_COMMON_H
