// zero_list.hip -- the norm, the update and the 8-bit state over lists of
// tensors (include/zero_shard.h, "lists of tensors"), for CDNA4 (gfx950).
//
// Every kernel here streams HBM: nothing is a contraction.  A list is a table
// in device memory: one 64-byte descriptor per tensor, then one 8-byte entry
// (tensor, chunk of the tensor) per workgroup of the norm, then one per
// workgroup of the update, so a workgroup finds its work with two dependent
// scalar loads whatever the number of tensors, and one launch covers the list.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>
#include <vector>

#include "zero_common.h"

#pragma clang fp contract(off)

namespace {

using namespace zero_detail;

// ------------------------------------------------------------------ the table

struct Desc {
  const void* grad;
  void* param;
  float* state;  // master (arrays), tiles (tiled, 8-bit)
  float* m;
  float* v;
  int64_t numel;
  int64_t block0;    // number of the tensor's first block of ZERO_STATE8_BLOCK elements in the list
  uint32_t formats;  // gradient, parameter, layout, group: one byte each
  uint32_t reserved;
  __host__ __device__ int gdt() const { return static_cast<int>(formats & 0xFFu); }
  __host__ __device__ int pdt() const { return static_cast<int>((formats >> 8) & 0xFFu); }
  __host__ __device__ int layout() const { return static_cast<int>((formats >> 16) & 0xFFu); }
  __host__ __device__ int group() const { return static_cast<int>(formats >> 24); }
};
static_assert(sizeof(Desc) == 64, "one scalar load of 16 dwords");

// The whole descriptor in one scalar load (member by member, the compiler
// loads what it needs next and waits for each).
__device__ __forceinline__ Desc load_desc(const Desc* descs, uint32_t tensor) {
  typedef uint32_t u32x16 __attribute__((ext_vector_type(16), aligned(16)));
  return __builtin_bit_cast(Desc, *reinterpret_cast<const u32x16*>(descs + tensor));
}

struct Entry {
  uint32_t tensor, chunk;
};

constexpr int64_t kMaxTensorNumel = int64_t(1) << 40;
constexpr int64_t kMaxNormBlocks = int64_t(1) << 23;  // one launch: its threads are counted in 32 bits
constexpr int64_t kMaxUpdateBlocks = int64_t(1) << 30;
// Elements per workgroup of the norm.
constexpr int64_t kNormPer = 16384;
constexpr int64_t kTile8 = ZERO_STATE8_TILE;
constexpr int kBlock8 = ZERO_STATE8_BLOCK;
constexpr int64_t kTile8Blocks = kTile8 / kBlock8;
constexpr int64_t kTile8Bytes = 6 * kTile8 + 8 * kTile8Blocks;
static_assert(kTile8Bytes % 128 == 0, "tiles keep the cache lines of their parts whole");

int64_t elem_bytes(int dt) { return dt == ZERO_FP32 ? 4 : 2; }
bool list_dtype_ok(int dt) { return dtype_ok(dt) || dt == ZERO_FP32; }

bool off(const void* p, uintptr_t align) { return (reinterpret_cast<uintptr_t>(p) & (align - 1)) != 0; }

uint64_t fold(uint64_t h, uint64_t x) {  // FNV-1a over the bytes of x
  for (int k = 0; k < 64; k += 8) h = (h ^ ((x >> k) & 0xFFu)) * 0x100000001B3ull;
  return h;
}
constexpr uint64_t kFoldStart = 0xCBF29CE484222325ull;

uint64_t list_check(const zero_list& l) {
  uint64_t h = kFoldStart;
  for (int64_t x : {l.table_bytes, l.grads_bytes, l.numel, l.norm_blocks, l.update_blocks, l.norm_offset,
                    l.update_offset, static_cast<int64_t>(l.shape), static_cast<int64_t>(l.n_tensors),
                    static_cast<int64_t>(l.n_groups), static_cast<int64_t>(l.state), static_cast<int64_t>(l.flags)})
    h = fold(h, static_cast<uint64_t>(x));
  return h;
}

// Sizes of the table's parts; false if a size or layout is out of range.
bool table_shape(const char* fn, const zero_list_tensor* t, int32_t n, zero_list* out) {
  if (n < 0 || (n > 0 && !t)) {
    fail(ZERO_ERR_INVALID, "%s: bad tensor list (n_tensors=%d)", fn, n);
    return false;
  }
  zero_list l{};
  l.n_tensors = n;
  l.shape = fold(kFoldStart, static_cast<uint64_t>(n));
  for (int32_t k = 0; k < n; ++k) {
    if (t[k].numel < 0 || t[k].numel > kMaxTensorNumel) {
      fail(ZERO_ERR_INVALID, "%s: tensor %d: numel %lld out of range", fn, k, static_cast<long long>(t[k].numel));
      return false;
    }
    if (t[k].layout < ZERO_STATE_NONE || t[k].layout > ZERO_STATE_8BIT) {
      fail(ZERO_ERR_INVALID, "%s: tensor %d: unknown state layout %d", fn, k, t[k].layout);
      return false;
    }
    const int32_t state = t[k].layout == ZERO_STATE_NONE ? 0 : t[k].layout == ZERO_STATE_8BIT ? 8 : 32;
    if (k > 0 && state != l.state) {
      fail(ZERO_ERR_INVALID, "%s: tensor %d: one list holds one kind of state (none, fp32 or 8-bit)", fn, k);
      return false;
    }
    l.state = state;
    l.shape = fold(l.shape, static_cast<uint64_t>(t[k].numel));
    l.numel += t[k].numel;
    l.norm_blocks += ceil_div(t[k].numel, kNormPer);
    if (state != 0) l.update_blocks += ceil_div(t[k].numel, state == 8 ? kTile8 : kTile);
    if (l.numel > kMaxPsi || l.norm_blocks > kMaxNormBlocks || l.update_blocks > kMaxUpdateBlocks) {
      fail(ZERO_ERR_INVALID, "%s: the list is too large", fn);
      return false;
    }
  }
  l.grads_bytes = static_cast<int64_t>(n) * sizeof(Desc);
  l.norm_offset = l.grads_bytes;
  l.update_offset = l.norm_offset + l.norm_blocks * static_cast<int64_t>(sizeof(Entry));
  l.table_bytes = l.update_offset + l.update_blocks * static_cast<int64_t>(sizeof(Entry));
  if (l.table_bytes == 0) l.table_bytes = sizeof(Desc);  // an empty list still has a table
  *out = l;
  return true;
}

struct Range {
  uintptr_t lo, hi;
  bool written;
  int32_t tensor;
};

// Checks one tensor and collects the memory it covers.
int check_tensor(const char* fn, const zero_list_tensor& t, int32_t k, int32_t n_groups, std::vector<Range>* ranges,
                 int32_t* flags) {
  if (!list_dtype_ok(t.gdt)) return fail(ZERO_ERR_INVALID, "%s: tensor %d: unknown gradient dtype %d", fn, k, t.gdt);
  if (!list_dtype_ok(t.pdt)) return fail(ZERO_ERR_INVALID, "%s: tensor %d: unknown parameter dtype %d", fn, k, t.pdt);
  if (t.group < 0 || t.group >= n_groups)
    return fail(ZERO_ERR_INVALID, "%s: tensor %d: group %d outside [0, %d)", fn, k, t.group, n_groups);
  if (off(t.grad, elem_bytes(t.gdt)) || off(t.param, elem_bytes(t.pdt)))
    return fail(ZERO_ERR_INVALID, "%s: tensor %d: gradient or parameter not aligned to its element size", fn, k);
  const bool arrays = t.layout == ZERO_STATE_ARRAYS;
  if (!arrays && (t.m || t.v))
    return fail(ZERO_ERR_INVALID, "%s: tensor %d: m and v belong to separate arrays only", fn, k);
  if (t.layout == ZERO_STATE_NONE && t.state)
    return fail(ZERO_ERR_INVALID, "%s: tensor %d: a state without a layout", fn, k);
  if ((t.layout == ZERO_STATE_TILED || t.layout == ZERO_STATE_8BIT) && t.numel > 0 && !t.state)
    return fail(ZERO_ERR_INVALID, "%s: tensor %d: NULL state", fn, k);
  if (arrays ? off(t.state, 4) || off(t.m, 4) || off(t.v, 4) : off(t.state, 16))
    return fail(ZERO_ERR_INVALID, "%s: tensor %d: misaligned state", fn, k);
  if (t.numel == 0) return ZERO_OK;
  if (!t.param) *flags &= ~ZERO_LIST_HAS_PARAMS;
  if (!t.state || (arrays && (!t.m || !t.v))) *flags &= ~ZERO_LIST_WHOLE_STATE;
  int64_t state_bytes = 4 * t.numel;
  if (t.layout == ZERO_STATE_TILED) state_bytes = 4 * zero_state_tiled_numel(t.numel);
  if (t.layout == ZERO_STATE_8BIT) state_bytes = zero_state8_bytes(t.numel);
  const struct {
    const void* p;
    int64_t bytes;
    bool written;
  } parts[] = {{t.grad, t.numel * elem_bytes(t.gdt), false},
               {t.param, t.numel * elem_bytes(t.pdt), true},
               {t.state, state_bytes, true},
               {t.m, 4 * t.numel, true},
               {t.v, 4 * t.numel, true}};
  for (const auto& part : parts) {
    if (!part.p) continue;
    const uintptr_t lo = reinterpret_cast<uintptr_t>(part.p);
    if (lo + static_cast<uintptr_t>(part.bytes) < lo)
      return fail(ZERO_ERR_INVALID, "%s: tensor %d: a buffer passes the end of the address space", fn, k);
    ranges->push_back({lo, lo + static_cast<uintptr_t>(part.bytes), part.written, k});
  }
  return ZERO_OK;
}

// Two tensors of a list run on workgroups in any order: nothing that one
// writes may be another's.
int check_overlap(const char* fn, std::vector<Range>* ranges) {
  std::sort(ranges->begin(), ranges->end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
  uintptr_t read_end = 0, write_end = 0;
  for (const Range& r : *ranges) {
    if (r.lo < write_end || (r.written && r.lo < read_end))
      return fail(ZERO_ERR_INVALID, "%s: tensor %d: a buffer overlaps one that the update writes", fn, r.tensor);
    (r.written ? write_end : read_end) = std::max(r.written ? write_end : read_end, r.hi);
  }
  return ZERO_OK;
}

// Checks the tensors and writes their descriptors; *flags receives ZERO_LIST_*.
int write_descs(const char* fn, const zero_list_tensor* t, int32_t n, int32_t n_groups, Desc* out, int32_t* flags) {
  std::vector<Range> ranges;
  ranges.reserve(5 * static_cast<size_t>(n));
  *flags = ZERO_LIST_HAS_PARAMS | ZERO_LIST_WHOLE_STATE;
  for (int32_t k = 0; k < n; ++k) {
    const int rc = check_tensor(fn, t[k], k, n_groups, &ranges, flags);
    if (rc != ZERO_OK) return rc;
  }
  const int rc = check_overlap(fn, &ranges);
  if (rc != ZERO_OK) return rc;
  int64_t block0 = 0;
  for (int32_t k = 0; k < n; ++k) {
    Desc d{};
    d.grad = t[k].grad;
    d.param = t[k].param;
    d.state = static_cast<float*>(t[k].state);
    d.m = t[k].m;
    d.v = t[k].v;
    if (t[k].layout == ZERO_STATE_TILED && d.state) {
      d.m = d.state + kTile;
      d.v = d.state + 2 * kTile;
    }
    d.numel = t[k].numel;
    d.block0 = block0;
    d.formats = static_cast<uint32_t>(t[k].gdt) | static_cast<uint32_t>(t[k].pdt) << 8 |
                static_cast<uint32_t>(t[k].layout) << 16 | static_cast<uint32_t>(t[k].group) << 24;
    std::memcpy(out + k, &d, sizeof d);
    block0 += ceil_div(t[k].numel, kTile8) * kTile8Blocks;
  }
  return ZERO_OK;
}

void write_entries(const zero_list_tensor* t, int32_t n, int64_t per, char* out) {
  for (int32_t k = 0; k < n; ++k)
    for (int64_t c = 0, chunks = ceil_div(t[k].numel, per); c < chunks; ++c) {
      const Entry e{static_cast<uint32_t>(k), static_cast<uint32_t>(c)};
      std::memcpy(out, &e, sizeof e);
      out += sizeof e;
    }
}

// A planned list with its table in place.
int list_ok(const char* fn, const zero_list* l) {
  if (!l) return fail(ZERO_ERR_INVALID, "%s: list NULL", fn);
  if (l->check != list_check(*l)) return fail(ZERO_ERR_INVALID, "%s: the list was not planned", fn);
  if (l->n_tensors > 0 && (!l->table_dev || !aligned16(l->table_dev)))
    return fail(ZERO_ERR_INVALID, "%s: the list's device table is NULL or not 16-byte aligned", fn);
  return ZERO_OK;
}

// ------------------------------------------------------------------ gradients and parameters

// A descriptor's addresses are global memory: said so, the compiler uses global
// (not flat) accesses, which do not also wait for LDS.
#define GLOBAL __attribute__((address_space(1)))
typedef GLOBAL float* gfloat;
typedef GLOBAL uint8_t* gbyte;
typedef GLOBAL uint16_t* gu16;

// Vectors of tensors that start anywhere: the hardware takes any element
// alignment in one access (global memory in unaligned mode, the default).
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));

__device__ __forceinline__ f32x4 load4(gfloat p) {
  return __builtin_nontemporal_load(reinterpret_cast<GLOBAL f32x4_any*>(p));
}
__device__ __forceinline__ void store4(gfloat p, f32x4 x) {
  __builtin_nontemporal_store(static_cast<f32x4_any>(x), reinterpret_cast<GLOBAL f32x4_any*>(p));
}

__device__ __forceinline__ float widen_any(uint32_t h, int dt) {
  return dt == ZERO_BF16 ? widen<ZERO_BF16>(h) : widen<ZERO_FP16>(h);
}

// Four consecutive gradients, as they lie (16-bit formats: in the lower half).
__device__ __forceinline__ u32x4 load_grad4(const void* grad, int dt, int64_t e) {
  if (dt == ZERO_FP32) return __builtin_nontemporal_load((GLOBAL u32x4_any*)((gfloat)grad + e));
  const u32x2 w = __builtin_nontemporal_load((GLOBAL u32x2_any*)((gu16)grad + e));
  return u32x4{w[0], w[1], 0u, 0u};
}

__device__ __forceinline__ f32x4 widen4(u32x4 w, int dt) {
  if (dt == ZERO_FP32) return __builtin_bit_cast(f32x4, w);
  if (dt == ZERO_BF16)
    return f32x4{widen<ZERO_BF16>(w[0] & 0xFFFFu), widen<ZERO_BF16>(w[0] >> 16), widen<ZERO_BF16>(w[1] & 0xFFFFu),
                 widen<ZERO_BF16>(w[1] >> 16)};
  return f32x4{widen<ZERO_FP16>(w[0] & 0xFFFFu), widen<ZERO_FP16>(w[0] >> 16), widen<ZERO_FP16>(w[1] & 0xFFFFu),
               widen<ZERO_FP16>(w[1] >> 16)};
}

__device__ __forceinline__ float load_grad1(const void* grad, int dt, int64_t e) {
  if (dt == ZERO_FP32) return ((gfloat)grad)[e];
  return widen_any(((gu16)grad)[e], dt);
}

__device__ __forceinline__ void store_param4(void* param, int dt, int64_t e, f32x4 p) {
  if (dt == ZERO_FP32) {
    store4((gfloat)param + e, p);
    return;
  }
  u32x2_any q;
  if (dt == ZERO_BF16) {
    // v_cvt_pk_bf16_f32, the same bits as bf16_rne for every input
    typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
    q = __builtin_bit_cast(u32x2, __builtin_convertvector(p, bf16x4));
  } else {
    q[0] = narrow<ZERO_FP16>(p[0]) | (narrow<ZERO_FP16>(p[1]) << 16);
    q[1] = narrow<ZERO_FP16>(p[2]) | (narrow<ZERO_FP16>(p[3]) << 16);
  }
  __builtin_nontemporal_store(q, (GLOBAL u32x2_any*)((gu16)param + e));
}

__device__ __forceinline__ void store_param1(void* param, int dt, int64_t e, float p) {
  if (dt == ZERO_FP32) {
    ((gfloat)param)[e] = p;
  } else {
    const uint32_t q = dt == ZERO_BF16 ? narrow<ZERO_BF16>(p) : narrow<ZERO_FP16>(p);
    ((gu16)param)[e] = static_cast<uint16_t>(q);
  }
}

// ------------------------------------------------------------------ scalars

// Scalars of every group by value (host form) or from the device.
struct GroupTable {
  AdamScalars s[ZERO_LIST_MAX_GROUPS];
};

// From the device: every lane reads the same bytes and no kernel writes them
// while this one runs, so they are constant memory here and come through the
// scalar cache.
template <typename T>
__device__ __forceinline__ T uniform_load(const T* p) {
  return *(const __attribute__((address_space(4))) T*)(uintptr_t)p;
}

__device__ __forceinline__ bool group_scalars(const GroupTable& host, const zero_step_state* st,
                                              const zero_group_scalars* groups, int group, AdamScalars* out) {
  if (st == nullptr) {
    *out = host.s[group];
    return true;
  }
  if (uniform_load(&st->skip)) return false;
  const float* s = groups[group].scalars;
  *out = AdamScalars{uniform_load(s),     uniform_load(s + 1), uniform_load(s + 2),
                     uniform_load(s + 3), uniform_load(s + 4), uniform_load(s + 5),
                     uniform_load(s + 6), uniform_load(s + 7), uniform_load(s + 8)};
  return true;
}

// ------------------------------------------------------------------ norm

// Adds a square, exact in fp64 (at most 2·24 significant bits), so that one
// fused operation rounds as the product and the sum would.
__device__ __forceinline__ void square(float x, double& acc) {
  const double d = static_cast<double>(x);
  acc = __builtin_fma(d, d, acc);
}

// A sum of squares of fp32 values is not finite exactly if one of them is not:
// finite squares stay below 2^256, and no list is long enough to bring their
// sum near 2^1024.
__device__ __forceinline__ uint32_t not_finite(double sum) { return __builtin_isfinite(sum) ? 0u : 1u; }

// 16 bytes of gradients: four or eight values.
template <int DT>
__device__ __forceinline__ void square16(u32x4 w, double& acc) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    if constexpr (DT == ZERO_FP32) {
      square(__uint_as_float(w[c]), acc);
    } else {
      square(widen<DT>(w[c] & 0xFFFFu), acc);
      square(widen<DT>(w[c] >> 16), acc);
    }
  }
}

// Elements [lo, hi) of one tensor by NT threads: whole 16-byte vectors wherever
// they start (kNormUnroll in flight per thread), then the last few elements.
constexpr int kNormUnroll = 4;
template <int DT, int NT>
__device__ __forceinline__ void square_range(const void* grad, int64_t lo, int64_t hi, int thread, double& acc) {
  constexpr int kPer = DT == ZERO_FP32 ? 4 : 8;
  const gbyte at = (gbyte)grad + lo * (16 / kPer);
  const int nv = static_cast<int>((hi - lo) / kPer);
  auto load = [&](int j) -> u32x4 { return __builtin_nontemporal_load((GLOBAL u32x4_any*)(at + 16 * j)); };
  int j = thread;
  for (; j + (kNormUnroll - 1) * NT < nv; j += kNormUnroll * NT) {
    u32x4 w[kNormUnroll];
#pragma unroll
    for (int u = 0; u < kNormUnroll; ++u) w[u] = load(j + u * NT);
#pragma unroll
    for (int u = 0; u < kNormUnroll; ++u) square16<DT>(w[u], acc);
  }
  for (; j < nv; j += NT) square16<DT>(load(j), acc);
  const int64_t e = lo + static_cast<int64_t>(nv) * kPer + thread;
  if (e < hi) square(load_grad1(grad, DT, e), acc);
}

// The chunk of entry `en` by NT threads.
template <int NT>
__device__ __forceinline__ void square_chunk(const Desc* descs, Entry en, int thread, double& acc) {
  const Desc d = load_desc(descs, en.tensor);
  if (d.grad == nullptr) return;
  const int64_t lo = static_cast<int64_t>(en.chunk) * kNormPer;
  const int64_t hi = lo + kNormPer < d.numel ? lo + kNormPer : d.numel;
  if (d.gdt() == ZERO_BF16) {
    square_range<ZERO_BF16, NT>(d.grad, lo, hi, thread, acc);
  } else if (d.gdt() == ZERO_FP16) {
    square_range<ZERO_FP16, NT>(d.grad, lo, hi, thread, acc);
  } else {
    square_range<ZERO_FP32, NT>(d.grad, lo, hi, thread, acc);
  }
}

// Workgroup b sums the squares of one chunk of one tensor's gradients.  Bound
// by HBM reads: the 195M bf16 gradients of the GPT-2 rank's 47 pieces take
// 59-61 us with the fold (6.4-6.6 TB/s), 60M fp32 ones in 500 ragged tensors
// 38-40 us; the fold, a launch of its own, is 4.5-5 us of either.  Measured in
// one process: two vectors in flight per thread and a cap of 8 wavefronts per
// SIMD +4 and +5%, eight and 3 -1.5 and +2%; caps of 3, 5, 6 and 8 +2 to +4%;
// chunks of 8192 elements +1%, 12,288 +7 and 0%, 32,768 0 and +4%.
STREAMING_KERNEL void list_sqnorm_kernel(const Desc* __restrict__ descs, const Entry* __restrict__ entries,
                                         double* __restrict__ part_sum, uint32_t* __restrict__ part_bad) {
  double acc = 0.0;
  square_chunk<kBlock>(descs, entries[blockIdx.x], static_cast<int>(threadIdx.x), acc);
  uint32_t bad = not_finite(acc);
  block_reduce(acc, bad);
  if (threadIdx.x == 0) {
    part_sum[blockIdx.x] = acc;
    part_bad[blockIdx.x] = bad;
  }
}

// A small list in one workgroup, its wavefronts taking the chunks in turn, with
// no partials to fold: one launch instead of two.  Measured on MI355X, a call
// among others: 65,536 bf16 elements in 16 tensors 5.6 us against 8.8 with two
// launches, 131,072 5.6 (fp32 6.0), 262,144 8.5-9.9; 40,000 in 64 and in 100
// tensors 6.0 against 9.2, 131,072 in 128 7.3-8.4.
constexpr int kSmallThreads = 1024;
constexpr int64_t kSmallChunks = 64, kSmallNumel = 131072;
__global__ __launch_bounds__(kSmallThreads) void list_sqnorm_small_kernel(const Desc* __restrict__ descs,
                                                                          const Entry* __restrict__ entries,
                                                                          int32_t chunks, double* __restrict__ out_sum,
                                                                          int32_t* __restrict__ out_bad) {
  double acc = 0.0;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int c = wave; c < chunks; c += kSmallThreads / 64)
    square_chunk<64>(descs, entries[c], static_cast<int>(threadIdx.x & 63), acc);
  uint32_t bad = not_finite(acc);
  block_reduce<kSmallThreads>(acc, bad);
  if (threadIdx.x == 0) {
    *out_sum = acc;
    *out_bad = static_cast<int32_t>(bad);
  }
}

// ------------------------------------------------------------------ AdamW, fp32 state

// One 256-thread workgroup per 1024 elements of a tensor, thread t owning
// elements 4t .. 4t+3, with the flat tiled update's mapping, launches and
// occupancy cap.  Both state layouts are the same addresses but for the
// distance of two chunks: 1024 floats (arrays) or a whole tile of
// [master | m | v].  Bound by HBM, 28 bytes an element with 16-bit gradients
// and parameters: the 195M parameters of the GPT-2 rank's pieces (tiled) take
// 823-829 us (6.6 TB/s, the flat update's rate: the two table lookups ahead of
// the data hide behind the other workgroups), 60M in 500 ragged tensors off the
// 16-byte lines (arrays) 271-275 us (6.1-6.2 TB/s).  Measured in one process on the
// Llama-7B rank's 842M (tiled, 3.59 ms) and on the ragged ones: 3 wavefronts
// per SIMD -0.5% and +1.7%, 5 +0.8% and +2.8%, 8 +2.1% and +4.2%; launches of
// 2^24 elements +1.5% and +1.9%, of 2^26 +0.4% and -0.1%.
STREAMING_KERNEL void list_adamw_kernel(const Desc* __restrict__ descs, const Entry* __restrict__ entries,
                                        GroupTable host, const zero_step_state* __restrict__ st,
                                        const zero_group_scalars* __restrict__ groups) {
  const Entry en = entries[xcd_grouped(blockIdx.x, gridDim.x)];
  const Desc d = load_desc(descs, en.tensor);
  if (d.grad == nullptr) return;
  const int64_t at = static_cast<int64_t>(en.chunk) * (d.layout() == ZERO_STATE_TILED ? 3 * kTile : kTile) +
                     4 * static_cast<int64_t>(threadIdx.x);
  const int64_t e = static_cast<int64_t>(en.chunk) * kTile + 4 * static_cast<int64_t>(threadIdx.x);
  const gfloat mp = (gfloat)d.state + at, mm = (gfloat)d.m + at, mv = (gfloat)d.v + at;
  AdamScalars s;
  if (e + 4 <= d.numel) {
    const u32x4 g4 = load_grad4(d.grad, d.gdt(), e);
    f32x4 p = load4(mp), m = load4(mm), v = load4(mv);
    if (!group_scalars(host, st, groups, d.group(), &s)) return;
    const f32x4 g = widen4(g4, d.gdt());
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float pc = p[c], mc = m[c], vc = v[c];
      adam_element(g[c], pc, mc, vc, s);
      p[c] = pc;
      m[c] = mc;
      v[c] = vc;
    }
    store4(mp, p);
    store4(mm, m);
    store4(mv, v);
    store_param4(d.param, d.pdt(), e, p);
  } else if (e < d.numel) {
    if (!group_scalars(host, st, groups, d.group(), &s)) return;
    for (int64_t i = e; i < d.numel; ++i) {
      const int64_t k = i - e;
      float p = mp[k], m = mm[k], v = mv[k];
      adam_element(load_grad1(d.grad, d.gdt(), i), p, m, v, s);
      mp[k] = p;
      mm[k] = m;
      mv[k] = v;
      store_param1(d.param, d.pdt(), i, p);
    }
  }
}

// ------------------------------------------------------------------ 8-bit moments

// Hash of a block's number: SplitMix64's output function (Steele, Lea & Flood
// 2014).  Its arguments are the same for a whole wavefront.
__host__ __device__ __forceinline__ uint64_t mix64(uint64_t z) {
  z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
  z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
  return z ^ (z >> 31);
}
constexpr uint64_t kGolden = 0x9E3779B97F4A7C15ull;
constexpr uint32_t kWeyl = 0x9E3779B9u;

constexpr float kTopM = 448.0f, kTopV = 1.875f;
constexpr float kSmallestPeak = 0x1p-110f;
// A second moment whose block is held as zeros reads as 0: eps alone then
// divides the first.
constexpr float kLeastEps8 = 1e-16f;

// Kernels with a cap of their own on the wavefronts per SIMD (STREAMING_KERNEL
// has 4).
#define WAVES_KERNEL(n) __global__ __launch_bounds__(kBlock) __attribute__((amdgpu_waves_per_eu(1, n)))

// A wavefront takes a block, lane l holding elements 4l .. 4l+3, so that every
// access of a wavefront is one contiguous span and a block's peaks need no
// shared memory; a tile's 16 blocks are four 256-thread workgroups.
constexpr int kTileParts = static_cast<int>(kTile8Blocks / (kBlock / 64));
static_assert(kBlock8 == 4 * 64, "a wavefront covers a block");

// What four codes stand for, without their scale.  An m code is an OCP e4m3
// number; a v code is the top of an fp32 pattern whose exponent lies 96 lower
// (its subnormals are fp32's).
__device__ __forceinline__ f32x4 decode_m(uint32_t c) {
  const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(c), false);
  const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(c), true);
  return f32x4{lo[0], lo[1], hi[0], hi[1]};
}
__device__ __forceinline__ f32x4 decode_v(uint32_t c) {
  f32x4 x;
#pragma unroll
  for (int k = 0; k < 4; ++k) x[k] = __uint_as_float(((c >> (8 * k)) & 0xFFu) << 20) * 0x1p96f;
  return x;
}

// Codes from positions: the last factor brings a scaled value down to where
// its code is the top bits of the fp32 pattern, subnormals included; adding
// the dither (20 bits: the part of a step that is cut off) rounds up with its
// probability.  code_m leaves the sign out; v is not negative (or NaN).
__device__ __forceinline__ uint32_t code_m(float m, float inv, uint32_t add) {
  const uint32_t c = ((__float_as_uint((m * inv) * 0x1p-120f) & 0x7FFFFFFFu) + add) >> 20;
  return c < 126u ? c : 126u;
}
// `least`: 1 in a block that is not held as zeros, else 0.
__device__ __forceinline__ uint32_t code_v(float v, float inv, uint32_t least, uint32_t add) {
  const uint32_t c = (__float_as_uint((v * inv) * 0x1p-96f) + add) >> 20;
  const uint32_t v_bits = __float_as_uint(v);
  const uint32_t lo = v_bits < least ? v_bits : least;
  const uint32_t up = c > lo ? c : lo;
  return up < 255u ? up : 255u;
}
// The signs of four values, each at the top of its byte.
__device__ __forceinline__ uint32_t signs(f32x4 m) {
  const uint32_t lo = __builtin_amdgcn_perm(__float_as_uint(m[1]), __float_as_uint(m[0]), 0x0C0C0703u);
  const uint32_t hi = __builtin_amdgcn_perm(__float_as_uint(m[3]), __float_as_uint(m[2]), 0x07030C0Cu);
  return (lo | hi) & 0x80808080u;
}

// The larger of a lane's value and that of the lane of its row that CTRL names.
template <int CTRL>
__device__ __forceinline__ uint32_t max_dpp(uint32_t x) {
  const uint32_t y = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), CTRL, 0xF, 0xF, true));
  return x > y ? x : y;
}

// The peaks of a block, as bit patterns (so that a NaN outweighs all), from
// those of its lanes: lanes 0 .. 31 end with m's and lanes 32 .. 63 with v's,
// both moments in the same six steps.
__device__ __forceinline__ uint32_t max_of(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t block_peaks(uint32_t m, uint32_t v) {
  const auto halves = __builtin_amdgcn_permlane32_swap(m, v, false, false);
  uint32_t x = max_of(halves[0], halves[1]);
  const auto rows = __builtin_amdgcn_permlane16_swap(x, x, false, false);
  x = max_of(rows[0], rows[1]);
  x = max_dpp<0x128>(x);     // row_ror:8
  x = max_dpp<0xB1>(x);      // quad_perm:[1,0,3,2]
  x = max_dpp<0x4E>(x);      // quad_perm:[2,3,0,1]
  return max_dpp<0x141>(x);  // row_half_mirror
}

__device__ __forceinline__ float read_lane(float x, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), lane));
}

// The codes of this lane's four elements (zeros past the tensor's end) and a
// scale: m's in lanes 0 .. 31, v's in the others, so that one division serves
// both.  dither(k): what element k adds to the positions of m and v.
struct Codes {
  uint32_t m, v;
  float scale;
};
template <typename F>
__device__ __forceinline__ Codes encode_block(f32x4 m, f32x4 v, int lane, F&& dither) {
  float top_m = fabsf(m[0]);
  uint32_t top_v = __float_as_uint(v[0]);
#pragma unroll
  for (int k = 1; k < 4; ++k) {
    top_m = __builtin_elementwise_maximum(top_m, fabsf(m[k]));  // a NaN outweighs all here too
    top_v = max_of(top_v, __float_as_uint(v[k]));
  }
  const float peak = __uint_as_float(block_peaks(__float_as_uint(top_m), top_v));
  const bool some = !(peak < kSmallestPeak);
  Codes c;
  c.scale = some ? peak * (lane < 32 ? 1.0f / kTopM : 1.0f / kTopV) : 0.0f;
  const float inv = some ? (lane < 32 ? kTopM : kTopV) / peak : 0.0f;
  const float inv_m = read_lane(inv, 0), inv_v = read_lane(inv, 32);
  const uint32_t least = static_cast<uint32_t>(__ballot(some) >> 32) & 1u;
  c.m = signs(m);
  c.v = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const u32x2 add = dither(k);
    c.m |= code_m(m[k], inv_m, add[0]) << (8 * k);
    c.v |= code_v(v[k], inv_v, least, add[1]) << (8 * k);
  }
  return c;
}

// The parts of one tile.
struct Tile8 {
  gfloat master;
  gbyte m, v;
  gfloat scale_m, scale_v;
};
__device__ __forceinline__ Tile8 tile8(float* state, int64_t tile) {
  const gbyte base = (gbyte)state + tile * kTile8Bytes;
  return Tile8{(gfloat)base, base + 4 * kTile8, base + 5 * kTile8, (gfloat)(base + 6 * kTile8),
               (gfloat)(base + 6 * kTile8) + kTile8Blocks};
}

// The codes of `have` (0 .. 4) elements, one a byte.
__device__ __forceinline__ void store_codes(gbyte to, uint32_t word, int have) {
  if (have == 4) {
    __builtin_nontemporal_store(word, (GLOBAL uint32_t*)to);
    return;
  }
  for (int k = 0; k < have; ++k) to[k] = static_cast<uint8_t>(word >> (8 * k));
}
__device__ __forceinline__ uint32_t load_codes(gbyte from, int have) {
  if (have == 4) return __builtin_nontemporal_load((GLOBAL uint32_t*)from);
  uint32_t w = 0;
  for (int k = 0; k < have; ++k) w |= static_cast<uint32_t>(from[k]) << (8 * k);
  return w;
}

// `have` (0 .. 4) elements of an fp32 array.
__device__ __forceinline__ f32x4 load_have(gfloat p, int have) {
  if (have == 4) return load4(p);
  f32x4 x = {0, 0, 0, 0};
  for (int k = 0; k < have; ++k) x[k] = p[k];
  return x;
}
__device__ __forceinline__ void store_have(gfloat p, int have, f32x4 x) {
  if (have == 4) {
    store4(p, x);
    return;
  }
  for (int k = 0; k < have; ++k) p[k] = x[k];
}

// One block of a tensor and this lane's place in it.
struct Block8 {
  Tile8 t;
  int64_t first;  // the block's first element in the tensor
  int64_t numel;
  int block, lane;                                                  // the block's number in the tile
  __device__ int at() const { return block * kBlock8 + 4 * lane; }  // in the tile
  __device__ int64_t elem() const { return first + 4 * lane; }      // in the tensor
  // How many of the lane's elements are the tensor's; FULL: all of the block's.
  template <bool FULL>
  __device__ int have() const {
    if (FULL) return 4;
    const int64_t left = numel - elem();
    return left >= 4 ? 4 : left > 0 ? static_cast<int>(left) : 0;
  }
};

// Block `block` of tile `chunk`, for the whole wavefront.
__device__ __forceinline__ Block8 block_of(const Desc& d, uint32_t chunk, int block) {
  Block8 b;
  b.t = tile8(d.state, chunk);
  b.block = __builtin_amdgcn_readfirstlane(block);
  b.lane = threadIdx.x & 63;
  b.first = static_cast<int64_t>(chunk) * kTile8 + b.block * kBlock8;
  b.numel = d.numel;
  return b;
}

// Lanes 0 and 32 hold the block's scales.
__device__ __forceinline__ void store_scales(const Block8& w, float scale) {
  if ((w.lane & 31) == 0) (w.lane < 32 ? w.t.scale_m : w.t.scale_v)[w.block] = scale;
}

// One element with the new moments in full precision: adam_element's moments,
// bit for bit, and its parameter but for rounding: the root and the quotients
// are the hardware's approximations (1 ulp each) and two products are fused
// with their sums.  That changes the step p takes by at most 14·2^-24 of
// itself, where the moments it is made of carry four bits.  Measured in one
// process: with adam_element's correctly rounded ones the update takes 2.45
// instead of 2.07 ms (842M parameters) and 196 instead of 188 us (60M ragged
// fp32 ones), and at the best occupancy cap for each 2.39 ms (8 wavefronts per
// SIMD) and 193 us (7).
__device__ __forceinline__ void adam8_element(float g, float& p, float& m, float& v, const AdamScalars& s,
                                              float inv_bc2) {
  g = g * s.gscale;
  const float m_keep = s.b1 * m;
  const float m_add = s.omb1 * g;
  m = m_keep + m_add;
  const float gg = g * g;
  const float v_keep = s.b2 * v;
  const float v_add = s.omb2 * gg;
  v = v_keep + v_add;
  const float d = __builtin_fmaf(__builtin_amdgcn_sqrtf(v), inv_bc2, s.eps);
  const float u = s.step_size * (m * __builtin_amdgcn_rcpf(d));
  p = __builtin_fmaf(p, s.decay, -u);
}

// A lane's gradients as they lie (load_grad4's form).
template <int DT>
__device__ __forceinline__ u32x4 load_grads(const void* grad, int64_t e, int have) {
  if (have == 4) return load_grad4(grad, DT, e);
  u32x4 g = {0, 0, 0, 0};
  for (int k = 0; k < have; ++k) {
    if (DT == ZERO_FP32) {
      g[k] = ((GLOBAL uint32_t*)grad)[e + k];
    } else {
      g[k >> 1] |= static_cast<uint32_t>(((gu16)grad)[e + k]) << (16 * (k & 1));
    }
  }
  return g;
}

template <bool FULL>
__device__ __forceinline__ void adamw8_block(const Desc& d, const Block8& w, const GroupTable& host, uint64_t seed,
                                             uint64_t step, const zero_step_state* st,
                                             const zero_group_scalars* groups) {
  const int have = w.have<FULL>(), at = w.at();
  const u32x4 g4 = d.gdt() == ZERO_FP32 ? load_grads<ZERO_FP32>(d.grad, w.elem(), have)
                                        : load_grads<ZERO_BF16>(d.grad, w.elem(), have);
  f32x4 p = load_have(w.t.master + at, have);
  const uint32_t mc = load_codes(w.t.m + at, have), vc = load_codes(w.t.v + at, have);
  const float sm = w.t.scale_m[w.block], sv = w.t.scale_v[w.block];
  AdamScalars s;  // fetched while the data is on its way
  if (!group_scalars(host, st, groups, d.group(), &s)) return;
  s.eps = fmaxf(s.eps, kLeastEps8);
  if (st != nullptr) step = static_cast<uint64_t>(uniform_load(&st->adam_step));
  const uint64_t block = static_cast<uint64_t>(d.block0 + w.first / kBlock8);
  const uint32_t key = static_cast<uint32_t>(mix64(mix64(seed + kGolden * step) + kGolden * (block + 1)));
  const uint32_t r0 = key + 4u * static_cast<uint32_t>(w.lane) * kWeyl;
  const float inv_bc2 = __builtin_amdgcn_rcpf(s.bc2_sqrt);
  const f32x4 g = widen4(g4, d.gdt());
  f32x4 m = decode_m(mc) * sm, v = decode_v(vc) * sv;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float pk = p[k], mk = m[k], vk = v[k];
    adam8_element(g[k], pk, mk, vk, s, inv_bc2);
    p[k] = pk;
    m[k] = FULL || k < have ? mk : 0.0f;
    v[k] = FULL || k < have ? vk : 0.0f;
  }
  store_have(w.t.master + at, have, p);
  if (have == 4) {
    store_param4(d.param, d.pdt(), w.elem(), p);
  } else {
    for (int k = 0; k < have; ++k) store_param1(d.param, d.pdt(), w.elem() + k, p[k]);
  }
  const Codes c = encode_block(m, v, w.lane, [&](int k) {
    const uint32_t r = r0 + static_cast<uint32_t>(k) * kWeyl;
    return u32x2{r >> 12, r & 0xFFFFFu};
  });
  store_codes(w.t.m + at, c.m, have);
  store_codes(w.t.v + at, c.v, have);
  store_scales(w, c.scale);
}

// Bound by HBM: 16 bytes an element (and 1/16 of scales) with 16-bit gradients
// and parameters.  The 842M parameters of the Llama-7B rank's pieces take
// 2.06-2.08 ms (6.5 TB/s, the fp32 update's rate), 60M ragged fp32 ones 188 us
// (6.4 TB/s).  Measured in one process: 5, 6, 7 and 8 wavefronts per SIMD 2.11,
// 2.08, 2.07 and 2.06 ms, and 186, 188, 190 and 192 us; four blocks a wavefront
// (a quarter of the reductions and divisions, 104 registers) 2.13 ms and 197 us
// at its best cap of 3; XCD groups of 8 to 96 workgroups within 1 and 2%.
// Without the non-temporal hint on the codes 9-13% slower.  The instructions
// have to be few: at this rate HBM leaves a SIMD 98 issue slots for a lane's
// element, of which 58 are used (counters); a form with separate reductions by
// shuffles, two divisions a block and correctly rounded quotients took 3.3 ms.
WAVES_KERNEL(6) void list_adamw8_kernel(const Desc* __restrict__ descs, const Entry* __restrict__ entries,
                                        GroupTable host, uint64_t seed, uint64_t step,
                                        const zero_step_state* __restrict__ st,
                                        const zero_group_scalars* __restrict__ groups) {
  const int64_t b = xcd_grouped(blockIdx.x, gridDim.x);
  const Entry en = entries[b / kTileParts];
  const Desc d = load_desc(descs, en.tensor);
  if (d.grad == nullptr) return;
  const Block8 w = block_of(d, en.chunk, static_cast<int>(b % kTileParts) * (kBlock / 64) + (threadIdx.x >> 6));
  if (w.first >= d.numel) return;
  if (w.first + kBlock8 <= d.numel) {
    adamw8_block<true>(d, w, host, seed, step, st, groups);
  } else {
    adamw8_block<false>(d, w, host, seed, step, st, groups);
  }
}

// ------------------------------------------------------------------ conversion

// Offset of element e of a tensor's fp32 state.
__device__ __forceinline__ int64_t state32_at(const Desc& d, int64_t e) {
  return d.layout() == ZERO_STATE_TILED ? e / kTile * (3 * kTile) + e % kTile : e;
}

// A lane's four elements never straddle two tiles of the fp32 state, whose
// NULL parts read as zeros.
template <bool FULL>
__device__ __forceinline__ void pack_block(const Desc& f, const Block8& w) {
  const int have = w.have<FULL>(), at = w.at();
  const int64_t at32 = state32_at(f, w.elem());
  const f32x4 zero = {0, 0, 0, 0};
  const f32x4 m = f.m ? load_have((gfloat)f.m + at32, have) : zero;
  const f32x4 v = f.v ? load_have((gfloat)f.v + at32, have) : zero;
  const f32x4 p = f.state ? load_have((gfloat)f.state + at32, have) : zero;
  const f32x4 size_v = {fabsf(v[0]), fabsf(v[1]), fabsf(v[2]), fabsf(v[3])};
  // half a step: nearest
  const Codes c = encode_block(m, size_v, w.lane, [](int) { return u32x2{0x80000u, 0x80000u}; });
  store_have(w.t.master + at, have, p);
  store_codes(w.t.m + at, c.m, have);
  store_codes(w.t.v + at, c.v, have);
  store_scales(w, c.scale);
}

// U adjacent blocks, all loads ahead of the stores; a NULL part is not written.
template <int U, bool FULL>
__device__ __forceinline__ void unpack_blocks(const Desc& f, const Block8 (&w)[U]) {
  f32x4 p[U];
  uint32_t mc[U], vc[U];
  float sm[U], sv[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    mc[u] = load_codes(w[u].t.m + w[u].at(), w[u].template have<FULL>());
    vc[u] = load_codes(w[u].t.v + w[u].at(), w[u].template have<FULL>());
    sm[u] = w[u].t.scale_m[w[u].block];
    sv[u] = w[u].t.scale_v[w[u].block];
  }
  if (f.state) {
#pragma unroll
    for (int u = 0; u < U; ++u) p[u] = load_have(w[u].t.master + w[u].at(), w[u].template have<FULL>());
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int have = w[u].template have<FULL>();
    const int64_t at32 = state32_at(f, w[u].elem());
    if (f.m) store_have((gfloat)f.m + at32, have, decode_m(mc[u]) * sm[u]);
    if (f.v) store_have((gfloat)f.v + at32, have, decode_v(vc[u]) * sv[u]);
    if (f.state) store_have((gfloat)f.state + at32, have, p[u]);
  }
}

// A wavefront of an unpacking workgroup: U adjacent blocks.
template <int U>
__device__ __forceinline__ void unpack_wave(const Desc* descs32, const Desc* descs8, const Entry* entries8) {
  constexpr int kParts = kTileParts / U;  // workgroups per tile
  const int64_t b = xcd_grouped(blockIdx.x, gridDim.x);
  const Entry en = entries8[b / kParts];
  const Desc d = load_desc(descs8, en.tensor), f = load_desc(descs32, en.tensor);
  Block8 w[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    w[u] = block_of(d, en.chunk, (static_cast<int>(b % kParts) * (kBlock / 64) + (threadIdx.x >> 6)) * U + u);
  if (w[0].first >= d.numel) return;
  if (w[U - 1].first + kBlock8 <= d.numel) {
    unpack_blocks<U, true>(f, w);
  } else {
    unpack_blocks<U, false>(f, w);
  }
}

// Bound by HBM, 18 bytes an element either way, scales apart.  What differs is
// how many bytes in flight suit each mix of reads and writes (measured on
// MI355X in one process; the GPT-2 rank's 195M parameters, tiled, the
// Llama-7B rank's 842M, 60M in ragged arrays):
//   pack: one block a wavefront, 4 wavefronts per SIMD 518-521 us (6.7 TB/s)
//     for 195M, 3 556, 6 522, 8 531; four blocks at 2 531, at 4 563;
//   unpack of master and moments: one block, 3 per SIMD 545 us (6.4 TB/s) for
//     195M and 174 us for 60M, 4 576 and 172; four blocks at 4 595 and 186;
//   unpack of moments alone: four blocks, 2 per SIMD 1.36 ms (6.2 TB/s) for
//     842M and 95-97 us for 60M, at 4 1.47 and 108; one block at 3 and 4
//     1.83-2.18 and 124-147, at 8 1.47 and 104.  Lists of few tiles (one per
//     compute unit) take the one-block form here too: 40,000 elements 3.2 us
//     on the GPU against 4.6.
constexpr int64_t kFewTiles = 256;

STREAMING_KERNEL void list_pack8_kernel(const Desc* __restrict__ descs32, const Desc* __restrict__ descs8,
                                        const Entry* __restrict__ entries8) {
  const int64_t b = xcd_grouped(blockIdx.x, gridDim.x);
  const Entry en = entries8[b / kTileParts];
  const Desc d = load_desc(descs8, en.tensor), f = load_desc(descs32, en.tensor);
  const Block8 w = block_of(d, en.chunk, static_cast<int>(b % kTileParts) * (kBlock / 64) + (threadIdx.x >> 6));
  if (w.first >= d.numel) return;
  if (w.first + kBlock8 <= d.numel) {
    pack_block<true>(f, w);
  } else {
    pack_block<false>(f, w);
  }
}

WAVES_KERNEL(3) void list_unpack8_kernel(const Desc* __restrict__ descs32, const Desc* __restrict__ descs8,
                                         const Entry* __restrict__ entries8) {
  unpack_wave<1>(descs32, descs8, entries8);
}

WAVES_KERNEL(2) void list_unpack8_moments_kernel(const Desc* __restrict__ descs32, const Desc* __restrict__ descs8,
                                                 const Entry* __restrict__ entries8) {
  unpack_wave<4>(descs32, descs8, entries8);
}

// ------------------------------------------------------------------ decision

struct GroupHparams {
  struct {
    double lr, beta1, beta2, eps, wd;
  } g[ZERO_LIST_MAX_GROUPS];
};

// Thread 0 decides; then thread k derives the scalars of group k.
__global__ __launch_bounds__(64) void list_decision_kernel(const double* __restrict__ sq,
                                                           const int32_t* __restrict__ flags, int32_t n_ranks,
                                                           double max_norm, GroupHparams hp, int32_t n_groups,
                                                           zero_step_state* __restrict__ st,
                                                           zero_group_scalars* __restrict__ groups) {
  __shared__ double gscale;
  __shared__ int64_t t;
  __shared__ bool taken;
  if (threadIdx.x == 0) {
    taken = take_decision(sq, flags, n_ranks, max_norm, st);
    t = st->adam_step;
    gscale = st->grad_scale;
  }
  __syncthreads();
  const int k = static_cast<int>(threadIdx.x);
  if (!taken || k >= n_groups) return;
  const auto& h = hp.g[k];
  float out[9];
  device_scalars(h.lr, h.beta1, h.beta2, h.eps, h.wd, t, gscale, out);
  for (int i = 0; i < 9; ++i) groups[k].scalars[i] = out[i];
  if (k == 0)
    for (int i = 0; i < 9; ++i) st->scalars[i] = out[i];
}
static_assert(ZERO_LIST_MAX_GROUPS <= 64, "one wavefront derives every group's scalars");

// ------------------------------------------------------------------ launches

const Desc* descs_of(const zero_list* l) { return static_cast<const Desc*>(l->table_dev); }
const Entry* entries_of(const zero_list* l, int64_t offset) {
  return reinterpret_cast<const Entry*>(static_cast<const char*>(l->table_dev) + offset);
}

// Elements per launch with 8-bit state: about the bytes of the fp32 update's
// 2^25 elements.  Measured in one process: 842M parameters 2.09 ms with 2^25,
// 2.08 with 2^26, 2.07 with 2^27; 60M 194, 188 and 188 us.
constexpr int64_t kElemsPerLaunch8 = int64_t(1) << 26;

// Issues launch(first entry, count) for each launch over the list.
template <typename F>
int for_each_list_launch(const zero_list* l, int64_t per, const char* fn, F&& launch) {
  const int64_t most = (l->state == 8 ? kElemsPerLaunch8 : kUpdateElemsPerLaunch) / per;
  for (int64_t b = 0; b < l->update_blocks; b += most) {
    launch(entries_of(l, l->update_offset) + b, dim3(static_cast<unsigned>(std::min(most, l->update_blocks - b))));
    const int rc = launch_status(fn);
    if (rc != ZERO_OK) return rc;
  }
  return ZERO_OK;
}

// A list that the update with `state` bits can take.
int update_list_ok(const char* fn, const zero_list* l, int32_t state) {
  const int rc = list_ok(fn, l);
  if (rc != ZERO_OK) return rc;
  if (l->n_tensors > 0 && l->state != state)
    return fail(ZERO_ERR_INVALID, "%s: the list holds %s state", fn,
                l->state == 8 ? "8-bit" : l->state == 32 ? "fp32" : "no");
  if (!(l->flags & ZERO_LIST_HAS_PARAMS)) return fail(ZERO_ERR_INVALID, "%s: a tensor has no param", fn);
  if (!(l->flags & ZERO_LIST_WHOLE_STATE)) return fail(ZERO_ERR_INVALID, "%s: a tensor's state is not whole", fn);
  return ZERO_OK;
}

int host_scalars(const char* fn, const zero_list* l, const zero_adamw_hparams* hp, GroupTable* out) {
  if (!hp) return fail(ZERO_ERR_INVALID, "%s: hparams NULL", fn);
  for (int32_t k = 0; k < l->n_groups; ++k) {
    const int rc = adam_scalars(fn, hp + k, out->s + k);
    if (rc != ZERO_OK) return rc;
  }
  return ZERO_OK;
}

int dev_scalars_ok(const char* fn, const zero_step_state* st, const zero_group_scalars* groups) {
  if (!st || !aligned16(st)) return fail(ZERO_ERR_INVALID, "%s: step state NULL or not 16-byte aligned", fn);
  if (!groups || !aligned16(groups)) return fail(ZERO_ERR_INVALID, "%s: group scalars NULL or not 16-byte aligned", fn);
  return ZERO_OK;
}

int launch_list_adamw(const char* fn, const zero_list* l, const GroupTable& host, const zero_step_state* st,
                      const zero_group_scalars* groups, void* stream) {
  return for_each_list_launch(l, kTile, fn, [&](const Entry* first, dim3 grid) {
    hipLaunchKernelGGL(list_adamw_kernel, grid, dim3(kBlock), 0, static_cast<hipStream_t>(stream), descs_of(l), first,
                       host, st, groups);
  });
}

int launch_list_adamw8(const char* fn, const zero_list* l, const GroupTable& host, uint64_t seed, uint64_t step,
                       const zero_step_state* st, const zero_group_scalars* groups, void* stream) {
  return for_each_list_launch(l, kTile8, fn, [&](const Entry* first, dim3 grid) {
    grid.x *= kTileParts;
    hipLaunchKernelGGL(list_adamw8_kernel, grid, dim3(kBlock), 0, static_cast<hipStream_t>(stream), descs_of(l), first,
                       host, seed, step, st, groups);
  });
}

int convert(const char* fn, const zero_list* l32, const zero_list* l8, bool pack, void* stream) {
  int rc = list_ok(fn, l32);
  if (rc == ZERO_OK) rc = list_ok(fn, l8);
  if (rc != ZERO_OK) return rc;
  if (l32->shape != l8->shape || l32->numel != l8->numel || l32->n_tensors != l8->n_tensors)
    return fail(ZERO_ERR_INVALID, "%s: the two lists' tensors differ in size", fn);
  if (l32->n_tensors > 0 && (l32->state != 32 || l8->state != 8))
    return fail(ZERO_ERR_INVALID, "%s: needs a list with fp32 state and one with 8-bit state", fn);
  const bool one = pack || (l32->flags & ZERO_LIST_WHOLE_STATE) != 0 || l8->update_blocks <= kFewTiles;
  const auto kernel = pack ? list_pack8_kernel : one ? list_unpack8_kernel : list_unpack8_moments_kernel;
  const unsigned parts = one ? kTileParts : kTileParts / 4;  // workgroups per tile
  return for_each_list_launch(l8, kTile8, fn, [&](const Entry* first, dim3 grid) {
    grid.x *= parts;
    hipLaunchKernelGGL(kernel, grid, dim3(kBlock), 0, static_cast<hipStream_t>(stream), descs_of(l32), descs_of(l8),
                       first);
  });
}

}  // namespace

// ====================================================================== C ABI

extern "C" {

int64_t zero_state8_bytes(int64_t n) { return n <= 0 || n > kMaxPsi ? 0 : ceil_div(n, kTile8) * kTile8Bytes; }

int64_t zero_list_table_bytes(const zero_list_tensor* tensors, int32_t n_tensors) {
  zero_list l;
  return table_shape("zero_list_table_bytes", tensors, n_tensors, &l) ? l.table_bytes : 0;
}

int zero_list_plan(const zero_list_tensor* tensors, int32_t n_tensors, int32_t n_groups, void* table_host,
                   int64_t table_bytes, zero_list* out) try {
  const char* fn = "zero_list_plan";
  if (!out || !table_host) return fail(ZERO_ERR_INVALID, "%s: NULL output", fn);
  if (n_groups < 1 || n_groups > ZERO_LIST_MAX_GROUPS)
    return fail(ZERO_ERR_INVALID, "%s: n_groups = %d outside [1, %d]", fn, n_groups, ZERO_LIST_MAX_GROUPS);
  zero_list l;
  if (!table_shape(fn, tensors, n_tensors, &l)) return ZERO_ERR_INVALID;
  if (table_bytes < l.table_bytes)
    return fail(ZERO_ERR_CAPACITY, "%s: table of %lld bytes, %lld needed", fn, static_cast<long long>(table_bytes),
                static_cast<long long>(l.table_bytes));
  std::vector<Desc> descs(static_cast<size_t>(n_tensors));
  const int rc = write_descs(fn, tensors, n_tensors, n_groups, descs.data(), &l.flags);
  if (rc != ZERO_OK) return rc;
  char* table = static_cast<char*>(table_host);
  std::memset(table, 0, static_cast<size_t>(std::min<int64_t>(l.table_bytes, sizeof(Desc))));
  if (n_tensors > 0) std::memcpy(table, descs.data(), static_cast<size_t>(l.grads_bytes));
  write_entries(tensors, n_tensors, kNormPer, table + l.norm_offset);
  if (l.state != 0) write_entries(tensors, n_tensors, l.state == 8 ? kTile8 : kTile, table + l.update_offset);
  l.n_groups = n_groups;
  l.check = list_check(l);
  *out = l;
  return ZERO_OK;
} catch (const std::bad_alloc&) {
  return fail(ZERO_ERR_CAPACITY, "zero_list_plan: out of host memory");
}

int zero_list_repoint(const zero_list_tensor* tensors, int32_t n_tensors, void* table_host, int64_t table_bytes,
                      const zero_list* list) try {
  const char* fn = "zero_list_repoint";
  if (!list || !table_host) return fail(ZERO_ERR_INVALID, "%s: NULL list or table", fn);
  if (list->check != list_check(*list)) return fail(ZERO_ERR_INVALID, "%s: the list was not planned", fn);
  zero_list l;
  if (!table_shape(fn, tensors, n_tensors, &l)) return ZERO_ERR_INVALID;
  if (l.shape != list->shape || l.state != list->state || l.n_tensors != list->n_tensors)
    return fail(ZERO_ERR_INVALID, "%s: the tensors are not the planned ones", fn);
  if (table_bytes < l.grads_bytes)
    return fail(ZERO_ERR_CAPACITY, "%s: table of %lld bytes, %lld needed", fn, static_cast<long long>(table_bytes),
                static_cast<long long>(l.grads_bytes));
  std::vector<Desc> descs(static_cast<size_t>(n_tensors));
  const int rc = write_descs(fn, tensors, n_tensors, list->n_groups, descs.data(), &l.flags);
  if (rc != ZERO_OK) return rc;
  if (l.flags != list->flags)
    return fail(ZERO_ERR_INVALID, "%s: params or state that the plan had are missing (or the reverse)", fn);
  if (n_tensors > 0) std::memcpy(table_host, descs.data(), static_cast<size_t>(l.grads_bytes));
  return ZERO_OK;
} catch (const std::bad_alloc&) {
  return fail(ZERO_ERR_CAPACITY, "zero_list_repoint: out of host memory");
}

size_t zero_list_grad_sqnorm_workspace_bytes(const zero_list* list) {
  if (!list || list->check != list_check(*list)) return 0;
  const size_t need = 12 * static_cast<size_t>(std::max<int64_t>(list->norm_blocks, 1));
  return (need + 255) / 256 * 256;
}

int zero_list_grad_sqnorm(const zero_list* list, void* ws_dev, size_t ws_bytes, double* sqnorm_dev,
                          int32_t* nonfinite_dev, void* stream) {
  const char* fn = "zero_list_grad_sqnorm";
  int rc = list_ok(fn, list);
  if (rc != ZERO_OK) return rc;
  if (!sqnorm_dev || !nonfinite_dev || !ws_dev) return fail(ZERO_ERR_INVALID, "%s: NULL output or workspace", fn);
  if (!aligned16(ws_dev)) return fail(ZERO_ERR_INVALID, "%s: workspace must be 16-byte aligned", fn);
  if (!aligned8(sqnorm_dev) || off(nonfinite_dev, 4)) return fail(ZERO_ERR_INVALID, "%s: misaligned output", fn);
  const size_t need = zero_list_grad_sqnorm_workspace_bytes(list);
  if (ws_bytes < need) return fail(ZERO_ERR_INVALID, "%s: workspace %zu bytes < %zu", fn, ws_bytes, need);
  if (list->norm_blocks <= kSmallChunks && list->numel <= kSmallNumel) {
    hipLaunchKernelGGL(list_sqnorm_small_kernel, dim3(1), dim3(kSmallThreads), 0, static_cast<hipStream_t>(stream),
                       descs_of(list), entries_of(list, list->norm_offset), static_cast<int32_t>(list->norm_blocks),
                       sqnorm_dev, nonfinite_dev);
    return launch_status(fn);
  }
  double* part_sum = static_cast<double*>(ws_dev);
  uint32_t* part_bad = reinterpret_cast<uint32_t*>(part_sum + list->norm_blocks);
  hipLaunchKernelGGL(list_sqnorm_kernel, dim3(static_cast<unsigned>(list->norm_blocks)), dim3(kBlock), 0,
                     static_cast<hipStream_t>(stream), descs_of(list), entries_of(list, list->norm_offset), part_sum,
                     part_bad);
  rc = launch_status(fn);
  if (rc != ZERO_OK) return rc;
  return zero_sqnorm_reduce(part_sum, part_bad, list->norm_blocks, sqnorm_dev, nonfinite_dev, stream);
}

int zero_list_adamw_step(const zero_list* list, const zero_adamw_hparams* hp, void* stream) {
  const char* fn = "zero_list_adamw_step";
  GroupTable host;
  int rc = update_list_ok(fn, list, 32);
  if (rc == ZERO_OK) rc = host_scalars(fn, list, hp, &host);
  return rc != ZERO_OK ? rc : launch_list_adamw(fn, list, host, nullptr, nullptr, stream);
}

int zero_list_adamw_step_dev(const zero_list* list, const zero_step_state* state_dev,
                             const zero_group_scalars* groups_dev, void* stream) {
  const char* fn = "zero_list_adamw_step_dev";
  int rc = update_list_ok(fn, list, 32);
  if (rc == ZERO_OK) rc = dev_scalars_ok(fn, state_dev, groups_dev);
  return rc != ZERO_OK ? rc : launch_list_adamw(fn, list, GroupTable{}, state_dev, groups_dev, stream);
}

int zero_list_adamw8_step(const zero_list* list, const zero_adamw_hparams* hp, uint64_t seed, void* stream) {
  const char* fn = "zero_list_adamw8_step";
  GroupTable host;
  int rc = update_list_ok(fn, list, 8);
  if (rc == ZERO_OK) rc = host_scalars(fn, list, hp, &host);
  if (rc != ZERO_OK) return rc;
  for (int32_t k = 0; k < list->n_groups; ++k) {
    if (!(static_cast<float>(hp[k].eps) >= kLeastEps8))
      return fail(ZERO_ERR_INVALID, "%s: group %d: eps below 1e-16", fn, k);
    if (hp[k].step != hp[0].step) return fail(ZERO_ERR_INVALID, "%s: the groups' steps differ", fn);
  }
  return launch_list_adamw8(fn, list, host, seed, static_cast<uint64_t>(hp[0].step), nullptr, nullptr, stream);
}

int zero_list_adamw8_step_dev(const zero_list* list, const zero_step_state* state_dev,
                              const zero_group_scalars* groups_dev, uint64_t seed, void* stream) {
  const char* fn = "zero_list_adamw8_step_dev";
  int rc = update_list_ok(fn, list, 8);
  if (rc == ZERO_OK) rc = dev_scalars_ok(fn, state_dev, groups_dev);
  return rc != ZERO_OK ? rc : launch_list_adamw8(fn, list, GroupTable{}, seed, 0, state_dev, groups_dev, stream);
}

int zero_list_decision_dev(const double* rank_sqnorms_dev, const int32_t* rank_flags_dev, int32_t n_ranks,
                           double max_norm, const zero_adamw_hparams* hp, int32_t n_groups,
                           zero_step_state* state_dev, zero_group_scalars* groups_dev, void* stream) {
  const char* fn = "zero_list_decision_dev";
  if (n_ranks < 1 || !rank_sqnorms_dev || !rank_flags_dev || !hp)
    return fail(ZERO_ERR_INVALID, "%s: NULL argument or n_ranks < 1", fn);
  if (n_groups < 1 || n_groups > ZERO_LIST_MAX_GROUPS)
    return fail(ZERO_ERR_INVALID, "%s: n_groups = %d outside [1, %d]", fn, n_groups, ZERO_LIST_MAX_GROUPS);
  if (!aligned8(rank_sqnorms_dev) || off(rank_flags_dev, 4)) return fail(ZERO_ERR_INVALID, "%s: misaligned norms", fn);
  const int rc = dev_scalars_ok(fn, state_dev, groups_dev);
  if (rc != ZERO_OK) return rc;
  GroupHparams g{};
  for (int32_t k = 0; k < n_groups; ++k) {
    zero_adamw_hparams h = hp[k];
    h.step = 1;
    h.grad_scale = 1.0;
    AdamScalars s;
    const int rc_k = adam_scalars(fn, &h, &s);
    if (rc_k != ZERO_OK) return rc_k;
    g.g[k] = {h.lr, h.beta1, h.beta2, h.eps, h.weight_decay};
  }
  hipLaunchKernelGGL(list_decision_kernel, dim3(1), dim3(64), 0, static_cast<hipStream_t>(stream), rank_sqnorms_dev,
                     rank_flags_dev, n_ranks, max_norm, g, n_groups, state_dev, groups_dev);
  return launch_status(fn);
}

int zero_list_state8_pack(const zero_list* from32, const zero_list* to8, void* stream) {
  return convert("zero_list_state8_pack", from32, to8, true, stream);
}

int zero_list_state8_unpack(const zero_list* from8, const zero_list* to32, void* stream) {
  return convert("zero_list_state8_unpack", to32, from8, false, stream);
}

}  // extern "C"
