// Runs the library's kernels on the CPU, for the checks of memory and arithmetic that a sanitizer can make there: every
// thread of a workgroup is a fiber, the lanes of a wavefront meet at each cross-lane operation, and workgroups run one
// after the other.  Only what the kernels of the embedding, the layer norm and the loss head use.  It says nothing of
// timing, of waits or of races between workgroups.
#ifndef LOCKSTEP_HIP_RUNTIME_H
#define LOCKSTEP_HIP_RUNTIME_H

#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <functional>
#include <vector>

#define __global__
#define __device__
#define __host__
#define __forceinline__ inline
#define __launch_bounds__(...)
#define __shared__ static

struct dim3 {
  unsigned x, y, z;
  dim3(int64_t x_ = 1, int64_t y_ = 1, int64_t z_ = 1) : x(x_), y(y_), z(z_) {}
};
struct float2 {
  float x, y;
};
struct alignas(8) uint2 {
  uint32_t x, y;
};
inline float2 make_float2(float x, float y) { return {x, y}; }
inline uint2 make_uint2(uint32_t x, uint32_t y) { return {x, y}; }
typedef void* hipStream_t;

namespace lockstep {

struct Vec {  // up to three operands of 16 bytes
  uint32_t w[12];
};

struct Fiber {
  void* stack = nullptr;  // where it goes on
  dim3 thread;
  int state = 0;  // 0 can run, 1 at a cross-lane operation, 2 at the barrier, 3 ended
  int kind = 0, site = 0;
  Vec in, out;
};

inline std::vector<Fiber>& fibers() {
  static std::vector<Fiber> f;
  return f;
}
inline void* home;
inline Fiber* now;
inline dim3 block, blocks, threads;
inline const std::function<void()>* body;
inline int barrier_or;

// Puts this stack's registers away and goes on where `to` left (x86-64: six registers and the return address).
extern "C" void lockstep_switch(void** from, void* to);
asm(".text\n.weak lockstep_switch\nlockstep_switch:\n"
    "push %rbp\npush %rbx\npush %r12\npush %r13\npush %r14\npush %r15\n"
    "mov %rsp, (%rdi)\nmov %rsi, %rsp\n"
    "pop %r15\npop %r14\npop %r13\npop %r12\npop %rbx\npop %rbp\nret\n");

inline void leave(int state) {
  Fiber* me = now;
  me->state = state;
  lockstep_switch(&me->stack, home);
}
inline void start() {
  (*body)();
  leave(3);
}

enum { kBallot = 1, kXor, kUp, kRead, kFirst, kMeet, kMfmaBf16, kMfmaF16 };

inline float bf16_value(uint16_t h) {
  const uint32_t u = static_cast<uint32_t>(h) << 16;
  float f;
  std::memcpy(&f, &u, 4);
  return f;
}
inline float f16_value(uint16_t h) {
  _Float16 f;
  std::memcpy(&f, &h, 2);
  return static_cast<float>(f);
}

// One operation of the lanes `on` of a wavefront.
inline void resolve(Fiber* wave, uint64_t on, int kind) {
  const int first = __builtin_ctzll(on);
  uint64_t ballot = 0;
  for (int l = 0; l < 64; ++l)
    if (on >> l & 1 && kind == kBallot && wave[l].in.w[0]) ballot |= 1ull << l;
  for (int l = 0; l < 64; ++l) {
    if (!(on >> l & 1)) continue;
    Fiber& f = wave[l];
    int from = l;
    switch (kind) {
      case kBallot:
        f.out.w[0] = static_cast<uint32_t>(ballot);
        f.out.w[1] = static_cast<uint32_t>(ballot >> 32);
        break;
      case kXor: from = l ^ static_cast<int>(f.in.w[2]); break;
      case kUp: from = l >= static_cast<int>(f.in.w[2]) ? l - static_cast<int>(f.in.w[2]) : l; break;
      case kRead: from = static_cast<int>(f.in.w[2]); break;
      case kFirst: from = first; break;
      case kMfmaBf16:
      case kMfmaF16: {
        if (on != ~0ull) std::abort();  // a matrix instruction needs the whole wavefront
        const auto value = kind == kMfmaBf16 ? bf16_value : f16_value;
        for (int q = 0; q < 4; ++q) {
          const int m = l / 16 * 4 + q, n = l % 16;
          float c;
          std::memcpy(&c, &f.in.w[8 + q], 4);
          double sum = c;
          for (int k = 0; k < 32; ++k) {
            const uint32_t a = wave[k / 8 * 16 + m].in.w[k % 8 / 2], b = wave[k / 8 * 16 + n].in.w[4 + k % 8 / 2];
            sum += static_cast<double>(value(static_cast<uint16_t>(k & 1 ? a >> 16 : a))) *
                   value(static_cast<uint16_t>(k & 1 ? b >> 16 : b));
          }
          c = static_cast<float>(sum);
          std::memcpy(&f.out.w[q], &c, 4);
        }
        break;
      }
    }
    if (kind >= kXor && kind <= kFirst) {
      if (!(on >> from & 1)) std::abort();  // a lane that takes no part
      std::memcpy(f.out.w, wave[from].in.w, 8);
    }
  }
  for (int l = 0; l < 64; ++l)
    if (on >> l & 1) wave[l].state = 0;
}

inline void run_block() {
  std::vector<Fiber>& f = fibers();
  const int n = static_cast<int>(threads.x);
  static std::vector<char> stacks;
  constexpr size_t kStack = 256 << 10;
  if (static_cast<int>(f.size()) != n) {
    f = std::vector<Fiber>(n);
    stacks.resize(kStack * n);
  }
  for (int t = 0; t < n; ++t) {
    void** top = reinterpret_cast<void**>(stacks.data() + kStack * (t + 1)) - 2;
    top = reinterpret_cast<void**>(reinterpret_cast<uintptr_t>(top) & ~uintptr_t(15));
    *--top = nullptr;  // what start() would return to: it never does
    *--top = reinterpret_cast<void*>(start);
    f[t].stack = top - 6;
    f[t].thread = dim3(t, 0, 0);
    f[t].state = 0;
  }
  for (;;) {
    bool ran = false;
    for (int t = 0; t < n; ++t)
      if (f[t].state == 0) {
        now = &f[t];
        lockstep_switch(&home, f[t].stack);
        ran = true;
      }
    bool moved = false, ended = true;
    for (int w = 0; w < n; w += 64) {  // lanes that wait at the first place of the code meet first
      int site = 1 << 30;
      for (int l = 0; l < 64; ++l)
        if (f[w + l].state == 1 && f[w + l].site < site) site = f[w + l].site;
      uint64_t on = 0;
      int kind = 0;
      for (int l = 0; l < 64; ++l)
        if (f[w + l].state == 1 && f[w + l].site == site) {
          on |= 1ull << l;
          kind = f[w + l].kind;
        }
      if (on) {
        resolve(&f[w], on, kind);
        moved = true;
      }
    }
    if (moved) continue;
    int any = 0;
    for (int t = 0; t < n; ++t)
      if (f[t].state == 2) {
        ended = false;
        any |= static_cast<int>(f[t].in.w[0]);
      }
    if (ended) return;
    barrier_or = any;
    for (int t = 0; t < n; ++t)
      if (f[t].state == 2) f[t].state = 0;
    (void)ran;
  }
}

template <typename F>
void launch(dim3 grid, dim3 group, F&& call) {
  if (static_cast<uint64_t>(grid.x) * grid.y * grid.z * group.x >= (1ull << 32) || group.x % 64 || group.x > 1024 || !grid.x)
    std::abort();
  const std::function<void()> f = call;
  body = &f;
  blocks = grid;
  threads = group;
  for (unsigned y = 0; y < grid.y; ++y)
    for (unsigned x = 0; x < grid.x; ++x) {
      block = dim3(x, y, 0);
      run_block();
    }
}

inline Vec ask(int kind, int site, const Vec& in) {
  now->in = in;
  now->kind = kind;
  now->site = site;
  leave(1);
  return now->out;
}
template <typename T>
T lanes(int kind, int site, T value, int arg) {
  static_assert(sizeof(T) <= 8, "one or two words");
  Vec v{};
  std::memcpy(v.w, &value, sizeof(T));
  v.w[2] = static_cast<uint32_t>(arg);
  v = ask(kind, site, v);
  std::memcpy(&value, v.w, sizeof(T));
  return value;
}
inline uint64_t ballot(bool p, int site) {
  Vec v{};
  v.w[0] = p;
  v = ask(kBallot, site, v);
  return v.w[0] | static_cast<uint64_t>(v.w[1]) << 32;
}
template <typename A, typename C>
C matrix(int kind, int site, A a, A b, C c) {
  Vec v{};
  std::memcpy(v.w, &a, 16);
  std::memcpy(v.w + 4, &b, 16);
  std::memcpy(v.w + 8, &c, 16);
  v = ask(kind, site, v);
  std::memcpy(&c, v.w, 16);
  return c;
}
inline int barrier(int value) {
  now->in.w[0] = static_cast<uint32_t>(value);
  leave(2);
  return barrier_or;
}

struct Buffer {
  const char* data;
  uint32_t bytes;
};
template <typename Lds>
void load_lds(const Buffer& r, Lds lds, uint32_t voffset, uint32_t soffset) {
  const uint64_t at = static_cast<uint64_t>(voffset) + soffset;
  char* to = (char*)lds + now->thread.x % 64 * 16;
  for (int k = 0; k < 16; k += 4) {  // past the end: zeros
    uint32_t w = 0;
    if (at + k + 4 <= r.bytes) std::memcpy(&w, r.data + at + k, 4);
    std::memcpy(to + k, &w, 4);
  }
}

}  // namespace lockstep

#define threadIdx (lockstep::now->thread)
#define blockIdx (lockstep::block)
#define gridDim (lockstep::blocks)
#define hipLaunchKernelGGL(kernel, grid, group, lds, stream, ...) \
  lockstep::launch(grid, group, [&, lockstep_stream = (stream)] { (void)lockstep_stream; kernel(__VA_ARGS__); })
#define __syncthreads() (void)lockstep::barrier(0)
#define __syncthreads_or(p) lockstep::barrier((p) ? 1 : 0)
#define __ballot(p) lockstep::ballot((p), __LINE__)
#define __shfl_xor(v, off, w) lockstep::lanes(lockstep::kXor, __LINE__, (v), (off))
#define __shfl_up(v, off, w) lockstep::lanes(lockstep::kUp, __LINE__, (v), (off))
#define __popcll(x) __builtin_popcountll(x)
#define __builtin_amdgcn_readlane(v, l) lockstep::lanes(lockstep::kRead, __LINE__, static_cast<int>(v), static_cast<int>(l))
#define __builtin_amdgcn_readfirstlane(v) lockstep::lanes(lockstep::kFirst, __LINE__, static_cast<int>(v), 0)
#define __builtin_amdgcn_wave_barrier() (void)lockstep::ask(lockstep::kMeet, __LINE__, lockstep::Vec{})
#define __builtin_amdgcn_fence(order, scope) (void)0
#define __builtin_amdgcn_s_waitcnt(counters) (void)0
#define __builtin_amdgcn_exp2f(x) exp2f(x)
#define __builtin_amdgcn_logf(x) log2f(x)
#define __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, x, y, z) lockstep::matrix(lockstep::kMfmaBf16, __LINE__, a, b, c)
#define __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, x, y, z) lockstep::matrix(lockstep::kMfmaF16, __LINE__, a, b, c)
#define __amdgpu_buffer_rsrc_t lockstep::Buffer
#define __builtin_amdgcn_make_buffer_rsrc(p, stride, n, flags) lockstep::Buffer{static_cast<const char*>(p), static_cast<uint32_t>(n)}
#define __builtin_amdgcn_raw_ptr_buffer_load_lds(r, lds, size, voffset, soffset, off, aux) lockstep::load_lds(r, lds, voffset, soffset)

inline float __uint_as_float(uint32_t u) {
  float f;
  std::memcpy(&f, &u, 4);
  return f;
}
inline uint32_t __float_as_uint(float f) {
  uint32_t u;
  std::memcpy(&u, &f, 4);
  return u;
}
inline uint32_t atomicAdd(uint32_t* p, uint32_t v) {
  const uint32_t old = *p;
  *p += v;
  return old;
}
inline uint32_t atomicOr(uint32_t* p, uint32_t v) {
  const uint32_t old = *p;
  *p |= v;
  return old;
}
template <typename A, typename B>
inline auto min(A a, B b) { return b < a ? b : a; }
using std::isfinite;

#endif
