// The kernels of the embedding, layer norm and loss head entry points, run on the CPU (lockstep/hip/hip_runtime.h) under
// sanitizers: buffers have exactly the sizes that the calls may touch, so a byte read or written past one is found, and
// results are compared with sums in 64 bits.
#include <cstdarg>
#include <memory>
#include <random>
#include <string>

#include "hip/hip_runtime.h"
#include "zero_shard.h"

namespace zero_detail {
static char message[256];
int fail(int code, const char* fmt, ...) {
  va_list args;
  va_start(args, fmt);
  std::vsnprintf(message, sizeof message, fmt, args);
  va_end(args);
  return code;
}
int launch_status(const char*) { return ZERO_OK; }
}  // namespace zero_detail

#define CHECK(x)                                                                \
  do {                                                                          \
    if (!(x)) {                                                                 \
      std::printf("line %d: %s (%s)\n", __LINE__, #x, zero_detail::message);    \
      std::exit(1);                                                             \
    }                                                                           \
  } while (0)

static std::mt19937_64 rng(11);
static int below(int n) { return static_cast<int>(rng() % static_cast<uint64_t>(n)); }
static double normal() { return std::normal_distribution<double>()(rng); }

static int bytes_of(int dt) { return dt == ZERO_FP32 ? 4 : 2; }
static double read(const void* p, int64_t i, int dt) {
  if (dt == ZERO_FP32) return static_cast<const float*>(p)[i];
  const uint16_t h = static_cast<const uint16_t*>(p)[i];
  return dt == ZERO_BF16 ? lockstep::bf16_value(h) : lockstep::f16_value(h);
}
static void write(void* p, int64_t i, int dt, double v) {
  const float f = static_cast<float>(v);
  if (dt == ZERO_FP32) {
    static_cast<float*>(p)[i] = f;
  } else if (dt == ZERO_FP16) {
    const _Float16 h = static_cast<_Float16>(f);
    std::memcpy(static_cast<uint16_t*>(p) + i, &h, 2);
  } else {
    uint32_t u;
    std::memcpy(&u, &f, 4);
    static_cast<uint16_t*>(p)[i] = static_cast<uint16_t>((u + 0x7FFF + (u >> 16 & 1)) >> 16);
  }
}
static double step_of(int dt, double v) {  // half a step of a result of this size
  const double rel = dt == ZERO_FP32 ? 0x1p-24 : dt == ZERO_BF16 ? 0x1p-9 : 0x1p-12;
  return std::fabs(v) * rel * 2 + (dt == ZERO_FP16 ? 0x1p-25 : 1e-40);
}

// Memory of exactly n bytes, starting `shift` bytes past a 16-byte line.
struct Memory {
  std::unique_ptr<char[]> all;
  char* data;
  explicit Memory(size_t n, size_t shift = 0) : all(new char[n + shift]), data(all.get() + shift) {
    std::memset(all.get(), 0xFF, n + shift);  // NaN in every format
  }
};

struct Rows {  // random rows whose last ends where their memory ends
  int64_t rows, cols, stride;
  int dt;
  Memory memory;
  zero_rows view;
  Rows(int64_t r, int64_t c, int d, int spare, int shift, double sigma)
      : rows(r), cols(c), stride(c + spare), dt(d),
        memory(r ? static_cast<size_t>(((r - 1) * stride + c) * bytes_of(d)) : 0, static_cast<size_t>(shift * bytes_of(d))),
        view{memory.data, r, c, stride, d, 0} {
    for (int64_t i = 0; i < r; ++i)
      for (int64_t j = 0; j < c; ++j) set(i, j, normal() * sigma);
  }
  double get(int64_t i, int64_t j) const { return read(memory.data, i * stride + j, dt); }
  void set(int64_t i, int64_t j, double v) { write(memory.data, i * stride + j, dt, v); }
  bool spare_untouched() const {
    for (int64_t i = 0; i + 1 < rows; ++i)
      for (int64_t j = cols; j < stride; ++j)
        for (int b = 0; b < bytes_of(dt); ++b)
          if (static_cast<unsigned char>(memory.data[(i * stride + j) * bytes_of(dt) + b]) != 0xFF) return false;
    return true;
  }
};

struct Ids {
  Memory memory;
  int bytes;
  std::vector<int64_t> value;
  Ids(int64_t n, int width, int kind, int64_t vocab) : memory(static_cast<size_t>(n) * width), bytes(width), value(n) {
    for (int64_t t = 0; t < n; ++t) {
      int64_t v = below(static_cast<int>(vocab));
      if (kind == 1) v = vocab / 2;                                                // all the same
      if (kind == 2) v = static_cast<int64_t>(std::exp(below(1000) / 1000.0 * std::log(vocab + 1.0))) - 1;  // skewed
      if (kind == 3 && below(3) == 0) v = below(2) ? -100 : vocab + below(5);      // some outside
      if (v >= vocab && kind == 2) v = vocab - 1;
      value[t] = v;
      if (width == 8) std::memcpy(memory.data + 8 * t, &v, 8);
      const int32_t w = static_cast<int32_t>(v);
      if (width == 4) std::memcpy(memory.data + 4 * t, &w, 4);
    }
  }
};

static void embedding(int64_t tokens, int64_t vocab, int64_t cols, int kind) {
  const int td = below(3), od = below(3), spare = below(2) * below(5), shift = below(3);
  Rows table(vocab, cols, td, spare, shift, 1.0), out(tokens, cols, od, spare, shift, 1.0), grad(vocab, cols, td, spare, shift, 1.0);
  Ids ids(tokens, below(2) ? 8 : 4, kind, vocab);
  const int64_t first = kind == 3 ? vocab / 4 : 0;
  std::printf("embedding %ld tokens, %ld x %ld, kind %d, formats %d %d, spare %d\n", (long)tokens, (long)vocab, (long)cols, kind, td, od, spare);
  std::fflush(stdout);
  CHECK(zero_embed_forward(&table.view, first, ids.memory.data, ids.bytes, 1.5, &out.view, nullptr) == ZERO_OK);
  CHECK(out.spare_untouched());
  for (int64_t t = 0; t < tokens; ++t)
    for (int64_t j = 0; j < cols; ++j) {
      const int64_t at = ids.value[t] - first;
      const double want = at >= 0 && at < vocab ? table.get(at, j) * 1.5 : 0.0;
      CHECK(std::fabs(out.get(t, j) - want) <= step_of(od, want));
    }
  for (int accumulate = 0; accumulate < 2; ++accumulate) {
    std::vector<double> sum(vocab * cols), size(vocab * cols);
    for (int64_t v = 0; v < vocab; ++v)
      for (int64_t j = 0; j < cols; ++j) sum[v * cols + j] = accumulate ? grad.get(v, j) : 0.0, size[v * cols + j] = std::fabs(sum[v * cols + j]);
    for (int64_t t = 0; t < tokens; ++t) {
      const int64_t at = ids.value[t] - first;
      if (at < 0 || at >= vocab) continue;
      for (int64_t j = 0; j < cols; ++j) {
        sum[at * cols + j] += 0.5 * out.get(t, j);
        size[at * cols + j] += std::fabs(0.5 * out.get(t, j));
      }
    }
    const size_t need = zero_embed_grad_workspace_bytes(tokens, vocab, cols);
    Memory ws(need);
    CHECK(zero_embed_grad(ids.memory.data, ids.bytes, first, &out.view, 0.5, &grad.view, accumulate, ws.data, need, nullptr) == ZERO_OK);
    CHECK(grad.spare_untouched());
    for (int64_t v = 0; v < vocab; ++v)
      for (int64_t j = 0; j < cols; ++j) {
        const double want = sum[v * cols + j];
        CHECK(std::fabs(grad.get(v, j) - want) <= step_of(td, want) + size[v * cols + j] * (tokens + 2) * 0x1p-24);
      }
  }
}

static void layernorm(int64_t n, int64_t cols, int center) {
  const int dt = below(3), gdt = below(3), wdt = below(2) ? ZERO_FP32 : dt, spare = below(2) * below(5), shift = below(3);
  std::printf("layer norm %ld x %ld, center %d, formats %d %d %d, spare %d\n", (long)n, (long)cols, center, dt, wdt, gdt, spare);
  std::fflush(stdout);
  Rows x(n, cols, dt, spare, shift, 1.0), y(n, cols, dt, spare, shift, 1.0), dy(n, cols, dt, spare, shift, 1.0), dx(n, cols, dt, spare, shift, 1.0);
  Rows weight(1, cols, wdt, 0, below(3), 1.0), bias(1, cols, wdt, 0, below(3), 1.0), dw(1, cols, gdt, 0, below(3), 1.0), db(1, cols, gdt, 0, below(3), 1.0);
  Memory mean(4 * n), rstd(4 * n);
  CHECK(zero_layernorm_forward(&x.view, weight.memory.data, bias.memory.data, wdt, 1e-3, center, &y.view,
                               center ? reinterpret_cast<float*>(mean.data) : nullptr, reinterpret_cast<float*>(rstd.data), nullptr) == ZERO_OK);
  std::vector<double> sw(cols), sb(cols), zw(cols), zb(cols);
  const size_t need = zero_layernorm_grad_workspace_bytes(n, cols);
  Memory ws(need);
  CHECK(zero_layernorm_grad(&x.view, &dy.view, weight.memory.data, wdt, center, center ? reinterpret_cast<float*>(mean.data) : nullptr,
                            reinterpret_cast<float*>(rstd.data), &dx.view, dw.memory.data, db.memory.data, gdt, 0, ws.data, need, nullptr) == ZERO_OK);
  CHECK(y.spare_untouched() && dx.spare_untouched());
  for (int64_t r = 0; r < n; ++r) {
    double m = 0, v = 0, level = 0, along = 0;
    if (center)
      for (int64_t j = 0; j < cols; ++j) m += x.get(r, j) / cols;
    for (int64_t j = 0; j < cols; ++j) v += (x.get(r, j) - m) * (x.get(r, j) - m) / cols;
    const double s = 1 / std::sqrt(v + 1e-3);
    for (int64_t j = 0; j < cols; ++j) {
      const double h = (x.get(r, j) - m) * s, want = h * weight.get(0, j) + bias.get(0, j), d = dy.get(r, j) * weight.get(0, j);
      CHECK(std::fabs(y.get(r, j) - want) <= step_of(dt, want) + 128 * 0x1p-24 * (4 + std::fabs(h)) * (1 + std::fabs(weight.get(0, j))));
      level += center ? d / cols : 0.0;
      along += d * h / cols;
      sw[j] += dy.get(r, j) * h, zw[j] += std::fabs(dy.get(r, j) * h);
      sb[j] += dy.get(r, j), zb[j] += std::fabs(dy.get(r, j));
    }
    for (int64_t j = 0; j < cols; ++j) {
      const double h = (x.get(r, j) - m) * s, d = dy.get(r, j) * weight.get(0, j), want = s * (d - level - h * along);
      CHECK(std::fabs(dx.get(r, j) - want) <= step_of(dt, want) + 512 * 0x1p-24 * s * (2 + std::fabs(d)) * (2 + std::fabs(h)));
    }
  }
  for (int64_t j = 0; j < cols; ++j) {
    CHECK(std::fabs(dw.get(0, j) - sw[j]) <= step_of(gdt, sw[j]) + (n + 64) * 0x1p-23 * (1 + zw[j]) * 8);
    CHECK(std::fabs(db.get(0, j) - sb[j]) <= step_of(gdt, sb[j]) + (n + 64) * 0x1p-24 * (1 + zb[j]));
  }
}

static void head(int64_t tokens, int64_t vocab, int64_t cols, int kind, bool gradients) {
  const int dt = below(2), spare = below(2) * below(9), shift = below(3) * 4, accumulate = below(2);
  std::printf("head %ld tokens, %ld x %ld, kind %d, format %d, spare %d, shift %d, gradients %d\n", (long)tokens, (long)vocab, (long)cols, kind, dt, spare, shift, gradients);
  std::fflush(stdout);
  Rows x(tokens, cols, dt, spare, shift, 1.0), table(vocab, cols, dt, spare, shift, 0.3), dx(tokens, cols, dt, spare, shift, 1.0), dw(vocab, cols, dt, spare, shift, 1.0);
  Ids labels(tokens, below(2) ? 8 : 4, kind, vocab);
  Memory losses(4 * tokens), loss(4), count(8), state_memory(sizeof(zero_step_state));
  zero_step_state* state = reinterpret_cast<zero_step_state*>(state_memory.data);
  state->loss_scale = 4.0;
  const size_t need = zero_loss_head_workspace_bytes(tokens, vocab, cols, gradients);
  // the library asks for 256-byte lines
  std::unique_ptr<char[]> room(new char[need + 256]);
  char* ws = room.get() + 256 - reinterpret_cast<uintptr_t>(room.get()) % 256;
  std::memset(room.get(), 0xFF, need + 256);
  std::vector<double> old(vocab * cols);
  for (int64_t v = 0; v < vocab; ++v)
    for (int64_t j = 0; j < cols; ++j) old[v * cols + j] = dw.get(v, j);
  float* l = reinterpret_cast<float*>(losses.data);
  int rc = gradients ? zero_loss_head_grad(&x.view, &table.view, labels.memory.data, labels.bytes, 0.5, state, l, reinterpret_cast<float*>(loss.data),
                                           reinterpret_cast<int64_t*>(count.data), &dx.view, &dw.view, accumulate, ws, need, nullptr)
                     : zero_loss_head(&x.view, &table.view, labels.memory.data, labels.bytes, l, reinterpret_cast<float*>(loss.data),
                                      reinterpret_cast<int64_t*>(count.data), ws, need, nullptr);
  CHECK(rc == ZERO_OK);
  CHECK(dx.spare_untouched() && dw.spare_untouched());
  int64_t many = 0;
  for (int64_t v : labels.value) many += v >= 0 && v < vocab;
  CHECK(*reinterpret_cast<int64_t*>(count.data) == many);
  const double factor = 0.5 * 4.0 / static_cast<double>(many ? many : 1);
  std::vector<double> want_dw(vocab * cols), size_dw(vocab * cols);
  double total = 0;
  for (int64_t t = 0; t < tokens; ++t) {
    const int64_t label = labels.value[t];
    if (label < 0 || label >= vocab) {
      CHECK(l[t] == 0.0f);
      for (int64_t j = 0; gradients && j < cols; ++j) CHECK(dx.get(t, j) == 0.0);
      continue;
    }
    std::vector<double> z(vocab), g(vocab);
    double top = -1e300, sum = 0;
    for (int64_t v = 0; v < vocab; ++v) {
      for (int64_t j = 0; j < cols; ++j) z[v] += x.get(t, j) * table.get(v, j);
      top = std::fmax(top, z[v]);
    }
    for (int64_t v = 0; v < vocab; ++v) sum += std::exp(z[v] - top);
    const double lse = top + std::log(sum);
    CHECK(std::fabs(l[t] - (lse - z[label])) <= 1e-4 + cols * 0x1p-20);
    total += lse - z[label];
    if (!gradients) continue;
    for (int64_t v = 0; v < vocab; ++v) g[v] = std::exp(z[v] - lse) - (v == label ? 1.0 : 0.0);
    for (int64_t j = 0; j < cols; ++j) {
      double want = 0, size = 0;
      for (int64_t v = 0; v < vocab; ++v) want += g[v] * table.get(v, j), size += std::fabs(g[v] * table.get(v, j));
      CHECK(std::fabs(dx.get(t, j) - want * factor) <= step_of(dt, want * factor) + (size + 0.01) * factor * 0x1p-7);
      for (int64_t v = 0; v < vocab; ++v) want_dw[v * cols + j] += g[v] * x.get(t, j) * factor, size_dw[v * cols + j] += std::fabs(g[v] * x.get(t, j)) * factor;
    }
  }
  CHECK(std::fabs(*reinterpret_cast<float*>(loss.data) - total / static_cast<double>(many ? many : 1)) <= 1e-4 + cols * 0x1p-20);
  for (int64_t i = 0; gradients && i < vocab * cols; ++i) {
    const double want = want_dw[i] + (accumulate ? old[i] : 0.0);
    CHECK(std::fabs(dw.get(i / cols, i % cols) - want) <= step_of(dt, want) + (size_dw[i] + 1e-4) * 0x1p-7);
  }
}

int main(int argc, char** argv) {
  const std::string part = argc > 1 ? argv[1] : "";
  if (part == "embedding") {
    for (int kind = 0; kind < 4; ++kind) {
      embedding(1, 1, 1, kind);
      embedding(5, 70, 8, kind);
      embedding(70, 200, 13, kind);
      embedding(512, 65, 9, kind);
      embedding(513, 65, 9, kind);
      embedding(700, 1, 3, kind);
      embedding(1500, 511, 11, kind);
      embedding(1500, 512, 2, kind);
      embedding(600, 300, 517, kind);
      embedding(2500, 70'000, 1, kind);
    }
    embedding(0, 70, 5, 0);
    embedding(20'000, 40, 3, 2);
  } else if (part == "norm") {
    for (int center = 0; center < 2; ++center)
      for (int64_t cols : {1, 7, 64, 511, 512, 513, 1023, 1024, 1025, 2047, 2048, 2049, 4103, 6145, 8191, 8200, 16384, 16383})
        layernorm(1 + below(cols > 3000 ? 3 : 9), cols, center);
    layernorm(2200, 5, 1);
    layernorm(600, 1030, 0);
  } else {
    for (int kind = 0; kind < 4; kind += 3) {
      head(1, 1, 1, kind, true);
      head(3, 257, 40, kind, true);
      head(30, 300, 65, kind, true);
      head(257, 100, 64, kind, true);
      head(20, 520, 70, kind, false);
      head(300, 70, 136, kind, false);
    }
    head(0, 30, 16, 0, true);
  }
  std::printf("kernel checks ok\n");
  return 0;
}
