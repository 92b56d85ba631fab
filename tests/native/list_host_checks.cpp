// Drives the host side of the list entry points under sanitizers: sizes, plans, repointing and every argument check.
// Nothing is launched: each device call here is refused first, or covers an empty list.
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <random>
#include <vector>

#include "zero_shard.h"

#define CHECK(x)                                                    \
  do {                                                              \
    if (!(x)) {                                                     \
      std::printf("line %d: %s (%s)\n", __LINE__, #x, zero_last_error()); \
      std::exit(1);                                                 \
    }                                                               \
  } while (0)

static void* at(uint64_t x) { return reinterpret_cast<void*>(x); }

static std::vector<zero_list_tensor> random_list(std::mt19937_64& rng, int n, int layout) {
  std::vector<zero_list_tensor> t(n);
  uint64_t next = 1 << 20;
  auto take = [&](uint64_t bytes, uint64_t align) {
    const uint64_t p = (next + align - 1) / align * align;
    next = p + bytes;
    return at(p);
  };
  for (auto& x : t) {
    std::memset(&x, 0, sizeof x);
    x.numel = rng() % 5 == 0 ? 0 : static_cast<int64_t>(rng() % 100000);
    x.gdt = static_cast<int32_t>(rng() % 3);
    x.pdt = static_cast<int32_t>(rng() % 3);
    x.layout = layout;
    x.group = static_cast<int32_t>(rng() % 3);
    const uint64_t n4 = 4 * static_cast<uint64_t>(x.numel);
    x.grad = rng() % 7 ? take(n4, x.gdt == ZERO_FP32 ? 4 : 2) : nullptr;
    x.param = take(n4, 4);
    if (layout == ZERO_STATE_ARRAYS) {
      x.state = take(n4, 4);
      x.m = static_cast<float*>(take(n4, 4));
      x.v = static_cast<float*>(take(n4, 4));
    } else if (layout == ZERO_STATE_TILED) {
      x.state = take(4 * static_cast<uint64_t>(zero_state_tiled_numel(x.numel)), 16);
    } else if (layout == ZERO_STATE_8BIT) {
      x.state = take(static_cast<uint64_t>(zero_state8_bytes(x.numel)), 16);
    }
  }
  return t;
}

int main() {
  std::mt19937_64 rng(7);
  for (int64_t n : {INT64_MIN, int64_t(-1), int64_t(0), int64_t(1), int64_t(4096), ZERO_MAX_NUMEL, INT64_MAX})
    CHECK(zero_state8_bytes(n) >= 0);
  for (int round = 0; round < 200; ++round) {
    for (int layout = ZERO_STATE_NONE; layout <= ZERO_STATE_8BIT; ++layout) {
      auto t = random_list(rng, static_cast<int>(rng() % 40), layout);
      const int32_t n = static_cast<int32_t>(t.size());
      const int64_t bytes = zero_list_table_bytes(t.data(), n);
      CHECK(bytes > 0);
      std::vector<char> table(bytes);  // exactly sized: a write past it is an error
      zero_list l;
      CHECK(zero_list_plan(t.data(), n, 3, table.data(), bytes, &l) == ZERO_OK);
      CHECK(l.table_bytes == bytes && l.n_tensors == n);
      CHECK(zero_list_plan(t.data(), n, 3, table.data(), bytes - 1, &l) == ZERO_ERR_CAPACITY);
      std::vector<char> grads(l.grads_bytes + 1);
      for (auto& x : t) x.grad = rng() % 2 ? x.grad : nullptr;
      CHECK(zero_list_repoint(t.data(), n, grads.data(), l.grads_bytes, &l) == ZERO_OK);
      CHECK(grads.back() == 0);  // nothing past the descriptors
      if (n > 0) CHECK(zero_list_repoint(t.data(), n - 1, grads.data(), l.grads_bytes, &l) == ZERO_ERR_INVALID);
      for (auto& x : t) {  // one bad entry at a time
        const zero_list_tensor good = x;
        x.gdt = 9;
        CHECK(zero_list_plan(t.data(), n, 3, table.data(), bytes, &l) == ZERO_ERR_INVALID);
        x = good;
        x.numel = INT64_MAX;
        CHECK(zero_list_table_bytes(t.data(), n) == 0);
        x = good;
        x.layout = INT32_MIN;
        CHECK(zero_list_table_bytes(t.data(), n) == 0);
        x = good;
        x.group = 3;
        CHECK(zero_list_plan(t.data(), n, 3, table.data(), bytes, &l) == ZERO_ERR_INVALID);
        x = good;
        if (x.numel > 0 && x.param) {
          x.param = at(UINT64_MAX - 3);
          CHECK(zero_list_plan(t.data(), n, 3, table.data(), bytes, &l) == ZERO_ERR_INVALID);
        }
        x = good;
      }
    }
  }
  CHECK(zero_list_table_bytes(nullptr, 1) == 0 && zero_list_table_bytes(nullptr, -1) == 0);
  // too many elements or workgroups
  std::vector<zero_list_tensor> big(600);
  for (auto& x : big) {
    std::memset(&x, 0, sizeof x);
    x.numel = int64_t(1) << 40;
  }
  CHECK(zero_list_table_bytes(big.data(), 600) == 0);

  char table[64];
  zero_list empty;
  CHECK(zero_list_plan(nullptr, 0, 1, table, sizeof table, &empty) == ZERO_OK);
  zero_adamw_hparams hp[64];
  for (auto& h : hp) h = {1e-3, 0.9, 0.999, 1e-8, 0.1, 1.0, 1};
  CHECK(zero_list_adamw_step(&empty, hp, nullptr) == ZERO_OK);
  CHECK(zero_list_adamw_step(&empty, nullptr, nullptr) == ZERO_ERR_INVALID);
  CHECK(zero_list_adamw8_step(&empty, hp, 0, nullptr) == ZERO_OK);
  CHECK(zero_list_state8_pack(&empty, &empty, nullptr) == ZERO_OK);
  CHECK(zero_list_state8_unpack(&empty, nullptr, nullptr) == ZERO_ERR_INVALID);
  CHECK(zero_list_adamw_step_dev(&empty, nullptr, nullptr, nullptr) == ZERO_ERR_INVALID);
  CHECK(zero_list_adamw8_step_dev(&empty, nullptr, nullptr, 0, nullptr) == ZERO_ERR_INVALID);
  CHECK(zero_list_grad_sqnorm(&empty, nullptr, 0, nullptr, nullptr, nullptr) == ZERO_ERR_INVALID);
  CHECK(zero_list_grad_sqnorm_workspace_bytes(nullptr) == 0);
  zero_list junk;
  std::memset(&junk, 0x5A, sizeof junk);
  CHECK(zero_list_adamw_step(&junk, hp, nullptr) == ZERO_ERR_INVALID);
  CHECK(zero_list_grad_sqnorm_workspace_bytes(&junk) == 0);
  double sq = 0.0;
  int32_t flag = 0;
  for (int g : {0, 65, -1, INT32_MAX})
    CHECK(zero_list_decision_dev(&sq, &flag, 1, 1.0, hp, g, static_cast<zero_step_state*>(at(16)),
                                 static_cast<zero_group_scalars*>(at(16)), nullptr) == ZERO_ERR_INVALID);
  hp[63].lr = NAN;
  CHECK(zero_list_decision_dev(&sq, &flag, 1, 1.0, hp, 64, static_cast<zero_step_state*>(at(16)),
                               static_cast<zero_group_scalars*>(at(16)), nullptr) == ZERO_ERR_INVALID);
  std::printf("list host checks ok\n");
  return 0;
}
