// Host-side checks of the dense operators' entry points (abi_dense.cpp) under
// AddressSanitizer and UndefinedBehaviorSanitizer, on the CPU, linked against
// stub launchers: sizes at the ends of their types, the workspace sums, and
// the optimiser's split of a long list into launches, whose arguments the
// stub checks entry by entry.
#include <climits>
#include <cstdint>
#include <cstdio>
#include <vector>

#include <hip/hip_runtime.h>

#include "dense_args.h"
#include "moe.h"

static int g_launches = 0, g_failed = 0;
static void check(bool ok, const char* what) {
  if (!ok) {
    ++g_failed;
    std::printf("FAILED: %s\n", what);
  }
}

static std::vector<moe::AdamwArgs> g_adamw;
static std::vector<uint32_t> g_chunks;
static int g_advanced = 0;

extern "C" {
int moe_norm_backward_parts(int64_t T, int32_t) { return (int)(T < 512 ? T : 512); }
moe_status_t moe_add_rmsnorm_launch(const moe::NormArgs*, int, int, hipStream_t) { ++g_launches; return MOE_OK; }
moe_status_t moe_rmsnorm_backward_launch(const moe::NormBwdArgs*, int, int, float*, hipStream_t) {
  ++g_launches;
  return MOE_OK;
}
size_t moe_gated_ffn_ws_impl(int64_t T, int32_t d, int32_t f, int, int) { return 256 + (size_t)T * (d + f) * 4; }
moe_status_t moe_gated_ffn_launch(const uint16_t*, int64_t, const uint16_t*, const uint16_t*, const uint16_t*, int64_t,
                                  int64_t, int32_t, int32_t, uint16_t*, uint16_t*, uint16_t*, void*, hipStream_t) {
  ++g_launches;
  return MOE_OK;
}
size_t moe_gated_ffn_backward_ws_impl(int64_t, int32_t, int32_t) { return 256; }
moe_status_t moe_gated_ffn_backward_launch(const uint16_t*, const uint16_t*, const uint16_t*, const uint16_t*,
                                           const uint16_t*, const uint16_t*, int64_t, int32_t, int32_t, uint16_t*,
                                           uint16_t*, void*, void*, int, void*, hipStream_t) {
  ++g_launches;
  return MOE_OK;
}
moe_status_t moe_adamw_launch(const moe::AdamwArgs* a, uint32_t chunks, int, int, int, hipStream_t) {
  g_adamw.push_back(*a);
  g_chunks.push_back(chunks);
  return MOE_OK;
}
moe_status_t moe_adamw_advance_launch(int32_t*, const float*, hipStream_t) {
  ++g_advanced;
  return MOE_OK;
}
}

static uint16_t* u16(uintptr_t p) { return reinterpret_cast<uint16_t*>(p); }

static void adamw_lists(const std::vector<int64_t>& n) {
  g_adamw.clear();
  g_chunks.clear();
  g_advanced = 0;
  std::vector<moe_adamw_tensor> t;
  for (size_t i = 0; i < n.size(); ++i) {
    const uintptr_t at = 0x10000 * (i + 1);
    t.push_back({(void*)at, nullptr, (void*)(at + 16), (void*)(at + 32), (void*)(at + 48), nullptr, nullptr, n[i]});
  }
  moe_adamw_config c{1e-3, 0.9, 0.99, 1e-8, 0.1, 32, MOE_OUT_BF16, MOE_OUT_BF16, 5};
  int32_t step = 0;
  check(moe_adamw_step(t.data(), (int32_t)t.size(), &c, &step, nullptr, nullptr) == MOE_OK, "adamw list");
  check(g_advanced == 1, "one advance");
  size_t next = 0;
  for (size_t l = 0; l < g_adamw.size(); ++l) {
    const moe::AdamwArgs& a = g_adamw[l];
    while (next < (size_t)a.first) check(n[next++] == 0, "only empty tensors are left out");
    check(a.count >= 1 && a.count <= moe::kAdamwTensors, "count");
    uint32_t at = 0;
    for (int k = 0; k < a.count; ++k, ++next) {
      check(a.t[k].p == t[next].param && a.t[k].n == n[next], "entry");
      check(a.start[k] == at, "start");
      at += (uint32_t)((n[next] + moe::kAdamwChunk - 1) / moe::kAdamwChunk);
    }
    check(a.start[a.count] == at && g_chunks[l] == at && at > 0 && at <= (uint32_t)INT_MAX, "chunks");
  }
  while (next < n.size()) check(n[next++] == 0, "every tensor is in a launch");
}

int main() {
  const uintptr_t P = 1 << 20;
  void* const ws = (void*)P;
  check(moe_add_rmsnorm(u16(P), 64, u16(P), 0, nullptr, 0, 0, nullptr, 0, 4, 64, 1e-6f, u16(P), nullptr, nullptr, nullptr,
                        nullptr) == MOE_OK && g_launches == 1, "norm");
  check(moe_add_rmsnorm(u16(P), INT64_MAX / 8, u16(P), 0, u16(P), 1, INT64_MAX / 8, u16(P), INT64_MAX / 8, INT32_MAX, 64,
                        1e-6f, u16(P), nullptr, nullptr, nullptr, nullptr) == MOE_OK, "norm, largest pitches");
  check(moe_add_rmsnorm(u16(P), 64, u16(P), 0, nullptr, 0, 0, nullptr, 0, INT64_MAX, 64, 1e-6f, u16(P), nullptr, nullptr,
                        nullptr, nullptr) == MOE_ERR_UNSUPPORTED, "norm, T");
  check(moe_add_rmsnorm_backward_workspace_bytes(INT64_MAX, 64) == 0, "norm ws, T");
  check(moe_add_rmsnorm_backward_workspace_bytes(INT32_MAX, 32768) == (size_t)512 * 32768 * 4, "norm ws");
  check(moe_gated_ffn_workspace_bytes(INT64_MAX, 64, 64, 0, 0) == 0, "ffn ws, T");
  check(moe_gated_ffn_workspace_bytes(4, INT32_MAX - 7, 64, 0, 0) == 0, "ffn ws, d");
  check(moe_gated_ffn_backward_workspace_bytes(INT64_MAX, 64, 64) == 0, "ffn backward ws, T");
  const int before = g_launches;
  check(moe_gated_ffn(u16(P), 64, u16(P), u16(P), nullptr, 0, INT64_MAX, 64, 64, nullptr, nullptr, u16(2 * P), ws,
                      SIZE_MAX, nullptr) == MOE_ERR_UNSUPPORTED, "ffn, T");
  check(moe_gated_ffn(u16(P), 64, u16(P), u16(P), nullptr, 0, 4, 64, INT32_MAX - 7, nullptr, nullptr, u16(2 * P), ws,
                      SIZE_MAX, nullptr) == MOE_ERR_UNSUPPORTED, "ffn, f");
  check(g_launches == before, "nothing launched");
  check(moe_gated_ffn(u16(P), 64, u16(P), u16(P), nullptr, 0, INT32_MAX, 64, 64, nullptr, nullptr, u16(2 * P), ws, SIZE_MAX,
                      nullptr) == MOE_OK, "ffn, largest T");
  // in place, the rows read and written must be the same ones
  const int placed = g_launches;
  check(moe_add_rmsnorm(u16(P), 64, u16(P), 0, u16(2 * P), 0, 80, u16(2 * P), 64, 4, 64, 1e-6f, u16(3 * P), nullptr,
                        nullptr, nullptr, nullptr) == MOE_ERR_INVALID_ARG, "s in r's place, another pitch");
  check(moe_add_rmsnorm(u16(P), 80, u16(P), 0, u16(2 * P), 0, 64, u16(P), 64, 4, 64, 1e-6f, u16(3 * P), nullptr, nullptr,
                        nullptr, nullptr) == MOE_ERR_INVALID_ARG, "s in x's place, another pitch");
  check(moe_add_rmsnorm_backward(u16(P), 80, u16(2 * P), 0, 64, u16(P), 0, (float*)P, nullptr, 0, 4, 64, u16(P), nullptr,
                                 (float*)P, ws, SIZE_MAX, nullptr) == MOE_ERR_INVALID_ARG, "dx in dy's place");
  check(g_launches == placed, "nothing launched in place");
  check(moe_add_rmsnorm(u16(P), 64, u16(P), 0, u16(2 * P), 0, 80, u16(2 * P), 80, 4, 64, 1e-6f, u16(3 * P), nullptr,
                        nullptr, nullptr, nullptr) == MOE_OK, "s in r's place");
  check(moe_add_rmsnorm_backward(u16(P), 64, u16(2 * P), 0, 64, u16(P), 0, (float*)P, nullptr, 0, 4, 64, u16(P), nullptr,
                                 (float*)P, ws, SIZE_MAX, nullptr) == MOE_OK, "dx in dy's place");
  // workgroup numbers past one launch dimension
  for (int64_t n : {(int64_t)1, moe::kGridX - 1, moe::kGridX, moe::kGridX + 1, (int64_t)INT32_MAX})
    check(moe::grid_x(n) * moe::grid_y(n) >= n && moe::grid_x(n) * moe::grid_y(n) - n < moe::kGridX &&
              moe::grid_x(n) * 1024 < ((int64_t)1 << 32) && moe::grid_y(n) <= 65535, "grid");
  adamw_lists({});
  adamw_lists({0, 0});
  adamw_lists({1});
  adamw_lists({8192, 8193, 0, 1});
  adamw_lists(std::vector<int64_t>(40, 10));
  adamw_lists(std::vector<int64_t>(41, 10));
  adamw_lists(std::vector<int64_t>(81, 0));
  std::vector<int64_t> mixed;
  for (int i = 0; i < 200; ++i) mixed.push_back(i % 3 ? 100 * i : 0);
  adamw_lists(mixed);
  const int64_t most = ((int64_t)1 << 40) - 1;
  adamw_lists(std::vector<int64_t>(20, most));      // 2^27 chunks each
  std::printf("ok: %d checks failed\n", g_failed);
  return g_failed != 0;
}
