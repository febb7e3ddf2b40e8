// Every call of the feed-forward block and the norms, refused for its arguments while the host has no
// memory for the error's text: each has to return its status, an exception may not leave it.
// Prints one line per call: its name and its status.
#include <cstdio>
#include <cstdlib>
#include <new>

#include "../../include/fp8z1.h"

static bool no_memory = false;

void* operator new(std::size_t n) {
  void* p = no_memory ? nullptr : std::malloc(n ? n : 1);
  if (!p) throw std::bad_alloc();
  return p;
}
void operator delete(void* p) noexcept { std::free(p); }
void operator delete(void* p, std::size_t) noexcept { std::free(p); }

#define CALL(name, ...)                       \
  do {                                        \
    no_memory = true;                         \
    const int rc = name(__VA_ARGS__);         \
    const char* const text = fp8z1_last_error(); \
    no_memory = false;                        \
    std::printf("%s %d %s\n", #name, rc, text); \
    std::fflush(stdout);                      \
  } while (0)

int main() {
  fp8z1_ffn f = {4, 2, 64, 32, FP8Z1_BF16, FP8Z1_ACT_SILU};
  fp8z1_ffn wrong = {4, 2, 64, 32, FP8Z1_E4M3, FP8Z1_ACT_SILU};
  fp8z1_norm n = {4, 64, FP8Z1_BF16, FP8Z1_F32, FP8Z1_GATE_NONE, 1e-6f, 1.0f, 1.0f, 0.0f, 0};
  fp8z1_norm wide = {4, 1 << 20, FP8Z1_BF16, FP8Z1_F32, FP8Z1_GATE_NONE, 1e-6f, 1.0f, 1.0f, 0.0f, 0};
  alignas(16) static uint8_t mem[64];  // an address; no call gets as far as to use it
  const int32_t* const off = reinterpret_cast<const int32_t*>(mem);
  float* const s = reinterpret_cast<float*>(mem);
  size_t bytes = 0;
  CALL(fp8z1_ffn_workspace_bytes, &wrong, &bytes);
  CALL(fp8z1_ffn_up, &f, mem, mem, s, mem, s, nullptr, nullptr, nullptr, mem, nullptr, 0, nullptr);
  CALL(fp8z1_ffn_up, &f, mem, mem, s, mem, s, off, mem, nullptr, mem, nullptr, 0, nullptr);
  CALL(fp8z1_ffn_down, &f, nullptr, mem, s, off, mem, nullptr, 0, nullptr);
  CALL(fp8z1_ffn_down, &f, mem, nullptr, s, off, mem, nullptr, 0, nullptr);
  CALL(fp8z1_ffn_down, &f, mem, mem, s, off, mem, mem + 4, 64, nullptr);
  CALL(fp8z1_ffn_down_bwd, &f, mem, mem, s, mem, mem, off, mem, mem, mem + 1, nullptr, 0, nullptr);
  CALL(fp8z1_ffn_up_bwd, &wrong, mem, mem, mem, s, mem, s, off, mem, nullptr, 0, nullptr);
  CALL(fp8z1_ffn_wgrad_workspace_bytes, 4, 0, 8, 8, &bytes);
  CALL(fp8z1_ffn_wgrad, 4, 1, 8, 8, FP8Z1_F32, mem, mem, off, FP8Z1_F32, mem, 0, nullptr, 0, nullptr);
  CALL(fp8z1_ffn_bwd_weights_workspace_bytes, nullptr, &bytes);
  CALL(fp8z1_ffn_bwd_weights, &f, mem, mem, mem, mem, mem, nullptr, FP8Z1_F32, mem, mem, mem, 0, nullptr, 0, nullptr);
  CALL(fp8z1_norm_join, &wide, mem, mem, s, nullptr, s, mem, mem, nullptr);
  CALL(fp8z1_norm_join, &n, mem, mem, s, nullptr, s, nullptr, nullptr, nullptr);
  CALL(fp8z1_norm_join, &n, mem + 1, mem, s, nullptr, s, mem, mem, nullptr);
  CALL(fp8z1_norm_join_bwd_workspace_bytes, &wide, &bytes);
  CALL(fp8z1_norm_join_bwd, &n, nullptr, nullptr, mem, mem, s, nullptr, s, mem, mem, s, nullptr, s, nullptr, 0, nullptr);
  return 0;
}
