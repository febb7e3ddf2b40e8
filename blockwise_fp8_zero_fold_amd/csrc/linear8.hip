// y = res + act(x W^T + bias) of rows in 8 bits.
#include "linear8.h"

namespace fp8z1 {

// (few rows are not tiled)
size_t linear8_workspace(int64_t T, int64_t E, int64_t N, int64_t K) {
  return few_rows8(T, E, N, K, 1) ? 0 : tiles8_bytes(T, E * N, K);
}

int linear8(const FfnArgs& p, int32_t dtype, void* workspace, size_t workspace_bytes, hipStream_t s, const char* what) {
  return launch8<kLinear>(p, dtype, workspace, workspace_bytes, s, what);
}

}  // namespace fp8z1
