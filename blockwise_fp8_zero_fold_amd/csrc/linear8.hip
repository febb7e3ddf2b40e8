// y = res + act(x W^T + bias) of rows in 8 bits.
#include "linear8.h"

namespace fp8z1 {

// (few rows are not tiled)
size_t linear8_workspace(int64_t T, int64_t E) { return few_rows8(T, E) ? 0 : part8_bytes(); }

int linear8(const FfnArgs& p, int32_t dtype, void* workspace, size_t workspace_bytes, hipStream_t s, const char* what) {
  return launch8<kLinear>(p, dtype, workspace, workspace_bytes, s, what);
}

}  // namespace fp8z1
