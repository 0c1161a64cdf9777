// fp8_api.cu -- the e4m3 part of the C ABI (include/mla_prolog.h): argument
// checks and dispatch of the row quantisation.
#include <cuda_runtime.h>
#include <stdint.h>
#include <stdio.h>

#include "../../include/mla_prolog.h"
#include "fp8.h"

using namespace mla;

namespace {

mla_status fail(cudaError_t e, const char* what) {
  char text[256];
  snprintf(text, sizeof(text), "%s: %s (%d)", what, cudaGetErrorString(e), (int)e);
  set_error_text(text);
  return MLA_ERR_CUDA;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// A stride between rows of `width` elements in units of `unit` elements (16
// bytes), rows not overlapping; not read for a single row.
bool stride_ok(int stride, int width, int unit, int rows) { return rows <= 1 || (stride >= width && stride % unit == 0); }

}  // namespace

extern "C" {

mla_status mla_fp8_quant_rows(const mla_fp8_quant_args* args, cudaStream_t stream) {
  if (!args) return MLA_ERR_INVALID_ARG;
  const mla_fp8_quant_args& a = *args;
  if (a.T < 0 || a.K <= 0 || (a.dtype != MLA_F16 && a.dtype != MLA_BF16) || !(a.eps >= 0.0f)) return MLA_ERR_INVALID_ARG;
  if (a.K % 16 != 0) return MLA_ERR_UNSUPPORTED;
  if (a.T == 0) return MLA_OK;
  if (!a.x || !a.q || !a.scale) return MLA_ERR_INVALID_ARG;
  if (!stride_ok(a.x_stride, a.K, 8, a.T) || !stride_ok(a.q_stride, a.K, 16, a.T)) return MLA_ERR_INVALID_ARG;
  const void* ptrs[] = {a.x, a.gamma, a.q, a.scale};
  for (const void* q : ptrs)
    if (!aligned16(q)) return MLA_ERR_MISALIGNED;
  Fp8RowsParams p = {};
  p.x = a.x; p.gamma = a.gamma; p.q = static_cast<uint8_t*>(a.q); p.scale = a.scale; p.T = a.T; p.K = a.K;
  p.x_stride = a.x_stride; p.q_stride = a.q_stride; p.eps = a.eps;
  cudaError_t e = fp8_rows_launch(a.dtype == MLA_BF16, p, stream);
  return e == cudaSuccess ? MLA_OK : fail(e, "fp8 row quantisation launch");
}

}  // extern "C"
