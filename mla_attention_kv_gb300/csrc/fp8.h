// fp8.h -- parameters and launchers of the e4m3 operators (row quantisation,
// block-scaled linear layer).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.h"

namespace mla {

constexpr int kFp8Block = 128;  // columns (and weight rows) that share a scale
constexpr float kE4m3Max = 448.0f;

struct Fp8RowsParams {
  const void* x;      // [T, K], row stride x_stride
  const void* gamma;  // [K], or null: no RMSNorm
  uint8_t* q;         // [T, K] e4m3, row stride q_stride
  float* scale;       // [ceil(K / 128), T]
  int T, K;
  long long x_stride, q_stride;
  float eps;
};
cudaError_t fp8_rows_launch(bool bf16, const Fp8RowsParams& p, cudaStream_t stream);

}  // namespace mla
