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

// ---------------------------------------------------------------- linear layer
struct Fp8LinearParams {
  const float* x_scale;  // [blocks of K, T]
  const float* w_scale;  // [blocks of N, blocks of K]
  void* out;             // [T, N], row stride out_stride (elements)
  unsigned* status;
  int T, K, N, out_stride;
  int dependent;  // launched while the kernel that makes the rows runs
  unsigned long long budget_ns;
};
// Few rows: weights as the 128-row operand, the K blocks split over a cluster.
cudaError_t fp8_narrow_prepare();
// w: the weight's tensor map, in boxes of 128 rows.
cudaError_t fp8_narrow_launch(bool bf16, const Fp8LinearParams& p, const CUtensorMap& w, const void* xq, int xq_stride, int num_sms,
                              cudaStream_t stream);
// Many rows: persistent CTAs on tiles of 128 rows x 256 weight rows.
cudaError_t fp8_wide_prepare();
cudaError_t fp8_wide_launch(bool bf16, const Fp8LinearParams& p, const CUtensorMap& w, const void* xq, int xq_stride, int num_sms,
                            cudaStream_t stream);
// The map of rows xq [T, K] with boxes of `box` rows.
bool fp8_row_map(CUtensorMap* map, const void* xq, int T, int K, int stride, int box);

}  // namespace mla
