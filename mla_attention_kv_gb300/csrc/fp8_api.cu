// fp8_api.cu -- the e4m3 part of the C ABI (include/mla_prolog.h): argument
// checks, the linear layer's handle and dispatch.
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include <new>

#include "../../include/mla_prolog.h"
#include "api_util.cuh"
#include "fp8.h"
#include "fp8_plan.h"
#include "tma.h"

using namespace mla;

struct mla_fp8_linear_s {
  mla_fp8_linear_config cfg;
  int device;
  int num_sms;
  int last_launches;
  unsigned long long budget_ns;
  void* ws;
  unsigned* status;
  uint8_t* xq;    // [max_tokens, K]
  float* xscale;  // [blocks of K, max_tokens]
  const float* w_scale;
  CUtensorMap w;
};

namespace {

// A stride between rows of `width` elements in units of `unit` elements (16
// bytes), rows not overlapping; not read for a single row.
bool stride_ok(int stride, int width, int unit, int rows) { return rows <= 1 || (stride >= width && stride % unit == 0); }

}  // namespace

extern "C" {

mla_status mla_fp8_quant_rows(const mla_fp8_quant_args* args, cudaStream_t stream) {
  if (!args) return MLA_ERR_INVALID_ARG;
  const mla_fp8_quant_args& a = *args;
  if (a.T < 0 || a.K <= 0 || (a.dtype != MLA_F16 && a.dtype != MLA_BF16) || !(a.eps >= 0.0f)) return MLA_ERR_INVALID_ARG;
  if (a.K % 16 != 0 || a.K > kMostCount || a.T > kMostCount) return MLA_ERR_UNSUPPORTED;
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

mla_status mla_fp8_linear_create(const mla_fp8_linear_config* cfg, const void* weight, const float* weight_scale, mla_fp8_linear** out) {
  if (!cfg || !out) return MLA_ERR_INVALID_ARG;
  *out = nullptr;
  const mla_fp8_linear_config& c = *cfg;
  if (c.in_features <= 0 || c.out_features <= 0 || c.max_tokens <= 0 || (c.dtype != MLA_F16 && c.dtype != MLA_BF16) || !weight ||
      !weight_scale)
    return MLA_ERR_INVALID_ARG;
  // (a grid has 65535 CTAs along the weight's 128-row tiles)
  if (c.in_features % 16 != 0 || c.in_features > kMostCount || c.out_features % 8 != 0 || c.out_features > 65535 * kFp8Block ||
      c.max_tokens > kMostCount)
    return MLA_ERR_UNSUPPORTED;
  if (!aligned16(weight) || !aligned16(weight_scale)) return MLA_ERR_MISALIGNED;
  mla_fp8_linear_s* h = new (std::nothrow) mla_fp8_linear_s();
  if (!h) return MLA_ERR_NO_MEMORY;
  memset(h, 0, sizeof(*h));
  h->cfg = c;
  h->w_scale = weight_scale;
  h->budget_ns = c.spin_budget_ns ? c.spin_budget_ns : 1000000000ull;
  cudaError_t e = cudaGetDevice(&h->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, h->device);
  if (e != cudaSuccess) {
    delete h;
    return fail(e, "device query");
  }
  if (!encode_tmap_2d(&h->w, CU_TENSOR_MAP_DATA_TYPE_UINT8, weight, (uint64_t)c.in_features, (uint64_t)c.out_features,
                      (uint64_t)c.in_features, kFp8Block, kFp8Block, CU_TENSOR_MAP_SWIZZLE_128B)) {
    delete h;
    return fail(cudaErrorInvalidValue, "weight tensor map");
  }
  // workspace: [status, 256 bytes] | scales | codes of the quantised rows
  const size_t blocks = ((size_t)c.in_features + kFp8Block - 1) / kFp8Block;
  const size_t q_off = 256 + ((blocks * c.max_tokens * sizeof(float) + 255) & ~(size_t)255);
  e = cudaMalloc(&h->ws, q_off + (size_t)c.max_tokens * c.in_features);
  if (e != cudaSuccess) {
    delete h;
    fail(e, "cudaMalloc workspace");
    return MLA_ERR_NO_MEMORY;
  }
  e = cudaMemset(h->ws, 0, 256);
  if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);  // a first call may come on a stream that does not wait for this one
  if (e == cudaSuccess) e = fp8_narrow_prepare();
  if (e == cudaSuccess) e = fp8_wide_prepare();
  if (e != cudaSuccess) {
    cudaFree(h->ws);
    delete h;
    return fail(e, "workspace and kernel attributes");
  }
  unsigned char* base = static_cast<unsigned char*>(h->ws);
  h->status = reinterpret_cast<unsigned*>(base);
  h->xscale = reinterpret_cast<float*>(base + 256);
  h->xq = base + q_off;
  *out = h;
  return MLA_OK;
}

mla_status mla_fp8_linear_destroy(mla_fp8_linear* h) {
  if (!h) return MLA_ERR_INVALID_ARG;
  cudaError_t e = cudaFree(h->ws);
  delete h;
  return e == cudaSuccess ? MLA_OK : fail(e, "cudaFree workspace");
}

mla_status mla_fp8_linear_status(mla_fp8_linear* h, cudaStream_t stream) {
  if (!h) return MLA_ERR_INVALID_ARG;
  DeviceGuard g(h->device);
  if (g.err != cudaSuccess) return fail(g.err, "cudaSetDevice");
  unsigned st = 0;
  const cudaError_t e = take_status(h->status, &st, stream);
  if (e != cudaSuccess) return fail(e, "read status");
  return st & kStatusTimeout ? MLA_ERR_DEVICE_TIMEOUT : MLA_OK;
}

int mla_fp8_linear_last_launches(mla_fp8_linear* h) { return h ? h->last_launches : -1; }

mla_status mla_fp8_linear_run(mla_fp8_linear* h, const mla_fp8_linear_args* args, cudaStream_t stream) {
  if (!h || !args) return MLA_ERR_INVALID_ARG;
  const mla_fp8_linear_args& a = *args;
  const mla_fp8_linear_config& c = h->cfg;
  if (a.T < 0 || !(a.eps >= 0.0f)) return MLA_ERR_INVALID_ARG;
  h->last_launches = 0;
  if (a.T == 0) return MLA_OK;
  if (a.T > c.max_tokens) return MLA_ERR_TOO_MANY_TOKENS;
  const int K = c.in_features, N = c.out_features;
  if (!a.out || !stride_ok(a.out_stride, N, 8, a.T)) return MLA_ERR_INVALID_ARG;
  if (a.x ? (a.x_q || a.x_scale || !stride_ok(a.x_stride, K, 8, a.T))
          : (!a.x_q || !a.x_scale || a.gamma || !stride_ok(a.x_q_stride, K, 16, a.T)))
    return MLA_ERR_INVALID_ARG;
  const void* ptrs[] = {a.x, a.gamma, a.x_q, a.x_scale, a.out};
  for (const void* q : ptrs)
    if (!aligned16(q)) return MLA_ERR_MISALIGNED;
  DeviceGuard g(h->device);
  if (g.err != cudaSuccess) return fail(g.err, "cudaSetDevice");
  const bool bf16 = c.dtype == MLA_BF16;
  const void* xq = a.x_q;
  int xq_stride = a.T > 1 ? a.x_q_stride : K;
  Fp8LinearParams p = {};
  p.x_scale = a.x_scale;
  cudaError_t e;
  if (a.x) {
    Fp8RowsParams r = {};
    r.x = a.x; r.gamma = a.gamma; r.q = h->xq; r.scale = h->xscale; r.T = a.T; r.K = K; r.x_stride = a.x_stride; r.q_stride = K;
    r.eps = a.eps;
    e = fp8_rows_launch(bf16, r, stream);
    if (e != cudaSuccess) return fail(e, "fp8 row quantisation launch");
    ++h->last_launches;
    xq = h->xq;
    xq_stride = K;
    p.x_scale = h->xscale;
    p.dependent = 1;
  }
  p.w_scale = h->w_scale; p.out = a.out; p.status = h->status; p.T = a.T; p.K = K; p.N = N;
  p.out_stride = a.T > 1 ? a.out_stride : N; p.budget_ns = h->budget_ns;
  e = fp8_narrow_is_faster(p, h->num_sms) ? fp8_narrow_launch(bf16, p, h->w, xq, xq_stride, h->num_sms, stream)
                                          : fp8_wide_launch(bf16, p, h->w, xq, xq_stride, h->num_sms, stream);
  if (e != cudaSuccess) return fail(e, "fp8 linear launch");
  ++h->last_launches;
  return MLA_OK;
}

}  // extern "C"
