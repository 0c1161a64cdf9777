// attn.h -- parameters and launchers of the attention operators (latent
// cache append, paged latent attention, prompt attention).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.h"

namespace mla {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kQkDim = kRank + kRope;  // 576: width of a cached key row

// ---------------------------------------------------------------- append
struct AppendParams {
  const void* ckv;  // [T, 512], row stride ckv_stride
  const void* kpe;  // [T, 64]
  const void* qpe;  // [T, H, 64] or null
  const int32_t* positions;  // null without rotation
  const void* gamma;         // null: rows as they are
  const float* cos_t;        // null: no rotation
  const float* sin_t;
  const int32_t* slots;
  void* latent_cache;
  void* kpe_cache;
  void* qpe_out;
  unsigned* status;
  int ckv_stride, kpe_stride, q_ts, q_hs, lat_rs, kpe_rs, qo_ts, qo_hs;
  int T, heads, nslots, max_pos;
  float eps;
};
cudaError_t append_launch(bool bf16, const AppendParams& p, cudaStream_t stream);

// ---------------------------------------------------------------- paged attention
// An item that worker i began and others went on with (rows = 0: none).
struct PagedJoin {
  int row;          // first row of [T * H]
  int rows;
  int last_worker;  // the worker with its last piece
  int pad;
};
struct PagedParams {
  const void* q_lat;
  const void* q_pe;
  const int32_t* cu_q;     // null: every sequence has n_uniform tokens
  const int32_t* kv_lens;
  const int32_t* table;
  const void* latent;
  const void* kpe;
  void* out;   // [T, H, 512]
  float* lse;  // [T, H] or null
  float* part_o;   // [workers][2][rows][512] fp32, unnormalised
  float* part_ml;  // [workers][2][rows][2]: running maximum (log2 units), sum
  PagedJoin* joins;  // [workers]
  unsigned* status;
  int ql_ts, ql_hs, qp_ts, qp_hs, table_stride, lat_rs, kpe_rs;
  int page, nblocks, nseq, T, heads, n_uniform;
  int workers;  // CTAs (or CTA pairs) that share the work
  float scale_log2;  // softmax scale * log2(e)
  unsigned long long budget_ns;
};
// mma.sync kernel: items of 16 or 32 query rows.
constexpr int kPagedMmaRows = 32;
inline int paged_mma_workers(int rows, int num_sms) { return rows == 16 ? 2 * num_sms : num_sms; }  // CTAs that are resident
cudaError_t paged_mma_prepare(bool bf16);  // kernel attributes, once per device
cudaError_t paged_mma_launch(bool bf16, const PagedParams& p, int rows, cudaStream_t stream);
// tcgen05 kernel: items of 128 query rows, two CTAs per worker.
constexpr int kPagedPairRows = 128;
struct PagedMaps {  // tensor maps of the last call's caches and what they were made from
  struct Key {
    const void* lat;
    const void* kpe;
    int lat_rs, kpe_rs, rows;
  } key;
  bool valid;
  CUtensorMap lat, kpe;
};
cudaError_t paged_pair_prepare(bool bf16);
cudaError_t paged_pair_launch(bool bf16, const PagedParams& p, PagedMaps* maps, cudaStream_t stream);
// Joins the partial results of items split over workers.
cudaError_t paged_combine_launch(bool bf16, const PagedParams& p, int rows, cudaStream_t stream);

// ---------------------------------------------------------------- prompt attention
struct PromptTensor {
  const void* ptr;
  int sb, sh, st;  // element strides: batch, head, token
};
struct PromptParams {
  PromptTensor q_nope, q_pe, k_nope, k_pe, value, out;
  float* lse;  // [b, H, s] or null
  const int32_t* cu;  // packed sequences [nseq + 1] over the s tokens of batch 0, or null
  unsigned* status;
  int b, s, nseq, heads, kv_heads, causal;
  int ctas;  // CTAs that share the work
  float scale_log2;
  unsigned long long budget_ns;
};
// Tensor maps of the last call of the tcgen05 kernel and what they were made
// from (a map is a function of address, sizes and strides alone).
struct PromptMaps {
  struct Key {
    PromptTensor t[3];
    int b, s, kv_heads;
  } key;
  bool valid;
  CUtensorMap map[3];  // k_nope, k_pe, value
};
cudaError_t prompt_tc_prepare(bool bf16);
cudaError_t prompt_tc_launch(bool bf16, const PromptParams& p, PromptMaps* maps, cudaStream_t stream);

}  // namespace mla
