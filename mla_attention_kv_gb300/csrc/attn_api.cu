// attn_api.cu -- the attention part of the C ABI (include/mla_prolog.h):
// handle, argument checks, workspace and kernel dispatch of the latent cache
// append, the paged latent attention and the prompt attention.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <new>

#include "../../include/mla_prolog.h"
#include "attn.h"

using namespace mla;

struct mla_attn_s {
  mla_attn_config cfg;
  int device;
  int num_sms;
  int last_launches;
  float scale_log2;
  unsigned long long budget_ns;
  void* ws;
  unsigned* status;
  float* part_o;
  float* part_ml;
  PagedJoin* joins;
  PagedMaps paged_maps;
  PromptMaps prompt_maps;
};

namespace {

mla_status fail(cudaError_t e, const char* what) {
  char text[256];
  snprintf(text, sizeof(text), "%s: %s (%d)", what, cudaGetErrorString(e), (int)e);
  set_error_text(text);
  return MLA_ERR_CUDA;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// A stride between rows of `width` elements: whole 16-byte units, rows not
// overlapping (the stride of a dimension of size 1 is not read).
bool stride_ok(int stride, int width, bool used) { return !used || (stride >= width && stride % 8 == 0); }

// Reads and clears the status word in one step (the second word keeps what was
// read): calls that overlap on another stream may set bits meanwhile.
__global__ void take_status_kernel(unsigned* status) { status[1] = atomicExch(status, 0u); }

// Makes the handle's device current for the length of a call.
struct DeviceGuard {
  int before = -1;
  cudaError_t err;
  explicit DeviceGuard(int device) {
    err = cudaGetDevice(&before);
    if (err == cudaSuccess && before != device)
      err = cudaSetDevice(device);
    else
      before = -1;
  }
  ~DeviceGuard() {
    if (before >= 0) cudaSetDevice(before);
  }
};

}  // namespace

extern "C" {

mla_status mla_attn_create(const mla_attn_config* cfg, mla_attn** out) {
  if (!cfg || !out) return MLA_ERR_INVALID_ARG;
  *out = nullptr;
  const mla_attn_config& c = *cfg;
  if (c.num_heads <= 0 || c.num_kv_heads < 0 || c.max_tokens <= 0 || c.max_pos <= 0 || !(c.eps >= 0.0f) ||
      !(c.scale >= 0.0f) || isinf(c.scale) || (c.dtype != MLA_F16 && c.dtype != MLA_BF16))
    return MLA_ERR_INVALID_ARG;
  const int kvh = c.num_kv_heads ? c.num_kv_heads : c.num_heads;
  if (c.kv_lora_rank != kRank || c.rope_dim != kRope || c.nope_dim != kNope || c.v_dim != kV ||
      c.num_heads % kvh != 0 || c.num_heads > 1024 || (long long)c.num_heads * c.max_tokens > 0x7fffffffLL / 2)
    return MLA_ERR_UNSUPPORTED;
  mla_attn_s* h = new (std::nothrow) mla_attn_s();
  if (!h) return MLA_ERR_NO_MEMORY;
  memset(h, 0, sizeof(*h));
  h->cfg = c;
  h->cfg.num_kv_heads = kvh;
  h->budget_ns = c.spin_budget_ns ? c.spin_budget_ns : 1000000000ull;
  h->scale_log2 = (c.scale > 0.0f ? c.scale : 1.0f / sqrtf((float)(kNope + kRope))) * kLog2e;
  cudaError_t e = cudaGetDevice(&h->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, h->device);
  if (e != cudaSuccess) {
    delete h;
    return fail(e, "device query");
  }
  // workspace: [status, 256 bytes] | a join record per worker | two partial results per worker
  const size_t rows_mma = (size_t)h->num_sms * 2 * kPagedMmaRows, rows_tc = (size_t)(h->num_sms / 2) * 2 * kPagedPairRows;
  const size_t rows = rows_mma > rows_tc ? rows_mma : rows_tc;
  const size_t join_off = 256, ml_off = join_off + (((size_t)h->num_sms * 2 * sizeof(PagedJoin) + 255) & ~(size_t)255), o_off = ml_off + ((rows * 2 * sizeof(float) + 255) & ~(size_t)255);
  e = cudaMalloc(&h->ws, o_off + rows * kRank * sizeof(float));
  if (e != cudaSuccess) {
    delete h;
    fail(e, "cudaMalloc workspace");
    return MLA_ERR_NO_MEMORY;
  }
  e = cudaMemset(h->ws, 0, ml_off);  // (status and records)
  if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);  // a first call may come on a stream that does not wait for this one
  if (e != cudaSuccess) {
    cudaFree(h->ws);
    delete h;
    return fail(e, "clear workspace");
  }
  unsigned char* base = static_cast<unsigned char*>(h->ws);
  h->status = reinterpret_cast<unsigned*>(base);
  h->joins = reinterpret_cast<PagedJoin*>(base + join_off);
  h->part_ml = reinterpret_cast<float*>(base + ml_off);
  h->part_o = reinterpret_cast<float*>(base + o_off);
  // (shared memory beyond the default is asked for once, not per call)
  const bool bf16 = c.dtype == MLA_BF16;
  e = paged_mma_prepare(bf16);
  if (e == cudaSuccess) e = paged_pair_prepare(bf16);
  if (e == cudaSuccess) e = prompt_tc_prepare(bf16);
  if (e != cudaSuccess) {
    cudaFree(h->ws);
    delete h;
    return fail(e, "kernel attributes");
  }
  *out = h;
  return MLA_OK;
}

mla_status mla_attn_destroy(mla_attn* h) {
  if (!h) return MLA_ERR_INVALID_ARG;
  cudaError_t e = cudaFree(h->ws);
  delete h;
  return e == cudaSuccess ? MLA_OK : fail(e, "cudaFree workspace");
}

mla_status mla_attn_status(mla_attn* h, cudaStream_t stream) {
  if (!h) return MLA_ERR_INVALID_ARG;
  DeviceGuard g(h->device);
  if (g.err != cudaSuccess) return fail(g.err, "cudaSetDevice");
  cudaError_t e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess) return fail(e, "cudaStreamSynchronize");
  unsigned st = 0;
  take_status_kernel<<<1, 1, 0, stream>>>(h->status);
  e = cudaGetLastError();
  if (e == cudaSuccess) e = cudaMemcpyAsync(&st, h->status + 1, sizeof(unsigned), cudaMemcpyDeviceToHost, stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess) return fail(e, "read status");
  if (st & kStatusBadPosition) return MLA_ERR_BAD_POSITION;
  if (st & kStatusTimeout) return MLA_ERR_DEVICE_TIMEOUT;
  if (st & kStatusBadSlot) return MLA_ERR_BAD_SLOT;
  if (st & kStatusBadLength) return MLA_ERR_BAD_LENGTH;
  return MLA_OK;
}

int mla_attn_last_launches(mla_attn* h) { return h ? h->last_launches : -1; }

mla_status mla_latent_append(mla_attn* h, const mla_latent_append_args* args, cudaStream_t stream) {
  if (!h || !args) return MLA_ERR_INVALID_ARG;
  const mla_latent_append_args& a = *args;
  if (a.T < 0 || a.page_size <= 0 || a.num_blocks <= 0 || (long long)a.page_size * a.num_blocks > 0x7fffffffLL)
    return MLA_ERR_INVALID_ARG;
  h->last_launches = 0;
  if (a.T == 0) return MLA_OK;
  if (a.T > h->cfg.max_tokens) return MLA_ERR_TOO_MANY_TOKENS;
  const int H = h->cfg.num_heads;
  if (!a.compressed_kv || !a.k_pe || !a.slot_mapping || !a.latent_cache || !a.kpe_cache ||
      (!a.cos_table != !a.sin_table) || (a.cos_table && !a.positions) || (a.q_pe && (!a.cos_table || !a.q_pe_out)))
    return MLA_ERR_INVALID_ARG;
  if (!stride_ok(a.compressed_kv_stride, kRank, a.T > 1) || !stride_ok(a.k_pe_stride, kRope, a.T > 1) ||
      !stride_ok(a.latent_row_stride, kRank, true) || !stride_ok(a.kpe_row_stride, kRope, true))
    return MLA_ERR_INVALID_ARG;
  if (a.q_pe && (!stride_ok(a.q_pe_token_stride, kRope, a.T > 1) || !stride_ok(a.q_pe_head_stride, kRope, H > 1) ||
                 !stride_ok(a.q_pe_out_token_stride, kRope, a.T > 1) || !stride_ok(a.q_pe_out_head_stride, kRope, H > 1)))
    return MLA_ERR_INVALID_ARG;
  if (a.q_pe && a.q_pe == a.q_pe_out &&
      ((a.T > 1 && a.q_pe_token_stride != a.q_pe_out_token_stride) || (H > 1 && a.q_pe_head_stride != a.q_pe_out_head_stride)))
    return MLA_ERR_INVALID_ARG;
  const void* ptrs[] = {a.compressed_kv, a.k_pe, a.slot_mapping, a.latent_cache, a.kpe_cache, a.gamma_kv, a.cos_table,
                        a.sin_table, a.positions, a.q_pe, a.q_pe ? a.q_pe_out : nullptr};
  for (const void* q : ptrs)
    if (!aligned16(q)) return MLA_ERR_MISALIGNED;
  DeviceGuard g(h->device);
  if (g.err != cudaSuccess) return fail(g.err, "cudaSetDevice");
  AppendParams p = {};
  p.ckv = a.compressed_kv; p.kpe = a.k_pe; p.qpe = a.q_pe; p.positions = a.positions; p.gamma = a.gamma_kv;
  p.cos_t = a.cos_table; p.sin_t = a.sin_table; p.slots = a.slot_mapping; p.latent_cache = a.latent_cache;
  p.kpe_cache = a.kpe_cache; p.qpe_out = a.q_pe_out; p.status = h->status; p.ckv_stride = a.compressed_kv_stride;
  p.kpe_stride = a.k_pe_stride; p.q_ts = a.q_pe_token_stride; p.q_hs = a.q_pe_head_stride; p.lat_rs = a.latent_row_stride;
  p.kpe_rs = a.kpe_row_stride; p.qo_ts = a.q_pe_out_token_stride; p.qo_hs = a.q_pe_out_head_stride; p.T = a.T; p.heads = H;
  p.nslots = a.page_size * a.num_blocks; p.max_pos = h->cfg.max_pos; p.eps = h->cfg.eps;
  cudaError_t e = append_launch(h->cfg.dtype == MLA_BF16, p, stream);
  if (e != cudaSuccess) return fail(e, "append launch");
  h->last_launches = 1;
  return MLA_OK;
}

mla_status mla_attn_paged_run(mla_attn* h, const mla_attn_paged_args* args, cudaStream_t stream) {
  if (!h || !args) return MLA_ERR_INVALID_ARG;
  const mla_attn_paged_args& a = *args;
  if (a.num_seqs < 0 || a.T < 0 || a.page_size <= 0 || a.num_blocks <= 0 || a.table_stride < 0 ||
      (long long)a.page_size * a.num_blocks > 0x7fffffffLL)
    return MLA_ERR_INVALID_ARG;
  h->last_launches = 0;
  if (a.num_seqs == 0 || a.T == 0) return MLA_OK;
  if (!a.cu_q && a.T % a.num_seqs != 0) return MLA_ERR_INVALID_ARG;
  if (a.T > h->cfg.max_tokens) return MLA_ERR_TOO_MANY_TOKENS;
  const int H = h->cfg.num_heads;
  if (!a.q_latent || !a.q_pe || !a.kv_lens || !a.block_table || !a.latent_cache || !a.kpe_cache || !a.out)
    return MLA_ERR_INVALID_ARG;
  if (!stride_ok(a.q_latent_token_stride, kRank, a.T > 1) || !stride_ok(a.q_latent_head_stride, kRank, H > 1) ||
      !stride_ok(a.q_pe_token_stride, kRope, a.T > 1) || !stride_ok(a.q_pe_head_stride, kRope, H > 1) ||
      !stride_ok(a.latent_row_stride, kRank, true) || !stride_ok(a.kpe_row_stride, kRope, true))
    return MLA_ERR_INVALID_ARG;
  const void* ptrs[] = {a.q_latent, a.q_pe, a.cu_q, a.kv_lens, a.block_table, a.latent_cache, a.kpe_cache, a.out, a.lse};
  for (const void* q : ptrs)
    if (!aligned16(q)) return MLA_ERR_MISALIGNED;
  DeviceGuard g(h->device);
  if (g.err != cudaSuccess) return fail(g.err, "cudaSetDevice");
  const bool bf16 = h->cfg.dtype == MLA_BF16;
  PagedParams p = {};
  p.q_lat = a.q_latent; p.q_pe = a.q_pe; p.cu_q = a.cu_q; p.kv_lens = a.kv_lens; p.table = a.block_table;
  p.latent = a.latent_cache; p.kpe = a.kpe_cache; p.out = a.out; p.lse = a.lse; p.part_o = h->part_o;
  p.part_ml = h->part_ml; p.joins = h->joins; p.status = h->status; p.ql_ts = a.q_latent_token_stride; p.ql_hs = a.q_latent_head_stride;
  p.qp_ts = a.q_pe_token_stride; p.qp_hs = a.q_pe_head_stride; p.table_stride = a.table_stride;
  p.lat_rs = a.latent_row_stride; p.kpe_rs = a.kpe_row_stride; p.page = a.page_size; p.nblocks = a.num_blocks;
  p.nseq = a.num_seqs; p.T = a.T; p.heads = H; p.n_uniform = a.cu_q ? 0 : a.T / a.num_seqs;
  p.scale_log2 = h->scale_log2; p.budget_ns = h->budget_ns;
  // (with ragged chunks the host knows only the average)
  const long long rows_per_seq = (long long)(a.T / a.num_seqs > 0 ? a.T / a.num_seqs : 1) * H;
  // 32 rows or fewer: the kernel built around the key stream (64 sequences of up to 4096 keys with 16 heads: 48 us, a
  // tcgen05 kernel for 128 rows 92 us); more: one pass of the tcgen05 kernel (64 sequences of up to 32768 keys with 128
  // heads: 250 us, four passes of the other 1344 us)
  const bool tc = rows_per_seq > kPagedMmaRows;
  const int rows = tc ? kPagedPairRows : rows_per_seq <= 16 ? 16 : kPagedMmaRows;
  p.workers = tc ? h->num_sms / 2 : paged_mma_workers(rows, h->num_sms);
  cudaError_t e = tc ? paged_pair_launch(bf16, p, &h->paged_maps, stream) : paged_mma_launch(bf16, p, rows, stream);
  if (e != cudaSuccess) return fail(e, "paged attention launch");
  e = paged_combine_launch(bf16, p, rows, stream);
  if (e != cudaSuccess) return fail(e, "paged attention combine launch");
  h->last_launches = 2;
  return MLA_OK;
}

mla_status mla_attn_prompt_run(mla_attn* h, const mla_attn_prompt_args* args, cudaStream_t stream) {
  if (!h || !args) return MLA_ERR_INVALID_ARG;
  const mla_attn_prompt_args& a = *args;
  if (a.b < 0 || a.s < 0 || (a.causal != 0 && a.causal != 1) || (a.cu_seqlens && (a.num_seqs < 0 || a.b > 1)))
    return MLA_ERR_INVALID_ARG;
  h->last_launches = 0;
  const long long T = (long long)a.b * a.s;
  if (T == 0 || (a.cu_seqlens && a.num_seqs == 0)) return MLA_OK;
  if (T > h->cfg.max_tokens) return MLA_ERR_TOO_MANY_TOKENS;
  if (!a.q_nope || !a.q_pe || !a.k_nope || !a.k_pe || !a.value || !a.out) return MLA_ERR_INVALID_ARG;
  const int H = h->cfg.num_heads, KH = h->cfg.num_kv_heads;
  PromptParams p = {};
  p.q_nope = {a.q_nope, a.q_nope_batch_stride, a.q_nope_head_stride, a.q_nope_token_stride};
  p.q_pe = {a.q_pe, a.q_pe_batch_stride, a.q_pe_head_stride, a.q_pe_token_stride};
  p.k_nope = {a.k_nope, a.k_nope_batch_stride, a.k_nope_head_stride, a.k_nope_token_stride};
  p.k_pe = {a.k_pe, a.k_pe_batch_stride, 0, a.k_pe_token_stride};
  p.value = {a.value, a.value_batch_stride, a.value_head_stride, a.value_token_stride};
  p.out = {a.out, a.out_batch_stride, a.out_head_stride, a.out_token_stride};
  const struct { PromptTensor* t; int width, heads; } all[] = {
      {&p.q_nope, kNope, H}, {&p.q_pe, kRope, H}, {&p.k_nope, kNope, KH}, {&p.k_pe, kRope, 1}, {&p.value, kV, KH}, {&p.out, kV, H}};
  for (const auto& x : all)
    if (!stride_ok(x.t->sb, x.width, a.b > 1) || !stride_ok(x.t->sh, x.width, x.heads > 1) || !stride_ok(x.t->st, x.width, a.s > 1))
      return MLA_ERR_INVALID_ARG;
  for (const auto& x : all) {
    if (!aligned16(x.t->ptr)) return MLA_ERR_MISALIGNED;
    if (a.b == 1) x.t->sb = x.width;
    if (x.heads == 1) x.t->sh = x.width;
    if (a.s == 1) x.t->st = x.width;
  }
  if (!aligned16(a.cu_seqlens) || !aligned16(a.lse)) return MLA_ERR_MISALIGNED;
  DeviceGuard g(h->device);
  if (g.err != cudaSuccess) return fail(g.err, "cudaSetDevice");
  p.lse = a.lse; p.cu = a.cu_seqlens; p.status = h->status; p.b = a.b; p.s = a.s; p.nseq = a.cu_seqlens ? a.num_seqs : a.b;
  p.heads = H; p.kv_heads = KH; p.causal = a.causal; p.ctas = h->num_sms; p.scale_log2 = h->scale_log2; p.budget_ns = h->budget_ns;
  cudaError_t e = prompt_tc_launch(h->cfg.dtype == MLA_BF16, p, &h->prompt_maps, stream);
  if (e != cudaSuccess) return fail(e, "prompt attention launch");
  h->last_launches = 1;
  return MLA_OK;
}

}  // extern "C"
