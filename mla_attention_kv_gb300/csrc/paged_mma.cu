// paged_mma.cu -- attention of new tokens over the paged latent cache, for
// items of 16 or 32 query rows, on mma.sync; and the kernel that joins
// partial results.
//
// Per query row r (a token and a head; q = [q_latent | q_pe], 576 wide) and
// cached token k (row [latent | k_pe], the latent also being the value):
//   s_k = scale * q . key_k,  out = sum_k softmax(s)_k * latent_k.
// One pass over the keys with a running maximum m and sum l per row:
//   m' = max(m, max s),  l' = l * 2^(m - m') + sum 2^(s - m'),
//   o' = o * 2^(m - m') + sum 2^(s - m') * latent       (s in log2 units)
// The 2^(s - m') are rounded to the I/O dtype (the operand type of the
// product with the latents); l sums them before that rounding, in fp32.
//
// With at most 32 rows an item reads 1152 bytes per key for at most
// 2 * 32 * 1088 FLOPs, well under the ratio at which the tensor cores
// matter, so the kernel is built around the key stream: two stages of keys
// filled by 16-byte cp.async (any page size; a page may end anywhere in a
// tile), each key row used from shared memory twice (as key and as value).
// What bounds it is the latency of the way through a tile (scores, softmax
// over the warps, output), so the work of a tile is spread over many warps:
// 16-row items run two CTAs of 8 warps per SM on tiles of 32 keys, 32-row
// items one CTA of 16 warps on tiles of 64.  Decode of 64 sequences of up to
// 4096 keys, 16 heads, fp16 (154 MB of cache): 47.7 us, 3.2 TB/s; 53 us when
// the queries were read from shared memory for every tile and a page's number
// checked where it is looked up (61 us with one CTA of 8 warps and tiles of
// 64).  Per tile of a CTA 5200 cycles: 1200 scores, 600 softmax, 850 output,
// 700 each for the issue of the next copies and for their arrival.
#include "attn.h"
#include "common.cuh"
#include "paged_plan.cuh"

namespace mla {
namespace {

constexpr int kPitch = kQkDim * 2 + 16;  // bytes per key / query row in shared memory: 73 16-byte units
constexpr int kSplit = 4;                // parts of the 576 columns that a tile's scores are summed from
constexpr int kRowsPerWarp = 4;          // key rows that a warp copies

// MT 16-row blocks of query rows; KT keys per tile.
template <int MT>
struct PmCfg {
  static constexpr int R = 16 * MT;
  static constexpr int KT = MT == 1 ? 32 : 64;
  static constexpr int kWarps = KT / 16 * kSplit;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kCtas = MT == 1 ? 2 : 1;  // per SM
  static constexpr int kCols = kRank / kWarps;   // output columns of a warp
  static constexpr int TPR = kThreads / R;       // softmax threads per row
  static constexpr int KPT = KT / TPR;           // keys per softmax thread
  static constexpr int kSPitch = KT + 4;         // floats
  static constexpr int kPPitch = KT + 8;         // 16-bit values
  static constexpr int kStageBytes = KT * kPitch;
  static constexpr int kQ = 0;
  static constexpr int kK = kQ + R * kPitch;
  static constexpr int kS = kK + 2 * kStageBytes;
  static constexpr int kP = kS + kSplit * R * kSPitch * 4;
  static constexpr int kRow = kP + R * kPPitch * 2;  // alpha [R], then 1 / l [R]
  static constexpr int kPlan = (kRow + 2 * R * 4 + 15) & ~15;
  static constexpr int kBytes = kPlan + (int)sizeof(PlanShared);
  static_assert(kRowsPerWarp * kWarps == KT, "copies of a tile");
  static_assert(TPR <= 32 && KPT * TPR == KT, "softmax threads");
};

// Where key k of sequence s lies: its block table entry and the row in that
// block (-1: there is no such key).  The entry is not looked at here, so that
// its load runs on under other work.
struct CachePlace {
  int blk, off;
};
__device__ __forceinline__ CachePlace cache_place(const PagedParams& p, int s, int k, int keys) {
  if (k >= keys) return {0, -1};
  const int pg = k / p.page;
  return {p.table[(size_t)s * p.table_stride + pg], k - pg * p.page};
}
// Its row index in the cache, or -1.
__device__ __forceinline__ int cache_row(const PagedParams& p, const CachePlace& c) {
  if (c.off < 0) return -1;
  if (c.blk < 0 || c.blk >= p.nblocks) {
    atomicOr(p.status, kStatusBadSlot);
    return -1;
  }
  return c.blk * p.page + c.off;
}

template <typename T, int MT>
__global__ void __launch_bounds__(PmCfg<MT>::kThreads, PmCfg<MT>::kCtas) paged_mma_kernel(const PagedParams p) {
  using E = Elem<T>;
  using S = PmCfg<MT>;
  constexpr int R = S::R, KT = S::KT, TPR = S::TPR, KPT = S::KPT, NT = S::kCols / 8;
  extern __shared__ __align__(16) unsigned char smem[];
  const uint32_t sb = smem_u32(smem);
  PlanShared* plan = reinterpret_cast<PlanShared*>(smem + S::kPlan);
  float* sS = reinterpret_cast<float*>(smem + S::kS);
  float* sAlpha = reinterpret_cast<float*>(smem + S::kRow);
  float* sInv = sAlpha + R;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int H = p.heads;

  grid_dep_launch_dependents();  // (the joining kernel may take its place)
  const long long total = plan_total(p, plan, R, blockIdx.x == 0);
  const int W = total > 0 ? plan_workers(total, p.workers, R) : 0;
  const int w = blockIdx.x;
  if (tid == 0) plan_open_join(p, w);
  if (w >= W) return;
  const long long x0 = plan_worker_begin(total, w, W), x1 = plan_worker_begin(total, w + 1, W);

  PlanCursor c;
  c.seek(p, plan, R, x0);
  for (bool more = true; more && c.lo < x1; more = c.next(p, R)) {
    const Seq q = c.q;
    const int row0 = c.j * R;  // first row of the item within its sequence
    const int live = min(R, q.n * H - row0);
    const int keys = q.keys_of_item(c.j, R, H);
    const int tiles = (keys + kKeyTile - 1) / kKeyTile;
    const long long a = x0 > c.lo ? x0 : c.lo, b = x1 < c.hi ? x1 : c.hi;
    // this worker's tiles of KT keys
    constexpr int kSub = kKeyTile / KT;
    const int t0 = c.tile_at(a, tiles, R) * kSub, t1 = min(c.tile_at(b, tiles, R) * kSub, (keys + KT - 1) / KT);
    const bool whole = c.lo >= x0 && c.hi <= x1;
    const int s = c.s;

    if (tid == 0 && c.hi >= x1) plan_post_join(p, c, R, w, x0, x1, total, W);

    // ---- key tiles: warp w copies rows 4w .. 4w + 3 of a stage
    auto rows_of = [&](int tile) {  // lanes 0-3 look up their rows
      return tile < t1 && lane < kRowsPerWarp ? cache_place(p, s, tile * KT + warp * kRowsPerWarp + lane, keys) : CachePlace{0, -1};
    };
    auto load = [&](int tile, const CachePlace& place) {
      const int rows = cache_row(p, place);
      const uint32_t st = sb + S::kK + (tile & 1) * S::kStageBytes + warp * kRowsPerWarp * kPitch;
#pragma unroll
      for (int r = 0; r < kRowsPerWarp; ++r) {
        const int row = __shfl_sync(~0u, rows, r);
        const T* src = static_cast<const T*>(p.latent) + (size_t)max(row, 0) * p.lat_rs;
        const uint32_t d = st + r * kPitch;
        cp_async16(d + lane * 16, src + lane * 8, row < 0 ? 0 : 16);
        cp_async16(d + 512 + lane * 16, src + 256 + lane * 8, row < 0 ? 0 : 16);
      }
      const int row = __shfl_sync(~0u, rows, lane >> 3);
      const T* src = static_cast<const T*>(p.kpe) + (size_t)max(row, 0) * p.kpe_rs;
      cp_async16(st + (lane >> 3) * kPitch + 1024 + (lane & 7) * 16, src + (lane & 7) * 8, row < 0 ? 0 : 16);
    };
    const CachePlace place0 = rows_of(t0), place1 = rows_of(t0 + 1);
    __syncthreads();  // the previous item's stages and queries are read
    // ---- queries (rows past the end are zero), together with the first tile
    for (int r = warp; r < R; r += S::kWarps) {
      const int tok = (row0 + r) / H, hd = (row0 + r) - tok * H;
      const bool ok = r < live;
      const T* ql = static_cast<const T*>(p.q_lat) + (ok ? (size_t)(q.begin + tok) * p.ql_ts + (size_t)hd * p.ql_hs : 0);
      const T* qp = static_cast<const T*>(p.q_pe) + (ok ? (size_t)(q.begin + tok) * p.qp_ts + (size_t)hd * p.qp_hs : 0);
      const uint32_t d = sb + S::kQ + r * kPitch;
      cp_async16(d + lane * 16, ql + lane * 8, ok ? 16 : 0);
      cp_async16(d + 512 + lane * 16, ql + 256 + lane * 8, ok ? 16 : 0);
      if (lane < 8) cp_async16(d + 1024 + lane * 16, qp + lane * 8, ok ? 16 : 0);
    }
    if (t0 < t1) load(t0, place0);
    cp_async_commit();
    if (t0 + 1 < t1) load(t0 + 1, place1);
    cp_async_commit();

    float acc[MT][NT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.f;
    const int srow = tid / TPR, sk0 = tid % TPR;  // softmax: row, first key (keys sk0 + TPR * i)
    const int limit = srow < live ? q.keys_of_row(row0 + srow, H) : 0;
    float m_run = -INFINITY, l_run = 0.f;

    // 16-row items: a warp's quarter of the queries stays in registers (32-row items would need 72 of a thread's 128)
    constexpr int kSteps = kQkDim / 16 / kSplit;
    const uint32_t qaddr = sb + S::kQ + (lane & 15) * kPitch + warp / (KT / 16) * 288 + (lane >> 4) * 16;
    uint32_t qf[MT == 1 ? kSteps : 1][4];
    if (MT == 1 && t0 < t1) {
      cp_async_wait<1>();
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        uint32_t* f = qf[MT == 1 ? k : 0];
        ldsm_x4(qaddr + k * 32, f[0], f[1], f[2], f[3]);
      }
    }
    for (int tile = t0; tile < t1; ++tile) {
      const CachePlace place = rows_of(tile + 2);
      cp_async_wait<1>();
      __syncthreads();
      const uint32_t st = sb + S::kK + (tile & 1) * S::kStageBytes;
      {  // scores: warp = (16 keys kg, quarter kq of the 576 columns)
        const int kg = warp % (KT / 16), kq = warp / (KT / 16);
        float sc[MT][2][4];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) sc[m][n][i] = 0.f;
        const uint32_t kaddr = st + (kg * 16 + (lane & 7) + ((lane >> 4) & 1) * 8) * kPitch + kq * 288 + ((lane >> 3) & 1) * 16;
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          uint32_t b0, b1, b2, b3;
          ldsm_x4(kaddr + k * 32, b0, b1, b2, b3);
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            uint32_t af[4];
            if (MT == 1) {
#pragma unroll
              for (int i = 0; i < 4; ++i) af[i] = qf[MT == 1 ? k : 0][i];
            } else {
              ldsm_x4(qaddr + m * 16 * kPitch + k * 32, af[0], af[1], af[2], af[3]);
            }
            mma16816<E::kBf16>(sc[m][0], af, b0, b1);
            mma16816<E::kBf16>(sc[m][1], af, b2, b3);
          }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            float* d = sS + (kq * R + m * 16 + (lane >> 2)) * S::kSPitch + kg * 16 + n * 8 + (lane & 3) * 2;
            *reinterpret_cast<float2*>(d) = make_float2(sc[m][n][0], sc[m][n][1]);
            *reinterpret_cast<float2*>(d + 8 * S::kSPitch) = make_float2(sc[m][n][2], sc[m][n][3]);
          }
      }
      __syncthreads();
      {  // softmax of the tile
        float v[KPT], mx = -INFINITY;
#pragma unroll
        for (int i = 0; i < KPT; ++i) {
          const int k = sk0 + i * TPR;
          const float* x4 = sS + srow * S::kSPitch + k;
          const float x = (x4[0] + x4[R * S::kSPitch]) + (x4[2 * R * S::kSPitch] + x4[3 * R * S::kSPitch]);
          v[i] = tile * KT + k < limit ? x * p.scale_log2 : -INFINITY;
          mx = fmaxf(mx, v[i]);
        }
#pragma unroll
        for (int d = TPR / 2; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, d));
        const float m_new = fmaxf(m_run, mx);
        const float mu = m_new == -INFINITY ? 0.f : m_new;  // (a row with no key so far)
        const float alpha = exp2f(m_run - mu);
        float ls = 0.f;
        T* prow = reinterpret_cast<T*>(smem + S::kP) + srow * S::kPPitch;
#pragma unroll
        for (int i = 0; i < KPT; ++i) {
          const float e = exp2f(v[i] - mu);
          ls += e;
          prow[sk0 + i * TPR] = E::from_f(e);
        }
        l_run = l_run * alpha + ls;
        m_run = m_new;
        if (sk0 == 0) sAlpha[srow] = alpha;
      }
      __syncthreads();
      {  // output: warp = kCols latent columns
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const float a0 = sAlpha[m * 16 + (lane >> 2)], a1 = sAlpha[m * 16 + (lane >> 2) + 8];
          if (__any_sync(~0u, a0 != 1.f || a1 != 1.f)) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              acc[m][n][0] *= a0;
              acc[m][n][1] *= a0;
              acc[m][n][2] *= a1;
              acc[m][n][3] *= a1;
            }
          }
        }
        const uint32_t paddr = sb + S::kP + (lane & 15) * (S::kPPitch * 2) + (lane >> 4) * 16;
        const uint32_t vaddr = st + (lane & 15) * kPitch + warp * (S::kCols * 2) + (lane >> 4) * 16;
#pragma unroll
        for (int k = 0; k < KT / 16; ++k) {
          uint32_t af[MT][4];
#pragma unroll
          for (int m = 0; m < MT; ++m)
            ldsm_x4(paddr + m * 16 * S::kPPitch * 2 + k * 32, af[m][0], af[m][1], af[m][2], af[m][3]);
#pragma unroll
          for (int n = 0; n < NT / 2; ++n) {
            uint32_t b0, b1, b2, b3;
            ldsm_x4_trans(vaddr + k * 16 * kPitch + n * 32, b0, b1, b2, b3);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              mma16816<E::kBf16>(acc[m][2 * n], af[m], b0, b1);
              mma16816<E::kBf16>(acc[m][2 * n + 1], af[m], b2, b3);
            }
          }
        }
      }
      __syncthreads();  // the stage is free
      if (tile + 2 < t1) load(tile + 2, place);
      cp_async_commit();
    }
    cp_async_wait<0>();

    // ---- results
    float l_all = l_run;
#pragma unroll
    for (int d = TPR / 2; d; d >>= 1) l_all += __shfl_xor_sync(~0u, l_all, d);
    if (whole) {
      if (sk0 == 0) {
        sInv[srow] = l_all == 0.f ? 0.f : 1.f / l_all;
        if (p.lse && srow < live)
          p.lse[(size_t)q.begin * H + row0 + srow] = l_all == 0.f ? -INFINITY : (m_run + log2f(l_all)) * kLn2;
      }
      __syncthreads();
      T* out = static_cast<T*>(p.out) + ((size_t)q.begin * H + row0) * kRank;
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const int r = m * 16 + (lane >> 2) + hf * 8;
          const float iv = sInv[r];
          if (r < live) {
            uint32_t* o = reinterpret_cast<uint32_t*>(out + (size_t)r * kRank + warp * S::kCols) + (lane & 3);
#pragma unroll
            for (int n = 0; n < NT; ++n) o[n * 4] = E::pack(acc[m][n][2 * hf] * iv, acc[m][n][2 * hf + 1] * iv);
          }
        }
    } else {
      const size_t slot = (size_t)w * 2 + (c.lo < x0 ? 0 : 1);
      if (sk0 == 0) {
        float* ml = p.part_ml + (slot * R + srow) * 2;
        ml[0] = m_run;
        ml[1] = l_all;
      }
      if (t0 < t1) {
        float* po = p.part_o + slot * R * kRank;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const int r = m * 16 + (lane >> 2) + hf * 8;
            float2* o = reinterpret_cast<float2*>(po + (size_t)r * kRank + warp * S::kCols) + (lane & 3);
#pragma unroll
            for (int n = 0; n < NT; ++n) o[n * 4] = make_float2(acc[m][n][2 * hf], acc[m][n][2 * hf + 1]);
          }
      }
    }
  }
}

// ---------------------------------------------------------------- combine
// Block (w1, y): the item that worker w1 began and others went on with (the
// record that w1 left); rows 8y .. 8y + 7 of it, one warp per row.  With
// weights u_i = 2^(m_i - m):
//   l = sum u_i l_i,  out = sum u_i o_i / l,  lse = (m + log2 l) * ln 2.
// Bound by latency: a lane reads the maximum and sum of one piece, and the
// rows of four pieces are in flight at a time.
template <typename T>
__global__ void __launch_bounds__(256) paged_combine_kernel(const PagedParams p, int R) {
  using E = Elem<T>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_dep_wait();  // (every block waits, so that this kernel never ends before the one that makes the pieces)
  const int w1 = blockIdx.x;
  const PagedJoin join = p.joins[w1];
  const int r = blockIdx.y * 8 + warp;
  if (r >= join.rows || !plan_join_fits(p, join, w1, R)) return;
  const int w2 = join.last_worker;
  const size_t row = (size_t)join.row + r;
  const int n = w2 - w1 + 1;
  auto slot = [&](int i) { return (size_t)(w1 + i) * 2 + (i == 0 ? 1 : 0); };
  auto ml = [&](int i) { return i < n ? reinterpret_cast<const float2*>(p.part_ml)[slot(i) * R + r] : make_float2(-INFINITY, 0.f); };
  float m = -INFINITY;
  for (int i = lane; i < n; i += 32) {
    const float2 a = ml(i);
    if (a.y != 0.f) m = fmaxf(m, a.x);
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
  float l = 0.f, o[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) o[i] = 0.f;
  for (int i0 = 0; i0 < n; i0 += 32) {
    const float2 a = ml(i0 + lane);
    const float f = a.y == 0.f ? 0.f : exp2f(a.x - m);  // (0: no key in this piece, its row is not written)
    l += f * a.y;
    const int end = min(32, n - i0);
    for (int j0 = 0; j0 < end; j0 += 4) {
      float4 x[4][4];
      float w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[j] = __shfl_sync(~0u, f, (j0 + j) & 31);
        if (j0 + j >= end) w[j] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) x[j][i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (w[j] != 0.f) {
          const float4* po = reinterpret_cast<const float4*>(p.part_o + (slot(i0 + j0 + j) * R + r) * kRank);
#pragma unroll
          for (int i = 0; i < 4; ++i) x[j][i] = po[i * 32 + lane];
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          o[4 * i] += w[j] * x[j][i].x;
          o[4 * i + 1] += w[j] * x[j][i].y;
          o[4 * i + 2] += w[j] * x[j][i].z;
          o[4 * i + 3] += w[j] * x[j][i].w;
        }
    }
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) l += __shfl_xor_sync(~0u, l, d);
  const float iv = l == 0.f ? 0.f : 1.f / l;
  uint2* d = reinterpret_cast<uint2*>(static_cast<T*>(p.out) + row * kRank);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    d[i * 32 + lane] = make_uint2(E::pack(o[4 * i] * iv, o[4 * i + 1] * iv), E::pack(o[4 * i + 2] * iv, o[4 * i + 3] * iv));
  if (p.lse && lane == 0) p.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

template <typename T, int MT>
cudaError_t prepare_mma() {
  return cudaFuncSetAttribute(paged_mma_kernel<T, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, PmCfg<MT>::kBytes);
}
template <typename T, int MT>
cudaError_t launch_mma(const PagedParams& p, cudaStream_t stream) {
  paged_mma_kernel<T, MT><<<p.workers, PmCfg<MT>::kThreads, PmCfg<MT>::kBytes, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t paged_mma_prepare(bool bf16) {
  const cudaError_t e = bf16 ? prepare_mma<__nv_bfloat16, 1>() : prepare_mma<__half, 1>();
  if (e != cudaSuccess) return e;
  return bf16 ? prepare_mma<__nv_bfloat16, 2>() : prepare_mma<__half, 2>();
}

cudaError_t paged_mma_launch(bool bf16, const PagedParams& p, int rows, cudaStream_t stream) {
  if (rows == 16)
    return bf16 ? launch_mma<__nv_bfloat16, 1>(p, stream) : launch_mma<__half, 1>(p, stream);
  return bf16 ? launch_mma<__nv_bfloat16, 2>(p, stream) : launch_mma<__half, 2>(p, stream);
}

cudaError_t paged_combine_launch(bool bf16, const PagedParams& p, int rows, cudaStream_t stream) {
  if (p.workers < 2) return cudaSuccess;
  // launched while the kernel before it runs (it waits for that one's end before it reads the pieces)
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(p.workers, (rows + 7) / 8);
  c.blockDim = dim3(256);
  c.stream = stream;
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &at;
  c.numAttrs = 1;
  return bf16 ? cudaLaunchKernelEx(&c, paged_combine_kernel<__nv_bfloat16>, p, rows)
              : cudaLaunchKernelEx(&c, paged_combine_kernel<__half>, p, rows);
}

}  // namespace mla
