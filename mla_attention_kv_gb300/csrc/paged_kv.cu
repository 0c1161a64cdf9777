// paged_kv.cu -- attention of new tokens over the paged k_nope / value / k_pe
// caches that the prolog writes, in 16 bits or as int8 codes with a scale per
// channel; and the kernel that joins partial results.
//
// Per query row r (a token and a head; q = [q_nope | q_pe], 192 wide) of KV
// head h and cached token j:
//   s_j = scale * (q_nope . k_nope_hj + q_pe . k_pe_j)
//   out = sum_j softmax(s)_j value_hj
// in one pass over the keys with a running maximum and sum, as in
// paged_mma.cu.  int8 codes stand for code * scale_c, so the key scales go
// into the queries and the value scales into the result:
//   s_j = sum_c (q_c k_scale_c) kcode_jc,  out_c = v_scale_c sum_j p_j vcode_jc.
//
// A key is read once per KV head (640 bytes with 16 bits: 256 + 256 of its
// own and 128 that the heads share, which come from L2 after the first) and
// used by n * G query rows, one of them in plain decoding with a head of its
// own: the kernel is bound by the cache's bytes.  So each warp is a worker
// with its own share of the keys, its own ring of stages filled by 16-byte
// cp.async (any page size; a page may end anywhere in a stage) and its own
// running softmax: nothing in the loop waits for another warp.  The products
// run on mma.sync with 16 query rows (a stage's chain of loads, not the
// tensor cores' rate, is what a warp waits for).
//
// int8: codes become fp16 exactly (byte ^ 0x80 as the low byte of 1024 + u,
// minus 1152).  The scaled queries are split in two fp16 parts, high and low,
// that take rows 0-7 and 8-15 of the same operand, so the products see them
// to about 2^-22 at no cost; an item then has 8 rows.  A thread's four
// consecutive codes of a key are four columns of one k-step in an order of
// its own, and the queries are laid out in the same order.
#include "attn.h"
#include "common.cuh"
#include "paged_kv_plan.cuh"

namespace mla {
namespace {

constexpr int kStages = 2;
constexpr int kStageBytes = 10240;  // keys 4 KB, rotated parts 2 KB, values 4 KB
constexpr int kPeOff = 4096, kVOff = 6144;
constexpr int kWarpBytes = kStages * kStageBytes;
constexpr int kKvThreads = kKvWarps * 32;
constexpr int kKvSmem = kKvWarps * kWarpBytes + (int)sizeof(PlanShared);
static_assert(kKvSmem <= 227 * 1024, "shared memory");

template <bool kI8>
struct KvCfg {
  static constexpr int R = kI8 ? kKvRowsI8 : kKvRows;
  static constexpr int E = kI8 ? 1 : 2;        // bytes per value
  static constexpr int Keys = kI8 ? 32 : 16;   // per stage
  static constexpr int CK = kNope * E / 16;    // 16-byte chunks of a key (and value) row
  static constexpr int CP = kRope * E / 16;    // of a rotated part
};

// Where chunk c of row r lies within a block of rows of 8 or 16 chunks (keys,
// values, 16-bit rotated parts) or of 4 (int8 rotated parts): any eight
// consecutive rows' chunks c fall on different banks.
template <int kChunks>
__device__ __forceinline__ uint32_t kv_at(int r, int c) {
  if (kChunks >= 8) return (uint32_t)(r * kChunks + (c ^ (r & 7))) * 16;
  return (uint32_t)(r * kChunks + (c ^ ((r >> 1) & 3))) * 16;
}

// Four int8 codes to fp16: lo = (byte i0, byte i1), hi = (byte i2, byte i3),
// chosen by the selectors (bytes 0-3 the codes, 4-7 the constant 0x64).
__device__ __forceinline__ uint32_t kv_half2(uint32_t biased, uint32_t selector) {
  const uint32_t u = __byte_perm(biased, 0x64646464u, selector);
  const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&u), __float2half2_rn(1152.f));
  return *reinterpret_cast<const uint32_t*>(&h);
}

// kWhole: pages are multiples of 16 rows, so that each 16 rows of a stage lie
// in one page.
template <typename T, bool kI8, bool kWhole>
__global__ void __launch_bounds__(kKvThreads, 1) paged_kv_kernel(const __grid_constant__ PagedKvParams p) {
  using E = Elem<T>;
  using S = KvCfg<kI8>;
  constexpr int R = S::R;
  constexpr bool kBf16 = !kI8 && E::kBf16;  // (codes are multiplied as fp16)
  extern __shared__ __align__(128) unsigned char smem[];
  PlanShared* plan = reinterpret_cast<PlanShared*>(smem + kKvWarps * kWarpBytes);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, q4 = lane & 3;
  const uint32_t ring = smem_u32(smem) + warp * kWarpBytes;
  const int G = p.plan.heads, H = G * p.kv_heads;

  grid_dep_launch_dependents();  // (the joining kernel may take its place)
  const long long total = kv_total(p, plan, R, blockIdx.x == 0);
  const int W = total > 0 ? kv_workers(total, p.plan.workers) : 0;
  const int w = warp * gridDim.x + blockIdx.x;  // (few workers: spread over the SMs)
  if (lane == 0) plan_open_join(p.plan, w);
  if (w >= W) return;
  const long long x0 = plan_worker_begin(total, w, W), x1 = plan_worker_begin(total, w + 1, W);

  KvCursor c;
  c.seek(p, plan, R, x0);
  for (bool more = true; more && c.lo < x1; more = c.next(p, R)) {
    const Seq sq = c.q;
    const int row0 = c.j * R;
    const int live = min(R, sq.n * G - row0);
    const int keys = sq.keys_of_item(c.j, R, G);
    const int tiles = (keys + kKvTile - 1) / kKvTile;
    const long long a = x0 > c.lo ? x0 : c.lo, b = x1 < c.hi ? x1 : c.hi;
    constexpr int kSub = kKvTile / S::Keys;
    const int t0 = c.tile_at(a, tiles) * kSub, t1 = min(c.tile_at(b, tiles) * kSub, (keys + S::Keys - 1) / S::Keys);
    const bool whole = c.lo >= x0 && c.hi <= x1;
    if (lane == 0 && c.hi >= x1) kv_post_join(p, c, R, w, x0, x1, total, W);

    // ---- stages.  A place is looked up two stages ahead of its use.
    constexpr int kParts = kWhole ? S::Keys / 16 : 1;  // of a stage that lie in one page each
    struct Place { int blk[kParts], off[kParts]; };
    const unsigned char* kb = static_cast<const unsigned char*>(p.k) + c.head * p.k_hs * S::E;
    const unsigned char* vb = static_cast<const unsigned char*>(p.v) + c.head * p.v_hs * S::E;
    const unsigned char* pb = static_cast<const unsigned char*>(p.kpe);
    const int32_t* table = p.plan.table + (size_t)c.s * p.plan.table_stride;
    auto check = [&](Place& pl) {
#pragma unroll
      for (int i = 0; i < kParts; ++i)
        if (pl.off[i] >= 0 && (pl.blk[i] < 0 || pl.blk[i] >= p.plan.nblocks)) {
          atomicOr(p.plan.status, kStatusBadSlot);
          pl.off[i] = -1;
        }
    };
    constexpr int kRowsAt = 32 / S::CK, kPeRowsAt = 32 / S::CP;
    // (kWhole) the next 16 rows to look up: their page and the first row there
    int npg = 0, noff = 0;
    if (kWhole) {
      npg = (int)((unsigned)(t0 * S::Keys) / (unsigned)p.plan.page);
      noff = t0 * S::Keys - npg * p.plan.page;
    }
    auto place_of = [&](int t) {
      Place pl;
      if constexpr (kWhole) {  // all lanes alike
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
          const bool ok = t < t1 && t * S::Keys + 16 * i < keys;
          pl.blk[i] = ok ? table[npg] : 0;
          pl.off[i] = ok ? noff : -1;
          noff += 16;
          if (noff == p.plan.page) noff = 0, ++npg;
        }
      } else {  // lane r looks up row r
        const int k = t * S::Keys + lane;
        const bool ok = t < t1 && lane < S::Keys && k < keys;
        const int pg = ok ? (int)((unsigned)k / (unsigned)p.plan.page) : 0;
        pl.blk[0] = ok ? table[pg] : 0;
        pl.off[0] = ok ? k - pg * p.plan.page : -1;
      }
      return pl;
    };
    auto load = [&](int t, Place pl) {
      check(pl);
      const uint32_t st = ring + (t % kStages) * kStageBytes;
      if constexpr (kWhole) {
        const int r0 = lane / S::CK, e0 = lane / S::CP;
        const long long kstep = (long long)kRowsAt * p.k_rs * S::E, vstep = (long long)kRowsAt * p.v_rs * S::E,
                        pstep = (long long)kPeRowsAt * p.kpe_rs * S::E;
#pragma unroll
        for (int h = 0; h < kParts; ++h) {
          const int rows = pl.off[h] < 0 ? 0 : keys - t * S::Keys - 16 * h;  // that there are
          const long long blk = pl.off[h] < 0 ? 0 : pl.blk[h], off = pl.off[h] < 0 ? 0 : pl.off[h];
          const unsigned char* ks = kb + (blk * p.k_bs + (off + r0) * p.k_rs) * S::E + lane % S::CK * 16;
          const unsigned char* vs = vb + (blk * p.v_bs + (off + r0) * p.v_rs) * S::E + lane % S::CK * 16;
          const unsigned char* ps = pb + (blk * p.kpe_bs + (off + e0) * p.kpe_rs) * S::E + lane % S::CP * 16;
#pragma unroll
          for (int i = 0; i < 16 / kRowsAt; ++i) {
            const int r = i * kRowsAt + r0, n = r < rows ? 16 : 0;
            const uint32_t d = st + kv_at<S::CK>(16 * h + r, lane % S::CK);
            cp_async16(d, ks, n);
            cp_async16(d + kVOff, vs, n);
            ks += kstep;
            vs += vstep;
          }
#pragma unroll
          for (int i = 0; i < 16 / kPeRowsAt; ++i) {
            const int r = i * kPeRowsAt + e0;
            cp_async16(st + kPeOff + kv_at<S::CP>(16 * h + r, lane % S::CP), ps, r < rows ? 16 : 0);
            ps += pstep;
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < S::Keys / kRowsAt; ++i) {
          const int r = i * kRowsAt + lane / S::CK, ch = lane % S::CK;
          const int blk = __shfl_sync(~0u, pl.blk[0], r), off = __shfl_sync(~0u, pl.off[0], r);
          const bool ok = off >= 0;
          const long long kx = ok ? blk * p.k_bs + (long long)off * p.k_rs : 0, vx = ok ? blk * p.v_bs + (long long)off * p.v_rs : 0;
          cp_async16(st + kv_at<S::CK>(r, ch), kb + kx * S::E + ch * 16, ok ? 16 : 0);
          cp_async16(st + kVOff + kv_at<S::CK>(r, ch), vb + vx * S::E + ch * 16, ok ? 16 : 0);
        }
#pragma unroll
        for (int i = 0; i < S::Keys / kPeRowsAt; ++i) {
          const int r = i * kPeRowsAt + lane / S::CP, ch = lane % S::CP;
          const int blk = __shfl_sync(~0u, pl.blk[0], r), off = __shfl_sync(~0u, pl.off[0], r);
          const bool ok = off >= 0;
          const long long x = ok ? blk * p.kpe_bs + (long long)off * p.kpe_rs : 0;
          cp_async16(st + kPeOff + kv_at<S::CP>(r, ch), pb + x * S::E + ch * 16, ok ? 16 : 0);
        }
      }
    };
    {
      Place first[kStages];
#pragma unroll
      for (int i = 0; i < kStages; ++i) first[i] = place_of(t0 + i);
#pragma unroll
      for (int i = 0; i < kStages; ++i) {
        if (t0 + i < t1) load(t0 + i, first[i]);
        cp_async_commit();
      }
    }

    // ---- queries, as operand fragments (rows past the item's end are zero)
    uint32_t qf[12][4];
    float row_scale = p.plan.scale_log2;
    auto q_row = [&](int r, const T*& qn, const T*& qp) {
      const int tok = (row0 + r) / G, hd = c.head * G + (row0 + r) - tok * G;
      qn = static_cast<const T*>(p.q_nope) + (long long)(sq.begin + tok) * p.qn_ts + (long long)hd * p.qn_hs;
      qp = static_cast<const T*>(p.q_pe) + (long long)(sq.begin + tok) * p.qp_ts + (long long)hd * p.qp_hs;
    };
    if constexpr (!kI8) {
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int r = g + hf * 8;
        const bool ok = r < live;
        const T *qn = nullptr, *qp = nullptr;
        if (ok) q_row(r, qn, qp);
#pragma unroll
        for (int k = 0; k < 12; ++k) {
          const T* src = k < 8 ? qn + k * 16 : qp + (k - 8) * 16;
          qf[k][hf] = ok ? *reinterpret_cast<const uint32_t*>(src + 2 * q4) : 0;
          qf[k][2 + hf] = ok ? *reinterpret_cast<const uint32_t*>(src + 8 + 2 * q4) : 0;
        }
      }
    } else {
      // q * scale, brought to a largest magnitude of 2^13 .. 2^14 by a power of two, as high + low fp16 parts
      float x[48], mx = 0.f;
      const bool ok = g < live;
      const T *qn = nullptr, *qp = nullptr;
      if (ok) q_row(g, qn, qp);
#pragma unroll
      for (int k = 0; k < 12; ++k) {
        const T* src = (k < 8 ? qn + k * 16 : qp + (k - 8) * 16) + 4 * q4;
        const float4 sc = *reinterpret_cast<const float4*>((k < 8 ? p.k_scale + c.head * kNope + k * 16 : p.kpe_scale + (k - 8) * 16) + 4 * q4);
        const uint2 v = ok ? *reinterpret_cast<const uint2*>(src) : make_uint2(0, 0);
        const T* e = reinterpret_cast<const T*>(&v);
        x[4 * k] = E::to_f(e[0]) * sc.x;
        x[4 * k + 1] = E::to_f(e[1]) * sc.y;
        x[4 * k + 2] = E::to_f(e[2]) * sc.z;
        x[4 * k + 3] = E::to_f(e[3]) * sc.w;
#pragma unroll
        for (int i = 0; i < 4; ++i) mx = fmaxf(mx, fabsf(x[4 * k + i]));
      }
      mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 2));
      const int up = mx > 0.f && mx < INFINITY ? min(13 - ilogbf(mx), 100) : 0;
      const float f = scalbnf(1.f, up);
      row_scale *= scalbnf(1.f, -up);
#pragma unroll
      for (int k = 0; k < 12; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float y0 = x[4 * k + 2 * i] * f, y1 = x[4 * k + 2 * i + 1] * f;
          const __half2 hi = __floats2half2_rn(y0, y1);
          const float2 hf = __half22float2(hi);
          const __half2 lo = __floats2half2_rn(y0 - hf.x, y1 - hf.y);
          qf[k][2 * i] = *reinterpret_cast<const uint32_t*>(&hi);
          qf[k][2 * i + 1] = *reinterpret_cast<const uint32_t*>(&lo);
        }
    }
    const int lim0 = g < live ? sq.keys_of_row(row0 + g, G) : 0;
    const int lim1 = !kI8 && g + 8 < live ? sq.keys_of_row(row0 + g + 8, G) : 0;

    float acc[16][4];
#pragma unroll
    for (int n = 0; n < 16; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;  // rows g and g + 8

    for (int t = t0; t < t1; ++t) {
      const Place ahead = place_of(t + kStages);
      cp_async_wait<kStages - 1>();
      __syncwarp();
      const uint32_t st = ring + (t % kStages) * kStageBytes;
      constexpr int NT = S::Keys / 8;
      float sc[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[n][i] = 0.f;
      if constexpr (!kI8) {
        const int r = (lane & 7) + ((lane >> 4) & 1) * 8, cc = (lane >> 3) & 1;
        float s2[NT][4];  // (a second set of sums: shorter chains)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) s2[n][i] = 0.f;
#pragma unroll
        for (int k = 0; k < 12; ++k) {
          uint32_t b0, b1, b2, b3;
          ldsm_x4(k < 8 ? st + kv_at<S::CK>(r, 2 * k + cc) : st + kPeOff + kv_at<S::CP>(r, 2 * (k - 8) + cc), b0, b1, b2, b3);
          mma16816<kBf16>(k & 1 ? s2[0] : sc[0], qf[k], b0, b1);
          mma16816<kBf16>(k & 1 ? s2[1] : sc[1], qf[k], b2, b3);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) sc[n][i] += s2[n][i];
      } else {
#pragma unroll
        for (int k = 0; k < 12; ++k) {
          uint32_t x[4];
          ldsm_x4(k < 8 ? st + kv_at<S::CK>(lane, k) : st + kPeOff + kv_at<S::CP>(lane, k - 8), x[0], x[1], x[2], x[3]);
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            const uint32_t u = x[n] ^ 0x80808080u;
            mma16816<false>(sc[n], qf[k], kv_half2(u, 0x4140), kv_half2(u, 0x4342));
          }
        }
      }
      // ---- softmax: row g in sc[.][0..1], row g + 8 in sc[.][2..3]
      const int k0 = t * S::Keys + 2 * q4;
      float x0m = -INFINITY, x1m = -INFINITY;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int k = k0 + n * 8 + i;
          const float u = kI8 ? sc[n][i] + sc[n][2 + i] : sc[n][i];
          sc[n][i] = k < lim0 ? u * row_scale : -INFINITY;
          x0m = fmaxf(x0m, sc[n][i]);
          if (!kI8) {
            sc[n][2 + i] = k < lim1 ? sc[n][2 + i] * row_scale : -INFINITY;
            x1m = fmaxf(x1m, sc[n][2 + i]);
          }
        }
#pragma unroll
      for (int d = 1; d <= 2; d <<= 1) {
        x0m = fmaxf(x0m, __shfl_xor_sync(~0u, x0m, d));
        if (!kI8) x1m = fmaxf(x1m, __shfl_xor_sync(~0u, x1m, d));
      }
      const float n0 = fmaxf(m0, x0m), n1 = fmaxf(m1, x1m);
      const float u0 = n0 == -INFINITY ? 0.f : n0, u1 = n1 == -INFINITY ? 0.f : n1;  // (a row with no key so far)
      const float a0 = n0 == m0 ? 1.f : exp2f(m0 - u0), a1 = n1 == m1 ? 1.f : exp2f(m1 - u1);
      m0 = n0;
      m1 = n1;
      if (__any_sync(~0u, a0 != 1.f || a1 != 1.f)) {
        l0 *= a0;
        l1 *= a1;
#pragma unroll
        for (int n = 0; n < 16; ++n) {
          acc[n][0] *= a0;
          acc[n][1] *= a0;
          acc[n][2] *= a1;
          acc[n][3] *= a1;
        }
      }
      uint32_t pf[NT / 2][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float e0 = exp2f(sc[n][0] - u0), e1 = exp2f(sc[n][1] - u0);
        l0 += e0 + e1;
        if constexpr (kI8) {
          const __half2 h = __floats2half2_rn(e0, e1);
          pf[n / 2][(n & 1) * 2] = *reinterpret_cast<const uint32_t*>(&h);
          pf[n / 2][(n & 1) * 2 + 1] = 0;
        } else {
          const float e2 = exp2f(sc[n][2] - u1), e3 = exp2f(sc[n][3] - u1);
          l1 += e2 + e3;
          pf[n / 2][(n & 1) * 2] = E::pack(e0, e1);
          pf[n / 2][(n & 1) * 2 + 1] = E::pack(e2, e3);
        }
      }
      // ---- output
      if constexpr (!kI8) {
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          uint32_t b0, b1, b2, b3;
          ldsm_x4_trans(st + kVOff + kv_at<S::CK>(lane & 15, 2 * n + (lane >> 4)), b0, b1, b2, b3);
          mma16816<kBf16>(acc[2 * n], pf[0], b0, b1);
          mma16816<kBf16>(acc[2 * n + 1], pf[0], b2, b3);
        }
      } else {
        // chunk n: acc[2n] has its even columns, acc[2n + 1] its odd ones
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          uint32_t x[4];
          ldsm_x4_trans(st + kVOff + kv_at<S::CK>(lane, n), x[0], x[1], x[2], x[3]);
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] ^= 0x80808080u;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            mma16816<false>(acc[2 * n], pf[k], kv_half2(x[2 * k], 0x4240), kv_half2(x[2 * k + 1], 0x4240));
            mma16816<false>(acc[2 * n + 1], pf[k], kv_half2(x[2 * k], 0x4341), kv_half2(x[2 * k + 1], 0x4341));
          }
        }
      }
      __syncwarp();  // the stage is free
      if (t + kStages < t1) load(t + kStages, ahead);
      cp_async_commit();
    }
    cp_async_wait<0>();
    __syncwarp();

    // ---- results
#pragma unroll
    for (int d = 1; d <= 2; d <<= 1) {
      l0 += __shfl_xor_sync(~0u, l0, d);
      l1 += __shfl_xor_sync(~0u, l1, d);
    }
    const size_t slot = (size_t)w * 2 + (c.lo < x0 ? 0 : 1);
#pragma unroll
    for (int hf = 0; hf < (kI8 ? 1 : 2); ++hf) {
      const int r = g + hf * 8;
      if (r >= live) continue;
      const float l = hf ? l1 : l0, m = hf ? m1 : m0;
      const int tok = (row0 + r) / G, hd = c.head * G + (row0 + r) - tok * G;
      const size_t orow = (size_t)(sq.begin + tok) * H + hd;
      const float iv = !whole ? 1.f : l == 0.f ? 0.f : 1.f / l;
      T* out = static_cast<T*>(p.plan.out) + orow * kV;
      float* po = p.plan.part_o + (slot * R + r) * kV;
      if (q4 == 0) {
        if (!whole) {
          float* ml = p.plan.part_ml + (slot * R + r) * 2;
          ml[0] = m;
          ml[1] = l;
        } else if (p.plan.lse) {
          p.plan.lse[orow] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
        }
      }
      if constexpr (!kI8) {
#pragma unroll
        for (int n = 0; n < 16; ++n) {
          const float y0 = acc[n][2 * hf] * iv, y1 = acc[n][2 * hf + 1] * iv;
          if (whole)
            *reinterpret_cast<uint32_t*>(out + n * 8 + 2 * q4) = E::pack(y0, y1);
          else
            *reinterpret_cast<float2*>(po + n * 8 + 2 * q4) = make_float2(y0, y1);
        }
      } else {
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          const int col = n * 16 + 4 * q4;
          const float4 vs = *reinterpret_cast<const float4*>(p.v_scale + c.head * kV + col);
          const float4 y = make_float4(acc[2 * n][0] * iv * vs.x, acc[2 * n + 1][0] * iv * vs.y, acc[2 * n][1] * iv * vs.z,
                                       acc[2 * n + 1][1] * iv * vs.w);
          if (whole)
            *reinterpret_cast<uint2*>(out + col) = make_uint2(E::pack(y.x, y.y), E::pack(y.z, y.w));
          else
            *reinterpret_cast<float4*>(po + col) = y;
        }
      }
    }
  }
}

// ---------------------------------------------------------------- joining
// The rows of an item that worker w1 began and others went on with: with
// weights u_i = 2^(m_i - m) of its pieces,
//   l = sum u_i l_i,  out = sum u_i o_i / l,  lse = (m + log2 l) * ln 2.
// `per` warps (1, 2, 4, 8 or 16) share a record's rows, a warp taking one row at a
// time with 16 pieces in flight.  Bound by latency, so the grid is what fits
// on the GPU at once: with a block for each eight possible rows 12 sequences
// with 12 rows per head took 47 us instead of 39.
constexpr int kJoinFlight = 16;
template <typename T>
__global__ void __launch_bounds__(256) paged_kv_join_kernel(const __grid_constant__ PagedKvParams p, int per, int R) {
  using E = Elem<T>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int G = p.plan.heads, H = G * p.kv_heads;
  grid_dep_wait();  // (every block waits, so that this kernel never ends before the one that makes the pieces)
  // (neighbouring records to a group: a long item leaves one record in many, at even distances)
  const int groups = gridDim.x * 8 / per, each = (p.plan.workers + groups - 1) / groups, first = (blockIdx.x * 8 + warp) / per * each;
  for (int c0 = 0; c0 < each; c0 += 32) {
   // (a lane looks at a record: most of them are empty)
   const int mine = first + c0 + lane;
   PagedJoin rec = {0, 0, 0, 0};
   if (c0 + lane < each && mine < p.plan.workers) rec = p.plan.joins[mine];
   const bool fits = rec.rows > 0 && rec.rows <= R && rec.row >= 0 && (long long)rec.row + rec.rows <= (long long)p.plan.T * G &&
                     rec.pad >= 0 && rec.pad < p.kv_heads && rec.last_worker >= mine && rec.last_worker < p.plan.workers;
   for (uint32_t left = __ballot_sync(~0u, fits); left; left &= left - 1) {
    const int from = __ffs(left) - 1, w1 = first + c0 + from;
    const PagedJoin j = {__shfl_sync(~0u, rec.row, from), __shfl_sync(~0u, rec.rows, from), __shfl_sync(~0u, rec.last_worker, from),
                         __shfl_sync(~0u, rec.pad, from)};
    const int n = j.last_worker - w1 + 1;
    auto slot = [&](int i) { return (size_t)(w1 + i) * 2 + (i == 0 ? 1 : 0); };
    for (int r = (blockIdx.x * 8 + warp) % per; r < j.rows; r += per) {
      const int tok = (j.row + r) / G;
      const size_t orow = (size_t)tok * H + j.pad * G + (j.row + r) - tok * G;
      auto ml = [&](int i) { return i < n ? reinterpret_cast<const float2*>(p.plan.part_ml)[slot(i) * R + r] : make_float2(-INFINITY, 0.f); };
      float m = -INFINITY;
      for (int i = lane; i < n; i += 32) {
        const float2 a = ml(i);
        if (a.y != 0.f) m = fmaxf(m, a.x);
      }
#pragma unroll
      for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
      float l = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int i0 = 0; i0 < n; i0 += 32) {
        const float2 a = ml(i0 + lane);
        const float f = a.y == 0.f ? 0.f : exp2f(a.x - m);
        l += f * a.y;
        const int end = min(32, n - i0);
        for (int j0 = 0; j0 < end; j0 += kJoinFlight) {
          float4 y[kJoinFlight];
          float u[kJoinFlight];
#pragma unroll
          for (int k = 0; k < kJoinFlight; ++k) {
            // (all loads are made, those past the end of the last piece: under a condition each would wait for the one
            // before.  A piece without keys has zeros.)
            const int i = min(j0 + k, end - 1);
            u[k] = __shfl_sync(~0u, f, i);
            if (j0 + k >= end) u[k] = 0.f;
            y[k] = reinterpret_cast<const float4*>(p.plan.part_o + (slot(i0 + i) * R + r) * kV)[lane];
          }
#pragma unroll
          for (int k = 0; k < kJoinFlight; ++k) {
            o.x += u[k] * y[k].x;
            o.y += u[k] * y[k].y;
            o.z += u[k] * y[k].z;
            o.w += u[k] * y[k].w;
          }
        }
      }
#pragma unroll
      for (int d = 16; d; d >>= 1) l += __shfl_xor_sync(~0u, l, d);
      const float iv = l == 0.f ? 0.f : 1.f / l;
      reinterpret_cast<uint2*>(static_cast<T*>(p.plan.out) + orow * kV)[lane] =
          make_uint2(E::pack(o.x * iv, o.y * iv), E::pack(o.z * iv, o.w * iv));
      if (p.plan.lse && lane == 0) p.plan.lse[orow] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
    }
   }
  }
}

template <typename T, bool kI8>
cudaError_t launch(const PagedKvParams& p, cudaStream_t stream) {
  const bool whole = p.plan.page % 16 == 0;
  if (whole)
    paged_kv_kernel<T, kI8, true><<<p.plan.workers / kKvWarps, kKvThreads, kKvSmem, stream>>>(p);
  else
    paged_kv_kernel<T, kI8, false><<<p.plan.workers / kKvWarps, kKvThreads, kKvSmem, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  constexpr int R = KvCfg<kI8>::R;
  // rows of an item (with ragged chunks the average, which is all the host knows)
  const long long rows = (long long)(p.plan.T / p.plan.nseq > 0 ? p.plan.T / p.plan.nseq : 1) * p.plan.heads;
  const int per = rows <= 1 ? 1 : rows <= 2 ? 2 : rows <= 4 ? 4 : rows <= 8 || R == 8 ? 8 : 16;
  const int blocks = (p.plan.workers * per + 15) / 8, most = p.plan.workers / kKvWarps * 2;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((blocks < most ? blocks : most) & ~1);  // (16 warps are two blocks)
  c.blockDim = dim3(256);
  c.stream = stream;
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, paged_kv_join_kernel<T>, p, per, R);
}

template <typename T>
cudaError_t prepare() {
  const void* k[4] = {(const void*)paged_kv_kernel<T, false, false>, (const void*)paged_kv_kernel<T, false, true>,
                      (const void*)paged_kv_kernel<T, true, false>, (const void*)paged_kv_kernel<T, true, true>};
  for (const void* f : k) {
    const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kKvSmem);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t paged_kv_prepare(bool bf16) { return bf16 ? prepare<__nv_bfloat16>() : prepare<__half>(); }

cudaError_t paged_kv_launch(bool bf16, bool i8, const PagedKvParams& p, cudaStream_t stream) {
  if (i8) return bf16 ? launch<__nv_bfloat16, true>(p, stream) : launch<__half, true>(p, stream);
  return bf16 ? launch<__nv_bfloat16, false>(p, stream) : launch<__half, false>(p, stream);
}

}  // namespace mla
