// paged_kv.cu -- attention of new tokens over the paged k_nope / value / k_pe
// caches that the prolog writes, in 16 bits or as int8 codes with a scale per
// channel; and the kernel that joins partial results of many rows.
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
// running softmax: nothing in the loop waits for another warp.  Pieces of
// an item that several workers share are joined in their order.  Few rows: by
// the worker that finishes last (its being last changes nothing in the result).
// More: by a second kernel, which spreads them over the GPU.  64 sequences of
// up to 4096 keys, 16 heads, one row each: 177 us, 182 with the second kernel;
// 12 rows per head in 20 pieces: 45 us with it, 69 without; 4 rows 37 and 42.
// The products run on mma.sync, in one of three forms:
//   up to 8 rows: S^T = K Q^T and O^T = V^T P^T, keys and value columns being
//     the 16 rows of an operand and the query rows its 8 columns.  P^T turns
//     from result to operand by a transposing move.  Half the products of the
//     last form, and 32 registers of output instead of 64;
//   int8, up to 4 rows: the same with the queries' high parts in columns 0-3 and
//     their low parts in columns 4-7, so that a key is multiplied once for
//     both (16 sequences of up to 4096 keys, 128 heads: 194 us, 205 without);
//   up to 16 rows (16-bit caches): S = Q K^T and O = P V.
// Eight warps per SM: eleven, which the first form has room for, bring more
// pieces to join and no more bandwidth (64 sequences of up to 4096 keys, 16
// heads: 182 us and 181).
//
// The softmax weights enter the second product in 16 bits (the type of the
// caches, fp16 with int8), which is the one rounding on the way; sums, maxima
// and results in progress have 32.  With a second part for what the rounding
// leaves, that product would be made twice; so the results' error against 64
// bits is 0.00024 with fp16 and 0.0021 with bf16, where 32-bit weights have 0.0002 and
// 0.0017, the rounding of the result itself.
//
// int8: the scaled queries are split in two fp16 parts, high and low, so the
// products see them to about 2^-22.  Codes become fp16 exactly (byte ^ 0x80 as
// the low byte of 1024 + u, minus 1152), so a sum is never larger than the
// products in it, whatever part of their range the codes use.  Scores of codes
// that keep an offset, code + 128, with 128 times the queries' sum taken off at
// the end, are 12 us faster (16 sequences of up to 4096 keys, 128 heads: 182 us,
// 194 so), but their sums are (|code| + 128) / |code| times as large, and with codes
// of 0 and 1 a score is off by several hundred 2^-23 of sum |q k|.  The integer
// pipe and these moves bound this form beside the bytes.  A thread's four
// consecutive codes of a key are four columns of one k-step in an order of its
// own, and the queries are laid out in the same order.
#include "attn.h"
#include "attn_tc.cuh"
#include "paged_kv_plan.cuh"

namespace mla {
namespace {

constexpr int kStages = 2;
constexpr int kJoinFlight = 16;  // pieces in flight when they are joined
constexpr int kStageBytes = 10240;  // keys 4 KB, rotated parts 2 KB, values 4 KB
constexpr int kPeOff = 4096, kVOff = 6144;
constexpr int kWarpBytes = kStages * kStageBytes;
constexpr int kKvThreads = kKvWarps * 32;
constexpr int kKvSmem = kKvWarps * kWarpBytes + (int)sizeof(PlanShared);
static_assert(kKvSmem <= 227 * 1024, "shared memory");

// kForm: how the products are made.
enum KvForm {
  kWide,   // up to 16 query rows per item
  kTrans,  // up to 8, transposed
  kSplit,  // int8, up to 4: columns 0-3 are the queries' high parts, columns 4-7 their low parts
};
template <bool kI8, KvForm kForm>
struct KvCfg {
  static constexpr int R = kForm == kWide ? kKvRows : kForm == kTrans ? kKvRowsT : kKvRowsSplit;
  static constexpr int E = kI8 ? 1 : 2;        // bytes per value
  static constexpr int Keys = kI8 ? 32 : 16;   // per stage
  static constexpr int CK = kNope * E / 16;    // 16-byte chunks of a key (and value) row
  static constexpr int CP = kRope * E / 16;    // of a rotated part
  static_assert(R * kV * 4 <= kWarpBytes, "results pass through the ring");
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

// The 8 x 8 matrix of 16-bit values that a warp holds (lane = row * 4 + pair), transposed.
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// One row of an item from its n pieces, of which piece(i) is the place: with
// weights u_i = 2^(m_i - m), m the largest m_i,
//   l = sum u_i l_i,  out = sum u_i o_i (four columns a lane), in a fixed order.
// kFlight (a divisor of 32) pieces are in flight, the first ones before the
// weights are known.
template <int kFlight, typename Piece>
__device__ __forceinline__ float4 kv_join_row(const PagedParams& p, int n, Piece piece, float* m_out, float* l_out) {
  const int lane = threadIdx.x & 31;
  const float4* part_o = reinterpret_cast<const float4*>(p.part_o) + lane;
  const float2* part_ml = reinterpret_cast<const float2*>(p.part_ml);
  float4 y[kFlight];
  // (all loads are made, those past the end of the last piece: under a condition each would wait for the one before)
  auto request = [&](int j0) {
#pragma unroll
    for (int k = 0; k < kFlight; ++k) y[k] = __ldcg(part_o + piece(min(j0 + k, n - 1)) * (kV / 4));
  };
  request(0);
  auto ml = [&](int i) { return i < n ? __ldcg(part_ml + piece(i)) : make_float2(-INFINITY, 0.f); };
  const float2 a0 = ml(lane);
  float m = a0.x;
  for (int i = 32 + lane; i < n; i += 32) m = fmaxf(m, ml(i).x);
#pragma unroll
  for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
  const float mu = m == -INFINITY ? 0.f : m;  // (no piece has keys)
  float l = 0.f, f = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j0 = 0; j0 < n; j0 += kFlight) {
    if (j0 % 32 == 0) {
      const float2 a = j0 == 0 ? a0 : ml(j0 + lane);
      f = ex2(a.x - mu);
      l += f * a.y;
    }
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      const float u = __shfl_sync(~0u, f, (j0 + k) & 31);
      if (j0 + k < n) {
        o.x += u * y[k].x;
        o.y += u * y[k].y;
        o.z += u * y[k].z;
        o.w += u * y[k].w;
      }
    }
    if (j0 + kFlight < n) request(j0 + kFlight);
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) l += __shfl_xor_sync(~0u, l, d);
  *m_out = m;
  *l_out = l;
  return o;
}

// kWhole: pages are multiples of 16 rows, so that each 16 rows of a stage lie
// in one page.
template <typename T, bool kI8, KvForm kForm, bool kWhole>
__global__ void __launch_bounds__(kKvThreads, 1) paged_kv_kernel(const __grid_constant__ PagedKvParams p) {
  using E = Elem<T>;
  using S = KvCfg<kI8, kForm>;
  constexpr bool kT = kForm != kWide, kTwo = kForm == kSplit;
  static_assert(kI8 ? kT : !kTwo, "int8 is transposed");
  constexpr int R = S::R;
  extern __shared__ __align__(128) unsigned char smem[];
  PlanShared* plan = reinterpret_cast<PlanShared*>(smem + kKvWarps * kWarpBytes);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, q4 = lane & 3;
  const uint32_t ring = smem_u32(smem) + warp * kWarpBytes;
  const int G = p.plan.heads, H = G * p.kv_heads;

  if (!p.join_here) grid_dep_launch_dependents();  // (the joining kernel may take its place)
  const long long total = kv_total(p, plan, R, blockIdx.x == 0);
  const int W = total > 0 ? kv_workers(total, p.plan.workers) : 0;
  const int w = warp * gridDim.x + blockIdx.x;  // (few workers: spread over the SMs)
  if (!p.join_here && lane == 0) plan_open_join(p.plan, w);
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
    if (!p.join_here && lane == 0 && c.hi >= x1) kv_post_join(p, c, R, w, x0, x1, total, W);

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
    auto q_row = [&](int r, const T*& qn, const T*& qp) {
      const int tok = (row0 + r) / G, hd = c.head * G + (row0 + r) - tok * G;
      qn = static_cast<const T*>(p.q_nope) + (long long)(sq.begin + tok) * p.qn_ts + (long long)hd * p.qn_hs;
      qp = static_cast<const T*>(p.q_pe) + (long long)(sq.begin + tok) * p.qp_ts + (long long)hd * p.qp_hs;
    };
    uint32_t qf[12][(kT && !kI8) || kTwo ? 2 : 4];
    float row_scale[2] = {p.plan.scale_log2, p.plan.scale_log2};
    if constexpr (!kI8) {
#pragma unroll
      for (int hf = 0; hf < (kT ? 1 : 2); ++hf) {
        const int r = g + hf * 8;
        const bool ok = r < live;
        const T *qn = nullptr, *qp = nullptr;
        if (ok) q_row(r, qn, qp);
#pragma unroll
        for (int k = 0; k < 12; ++k) {
          const T* src = k < 8 ? qn + k * 16 : qp + (k - 8) * 16;
          qf[k][hf] = ok ? *reinterpret_cast<const uint32_t*>(src + 2 * q4) : 0;
          qf[k][(kT ? 1 : 2) + hf] = ok ? *reinterpret_cast<const uint32_t*>(src + 8 + 2 * q4) : 0;
        }
      }
    } else {
      // q * scale, brought to a largest magnitude of 2^13 .. 2^14 by a power of two, as high + low fp16 parts
      float x[48], mx = 0.f;
      const int r = kTwo ? g & 3 : g;
      const bool ok = r < live;
      const T *qn = nullptr, *qp = nullptr;
      if (ok) q_row(r, qn, qp);
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
#pragma unroll
      for (int k = 0; k < 12; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) {  // (codes 0 and 2 of the four, then 1 and 3)
          const float y0 = x[4 * k + i] * f, y1 = x[4 * k + i + 2] * f;
          const __half2 hi = __floats2half2_rn(y0, y1);
          const float2 hf = __half22float2(hi);
          const __half2 lo = __floats2half2_rn(y0 - hf.x, y1 - hf.y);
          if constexpr (kTwo) {
            qf[k][i] = *reinterpret_cast<const uint32_t*>(g < 4 ? &hi : &lo);
          } else {
            qf[k][i] = *reinterpret_cast<const uint32_t*>(&hi);
            qf[k][2 + i] = *reinterpret_cast<const uint32_t*>(&lo);
          }
        }
      const float down = p.plan.scale_log2 * scalbnf(1.f, -up);
      const int ra = kTwo ? 2 * (q4 & 1) : 2 * q4;  // this lane's rows of the softmax (lane 4 r holds row r)
#pragma unroll
      for (int i = 0; i < 2; ++i) row_scale[i] = __shfl_sync(~0u, down, 4 * (ra + i));
    }
    // this lane's two rows of the softmax: 2 q4 and 2 q4 + 1 (kT), g and g + 8
    const int ra = kTwo ? 2 * (q4 & 1) : kT ? 2 * q4 : g, rb = kT ? ra + 1 : g + 8;
    const int lim0 = ra < live ? sq.keys_of_row(row0 + ra, G) : 0, lim1 = rb < live ? sq.keys_of_row(row0 + rb, G) : 0;
    const int lim_all = sq.keys_of_row(row0, G);  // keys that all rows see

    constexpr int NO = kT ? 8 : 16;
    float acc[NO][4];
#pragma unroll
    for (int n = 0; n < NO; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

    for (int t = t0; t < t1; ++t) {
      const Place ahead = place_of(t + kStages);
      cp_async_wait<kStages - 1>();
      __syncwarp();
      const uint32_t st = ring + (t % kStages) * kStageBytes;
      // ---- scores: sc[n] has (kT) keys 16 n + g, + 8 for rows ra, rb, or keys 8 n + 2 q4, + 1 for row ra, then for rb
      constexpr int NS = kT ? S::Keys / 16 : S::Keys / 8;
      float sc[NS][4], s2[NS][4];  // (two sets of sums: shorter chains)
#pragma unroll
      for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[n][i] = s2[n][i] = 0.f;
      if constexpr (kI8) {
#pragma unroll
        for (int k = 0; k < 12; ++k) {
          uint32_t x[4];
          ldsm_x4(k < 8 ? st + kv_at<S::CK>(lane, k) : st + kPeOff + kv_at<S::CP>(lane, k - 8), x[0], x[1], x[2], x[3]);
#pragma unroll
          for (int n = 0; n < 4; ++n) x[n] ^= 0x80808080u;
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const uint32_t af[4] = {kv_half2(x[2 * n], 0x4240), kv_half2(x[2 * n + 1], 0x4240), kv_half2(x[2 * n], 0x4341),
                                    kv_half2(x[2 * n + 1], 0x4341)};
            if constexpr (kTwo) {
              mma16816<false>(k & 1 ? s2[n] : sc[n], af, qf[k][0], qf[k][1]);
            } else {
              mma16816<false>(sc[n], af, qf[k][0], qf[k][1]);
              mma16816<false>(s2[n], af, qf[k][2], qf[k][3]);
            }
          }
        }
      } else if constexpr (kT) {
        const int r = (lane & 7) + ((lane >> 3) & 1) * 8, cc = lane >> 4;
#pragma unroll
        for (int k = 0; k < 12; ++k) {
          uint32_t af[4];
          ldsm_x4(k < 8 ? st + kv_at<S::CK>(r, 2 * k + cc) : st + kPeOff + kv_at<S::CP>(r, 2 * (k - 8) + cc), af[0], af[1], af[2], af[3]);
          mma16816<E::kBf16>(k & 1 ? s2[0] : sc[0], af, qf[k][0], qf[k][1]);
        }
      } else {
        const int r = (lane & 7) + ((lane >> 4) & 1) * 8, cc = (lane >> 3) & 1;
#pragma unroll
        for (int k = 0; k < 12; ++k) {
          uint32_t b0, b1, b2, b3;
          ldsm_x4(k < 8 ? st + kv_at<S::CK>(r, 2 * k + cc) : st + kPeOff + kv_at<S::CP>(r, 2 * (k - 8) + cc), b0, b1, b2, b3);
          mma16816<E::kBf16>(k & 1 ? s2[0] : sc[0], qf[k], b0, b1);
          mma16816<E::kBf16>(k & 1 ? s2[1] : sc[1], qf[k], b2, b3);
        }
      }
      // ---- softmax
      float x0m = -INFINITY, x1m = -INFINITY;
      // (value i of sc[n]: its row is the lane's second, its key that far from the stage's first)
      auto second = [](int i) { return kT ? (i & 1) : (i >> 1); };
      auto key_of = [&](int n, int i) { return kT ? 16 * n + g + 8 * (i >> 1) : 8 * n + 2 * q4 + (i & 1); };
#pragma unroll
      for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float x = sc[n][i] + s2[n][i];
          if (kTwo) x += __shfl_xor_sync(~0u, x, 2);  // (high and low parts; both lanes go on with the row)
          sc[n][i] = x * row_scale[second(i)];
        }
      if ((t + 1) * S::Keys > lim_all) {  // (the same for all lanes)
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (t * S::Keys + key_of(n, i) >= (second(i) ? lim1 : lim0)) sc[n][i] = -INFINITY;
      }
#pragma unroll
      for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (second(i)) x1m = fmaxf(x1m, sc[n][i]);
          else x0m = fmaxf(x0m, sc[n][i]);
        }
#pragma unroll
      for (int d = kT ? 4 : 1; d <= (kT ? 16 : 2); d <<= 1) {
        x0m = fmaxf(x0m, __shfl_xor_sync(~0u, x0m, d));
        x1m = fmaxf(x1m, __shfl_xor_sync(~0u, x1m, d));
      }
      const float n0 = fmaxf(m0, x0m), n1 = fmaxf(m1, x1m);
      const float u0 = n0 == -INFINITY ? 0.f : n0, u1 = n1 == -INFINITY ? 0.f : n1;  // (a row with no key so far)
      if (__any_sync(~0u, n0 != m0 || n1 != m1)) {
        const float a0 = ex2(m0 - u0), a1 = ex2(m1 - u1);
        l0 *= a0;
        l1 *= a1;
#pragma unroll
        for (int n = 0; n < NO; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[n][i] *= second(i) ? a1 : a0;
        m0 = n0;
        m1 = n1;
      }
#pragma unroll
      for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sc[n][i] = ex2(sc[n][i] - (second(i) ? u1 : u0));
          if (second(i)) l1 += sc[n][i];
          else l0 += sc[n][i];
        }
      // ---- output: acc[n] has (kT) value columns 16 n + g, + 8 (int8: 16 n + 2 g, + 1) for rows ra, rb, or columns
      // 8 n + 2 q4, + 1 for row ra, then for rb
      if constexpr (kT) {
        uint32_t pf[NS][2];
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t x;
            if constexpr (kI8)
              x = Elem<__half>::pack(sc[n][2 * i], sc[n][2 * i + 1]);
            else
              x = E::pack(sc[n][2 * i], sc[n][2 * i + 1]);
            pf[n][i] = movmatrix(x);
          }
        if constexpr (kI8) {
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            uint32_t x[4];
            ldsm_x4_trans(st + kVOff + kv_at<S::CK>(lane, n), x[0], x[1], x[2], x[3]);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] ^= 0x80808080u;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t af[4] = {kv_half2(x[2 * k], 0x4240), kv_half2(x[2 * k], 0x4341), kv_half2(x[2 * k + 1], 0x4240),
                                      kv_half2(x[2 * k + 1], 0x4341)};
              mma16816<false>(acc[n], af, pf[k][0], pf[k][1]);
            }
          }
        } else {
          const int r = (lane & 7) + (lane >> 4) * 8, cc = (lane >> 3) & 1;
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            uint32_t af[4];
            ldsm_x4_trans(st + kVOff + kv_at<S::CK>(r, 2 * n + cc), af[0], af[1], af[2], af[3]);
            mma16816<E::kBf16>(acc[n], af, pf[0][0], pf[0][1]);
          }
        }
      } else {
        const uint32_t pf[4] = {E::pack(sc[0][0], sc[0][1]), E::pack(sc[0][2], sc[0][3]), E::pack(sc[1][0], sc[1][1]),
                                E::pack(sc[1][2], sc[1][3])};
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          uint32_t b0, b1, b2, b3;
          ldsm_x4_trans(st + kVOff + kv_at<S::CK>(lane & 15, 2 * n + (lane >> 4)), b0, b1, b2, b3);
          mma16816<E::kBf16>(acc[2 * n], pf, b0, b1);
          mma16816<E::kBf16>(acc[2 * n + 1], pf, b2, b3);
        }
      }
      __syncwarp();  // the stage is free
      if (t + kStages < t1) load(t + kStages, ahead);
      cp_async_commit();
    }
    cp_async_wait<0>();
    __syncwarp();

    // ---- results, through the ring's place, so that a warp stores whole rows
#pragma unroll
    for (int d = kT ? 4 : 1; d <= (kT ? 16 : 2); d <<= 1) {
      l0 += __shfl_xor_sync(~0u, l0, d);
      l1 += __shfl_xor_sync(~0u, l1, d);
    }
    float* place = reinterpret_cast<float*>(smem + warp * kWarpBytes);
#pragma unroll
    for (int n = 0; n < NO; ++n) {
      if constexpr (!kT) {
        *reinterpret_cast<float2*>(place + ra * kV + n * 8 + 2 * q4) = make_float2(acc[n][0], acc[n][1]);
        *reinterpret_cast<float2*>(place + rb * kV + n * 8 + 2 * q4) = make_float2(acc[n][2], acc[n][3]);
      } else {
        const int c0 = n * 16 + (kI8 ? 2 * g : g), c1 = c0 + (kI8 ? 1 : 8);
        if (kTwo && q4 >= 2) continue;
        place[ra * kV + c0] = acc[n][0];
        place[rb * kV + c0] = acc[n][1];
        place[ra * kV + c1] = acc[n][2];
        place[rb * kV + c1] = acc[n][3];
      }
    }
    __syncwarp();
    float4 vs = make_float4(1.f, 1.f, 1.f, 1.f);
    if (kI8) vs = reinterpret_cast<const float4*>(p.v_scale + c.head * kV)[lane];
    auto store = [&](int r, float4 y, float m, float l) {  // row r's result, four columns a lane
      const int tok = (row0 + r) / G;
      const size_t orow = (size_t)(sq.begin + tok) * H + c.head * G + (row0 + r) - tok * G;
      const float iv = l == 0.f ? 0.f : 1.f / l;
      reinterpret_cast<uint2*>(static_cast<T*>(p.plan.out) + orow * kV)[lane] =
          make_uint2(E::pack(y.x * iv * vs.x, y.y * iv * vs.y), E::pack(y.z * iv * vs.z, y.w * iv * vs.w));
      if (p.plan.lse && lane == 0) p.plan.lse[orow] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
    };
    // (slot of worker v: its first place for an item that others began, its second for one that it begins)
    auto part = [&](int v, bool begins) { return (size_t)v * 2 + (begins ? 1 : 0); };
    float4* part_o = reinterpret_cast<float4*>(p.plan.part_o);
    float2* part_ml = reinterpret_cast<float2*>(p.plan.part_ml);
    for (int r = 0; r < live; ++r) {
      // (lane r / 2 holds row r in its first or second place, or lanes 4 r and 4 (r - 8))
      const int from = kT ? r >> 1 : (r & 7) * 4;
      const bool sec = kT ? r & 1 : r >= 8;
      const float l = __shfl_sync(~0u, sec ? l1 : l0, from), m = __shfl_sync(~0u, sec ? m1 : m0, from);
      const float4 y = reinterpret_cast<const float4*>(place + r * kV)[lane];
      if (whole) {
        store(r, y, m, l);
      } else {
        const size_t at = part(w, c.lo >= x0) * R + r;
        part_o[at * (kV / 4) + lane] = y;
        if (lane == 0) part_ml[at] = make_float2(m, l);
      }
    }
    __syncwarp();  // (the ring is filled again by the next item)
    if (whole || !p.join_here) continue;
    // ---- the last piece to arrive joins them all
    int w1, w2;
    kv_sharers(c, w, x0, x1, total, W, &w1, &w2);
    __threadfence();
    __syncwarp();
    unsigned before = 0;
    if (lane == 0) before = atomicInc(p.arrived + w1, w2 - w1);  // (0 again after the last)
    if (__shfl_sync(~0u, before, 0) != (unsigned)(w2 - w1)) continue;
    __threadfence();
    for (int r = 0; r < live; ++r) {
      float m, l;
      const float4 y = kv_join_row<kJoinFlight>(p.plan, w2 - w1 + 1, [&](int i) { return part(w1 + i, i == 0) * R + r; }, &m, &l);
      store(r, y, m, l);
    }
  }
}

// ---------------------------------------------------------------- joining
// The rows of an item that worker w1 began and others went on with:
//   out / l, lse = (m + log2 l) * ln 2.
// `per` warps (1, 2, 4, 8 or 16) share a record's rows, a warp taking one row at a
// time with 16 pieces in flight.  Bound by latency, so the grid is what fits
// on the GPU at once: a block for each eight possible rows costs 12 sequences
// with 12 rows per head 8 us more.
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
        float m, l;
        const float4 o = kv_join_row<kJoinFlight>(p.plan, n, [&](int i) { return slot(i) * R + r; }, &m, &l);
        const float iv = l == 0.f ? 0.f : 1.f / l;
        const float4 vs = p.v_scale ? reinterpret_cast<const float4*>(p.v_scale + j.pad * kV)[lane] : make_float4(1.f, 1.f, 1.f, 1.f);
        reinterpret_cast<uint2*>(static_cast<T*>(p.plan.out) + orow * kV)[lane] =
            make_uint2(E::pack(o.x * iv * vs.x, o.y * iv * vs.y), E::pack(o.z * iv * vs.z, o.w * iv * vs.w));
        if (p.plan.lse && lane == 0) p.plan.lse[orow] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
      }
    }
  }
}

template <typename T, bool kI8, KvForm kForm>
cudaError_t launch(PagedKvParams p, int num_sms, cudaStream_t stream) {
  using S = KvCfg<kI8, kForm>;
  p.plan.workers = paged_kv_workers(num_sms);
  const long long rows = paged_kv_rows(p);
  p.join_here = paged_kv_joins_here(rows);
  // What beginning and ending an item takes, in tiles of 32 keys, which a warp goes through in 3.3 us with 16 bits and 1.5
  // with int8.  int8, 16 sequences of up to 8192 keys, 8 heads: 8 rows 58.6, 47.3, 42.3, 41.8 us with 1, 2, 3, 4; 64
  // sequences of up to 512 keys, 16 heads, one row: 33.0, 31.7, 33.3, 34.4.  16 bits, up to 256 keys: 22.6, 24.2, 25.0.
  p.item_cost = !kI8 ? 1 : p.join_here ? 2 : 3;
  if (p.plan.page % 16 == 0)
    paged_kv_kernel<T, kI8, kForm, true><<<num_sms, kKvThreads, kKvSmem, stream>>>(p);
  else
    paged_kv_kernel<T, kI8, kForm, false><<<num_sms, kKvThreads, kKvSmem, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || p.join_here) return e;
  const int per = rows <= 1 ? 1 : rows <= 2 ? 2 : rows <= 4 ? 4 : rows <= 8 || S::R == 8 ? 8 : 16;
  const int blocks = (p.plan.workers * per + 15) / 8, most = num_sms * 2;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((blocks < most ? blocks : most) & ~1);  // (16 warps are two blocks)
  c.blockDim = dim3(256);
  c.stream = stream;
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, paged_kv_join_kernel<T>, p, per, S::R);
}

template <typename T, bool kI8, KvForm kForm>
cudaError_t prepare_one() {
  const cudaError_t e = cudaFuncSetAttribute(paged_kv_kernel<T, kI8, kForm, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kKvSmem);
  return e == cudaSuccess ? cudaFuncSetAttribute(paged_kv_kernel<T, kI8, kForm, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kKvSmem) : e;
}
template <typename T>
cudaError_t prepare() {
  cudaError_t e = prepare_one<T, false, kWide>();
  if (e == cudaSuccess) e = prepare_one<T, false, kTrans>();
  if (e == cudaSuccess) e = prepare_one<T, true, kTrans>();
  if (e == cudaSuccess) e = prepare_one<T, true, kSplit>();
  return e;
}
template <typename T>
cudaError_t launch_any(bool i8, const PagedKvParams& p, int num_sms, cudaStream_t stream) {
  const long long rows = paged_kv_rows(p);
  if (i8) return rows <= kKvRowsSplit ? launch<T, true, kSplit>(p, num_sms, stream) : launch<T, true, kTrans>(p, num_sms, stream);
  return rows <= kKvRowsT ? launch<T, false, kTrans>(p, num_sms, stream) : launch<T, false, kWide>(p, num_sms, stream);
}

}  // namespace

cudaError_t paged_kv_prepare(bool bf16) { return bf16 ? prepare<__nv_bfloat16>() : prepare<__half>(); }

cudaError_t paged_kv_launch(bool bf16, bool i8, const PagedKvParams& p, int num_sms, cudaStream_t stream) {
  return bf16 ? launch_any<__nv_bfloat16>(i8, p, num_sms, stream) : launch_any<__half>(i8, p, num_sms, stream);
}

}  // namespace mla
