// attention_bwd.cuh -- gradients of the masked attention (sm_100a).
//
// With P_ij = exp(scale q_i.k_j - lse_i) for the keys that row i sees (else 0)
// and D_i = dO_i . O_i:
//   dV_j = sum_i P_ij dO_i         dP_ij = dO_i . v_j    dS_ij = P_ij (dP_ij - D_i)
//   dQ_i = scale sum_j dS_ij k_j   dK_j  = scale sum_i dS_ij q_i
// and the query heads that share a K/V head add up in its dK and dV.
//
// `prep` forms D (one pass over O and dO; for rows of few keys anew from P and dP,
// since there the rounding of O to bf16 weighs as much as that of dS) and lays the
// rows' (lse, D), intervals and their hulls per 128-row tile out in the workspace,
// padded to whole tiles.  The main kernel then runs two kinds of blocks: `dkdv` owns
// 128 keys of a K/V head and walks the query tiles that see them, over all heads of
// the group; `dq` owns 128 query rows of a head and walks their key tiles.  Both
// recompute S and dP, 7 products of 128 x 128 x 128 per pair of tiles where one walk
// would need 5: the price of sums that stay in tensor memory, need no atomics and
// come out the same on every run.  The kinds share a launch so that the shorter dq
// blocks fill the SMs that the dkdv blocks leave (1,127 rows x 8 heads: 72 blocks of
// each kind side by side).  Where there are few key tiles, a tile's walk is cut into
// `parts`, whose fp32 sums go to the workspace and are added in order by a third
// kernel (9,001 + 5,097 rows, 14 heads over 2 K/V heads: 222 walks of up to 777 steps).
//
// Measured: that case by itself, at 1,965 MHz, 2.11 ms for the main kernel, 1,270 TFLOP/s of
// products done and 909 of the five that a single walk would need; adding its parts 16 us.
// In a loop with the forward call, under the 1 kW power cap at 1,650 MHz, the whole call
// takes 2.48 ms, 1,085 and 775 TFLOP/s.  1,127 causal
// rows x 8 heads 19.5 us, three or four steps of each walk after another.
//
// dkdv works on S^T = K Q^T and dP^T = V dO^T (keys on the 128 TMEM lanes), so
// that P^T and dS^T are, rounded to bf16 in place, the A operands of
// dV += P^T dO and dK += dS^T Q straight from tensor memory; dq works on S and dP
// (queries on the lanes) for dQ += dS K alike.  The four or three 128-column fp32
// accumulators fill tensor memory (512 columns).  P and dS are rounded to bf16 as
// MMA operands; every sum is fp32.
//
// Warps 0-15 do the element-wise part, warp w on the 16 lanes
// 32 (w % 4) + 16 ((w / 4) % 2) and the columns 64 (w / 8): with the 16x256b shape
// thread (t0 = lane % 4, t1 = lane / 4) holds lanes t1, t1 + 8 and columns
// 8 r + 2 t0, + 1.  Warp 16 loads by TMA, warp 17 issues the MMAs.  The issuing
// thread orders its work so that the tensor core runs two products while the
// other warps run one element-wise phase:
//   dkdv: .. dV(i) S(i+1) | dK(i) dP(i+1) ..   against   dS(i) | P(i+1)
//   dq:   S(j+1) | dP(j+1) dQ(j)               against   dS(j) | P(j+1)
//
// Masked places (see attention.cuh): P is set to 0 there by the rows' intervals
// and dS with it, never by a product.  The tiles that are B operands of a product
// with such zeros (dO and Q in dkdv, K in dq) may hold inf or NaN in masked rows.
// dq: such a row of K makes its column of S non-finite, so in tiles with masked
// pairs each warp looks at the S it holds anyway (one packed FMA per two values)
// and, if need be, clears K's rows of its half before it hands dS on.  dkdv: looking
// at dP before P is handed on would cost such tiles half their time again, so the
// CTA runs a second time with that look if its dK or dV come out non-finite.  A
// pair that is seen and not finite gets a NaN P or dS.
#pragma once

#include "attention.cuh"

namespace h3 {
namespace attn_bwd {

using attn::BM;
using attn::BN;
using attn::HD;
using attn::HALF_BYTES;
using attn::IDESC_O;
using attn::IDESC_S;
using attn::TILE_BYTES;
using attn::any_nonfinite;
using attn::zero_nonfinite;
using attn::mma_wait;
using attn::warp_wait;
using attn::warp_wait_exact;

constexpr int WARPS = 16;                     // element-wise warps
constexpr int W_PROD = WARPS;
constexpr int W_MMA = WARPS + 1;
constexpr int THREADS = 32 * (WARPS + 2);

struct Params {
  int n_q, n_k, n_heads, group, n_qt;         // n_qt: query tiles of 128 rows
  float scale, scale_log2;
  const float2* stat;                         // [B][H][n_qt * 128] (lse log2 e, D)
  const int2* rng;                            // [B][n_qt * 128] intervals (lo, length), (0, 0) past the end
  const int4* hull;                           // [B][n_qt] (min lo, max hi, max lo, min hi)
  __nv_bfloat16 *dq, *dk, *dv;
  long long dq_stride, dk_stride, dv_stride;  // row strides, elements
  int n_kv_heads, n_kt, batch;                // n_kt: key tiles of 128 rows
  int parts;                                  // pieces of a key tile's walk
  float* partial;                             // parts > 1: [parts][B][n_kv_heads][n_kt][dV, dK][128][128]
  unsigned long long wait_limit_ns, drain_limit_ns;
  int err_slot;
};

// ------------------------------------------------------------------ prep ----

// D (16 x 8) += A (16 x 16) B (16 x 8): one warp, bf16 operands, fp32 sums.
__device__ __forceinline__ void mma_16x8x16(float (&d)[4], const uint4 a, const uint2 b) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y));
}

// D of rows with at most this many keys comes from P and dP.  Against 64 bits that
// takes the error of dQ and dK, which the roundings of dS and of the outputs alone
// make 1.41 times that of the outputs' rounding, from 1.45 - 1.6 down to 1.41 - 1.44 of it
// (documents of 20 to 2,000 rows, causal and full; up to 1.47 elsewhere.  Measured, not
// bounds).
constexpr int SHORT_ROW = 32;

struct PrepInputs {
  const __nv_bfloat16 *q, *k, *v;
  long long q_stride, k_stride, v_stride;
  int group;
  float scale_log2;
};

struct ShortRows {
  int2 range[BM];            // {0, 0} for the others
  float lse_log2[BM];
  float part[BM][8];         // [row][warp]
};

// The block: D_i = sum_j P_ij (dO_i . v_j) of the tile's short rows, into sm.part.
// 16 rows against 8 keys at a time on a warp's matrix unit, the steps dealt to the
// warps in turn (of a causal mask only 32 rows are short: 8 steps of the whole tile).
// Lane t of four holds elements 8 t .. 8 t + 7 of 32, one 16-byte load, for both
// operands: the order of a product's terms is free.
__device__ __forceinline__ void short_rows(ShortRows& sm, const PrepInputs& in, const __nv_bfloat16* dout,
                                           long long do_stride, int n_q, int n_k, int batch, int head, int tile) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int kv_col = head / in.group * HD + 8 * t;
  int step = 0;
  for (int row0 = 0; row0 < BM; row0 += 16) {
    const int2 r[2] = {sm.range[row0 + g], sm.range[row0 + g + 8]};
    auto next_key = [&](int from) {                // the first key from `from` on that a short row sees
      int k = 0x7fffffff;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (r[h].y > from) k = min(k, max(r[h].x, from));
      return __reduce_min_sync(0xffffffffu, k);
    };
    float d[2] = {0.f, 0.f};
    for (int key0 = next_key(0); key0 != 0x7fffffff; key0 = next_key(key0 + 8)) {
      if ((step++ & 7) != warp) continue;
      const long long kv = static_cast<long long>(batch) * n_k + min(key0 + g, n_k - 1);
      const __nv_bfloat16 *kr = in.k + kv * in.k_stride + kv_col, *vr = in.v + kv * in.v_stride + kv_col;
      const long long q0 = static_cast<long long>(batch) * n_q + min(tile * BM + row0 + g, n_q - 1);
      const long long q1 = static_cast<long long>(batch) * n_q + min(tile * BM + row0 + g + 8, n_q - 1);
      const int col = head * HD + 8 * t;
      const __nv_bfloat16 *qa = in.q + q0 * in.q_stride + col, *qb = in.q + q1 * in.q_stride + col;
      const __nv_bfloat16 *da = dout + q0 * do_stride + col, *db = dout + q1 * do_stride + col;
      auto load = [](const __nv_bfloat16* p) { return *reinterpret_cast<const uint4*>(p); };
      float s[4] = {0.f, 0.f, 0.f, 0.f}, dp[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
      for (int c = 0; c < HD; c += 64) {
        uint4 w[2][6];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          w[u][0] = load(qa + c + 32 * u);
          w[u][1] = load(qb + c + 32 * u);
          w[u][2] = load(kr + c + 32 * u);
          w[u][3] = load(da + c + 32 * u);
          w[u][4] = load(db + c + 32 * u);
          w[u][5] = load(vr + c + 32 * u);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint4(&x)[6] = w[u];
          mma_16x8x16(s, {x[0].x, x[1].x, x[0].y, x[1].y}, {x[2].x, x[2].y});
          mma_16x8x16(dp, {x[3].x, x[4].x, x[3].y, x[4].y}, {x[5].x, x[5].y});
          mma_16x8x16(s, {x[0].z, x[1].z, x[0].w, x[1].w}, {x[2].z, x[2].w});
          mma_16x8x16(dp, {x[3].z, x[4].z, x[3].w, x[4].w}, {x[5].z, x[5].w});
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {                // row g + 8 (e / 2), key 2 t + e % 2
        const int h = e >> 1, key = key0 + 2 * t + (e & 1);
        if (key >= r[h].x && key < r[h].y)
          d[h] = fmaf(ex2_approx(fmaf(s[e], in.scale_log2, -sm.lse_log2[row0 + g + 8 * h])), dp[e], d[h]);
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      d[h] += __shfl_xor_sync(0xffffffffu, d[h], 1);
      d[h] += __shfl_xor_sync(0xffffffffu, d[h], 2);
      if (t == 0) sm.part[row0 + g + 8 * h][warp] = d[h];
    }
  }
}

// One block per (query tile, head, batch): 16 lanes per row, 16 rows at a time, four
// such steps' loads in flight.  Blocks of head 0 also write the tile's intervals and
// hull.  Bound by the reads of O and dO (14,098 rows x 14 heads 18.0 us, 0.87 of the
// copy rate); with few blocks by the two round trips to memory, and a third and a
// fourth where there are short rows (1,127 rows x 8 heads 4.1, with them 6.9 us).
__global__ void __launch_bounds__(256, 3) prep_kernel(const __grid_constant__ PrepInputs in,
                                                      const __nv_bfloat16* __restrict__ o,
                                                      const __nv_bfloat16* __restrict__ dout,
                                                      const float* __restrict__ lse, const int2* __restrict__ ranges,
                                                      int n_q, int n_k, int n_heads, int n_qt, long long o_stride,
                                                      long long do_stride, float2* __restrict__ stat,
                                                      int2* __restrict__ rng, int4* __restrict__ hull) {
  begin_after_predecessor(o, dout, lse, ranges);
  const int tile = blockIdx.x, head = blockIdx.y, batch = blockIdx.z;
  const int sub = threadIdx.x & 15, first = tile * BM + (threadIdx.x >> 4);
  const long long bh = static_cast<long long>(batch) * n_heads + head;
  const long long row0 = static_cast<long long>(batch) * n_q;
  __shared__ ShortRows few;
  int2 range = make_int2(0, 0);
  bool is_short = false;
  if (threadIdx.x < BM && tile * BM + threadIdx.x < n_q) {
    range = attn::clamp_range(ranges[row0 + tile * BM + threadIdx.x], n_k);
    is_short = range.x < range.y && range.y - range.x <= SHORT_ROW;
    few.lse_log2[threadIdx.x] = lse[bh * n_q + tile * BM + threadIdx.x] * 1.4426950408889634f;
  }
  if (threadIdx.x < BM) few.range[threadIdx.x] = is_short ? range : make_int2(0, 0);
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint4 a[4], b[4];
    float l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = min(first + (4 * half + i) * 16, n_q - 1);   // rows past the end: read, not used
      a[i] = __ldcs(reinterpret_cast<const uint4*>(o + (row0 + row) * o_stride + head * HD + 8 * sub));
      b[i] = *reinterpret_cast<const uint4*>(dout + (row0 + row) * do_stride + head * HD + 8 * sub);
      l[i] = lse[bh * n_q + row];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = first + (4 * half + i) * 16;
      const uint32_t wa[4] = {a[i].x, a[i].y, a[i].z, a[i].w}, wb[4] = {b[i].x, b[i].y, b[i].z, b[i].w};
      float2 s = make_float2(0.f, 0.f);
#pragma unroll
      for (int m = 0; m < 4; ++m)
        s = __ffma2_rn(make_float2(__uint_as_float(wa[m] << 16), __uint_as_float(wa[m] & 0xffff0000u)),
                       make_float2(__uint_as_float(wb[m] << 16), __uint_as_float(wb[m] & 0xffff0000u)), s);
      float d = s.x + s.y;
#pragma unroll
      for (int k = 8; k > 0; k >>= 1) d += __shfl_xor_sync(0xffffffffu, d, k);
      // rows without keys (lse = -inf) are masked everywhere
      if (sub == 0)
        stat[bh * n_qt * BM + row] = row < n_q ? make_float2(l[i] * 1.4426950408889634f, d) : make_float2(0.f, 0.f);
    }
  }
  if (__syncthreads_or(is_short)) {                // over what was written above
    short_rows(few, in, dout, do_stride, n_q, n_k, batch, head, tile);
    __syncthreads();
    if (is_short) {
      float d = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) d += few.part[threadIdx.x][w];
      stat[bh * n_qt * BM + tile * BM + threadIdx.x].y = d;
    }
  }
  if (head == 0) {
    __shared__ int part[4][4];
    if (threadIdx.x < BM) {
      const int2 r = range;
      rng[(static_cast<long long>(batch) * n_qt + tile) * BM + threadIdx.x] = make_int2(r.x, r.y - r.x);
      const bool some = r.x < r.y;
      const int lo = __reduce_min_sync(0xffffffffu, some ? r.x : 0x7fffffff);
      const int hi = __reduce_max_sync(0xffffffffu, some ? r.y : 0);
      const int all_lo = __reduce_max_sync(0xffffffffu, r.x), all_hi = __reduce_min_sync(0xffffffffu, r.y);
      if ((threadIdx.x & 31) == 0) {
        int* p = part[threadIdx.x >> 5];
        p[0] = lo;
        p[1] = hi;
        p[2] = all_lo;
        p[3] = all_hi;
      }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      int4 h = make_int4(0x7fffffff, 0, 0, 0x7fffffff);
      for (int q = 0; q < 4; ++q) {
        h.x = min(h.x, part[q][0]);
        h.y = max(h.y, part[q][1]);
        h.z = max(h.z, part[q][2]);
        h.w = min(h.w, part[q][3]);
      }
      hull[static_cast<long long>(batch) * n_qt + tile] = h;
    }
  }
}

// --------------------------------------------------------------- helpers ----

__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* map, uint32_t bar, int col, int row,
                                          int batch) {
  tma_load_3d(dst, map, bar, col, row, batch);
  tma_load_3d(dst + HALF_BYTES, map, bar, col + 64, row, batch);
}

// D = A B^T of two K-major 128 x 128 tiles in shared memory.
__device__ __forceinline__ void issue_abt(uint32_t d, uint32_t a, uint32_t b) {
#pragma unroll
  for (int kk = 0; kk < 8; ++kk) {
    const uint32_t off = (kk >> 2) * HALF_BYTES + (kk & 3) * 32;
    mma_ss(d, smem_desc_sw128(a + off, 16, 1024), smem_desc_sw128(b + off, 16, 1024), IDESC_S, kk > 0 ? 1u : 0u);
  }
}

// D += A B: A in tensor memory (bf16 pairs: 64 of the 128 K values in columns
// 0-31, the others in 64-95), B a 128 x 128 tile in shared memory, MN-major.
__device__ __forceinline__ void issue_ab(uint32_t d, uint32_t a, uint32_t b, bool accumulate) {
#pragma unroll
  for (int kk = 0; kk < 8; ++kk)
    mma_ts(d, a + (kk >> 2) * 64 + (kk & 3) * 8, smem_desc_sw128(b + kk * 2048, HALF_BYTES, 1024), IDESC_O,
           (accumulate || kk > 0) ? 1u : 0u);
}

// This warp's 16 lanes x 64 columns of an accumulator -> v.
__device__ __forceinline__ void load_acc(uint32_t taddr, uint32_t (&v)[32]) {
  __syncwarp();
  tmem_ld16x256(taddr, v);
  tmem_wait_ld(v);
}

// They, times `scale`, rounded to bf16 rows `row_a`, `row_a + 8` (< n_rows) of an
// output at `out`.
__device__ __forceinline__ void store_tile(const uint32_t (&v)[32], float scale, __nv_bfloat16* out, long long stride,
                                           int row_a, int n_rows, int t0) {
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const int col = 8 * r + 2 * t0;
    if (row_a < n_rows)
      *reinterpret_cast<uint32_t*>(out + row_a * stride + col) =
          pack_bf16x2(__uint_as_float(v[4 * r]) * scale, __uint_as_float(v[4 * r + 1]) * scale);
    if (row_a + 8 < n_rows)
      *reinterpret_cast<uint32_t*>(out + (row_a + 8) * stride + col) =
          pack_bf16x2(__uint_as_float(v[4 * r + 2]) * scale, __uint_as_float(v[4 * r + 3]) * scale);
  }
}

// They as fp32, rows of 128.
__device__ __forceinline__ void store_partial(const uint32_t (&v)[32], float* out, int row_a, int t0) {
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    *reinterpret_cast<uint2*>(out + row_a * HD + 8 * r + 2 * t0) = make_uint2(v[4 * r], v[4 * r + 1]);
    *reinterpret_cast<uint2*>(out + (row_a + 8) * HD + 8 * r + 2 * t0) = make_uint2(v[4 * r + 2], v[4 * r + 3]);
  }
}

// Rounded values of this warp's 16 x 64 piece -> tensor memory, then one arrival.
__device__ __forceinline__ void publish(uint32_t taddr, const uint32_t (&pk)[16], uint32_t bar, int lane) {
  __syncwarp();
  tmem_st16x128(taddr, pk);
  tmem_wait_st();
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

__device__ __forceinline__ bool nonfinite(uint32_t v) { return (v & 0x7f800000u) == 0x7f800000u; }

// ------------------------------------------------------------------ dkdv ----

namespace dkdv {
constexpr uint32_t SMEM_K = 0, SMEM_V = TILE_BYTES;
constexpr uint32_t SMEM_Q = 2 * TILE_BYTES, SMEM_DO = 4 * TILE_BYTES;   // two slots each
constexpr uint32_t SMEM_STAT = 6 * TILE_BYTES;                          // two slots of 128 (lse, D)
constexpr uint32_t SMEM_RNG = SMEM_STAT + 2 * 1024;                     // two slots of 128 intervals
constexpr uint32_t SMEM_BAR = SMEM_RNG + 2 * 1024;
// barriers: kv_full, q_full[2], q_empty[2], do_full[2], do_empty[2], s_full, p_full, dp_full,
//           ds_full, out_full, mma_done
constexpr int NUM_BARS = 15;
constexpr uint32_t SMEM_MISC = SMEM_BAR + NUM_BARS * 8;                 // tmem base, abort, first, last, run again
constexpr uint32_t SMEM_BYTES = SMEM_MISC + 24 + 1024;
constexpr uint32_t TMEM_S = 0, TMEM_DP = 128, TMEM_DV = 256, TMEM_DK = 384;
}  // namespace dkdv

// One block per (128 keys, K/V head, batch, part).
__device__ __forceinline__ void dkdv_block(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                           const CUtensorMap& tm_do, const Params& p, uint8_t* smem_raw, int kt,
                                           int kvh, int batch, int part) {
  using namespace dkdv;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const gbase = smem_raw + (base - raw);
  const uint32_t bar0 = base + SMEM_BAR;
  const uint32_t bar_kv = bar0;
  auto bar_q_full = [&](int s) { return bar0 + 8u * (1 + s); };
  auto bar_q_empty = [&](int s) { return bar0 + 8u * (3 + s); };
  auto bar_do_full = [&](int s) { return bar0 + 8u * (5 + s); };
  auto bar_do_empty = [&](int s) { return bar0 + 8u * (7 + s); };
  const uint32_t bar_s = bar0 + 72u, bar_p = bar0 + 80u, bar_dp = bar0 + 88u, bar_ds = bar0 + 96u;
  const uint32_t bar_out = bar0 + 104u, bar_done = bar0 + 112u;
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(gbase + SMEM_MISC);
  volatile uint32_t* const abort_flag = reinterpret_cast<volatile uint32_t*>(gbase + SMEM_MISC + 4);
  int* const span = reinterpret_cast<int*>(gbase + SMEM_MISC + 8);
  volatile uint32_t* const again = reinterpret_cast<volatile uint32_t*>(gbase + SMEM_MISC + 16);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int k0 = kt * BN;
  const uint64_t limit = p.wait_limit_ns;
  const int eslot = p.err_slot;
  const int4* const hulls = p.hull + static_cast<long long>(batch) * p.n_qt;
  auto init_bars = [&] {
    for (int i = 0; i < NUM_BARS; ++i) mbar_init(bar0 + 8u * i, i == 10 || i == 12 ? WARPS : 1);
    mbar_fence_init();
  };

  if (threadIdx.x == 0) {
    init_bars();
    span[0] = 0x7fffffff;
    span[1] = -1;
    *abort_flag = 0u;
    *again = 0u;
  }
  __syncthreads();
  // the query tiles, first to last, with a row that sees one of these keys
  {
    int first = 0x7fffffff, last = -1;
    for (int i = threadIdx.x; i < p.n_qt; i += THREADS) {
      const int4 h = hulls[i];
      if (h.x < k0 + BN && h.y > k0) {
        first = min(first, i);
        last = i;
      }
    }
    first = __reduce_min_sync(0xffffffffu, first);
    last = __reduce_max_sync(0xffffffffu, last);
    if (lane == 0 && last >= 0) {
      atomicMin(&span[0], first);
      atomicMax(&span[1], last);
    }
  }
  __syncthreads();
  const int qt0 = span[0], nt = span[1] - span[0] + 1;
  // the steps (head, query tile) of this part, heads outermost
  const int all = span[1] < 0 ? 0 : nt * p.group;
  const int it0 = static_cast<int>(static_cast<long long>(all) * part / p.parts);
  const int iters = static_cast<int>(static_cast<long long>(all) * (part + 1) / p.parts) - it0;
  const int qt_first = all > 0 ? qt0 + it0 % nt : 0, head_first = kvh * p.group + (all > 0 ? it0 / nt : 0);
  float* const sums = p.partial + ((((static_cast<long long>(part) * p.batch + batch) * p.n_kv_heads + kvh) * p.n_kt + kt) *
                                   2) * BN * HD;      // parts > 1: dV, then dK
  if (iters == 0) {                              // no row sees these keys
    if (p.parts > 1) {
      for (int i = threadIdx.x; i < 2 * BN * HD / 4; i += THREADS)
        reinterpret_cast<uint4*>(sums)[i] = make_uint4(0u, 0u, 0u, 0u);
      return;
    }
    for (int i = threadIdx.x; i < BN * (HD / 8); i += THREADS) {
      const int key = k0 + i / (HD / 8), col = kvh * HD + 8 * (i % (HD / 8));
      if (key < p.n_k) {
        const long long r = static_cast<long long>(batch) * p.n_k + key;
        *reinterpret_cast<uint4*>(p.dk + r * p.dk_stride + col) = make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint4*>(p.dv + r * p.dv_stride + col) = make_uint4(0u, 0u, 0u, 0u);
      }
    }
    return;
  }
  // whether some row of query tile i does not see all of these keys
  auto edge_tile = [&](int i) { const int4 h = hulls[i]; return h.z > k0 || h.w < k0 + BN; };
  if (warp == W_MMA) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  for (int run = 0; run < 2; ++run) {
  if (warp == W_PROD) {
    if (lane == 0) {
      mbar_arrive_expect_tx(bar_kv, 2 * TILE_BYTES);
      load_tile(base + SMEM_K, &tm_k, bar_kv, kvh * HD, k0, batch);
      load_tile(base + SMEM_V, &tm_v, bar_kv, kvh * HD, k0, batch);
      int issued_q = 0, issued_do = 0, qt = qt_first, head = head_first;
      for (int it = 0; it < iters; ++it) {
        const int s = it & 1;
        const uint32_t par = ((it >> 1) - 1) & 1;
        // dO's slot frees first (after dV), Q's with dK
        if (it > 1 && !mbar_wait_bounded(bar_do_empty(s), par, abort_flag, limit, eslot)) break;
        mbar_arrive_expect_tx(bar_do_full(s), TILE_BYTES);
        load_tile(base + SMEM_DO + s * TILE_BYTES, &tm_do, bar_do_full(s), head * HD, qt * BM, batch);
        issued_do = it + 1;
        if (it > 1 && !mbar_wait_bounded(bar_q_empty(s), par, abort_flag, limit, eslot)) break;
        mbar_arrive_expect_tx(bar_q_full(s), TILE_BYTES + 2048);
        load_tile(base + SMEM_Q + s * TILE_BYTES, &tm_q, bar_q_full(s), head * HD, qt * BM, batch);
        bulk_load(base + SMEM_STAT + s * 1024,
                  p.stat + ((static_cast<long long>(batch) * p.n_heads + head) * p.n_qt + qt) * BM, 1024, bar_q_full(s));
        bulk_load(base + SMEM_RNG + s * 1024, p.rng + (static_cast<long long>(batch) * p.n_qt + qt) * BM, 1024,
                  bar_q_full(s));
        issued_q = it + 1;
        if (++qt == qt0 + nt) qt = qt0, ++head;
      }
      // every load that was started lands before the CTA ends
      volatile uint32_t never = 0u;
      mbar_wait_bounded(bar_kv, 0, &never, p.drain_limit_ns, eslot);
      for (int it = max(issued_q - 2, 0); it < issued_q; ++it)
        mbar_wait_bounded(bar_q_full(it & 1), (it >> 1) & 1, &never, p.drain_limit_ns, eslot);
      for (int it = max(issued_do - 2, 0); it < issued_do; ++it)
        mbar_wait_bounded(bar_do_full(it & 1), (it >> 1) & 1, &never, p.drain_limit_ns, eslot);
    }
  } else if (warp == W_MMA) {
    if (lane == 0) {
      auto q_tile = [&](int s) { return base + SMEM_Q + s * TILE_BYTES; };
      auto do_tile = [&](int s) { return base + SMEM_DO + s * TILE_BYTES; };
      bool ok = mma_wait(bar_kv, 0, abort_flag, limit, eslot) &&
                mma_wait(bar_q_full(0), 0, abort_flag, limit, eslot);
      if (ok) {
        tc_fence_after();
        issue_abt(tmem + TMEM_S, base + SMEM_K, q_tile(0));
        tc_commit(bar_s);
        ok = mma_wait(bar_do_full(0), 0, abort_flag, limit, eslot);
      }
      if (ok) {
        tc_fence_after();
        issue_abt(tmem + TMEM_DP, base + SMEM_V, do_tile(0));
        tc_commit(bar_dp);
      }
      for (int it = 0; ok && it < iters; ++it) {
        const int s = it & 1, sn = s ^ 1;
        const uint32_t par = it & 1, par_next = ((it + 1) >> 1) & 1;
        const bool more = it + 1 < iters;
        // dV(i) and, into the S columns it has just read P from, S(i + 1)
        if (more ? !mbar_spin2_bounded(bar_p, par, bar_q_full(sn), par_next, abort_flag, limit, eslot)
                 : !mma_wait(bar_p, par, abort_flag, limit, eslot))
          break;
        tc_fence_after();
        issue_ab(tmem + TMEM_DV, tmem + TMEM_S, do_tile(s), it > 0);
        tc_commit(bar_do_empty(s));
        if (more) {
          issue_abt(tmem + TMEM_S, base + SMEM_K, q_tile(sn));
          tc_commit(bar_s);
        }
        // dK(i) and dP(i + 1)
        if (more ? !mbar_spin2_bounded(bar_ds, par, bar_do_full(sn), par_next, abort_flag, limit, eslot)
                 : !mma_wait(bar_ds, par, abort_flag, limit, eslot))
          break;
        tc_fence_after();
        issue_ab(tmem + TMEM_DK, tmem + TMEM_DP, q_tile(s), it > 0);
        tc_commit(bar_q_empty(s));
        if (more) {
          issue_abt(tmem + TMEM_DP, base + SMEM_V, do_tile(sn));
          tc_commit(bar_dp);
        } else {
          tc_commit(bar_out);
        }
      }
      tc_commit(bar_done);
      volatile uint32_t never = 0u;
      mma_wait(bar_done, 0, &never, p.drain_limit_ns, eslot);
    }
  } else {
    const int t0 = lane & 3, t1 = lane >> 2;
    const int lane16 = 32 * (warp & 3) + 16 * ((warp >> 2) & 1);
    const int half = warp >> 3;                    // queries 64 half .. 64 half + 63 of the tile
    const uint32_t lb = static_cast<uint32_t>(lane16) << 16;
    const uint32_t t_s = tmem + lb + TMEM_S + 64 * half, t_dp = tmem + lb + TMEM_DP + 64 * half;
    const int key_a = k0 + lane16 + t1, key_b = key_a + 8;
    const float sl2 = p.scale_log2;
    bool ok = true;
    int qt = qt_first;
    for (int it = 0; ok && it < iters; ++it) {
      const int s = it & 1;
      // this thread's query columns: (lse, D) and intervals of two queries at a time
      const float4* const stat = reinterpret_cast<const float4*>(gbase + SMEM_STAT + s * 1024 + half * 512) + t0;
      const int4* const rng = reinterpret_cast<const int4*>(gbase + SMEM_RNG + s * 1024 + half * 512) + t0;
      const bool edge = edge_tile(qt);              // some row does not see all of these keys
      if (++qt == qt0 + nt) qt = qt0;
      bool partial = false, none = false;           // of this warp's 16 keys x 64 queries
      bool odd = false;                             // some S or dP in sight is not finite
      if (!warp_wait(bar_q_full(s), (it >> 1) & 1, abort_flag, limit, eslot) ||
          !warp_wait(bar_s, it & 1, abort_flag, limit, eslot)) { ok = false; break; }
      tc_fence_after();
      uint32_t sr[32];
      if (edge) {
        const int kw = k0 + lane16;
        const int4 g = (rng - t0)[lane];            // (lo, length) of two of the 64 queries
        const bool all = max(g.x, g.z) <= kw && min(g.x + g.y, g.z + g.w) >= kw + 16;
        const bool any = (g.x < kw + 16 && g.x + g.y > kw) || (g.z < kw + 16 && g.z + g.w > kw);
        partial = !__all_sync(0xffffffffu, all);
        none = !__any_sync(0xffffffffu, any);
        if (run == 1) {
          if (!warp_wait(bar_dp, it & 1, abort_flag, limit, eslot)) { ok = false; break; }
          tc_fence_after();
          tmem_ld16x256(t_dp, sr);
          tmem_wait_ld(sr);
          odd = any_nonfinite(sr);
          tmem_ld16x256(t_s, sr);
          tmem_wait_ld(sr);
          odd |= any_nonfinite(sr);
          if (odd) {                                // S(i) and dP(i) have read Q and dO, dV(i) and dK(i) have not
            zero_nonfinite(gbase + SMEM_Q + s * TILE_BYTES, 64 * half, 64, lane);
            zero_nonfinite(gbase + SMEM_DO + s * TILE_BYTES, 64 * half, 64, lane);
          }
        }
        if (none) {                                 // P = dS = 0
          const uint32_t zero[16] = {};
          publish(t_s, zero, bar_p, lane);
          if (!warp_wait(bar_dp, it & 1, abort_flag, limit, eslot)) { ok = false; break; }
          tc_fence_after();
          publish(t_dp, zero, bar_ds, lane);
          continue;
        }
      }
      tmem_ld16x256(t_s, sr);
      tmem_wait_ld(sr);
      float x[32];                                  // P^T: registers as loaded (4 r: key a, 4 r + 2: key b)
      const float2 c2 = make_float2(sl2, sl2);
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const float4 st = stat[4 * r];
        const float2 ml = make_float2(-st.x, -st.z);
        const float2 ya = __ffma2_rn(make_float2(__uint_as_float(sr[4 * r]), __uint_as_float(sr[4 * r + 1])), c2, ml);
        const float2 yb = __ffma2_rn(make_float2(__uint_as_float(sr[4 * r + 2]), __uint_as_float(sr[4 * r + 3])), c2, ml);
        x[4 * r] = ex2_approx(ya.x);
        x[4 * r + 1] = ex2_approx(ya.y);
        x[4 * r + 2] = ex2_approx(yb.x);
        x[4 * r + 3] = ex2_approx(yb.y);
      }
      if (partial) {
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          const int4 g = rng[4 * r];                // (lo, length) of two queries
          auto seen = [](int key, int lo, int len) { return static_cast<unsigned>(key - lo) < static_cast<unsigned>(len); };
          if (!seen(key_a, g.x, g.y)) x[4 * r] = 0.f;
          if (!seen(key_a, g.z, g.w)) x[4 * r + 1] = 0.f;
          if (!seen(key_b, g.x, g.y)) x[4 * r + 2] = 0.f;
          if (!seen(key_b, g.z, g.w)) x[4 * r + 3] = 0.f;
        }
      }
      if (odd) {                                    // seen pairs that are not finite: dV and dK must not hide them
#pragma unroll 1
        for (int which = 0; which < 2; ++which) {
          __syncwarp();
          tmem_ld16x256(which == 0 ? t_dp : t_s, sr);
          tmem_wait_ld(sr);
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const int4 g = rng[4 * (e >> 2)];
            const int key = (e & 2) ? key_b : key_a, lo = (e & 1) ? g.z : g.x, len = (e & 1) ? g.w : g.y;
            if (nonfinite(sr[e]) && static_cast<unsigned>(key - lo) < static_cast<unsigned>(len))
              x[e] = __int_as_float(0x7fc00000);
          }
        }
      }
      uint32_t pk[16];
#pragma unroll
      for (int r = 0; r < 16; ++r) pk[r] = pack_bf16x2(x[2 * r], x[2 * r + 1]);
      publish(t_s, pk, bar_p, lane);
      if (!warp_wait(bar_dp, it & 1, abort_flag, limit, eslot)) { ok = false; break; }
      tc_fence_after();
      tmem_ld16x256(t_dp, sr);
      tmem_wait_ld(sr);
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const float4 st = stat[4 * r];
        const float2 md = make_float2(-st.y, -st.w);
        const float2 da = __fmul2_rn(
            make_float2(x[4 * r], x[4 * r + 1]),
            __fadd2_rn(make_float2(__uint_as_float(sr[4 * r]), __uint_as_float(sr[4 * r + 1])), md));
        const float2 db = __fmul2_rn(
            make_float2(x[4 * r + 2], x[4 * r + 3]),
            __fadd2_rn(make_float2(__uint_as_float(sr[4 * r + 2]), __uint_as_float(sr[4 * r + 3])), md));
        // where P is 0 a masked pair's inf or NaN must not come through
        x[4 * r] = partial && x[4 * r] == 0.f ? 0.f : da.x;
        x[4 * r + 1] = partial && x[4 * r + 1] == 0.f ? 0.f : da.y;
        x[4 * r + 2] = partial && x[4 * r + 2] == 0.f ? 0.f : db.x;
        x[4 * r + 3] = partial && x[4 * r + 3] == 0.f ? 0.f : db.y;
      }
#pragma unroll
      for (int r = 0; r < 16; ++r) pk[r] = pack_bf16x2(x[2 * r], x[2 * r + 1]);
      publish(t_dp, pk, bar_ds, lane);
    }
    if (ok && warp_wait_exact(bar_out, 0, abort_flag, limit, eslot)) {
      tc_fence_after();
      const long long r0 = static_cast<long long>(batch) * p.n_k;
      const int col = kvh * HD + 64 * half;
      uint32_t v[32];
      load_acc(tmem + lb + TMEM_DV + 64 * half, v);
      bool finite = !any_nonfinite(v);
      if (p.parts > 1)
        store_partial(v, sums + 64 * half, lane16 + t1, t0);
      else
        store_tile(v, 1.f, p.dv + r0 * p.dv_stride + col, p.dv_stride, key_a, p.n_k, t0);
      load_acc(tmem + lb + TMEM_DK + 64 * half, v);
      finite &= !any_nonfinite(v);
      if (p.parts > 1)
        store_partial(v, sums + BN * HD + 64 * half, lane16 + t1, t0);
      else
        store_tile(v, p.scale, p.dk + r0 * p.dk_stride + col, p.dk_stride, key_a, p.n_k, t0);
      if (!finite && lane == 0) *again = 1u;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (run == 1 || *again == 0u || *abort_flag != 0u) break;
  // second run: loads, products and waits of the first have ended; the commits
  // that nothing waited for arrive, then the barriers start over
  if (threadIdx.x == 0) {
    volatile uint32_t never = 0u;
    for (int s = 0; s < 2; ++s) {
      const int uses = (iters - s + 1) / 2;
      if (uses == 0) continue;
      mbar_wait_bounded(bar_q_empty(s), (uses - 1) & 1, &never, p.drain_limit_ns, eslot);
      mbar_wait_bounded(bar_do_empty(s), (uses - 1) & 1, &never, p.drain_limit_ns, eslot);
    }
    for (int i = 0; i < NUM_BARS; ++i) mbar_inval(bar0 + 8u * i);
    init_bars();
  }
  __syncthreads();
  tc_fence_after();
  }
  if (warp == W_MMA) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// -------------------------------------------------------------------- dq ----

namespace dq {
constexpr int SLOTS = 5;                                         // K and V tiles in turn
constexpr uint32_t SMEM_Q = 0, SMEM_DO = TILE_BYTES, SMEM_KV = 2 * TILE_BYTES;
constexpr uint32_t SMEM_BAR = SMEM_KV + SLOTS * TILE_BYTES;
// barriers: q_full, kv_full[5], kv_empty[5], s_full[2], dp_full, ds_full, out_full, mma_done
constexpr int NUM_BARS = 1 + 2 * SLOTS + 2 + 4;
constexpr uint32_t SMEM_MISC = SMEM_BAR + NUM_BARS * 8;          // tmem base, abort
constexpr uint32_t SMEM_BYTES = SMEM_MISC + 8 + 1024;
constexpr uint32_t TMEM_S = 0, TMEM_DP = 256, TMEM_DQ = 384;     // S in two buffers
}  // namespace dq

// One block per (128 query rows, head, batch).
__device__ __forceinline__ void dq_block(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                         const CUtensorMap& tm_do, const Params& p, uint8_t* smem_raw, int qt, int head,
                                         int batch) {
  using namespace dq;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const gbase = smem_raw + (base - raw);
  const uint32_t bar0 = base + SMEM_BAR;
  const uint32_t bar_q = bar0;
  auto bar_full = [&](int s) { return bar0 + 8u * (1 + s); };
  auto bar_empty = [&](int s) { return bar0 + 8u * (1 + SLOTS + s); };
  auto bar_s = [&](int i) { return bar0 + 8u * (1 + 2 * SLOTS + i); };
  const uint32_t bar_dp = bar0 + 8u * (3 + 2 * SLOTS), bar_ds = bar_dp + 8u;
  const uint32_t bar_out = bar_dp + 16u, bar_done = bar_dp + 24u;
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(gbase + SMEM_MISC);
  volatile uint32_t* const abort_flag = reinterpret_cast<volatile uint32_t*>(gbase + SMEM_MISC + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q_row0 = qt * BM, kv_col = head / p.group * HD;
  const uint64_t limit = p.wait_limit_ns;
  const int eslot = p.err_slot;
  const int4 hull = p.hull[static_cast<long long>(batch) * p.n_qt + qt];
  __nv_bfloat16* const out = p.dq + static_cast<long long>(batch) * p.n_q * p.dq_stride + head * HD;

  if (hull.x >= hull.y) {                          // no row of the tile sees a key
    for (int i = threadIdx.x; i < BM * (HD / 8); i += THREADS) {
      const int row = q_row0 + i / (HD / 8);
      if (row < p.n_q)
        *reinterpret_cast<uint4*>(out + row * p.dq_stride + 8 * (i % (HD / 8))) = make_uint4(0u, 0u, 0u, 0u);
    }
    return;
  }
  const int tile0 = hull.x / BN, nkv = (hull.y + BN - 1) / BN - tile0;
  // whether some row does not see all keys of the j-th tile
  auto edge_tile = [&](int j) { return (tile0 + j) * BN < hull.z || (tile0 + j + 1) * BN > hull.w; };
  if (threadIdx.x == 0) {
    for (int i = 0; i < NUM_BARS; ++i)
      mbar_init(bar0 + 8u * i, i == 4 + 2 * SLOTS ? WARPS : 1);
    *abort_flag = 0u;
    mbar_fence_init();
  }
  if (warp == W_MMA) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == W_PROD) {
    if (lane == 0) {
      mbar_arrive_expect_tx(bar_q, 2 * TILE_BYTES);
      load_tile(base + SMEM_Q, &tm_q, bar_q, head * HD, q_row0, batch);
      load_tile(base + SMEM_DO, &tm_do, bar_q, head * HD, q_row0, batch);
      int issued = 0;
      for (int idx = 0; idx < 2 * nkv; ++idx) {
        const int s = idx % SLOTS, use = idx / SLOTS;
        if (use > 0 && !mbar_wait_bounded(bar_empty(s), (use - 1) & 1, abort_flag, limit, eslot)) break;
        mbar_arrive_expect_tx(bar_full(s), TILE_BYTES);
        load_tile(base + SMEM_KV + s * TILE_BYTES, (idx & 1) ? &tm_v : &tm_k, bar_full(s), kv_col,
                  (tile0 + (idx >> 1)) * BN, batch);
        issued = idx + 1;
      }
      volatile uint32_t never = 0u;
      mbar_wait_bounded(bar_q, 0, &never, p.drain_limit_ns, eslot);
      for (int idx = max(issued - SLOTS, 0); idx < issued; ++idx)
        mbar_wait_bounded(bar_full(idx % SLOTS), (idx / SLOTS) & 1, &never, p.drain_limit_ns, eslot);
    }
  } else if (warp == W_MMA) {
    if (lane == 0) {
      auto kv_tile = [&](int idx) { return base + SMEM_KV + (idx % SLOTS) * TILE_BYTES; };
      auto full_wait = [&](int idx) {
        return mma_wait(bar_full(idx % SLOTS), (idx / SLOTS) & 1, abort_flag, limit, eslot);
      };
      bool ok = mma_wait(bar_q, 0, abort_flag, limit, eslot) && full_wait(0);
      if (ok) {
        tc_fence_after();
        issue_abt(tmem + TMEM_S, base + SMEM_Q, kv_tile(0));
        tc_commit(bar_s(0));
        ok = full_wait(1);
      }
      if (ok) {
        tc_fence_after();
        issue_abt(tmem + TMEM_DP, base + SMEM_DO, kv_tile(1));
        tc_commit(bar_dp);
        tc_commit(bar_empty(1));
      }
      for (int j = 0; ok && j < nkv; ++j) {
        const bool more = j + 1 < nkv;
        const int kn = 2 * j + 2, vn = 2 * j + 3;
        if (more) {
          if (!full_wait(kn)) break;
          tc_fence_after();
          issue_abt(tmem + TMEM_S + 128 * ((j + 1) & 1), base + SMEM_Q, kv_tile(kn));
          tc_commit(bar_s((j + 1) & 1));
        }
        if (more ? !mbar_spin2_bounded(bar_ds, j & 1, bar_full(vn % SLOTS), (vn / SLOTS) & 1, abort_flag, limit, eslot)
                 : !mma_wait(bar_ds, j & 1, abort_flag, limit, eslot))
          break;
        tc_fence_after();
        if (more) {
          issue_abt(tmem + TMEM_DP, base + SMEM_DO, kv_tile(vn));
          tc_commit(bar_dp);
          tc_commit(bar_empty(vn % SLOTS));
        }
        issue_ab(tmem + TMEM_DQ, tmem + TMEM_S + 128 * (j & 1), kv_tile(2 * j), j > 0);
        tc_commit(more ? bar_empty((2 * j) % SLOTS) : bar_out);
      }
      tc_commit(bar_done);
      volatile uint32_t never = 0u;
      mma_wait(bar_done, 0, &never, p.drain_limit_ns, eslot);
    }
  } else {
    const int t0 = lane & 3, t1 = lane >> 2;
    const int lane16 = 32 * (warp & 3) + 16 * ((warp >> 2) & 1);
    const int half = warp >> 3;                    // keys 64 half .. 64 half + 63 of the tile
    const uint32_t lb = static_cast<uint32_t>(lane16) << 16;
    const uint32_t t_dp = tmem + lb + TMEM_DP + 64 * half;
    const int ra = lane16 + t1;                    // rows of the tile
    const long long qp = static_cast<long long>(p.n_qt) * BM;
    const float2* const stat = p.stat + (static_cast<long long>(batch) * p.n_heads + head) * qp + q_row0 + ra;
    const int2* const rng = p.rng + batch * qp + q_row0 + ra;
    const float2 st_a = stat[0], st_b = stat[8];
    const int2 rng_a = rng[0], rng_b = rng[8];
    const unsigned len_a = rng_a.y, len_b = rng_b.y;
    const float2 c2 = make_float2(p.scale_log2, p.scale_log2);
    const float2 la = make_float2(-st_a.x, -st_a.x), lbv = make_float2(-st_b.x, -st_b.x);
    const float2 da = make_float2(-st_a.y, -st_a.y), db = make_float2(-st_b.y, -st_b.y);
    bool ok = true;
    for (int j = 0; ok && j < nkv; ++j) {
      const int key0 = (tile0 + j) * BN;
      const uint32_t t_s = tmem + lb + TMEM_S + 128 * (j & 1) + 64 * half;
      bool partial = false, odd = false;            // of this warp's 16 rows x 64 keys
      if (!warp_wait(bar_s(j & 1), (j >> 1) & 1, abort_flag, limit, eslot)) { ok = false; break; }
      tc_fence_after();
      uint32_t sr[32];
      tmem_ld16x256(t_s, sr);
      tmem_wait_ld(sr);
      if (edge_tile(j)) {
        const int kw = key0 + 64 * half;
        const bool all = max(rng_a.x, rng_b.x) <= kw && min(rng_a.x + rng_a.y, rng_b.x + rng_b.y) >= kw + 64;
        const bool any = (rng_a.x < kw + 64 && rng_a.x + rng_a.y > kw) || (rng_b.x < kw + 64 && rng_b.x + rng_b.y > kw);
        partial = !__all_sync(0xffffffffu, all);
        odd = any_nonfinite(sr);                    // S(j) has read K(j), dQ(j) has not
        if (odd) zero_nonfinite(gbase + SMEM_KV + ((2 * j) % SLOTS) * TILE_BYTES, 64 * half, 64, lane);
        if (!__any_sync(0xffffffffu, any)) {        // dS = 0
          const uint32_t zero[16] = {};
          if (!warp_wait(bar_dp, j & 1, abort_flag, limit, eslot)) { ok = false; break; }
          tc_fence_after();
          publish(t_s, zero, bar_ds, lane);
          continue;
        }
      }
      float x[32];                                  // P, then dS (4 r: row a, 4 r + 2: row b)
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const float2 ya = __ffma2_rn(make_float2(__uint_as_float(sr[4 * r]), __uint_as_float(sr[4 * r + 1])), c2, la);
        const float2 yb = __ffma2_rn(make_float2(__uint_as_float(sr[4 * r + 2]), __uint_as_float(sr[4 * r + 3])), c2, lbv);
        x[4 * r] = ex2_approx(ya.x);
        x[4 * r + 1] = ex2_approx(ya.y);
        x[4 * r + 2] = ex2_approx(yb.x);
        x[4 * r + 3] = ex2_approx(yb.y);
      }
      if (odd) {                                    // a seen pair with a non-finite S: its dS, whatever P is
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (nonfinite(sr[e])) x[e] = __int_as_float(0x7fc00000);
      }
      if (!warp_wait(bar_dp, j & 1, abort_flag, limit, eslot)) { ok = false; break; }
      tc_fence_after();
      tmem_ld16x256(t_dp, sr);
      tmem_wait_ld(sr);
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const float2 va = __fmul2_rn(
            make_float2(x[4 * r], x[4 * r + 1]),
            __fadd2_rn(make_float2(__uint_as_float(sr[4 * r]), __uint_as_float(sr[4 * r + 1])), da));
        const float2 vb = __fmul2_rn(
            make_float2(x[4 * r + 2], x[4 * r + 3]),
            __fadd2_rn(make_float2(__uint_as_float(sr[4 * r + 2]), __uint_as_float(sr[4 * r + 3])), db));
        x[4 * r] = va.x;
        x[4 * r + 1] = va.y;
        x[4 * r + 2] = vb.x;
        x[4 * r + 3] = vb.y;
      }
      if (partial) {
        const int off_a = key0 + 64 * half + 2 * t0 - rng_a.x, off_b = key0 + 64 * half + 2 * t0 - rng_b.x;
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const int k = 8 * (e >> 2) + (e & 1);
          const bool seen = ((e >> 1) & 1) ? static_cast<unsigned>(off_b + k) < len_b
                                           : static_cast<unsigned>(off_a + k) < len_a;
          if (!seen) x[e] = 0.f;
        }
      }
      uint32_t pk[16];
#pragma unroll
      for (int r = 0; r < 16; ++r) pk[r] = pack_bf16x2(x[2 * r], x[2 * r + 1]);
      publish(t_s, pk, bar_ds, lane);
    }
    if (ok && warp_wait_exact(bar_out, 0, abort_flag, limit, eslot)) {
      tc_fence_after();
      uint32_t v[32];
      load_acc(tmem + lb + TMEM_DQ + 64 * half, v);
      store_tile(v, p.scale, out + 64 * half, p.dq_stride, q_row0 + ra, p.n_q, t0);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == W_MMA) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------ launches ----

constexpr uint32_t SMEM_BYTES = dkdv::SMEM_BYTES > dq::SMEM_BYTES ? dkdv::SMEM_BYTES : dq::SMEM_BYTES;

// dkdv blocks first (they are longer), then dq blocks; of each kind the heads
// fastest and the tiles in the order of falling walks under a causal mask: the first
// keys are seen most, the last rows see most.
__global__ void __launch_bounds__(THREADS, 1)
backward_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                const __grid_constant__ Params p) {
  begin_after_predecessor();
  extern __shared__ uint8_t smem_raw[];
  const unsigned n_dkdv = static_cast<unsigned>(p.n_kt) * p.parts * p.n_kv_heads * p.batch;
  unsigned i = blockIdx.x;
  if (i < n_dkdv) {
    const int part = i % p.parts;
    i /= p.parts;
    const int kvh = i % p.n_kv_heads;
    i /= p.n_kv_heads;
    dkdv_block(tm_q, tm_k, tm_v, tm_do, p, smem_raw, i % p.n_kt, kvh, i / p.n_kt, part);
  } else {
    i -= n_dkdv;
    const int head = i % p.n_heads;
    i /= p.n_heads;
    dq_block(tm_q, tm_k, tm_v, tm_do, p, smem_raw, p.n_qt - 1 - static_cast<int>(i % p.n_qt), head, i / p.n_qt);
  }
}

// dV and dK of split walks: the parts' sums in order, four columns per thread.
__global__ void __launch_bounds__(256) sum_parts_kernel(const __grid_constant__ Params p) {
  begin_after_predecessor();
  const long long tile_size = static_cast<long long>(2) * BN * HD;
  const long long tiles = static_cast<long long>(p.batch) * p.n_kv_heads * p.n_kt;
  const long long n = tiles * (tile_size / 4);
  for (long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; i < n;
       i += static_cast<long long>(gridDim.x) * 256) {
    const long long tile = i / (tile_size / 4);
    const int e = static_cast<int>(i % (tile_size / 4)) * 4;
    const bool is_dk = e >= BN * HD;
    const int row = (e % (BN * HD)) / HD, col = e % HD;
    const int key = static_cast<int>(tile % p.n_kt) * BN + row;
    if (key >= p.n_k) continue;
    const long long bh = tile / p.n_kt;
    const int kvh = static_cast<int>(bh % p.n_kv_heads), batch = static_cast<int>(bh / p.n_kv_heads);
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    const float* src = p.partial + tile * tile_size + e;
#pragma unroll 4
    for (int k = 0; k < p.parts; ++k, src += tiles * tile_size) {
      const float4 v = __ldcs(reinterpret_cast<const float4*>(src));
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
    const float f = is_dk ? p.scale : 1.f;
    __nv_bfloat16* out = is_dk ? p.dk : p.dv;
    const long long stride = is_dk ? p.dk_stride : p.dv_stride;
    *reinterpret_cast<uint2*>(out + (static_cast<long long>(batch) * p.n_k + key) * stride + kvh * HD + col) =
        make_uint2(pack_bf16x2(s.x * f, s.y * f), pack_bf16x2(s.z * f, s.w * f));
  }
}

}  // namespace attn_bwd
}  // namespace h3
