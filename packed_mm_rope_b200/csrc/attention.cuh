// attention.cuh -- full softmax attention over one packed sequence (sm_100a).
//
// "Inside MiniMax H3" sections 2 and 6: every modality's rows share one
// attention sequence and the open inference path runs FULL attention, whose
// cost dominates long videos; "MiniMax H3 -- one transformer ..." notes that
// attention is bidirectional.  So: O = softmax(Q K^T * scale) V per (batch,
// head), no mask, every row attends to every row.
//
// Design (one CTA per 256 query rows of one head, one CTA per SM):
//   warps 0-7   softmax for query tile 0 (rows   0..127)
//   warps 8-15  softmax for query tile 1 (rows 128..255)
//   warp  16    TMA producer: Q tiles once, then K_j, V_j into a ring
//   warp  17    TMEM allocator and single-thread tcgen05.mma issuer
// Tensor memory (512 columns x 128 lanes, fp32):
//   [  0,128)  S0 = Q0 K_j^T    (P0 = bf16 softmax numerators aliased on
//   [128,256)  S1 = Q1 K_j^T     its first 64 columns, two per column)
//   [256,384)  O0 accumulator   [384,512) O1 accumulator
// Per KV tile j the issuer runs  PV0(j), S0(j+1), PV1(j), S1(j+1): while one
// query tile's warps exponentiate their S tile the tensor core works on the
// other.  Each P tile is released in two 64-key halves with their own
// barriers, so the first half of P.V runs while the second half is still being
// exponentiated.  The issuing thread polls V(j) together with the first half of
// P0(j) and K(j+1) together with its second half: one barrier poll whose result
// is branched on costs it ~160 cycles, and the second pair sits on the chain
// P0(j) -> P.V -> S0(j+1) -> softmax.
//
// Softmax: four threads per query row.  Warp w of a query tile reads the 16
// TMEM lanes 32 (w % 4) + 16 ((w / 4) % 2) + [0, 16) with the 16x256b shape,
// so thread (t0 = lane % 4, t1 = lane / 4) holds rows t1 and t1 + 8 of those
// lanes and, of every 8-column block, columns 2 t0 and 2 t0 + 1; the four
// threads of a row (a quad) together hold its 128 keys.  Four warps per
// sub-partition hide each other's TMEM and barrier latencies (one thread per
// row leaves two).  Logits are handled in log2 units (x = s * scale * log2 e).
// Numerators are 2^(x - m) against a running reference m per row that is only
// raised when a thread's share of a 64-key half would overflow the headroom:
// the half's numerators are computed first (speculatively, against the current
// m) and kept unless a share exceeds 2^62 (four shares stay below 2^64).  Then
// the quad takes the half's true maximum by shuffles, O (in TMEM) and the row
// sums are multiplied by 2^(m_old - m_new), and the half is recomputed.  Any m
// gives the same quotient O / l; the limit only keeps numerators, sums and O
// far from fp32/bf16 overflow.  In practice m is set by the first half-tile
// and never moves again, so the hot loop has no max reduction at all: one
// packed fp32x2 FMA, two MUFU ex2, one packed add and one bf16x2 conversion per
// pair of logits.  The S tile of step j+1 is only issued after PV(j), so when
// a warp sees S(j) complete, O already holds PV(j-1) and a rescale for the
// first half can be applied in place; a rescale for the second half first
// waits for the first half of PV(j) to land (pva_done).  Each thread keeps its
// share of the row sums; the quad adds them once, in the epilogue.
//
// Shared memory (1024-byte aligned): Q0, Q1 (32 KB each) and a ring of
// KV_STAGES 32 KB slots; every 128 x 128 bf16 tile is two 128-row x 64-column
// halves in the TMA 128-byte-swizzle layout, which is the canonical K-major
// layout for Q and K and the MN-major layout for V as a B operand.
//
// Every mbarrier wait is bounded (global-time limit); a thread that gives up
// raises an abort flag that all other waits observe, the producer and the
// issuer drain what they already started, and TMEM is freed before exit.
//
// MASKED: query row i attends to the keys [lo_i, hi_i) of `ranges` only (keys
// and queries may differ in number, and groups of query heads may share a K/V
// head).  The CTA visits the key tiles of the hull of its rows' intervals.  In
// tiles that some row does not see in full, each warp tells by votes whether none
// of its 16 rows sees any of a 64-key half (P = 0 without a look at S), or each
// row sees all of it or nothing (a reference of +inf, hence numerators of 0, for
// the latter), or an interval ends inside: then logits outside a row's interval
// become -inf.  A row takes
// its reference m from its first half with a visible key; a row without one ends
// with l = 0, O = 0 and a log-sum-exp of -inf.
// P = 0 does not hide a V row that holds inf or NaN (0 x inf = NaN on the tensor
// core), nor a reference of +inf a logit of inf or NaN, but neither can go unseen:
// O is not finite then.  In that case the CTA runs a second time: logits are masked
// one by one, the softmax warps first clear such elements of V from every tile
// with masked pairs, and rows that do attend to such a key get a NaN logit there:
// masked places cannot change a row, and what a row attends to is never hidden.
// (Looking through V on every run, by the softmax warps or by two warps of their
// own, made such tiles 1.5 to 2 times as long.)
//
// Where there are few blocks, `parts` CTAs of a cluster share a block's walk over the
// keys.  Each leaves O, m and l of its keys in shared memory (the idle Q and K/V
// slots); each then brings a share of the rows to their common reference, adds the
// parts up out of the cluster's distributed shared memory, divides and stores.
//
// Measured with masks: documents of 9,001 + 5,097 rows x 14 heads over 2 K/V heads
// by itself, at 1,965 MHz, 653 us, 1,174 TFLOP/s on the pairs that are seen; in a loop
// with its gradients, under the 1 kW power cap at 1,650 MHz, 769 us, 997 TFLOP/s.
// Documents of 4,584, 82, 2,292 and 701 rows x 8 heads 134 - 141 us (800 TFLOP/s), two
// block prefixes over 7,660 rows, 8 over 2 heads, 126 - 130 us: their 240 blocks of 6 to
// 37 and 7 to 32 key tiles leave 46 and 41 steps per SM on average but 60 on the fullest,
// so a quarter and a third of the SMs' time is idle.  82 rows x 1 head 12 us, launch and
// one block's latency.
#pragma once

#include "common.cuh"
#include "rope.cuh"

namespace h3 {
namespace attn {

constexpr int BM = 128;          // query rows per tile (MMA M)
constexpr int BN = 128;          // key rows per tile  (S MMA N, PV MMA K)
constexpr int HD = 128;          // head dim
constexpr int KV_STAGES = 4;     // K/V ring slots of 32 KB
constexpr int SOFTMAX_WARPS = 16;                   // 8 per query tile, four threads per row
constexpr int W_PROD = SOFTMAX_WARPS;                // TMA producer
constexpr int W_MMA = SOFTMAX_WARPS + 1;             // TMEM allocator and MMA issuer
constexpr int THREADS = 32 * (SOFTMAX_WARPS + 2);    // 576
constexpr uint32_t TILE_BYTES = BM * HD * 2;     // 32768
constexpr uint32_t HALF_BYTES = TILE_BYTES / 2;  // 16384

constexpr uint32_t SMEM_Q = 0;
constexpr uint32_t SMEM_KV = 2 * TILE_BYTES;
constexpr uint32_t SMEM_BAR = SMEM_KV + KV_STAGES * TILE_BYTES;
// barriers: q_full[2], kv_full[S], kv_empty[S], s_full[2], p_full[2][2] (halves),
//           pva_done[2] (first half of PV landed), o_full[2], mma_done,
//           q_ready[2] (Q tile rotated in place, fused RoPE only)
//           v_clean (masked, second run: the V tile holds no inf or NaN any more)
constexpr int NUM_BARS = 2 + 2 * KV_STAGES + 2 + 4 + 2 + 2 + 1 + 2 + 1;
constexpr uint32_t SMEM_MISC = SMEM_BAR + NUM_BARS * 8;       // tmem base, abort, hull, run again; two key sets
constexpr uint32_t SMEM_RANGES = SMEM_MISC + 32 + 32;         // masked: intervals of the CTA's 256 rows
constexpr uint32_t SMEM_BYTES = SMEM_MISC + 32 + 32 + 1024;   // + alignment slack
constexpr uint32_t SMEM_ROW_ML = SMEM_RANGES + 2 * BM * 8;    // masked, parts > 1: (m, l) of the 256 rows
constexpr uint32_t SMEM_ROW_F = SMEM_ROW_ML + 2 * BM * 8;     // and the parts' factors of the rows stored here
constexpr uint32_t MASKED_SMEM_BYTES = SMEM_BYTES + 2 * BM * 8 + 2 * BM * 8 + 2 * BM * 4;
constexpr int MERGE_STRIDE = HD + 4;   // floats per row of the exchanged O: rows 16 bytes apart in the banks
static_assert(2 * BM * MERGE_STRIDE * 4 <= SMEM_BAR, "the exchanged rows must fit in the Q and K/V slots");
static_assert(SMEM_MISC % 16 == 0, "the key sets are read 16 bytes at a time");

constexpr uint32_t IDESC_S = idesc_bf16_f32(BM, BN, false, false);   // Q, K both K-major
constexpr uint32_t IDESC_O = idesc_bf16_f32(BM, HD, false, true);    // P from TMEM, V MN-major

constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t TMEM_S0 = 0, TMEM_O0 = 256;

// Waits of the single MMA-issuing thread spin with test_wait (never suspend):
// it is on the critical path of both query tiles.
__device__ __forceinline__ bool mma_wait(uint32_t bar, uint32_t parity, volatile uint32_t* abort,
                                         uint64_t limit, int err_slot) {
  return mbar_spin_bounded(bar, parity, abort, limit, err_slot);
}

// All lanes wait; the warp proceeds only if every lane saw the phase complete,
// so the .sync.aligned tcgen05 instructions that follow run converged.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile uint32_t* abort,
                                          uint64_t limit, int err_slot) {
  const bool r = mbar_wait_bounded(bar, parity, abort, limit, err_slot);
  return __all_sync(0xffffffffu, r);
}

// The same for a walk's last product (one wait per block), short limits included.
__device__ __forceinline__ bool warp_wait_exact(uint32_t bar, uint32_t parity, volatile uint32_t* abort,
                                                uint64_t limit, int err_slot) {
  const bool r = mbar_wait_exact(bar, parity, abort, limit, err_slot);
  return __all_sync(0xffffffffu, r);
}

struct Params {
  int n_rows;
  int n_heads;
  int n_kv_tiles;
  float scale_log2;               // softmax scale * log2(e)
  __nv_bfloat16* o;
  long long o_row_stride;         // elements
  long long o_batch_stride;       // elements
  float* lse;                     // [B][H][N] or null
  unsigned long long wait_limit_ns;
  unsigned long long drain_limit_ns;
  int err_slot;                   // error word of the launching stream
  // fused RoPE on Q (rope_cs == null: Q arrives rotated)
  const float2* rope_cs;          // [B][N][64] (cos, sin) per rotary pair
  int rope_layout;                // 0 adjacent pairs, 1 half-split
  // MASKED only
  const int2* ranges;             // [B][n_rows] key interval [lo, hi) of each query row
  int n_keys;
  int group;                      // query heads per K/V head
  int parts;                      // CTAs (a cluster) that share a block's keys: 1, 2, 4 or 8
};

template <bool V>
struct Flag {
  static constexpr bool value = V;
};

// Keys of the row's interval that exist: an empty interval is (0, 0).
__device__ __forceinline__ int2 clamp_range(int2 r, int n_keys) {
  r.x = max(r.x, 0);
  r.y = min(r.y, n_keys);
  return r.x < r.y ? r : make_int2(0, 0);
}

// Whether some lane of the warp holds an inf or NaN (multiplied by 0 and added
// up, one packed FMA per two values: NaN if any is not finite).
__device__ __forceinline__ bool any_nonfinite(const uint32_t (&v)[32]) {
  float2 acc = make_float2(0.f, 0.f);
  const float2 zero = acc;
#pragma unroll
  for (int i = 0; i < 16; ++i)
    acc = __ffma2_rn(make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), zero, acc);
  return __any_sync(0xffffffffu, !(acc.x + acc.y == 0.f));
}

// Sets the inf and NaN elements of `rows` (8 or 64, at a multiple of 8) rows of a
// 128 x 128 bf16 tile (two halves of 64 columns) to 0, ordered for the tensor
// core, and returns the rows' bits (one warp; the 128-byte swizzle moves 16-byte
// pieces within their row only).  Rare, so it is kept out of the callers' registers.
__device__ __noinline__ uint2 zero_nonfinite(uint8_t* tile, int row0, int rows, int lane) {
  uint32_t lo = 0u, hi = 0u;
#pragma unroll 1
  for (int i = lane; i < rows * 16; i += 32) {      // 8 pieces of 16 bytes per row and half
    const int row = (i % (rows * 8)) >> 3;
    uint4* q = reinterpret_cast<uint4*>(tile + (i / (rows * 8)) * HALF_BYTES + (row0 + row) * 128 + (i & 7) * 16);
    const uint4 u = *q;
    uint32_t w[4] = {u.x, u.y, u.z, u.w};
    bool found = false;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      if ((w[m] & 0x7f80u) == 0x7f80u) w[m] &= 0xffff0000u, found = true;
      if ((w[m] & 0x7f800000u) == 0x7f800000u) w[m] &= 0xffffu, found = true;
    }
    if (found) {
      *q = make_uint4(w[0], w[1], w[2], w[3]);
      if (row < 32) lo |= 1u << row;
      else hi |= 1u << (row - 32);
    }
  }
  __syncwarp();
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  return make_uint2(__reduce_or_sync(0xffffffffu, lo), __reduce_or_sync(0xffffffffu, hi));
}

template <bool MASKED>
__global__ void __launch_bounds__(THREADS, 1)
attention_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const Params p) {
  if (MASKED) begin_after_predecessor();
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const gbase = smem_raw + (base - raw);

  const uint32_t bar0 = base + SMEM_BAR;
  auto bar_q_full = [&](int i) { return bar0 + 8u * i; };
  auto bar_kv_full = [&](int s) { return bar0 + 8u * (2 + s); };
  auto bar_kv_empty = [&](int s) { return bar0 + 8u * (2 + KV_STAGES + s); };
  auto bar_s_full = [&](int i) { return bar0 + 8u * (2 + 2 * KV_STAGES + i); };
  auto bar_p_full = [&](int i, int half) { return bar0 + 8u * (4 + 2 * KV_STAGES + 2 * i + half); };
  auto bar_pva_done = [&](int i) { return bar0 + 8u * (8 + 2 * KV_STAGES + i); };
  auto bar_o_full = [&](int i) { return bar0 + 8u * (10 + 2 * KV_STAGES + i); };
  const uint32_t bar_mma_done = bar0 + 8u * (12 + 2 * KV_STAGES);
  auto bar_q_ready = [&](int i) { return bar0 + 8u * (13 + 2 * KV_STAGES + i); };
  const uint32_t bar_v_clean = bar0 + 8u * (15 + 2 * KV_STAGES);
  const bool fused_rope = !MASKED && p.rope_cs != nullptr;
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(gbase + SMEM_MISC);
  volatile uint32_t* const abort_flag = reinterpret_cast<volatile uint32_t*>(gbase + SMEM_MISC + 4);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  // masked: a flat grid, heads fastest, the tiles in the order of the sequence or, if the
  // last row sees at least as many keys as the first, in the reverse order.  Under a causal
  // mask that puts the longest walks of all heads first and the shortest last (8,192 causal
  // rows x 8 heads, 256 blocks: heads slowest leaves 1.5 times as long); with documents it
  // says nothing about the walks between the ends (two block prefixes of 1,201 / 4,096 and
  // 880 / 3,564 rows: walks of 28, 7, 32 and 10 key tiles, in that order).
  const int n_tiles = (p.n_rows + 2 * BM - 1) / (2 * BM);
  int head = blockIdx.y, batch = blockIdx.z, tile = blockIdx.x, part = 0;
  if constexpr (MASKED) {
    part = blockIdx.x % p.parts;       // the CTA's rank in its cluster
    const int block = blockIdx.x / p.parts;
    head = block % p.n_heads;
    tile = block / p.n_heads % n_tiles;
    batch = block / p.n_heads / n_tiles;
    if (gridDim.x > 148u) {            // more than run at once on a B200
      const int2 a = clamp_range(p.ranges[0], p.n_keys), b = clamp_range(p.ranges[p.n_rows - 1], p.n_keys);
      if (b.y - b.x >= a.y - a.x) tile = n_tiles - 1 - tile;
    }
  }
  const int q_row0 = tile * (2 * BM);
  const uint64_t limit = p.wait_limit_ns;
  const int eslot = p.err_slot;

  auto init_bars = [&] {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_q_full(i), 1);
      mbar_init(bar_s_full(i), 1);
      mbar_init(bar_p_full(i, 0), 8);    // one arrival per softmax warp of the tile
      mbar_init(bar_p_full(i, 1), 8);
      mbar_init(bar_pva_done(i), 1);
      mbar_init(bar_o_full(i), 1);
    }
    for (int s = 0; s < KV_STAGES; ++s) {
      mbar_init(bar_kv_full(s), 1);
      mbar_init(bar_kv_empty(s), 1);
    }
    mbar_init(bar_mma_done, 1);
    mbar_init(bar_q_ready(0), 8);
    mbar_init(bar_q_ready(1), 8);
    mbar_init(bar_v_clean, SOFTMAX_WARPS);
    mbar_fence_init();
  };
  volatile uint32_t* const again = reinterpret_cast<volatile uint32_t*>(gbase + SMEM_MISC + 24);   // masked
  int* const hull = reinterpret_cast<int*>(gbase + SMEM_MISC + 8);                                 // masked
  // masked: this thread's row's interval, on its way while the barriers are set up
  int2 range = make_int2(0, 0x7fffffff);           // rows past the end see all and are never stored
  if (MASKED && threadIdx.x < 2 * BM && q_row0 + threadIdx.x < p.n_rows)
    range = p.ranges[static_cast<long long>(batch) * p.n_rows + q_row0 + threadIdx.x];
  if (threadIdx.x == 0) {
    *abort_flag = 0u;
    *again = 0u;
    hull[0] = hull[2] = 0x7fffffff;
    hull[1] = hull[3] = 0;
    init_bars();
  }
  auto load_q = [&] {                              // producer thread
    for (int i = 0; i < 2; ++i) {
      const uint32_t dst = base + SMEM_Q + i * TILE_BYTES;
      mbar_arrive_expect_tx(bar_q_full(i), TILE_BYTES);
      tma_load_3d(dst, &tm_q, bar_q_full(i), head * HD, q_row0 + i * BM, batch);
      tma_load_3d(dst + HALF_BYTES, &tm_q, bar_q_full(i), head * HD + 64, q_row0 + i * BM, batch);
    }
  };
  int nkv = p.n_kv_tiles;
  int tile0 = 0;                     // first key tile of this CTA
  int full_lo = 0, full_hi = 0;      // masked: keys [full_lo, full_hi) are seen by every row of the CTA
  if constexpr (MASKED) {
    // Q and tensor memory meanwhile
    if (warp == W_MMA) {
      tmem_alloc(smem_u32(tmem_slot), TMEM_COLS);
      tmem_relinquish();
    }
    __syncthreads();
    if (warp == W_PROD && lane == 0) load_q();
    // hull of the rows' intervals, and the keys that all of them see
    if (threadIdx.x < 2 * BM) {
      int2 r = make_int2(0x7fffffff, 0);           // rows past the end: no say in the hull
      int all_lo = 0, all_hi = 0x7fffffff;
      if (q_row0 + threadIdx.x < p.n_rows) {
        range = r = clamp_range(range, p.n_keys);
        all_lo = r.x;
        all_hi = r.y;
        if (r.x >= r.y) r = make_int2(0x7fffffff, 0);
      }
      reinterpret_cast<int2*>(gbase + SMEM_RANGES)[threadIdx.x] = range;
      const int lo = __reduce_min_sync(0xffffffffu, r.x), hi = __reduce_max_sync(0xffffffffu, r.y);
      all_hi = __reduce_min_sync(0xffffffffu, all_hi);
      all_lo = __reduce_max_sync(0xffffffffu, all_lo);
      if (lane == 0) {
        atomicMin(&hull[0], lo);
        atomicMax(&hull[1], hi);
        atomicMin(&hull[2], all_hi);
        atomicMax(&hull[3], all_lo);
      }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    full_hi = hull[2];
    full_lo = hull[3];
    nkv = 0;
    if (hull[0] < hull[1]) {
      tile0 = hull[0] / BN;
      nkv = (hull[1] + BN - 1) / BN - tile0;
    }
    if (nkv == 0) {                                // no row attends to anything
      if (part == 0) {
        for (int i = threadIdx.x; i < 2 * BM * (HD / 8); i += THREADS) {
          const int row = q_row0 + i / (HD / 8);
          if (row < p.n_rows)
            *reinterpret_cast<uint4*>(p.o + batch * p.o_batch_stride + static_cast<long long>(row) * p.o_row_stride +
                                      head * HD + 8 * (i % (HD / 8))) = make_uint4(0u, 0u, 0u, 0u);
        }
        if (p.lse != nullptr && threadIdx.x < 2 * BM && q_row0 + threadIdx.x < p.n_rows)
          p.lse[(static_cast<long long>(batch) * p.n_heads + head) * p.n_rows + q_row0 + threadIdx.x] = -INFINITY;
      }
      if (warp == W_PROD && lane == 0) {           // Q's copies end before the CTA does
        volatile uint32_t never = 0u;
        for (int i = 0; i < 2; ++i) mbar_wait_bounded(bar_q_full(i), 0, &never, p.drain_limit_ns, eslot);
      }
      if (warp == W_MMA) tmem_dealloc(*tmem_slot, TMEM_COLS);
      return;
    }
    const int j0 = nkv * part / p.parts;           // this CTA's share of the key tiles, maybe none
    nkv = nkv * (part + 1) / p.parts - j0;
    tile0 += j0;
  }
  if constexpr (!MASKED) {
    if (warp == W_MMA) {
      tmem_alloc(smem_u32(tmem_slot), TMEM_COLS);
      tmem_relinquish();
    }
    if (warp == W_PROD && lane == 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  }
  const uint32_t tmem = *tmem_slot;

  // masked: whether some row of the CTA does not see all of the j-th key tile
  auto edge_tile = [&](int j) { return (tile0 + j) * BN < full_lo || (tile0 + j + 1) * BN > full_hi; };

  for (int run = 0; run < (MASKED ? 2 : 1) && nkv > 0; ++run) {
  if (warp == W_PROD) {
    // ------------------------------------------------------------ TMA ----
    if (lane == 0) {
      const int kv_col0 = (MASKED ? head / p.group : head) * HD;
      if (!MASKED || run > 0) load_q();
      int issued = 0;
      for (int idx = 0; idx < 2 * nkv; ++idx) {
        const int s = idx % KV_STAGES;
        const int use = idx / KV_STAGES;
        if (use > 0 && !mbar_wait_bounded(bar_kv_empty(s), (use - 1) & 1, abort_flag, limit, eslot)) break;
        const CUtensorMap* tm = (idx & 1) ? &tm_v : &tm_k;
        const int row = (tile0 + (idx >> 1)) * BN;
        const uint32_t dst = base + SMEM_KV + s * TILE_BYTES;
        mbar_arrive_expect_tx(bar_kv_full(s), TILE_BYTES);
        tma_load_3d(dst, tm, bar_kv_full(s), kv_col0, row, batch);
        tma_load_3d(dst + HALF_BYTES, tm, bar_kv_full(s), kv_col0 + 64, row, batch);
        issued = idx + 1;
      }
      // Drain: every load this thread started must land before the CTA exits.
      // The drain ignores the abort flag (a never-raised local flag).
      volatile uint32_t never = 0u;
      for (int i = 0; i < 2; ++i) mbar_wait_bounded(bar_q_full(i), 0, &never, p.drain_limit_ns, eslot);
      for (int idx = (issued > KV_STAGES ? issued - KV_STAGES : 0); idx < issued; ++idx)
        mbar_wait_bounded(bar_kv_full(idx % KV_STAGES), (idx / KV_STAGES) & 1, &never,
                          p.drain_limit_ns, eslot);
    }
  } else if (warp == W_MMA) {
    // ------------------------------------------------------------ MMA ----
    if (lane == 0) {
      auto q_addr = [&](int i) { return base + SMEM_Q + i * TILE_BYTES; };
      auto kv_addr = [&](int s) { return base + SMEM_KV + s * TILE_BYTES; };
      // S_i = Q_i K^T : 8 MMAs of K=16 over the two 64-column swizzled halves
      auto issue_s = [&](int i, int ks) {
        const uint32_t d = tmem + TMEM_S0 + i * 128;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint32_t off = (kk >> 2) * HALF_BYTES + (kk & 3) * 32;
          mma_ss(d, smem_desc_sw128(q_addr(i) + off, 16, 1024),
                 smem_desc_sw128(kv_addr(ks) + off, 16, 1024), IDESC_S, kk > 0 ? 1u : 0u);
        }
      };
      // O_i += P_i V over keys [64*half, 64*half + 64): A = P_i from TMEM (8
      // columns per K=16 step), B = V rows from shared memory, MN-major
      auto issue_pv = [&](int i, int vs, int half, bool acc) {
        const uint32_t d = tmem + TMEM_O0 + i * 128;
        const uint32_t a = tmem + TMEM_S0 + i * 128;
#pragma unroll
        for (int k4 = 0; k4 < 4; ++k4) {
          const int kk = 4 * half + k4;
          mma_ts(d, a + kk * 8, smem_desc_sw128(kv_addr(vs) + kk * 2048, HALF_BYTES, 1024),
                 IDESC_O, (acc || kk > 0) ? 1u : 0u);
        }
      };
      // P_i(j) in two halves; the first half's completion is announced on pva_done.
      // x / y (non-zero): a barrier the caller needs, polled together with the
      // second / first half of P so that the two polls' latencies overlap
      auto issue_pv_tile = [&](int i, int vs, int j, uint32_t x, uint32_t x_par, uint32_t y = 0u,
                               uint32_t y_par = 0u) -> bool {
        if (y != 0u ? !mbar_spin2_bounded(bar_p_full(i, 0), j & 1, y, y_par, abort_flag, limit, eslot)
                    : !mma_wait(bar_p_full(i, 0), j & 1, abort_flag, limit, eslot))
          return false;
        tc_fence_after();
        issue_pv(i, vs, 0, j > 0);
        tc_commit(bar_pva_done(i));
        if (x != 0u ? !mbar_spin2_bounded(bar_p_full(i, 1), j & 1, x, x_par, abort_flag, limit, eslot)
                    : !mma_wait(bar_p_full(i, 1), j & 1, abort_flag, limit, eslot))
          return false;
        tc_fence_after();
        issue_pv(i, vs, 1, true);
        return true;
      };
      // with fused RoPE the softmax warpgroups rotate Q in place first
      auto bar_q = [&](int i) { return fused_rope ? bar_q_ready(i) : bar_q_full(i); };
      bool ok = mma_wait(bar_q(0), 0, abort_flag, limit, eslot) &&
                mma_wait(bar_kv_full(0), 0, abort_flag, limit, eslot);
      if (ok) {
        tc_fence_after();
        issue_s(0, 0);
        tc_commit(bar_s_full(0));
        ok = mma_wait(bar_q(1), 0, abort_flag, limit, eslot);
      }
      if (ok) {
        tc_fence_after();
        issue_s(1, 0);
        tc_commit(bar_s_full(1));
        tc_commit(bar_kv_empty(0));
      }
      for (int j = 0; ok && j < nkv; ++j) {
        const int vidx = 2 * j + 1, vs = vidx % KV_STAGES;
        const int kidx = 2 * j + 2, ks = kidx % KV_STAGES;
        const bool more = j + 1 < nkv;
        // V(j) is waited for together with the first half of P0(j), K(j + 1)
        // together with its second half
        if (!issue_pv_tile(0, vs, j, more ? bar_kv_full(ks) : 0u, (kidx / KV_STAGES) & 1, bar_kv_full(vs),
                           (vidx / KV_STAGES) & 1))
          break;
        if (more) {
          tc_fence_after();
          issue_s(0, ks);
          tc_commit(bar_s_full(0));
        } else {
          tc_commit(bar_o_full(0));
        }
        if (!issue_pv_tile(1, vs, j, 0u, 0u)) break;
        tc_commit(bar_kv_empty(vs));
        if (more) {
          issue_s(1, ks);
          tc_commit(bar_s_full(1));
          tc_commit(bar_kv_empty(ks));
        } else {
          tc_commit(bar_o_full(1));
        }
      }
      // Drain: all MMAs issued above complete before TMEM is released.
      tc_commit(bar_mma_done);
      volatile uint32_t never = 0u;
      mma_wait(bar_mma_done, 0, &never, p.drain_limit_ns, eslot);
    }
  } else {
    // -------------------------------------------------------- softmax ----
    // Eight warps per query tile, four threads per row: warp w reads the 16
    // TMEM lanes 32 (w % 4) + 16 ((w / 4) % 2) + [0, 16) with the 16x256b
    // shape, so thread (t0 = lane % 4, t1 = lane / 4) holds rows t1 and t1 + 8
    // of that group and, of every 8-column block, columns 2 t0 and 2 t0 + 1.
    // The four threads of a row agree on its reference through shuffles.
    const int wg = warp >> 3;                      // query tile 0 or 1
    const int t0 = lane & 3, t1 = lane >> 2;
    const int lane16 = 32 * (warp & 3) + 16 * ((warp >> 2) & 1);
    const uint32_t lb = static_cast<uint32_t>(lane16) << 16;
    const uint32_t t_s = tmem + lb + TMEM_S0 + wg * 128;
    const uint32_t t_o = tmem + lb + TMEM_O0 + wg * 128;
    const float sl2 = p.scale_log2;
    const int tail = p.n_rows - (nkv - 1) * BN;    // valid keys in the last tile (1..128)
    const int row_a = q_row0 + wg * BM + lane16 + t1;
    const int row_b = row_a + 8;
    // masked: the intervals of row_a and row_b (8 rows on)
    const int2* const rng = reinterpret_cast<const int2*>(gbase + SMEM_RANGES) + wg * BM + lane16 + t1;
    const volatile uint32_t* const unclean = reinterpret_cast<uint32_t*>(gbase + SMEM_MISC + 32);   // key sets of V
    float m_a = -INFINITY, m_b = -INFINITY;        // log2 units, identical in a row's 4 threads
    float l_a = 0.f, l_b = 0.f;                    // this thread's share of the row sums
    bool ok = true;
    constexpr float PART_LIMIT = 4611686018427387904.0f;   // 2^62: four shares stay below 2^64

    auto quad_max = [](float v) {
      v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
      return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
    };
    auto quad_or = [](bool v) {
      int x = v ? 1 : 0;
      x |= __shfl_xor_sync(0xffffffffu, x, 1);
      x |= __shfl_xor_sync(0xffffffffu, x, 2);
      return x != 0;
    };
    // logits of 64 keys starting at key c0 of the tile (registers as loaded);
    // keys past the end -> -inf; masked: keys outside the row's interval -> -inf
    auto to_logits = [&](const uint32_t (&r)[32], int c0, bool last, float (&x)[32]) {
#pragma unroll
      for (int e = 0; e < 32; ++e) x[e] = __uint_as_float(r[e]);
      if (!MASKED && last && tail < BN) {
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const int key = c0 + 8 * (e >> 2) + 2 * t0 + (e & 1);
          if (key >= tail) x[e] = -INFINITY;
        }
      }
    };
    auto mask_logits = [&](int key0, const volatile uint32_t* bad, float (&x)[32]) {
      const int2 a = rng[0], b = rng[8];
      const unsigned len_a = a.y - a.x, len_b = b.y - b.x;
      const int off_a = key0 + 2 * t0 - a.x, off_b = key0 + 2 * t0 - b.x;
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        const int k = 8 * (e >> 2) + (e & 1);
        const bool seen = ((e >> 1) & 1) ? static_cast<unsigned>(off_b + k) < len_b
                                         : static_cast<unsigned>(off_a + k) < len_a;
        if (!seen) x[e] = -INFINITY;
      }
      if (bad != nullptr && (bad[0] | bad[1]) != 0u) {   // a key of this half has inf or NaN in V
        const uint32_t bad_lo = bad[0], bad_hi = bad[1];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const int k = 8 * (e >> 2) + (e & 1);
          const bool seen = ((e >> 1) & 1) ? static_cast<unsigned>(off_b + k) < len_b
                                           : static_cast<unsigned>(off_a + k) < len_a;
          const uint32_t bit = (k < 32 ? bad_lo : bad_hi) >> ((k & 31) + 2 * t0) & 1u;
          if (bit && seen) x[e] = __int_as_float(0x7fc00000);
        }
      }
    };
    // numerators of the 16 keys of each row: bf16 pairs (register order of the
    // 16x128b store) and this thread's sums
    auto exps = [&](const float (&x)[32], uint32_t (&pk)[16], float& sa, float& sb, bool none_a = false,
                    bool none_b = false) {
      const float2 c2 = make_float2(sl2, sl2);
      const float ra = none_a ? -INFINITY : -m_a, rb = none_b ? -INFINITY : -m_b;
      const float2 ma = make_float2(ra, ra), mb = make_float2(rb, rb);
      float2 acc_a = make_float2(0.f, 0.f), acc_b = make_float2(0.f, 0.f);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float2 ya = __ffma2_rn(make_float2(x[4 * q], x[4 * q + 1]), c2, ma);
        const float2 yb = __ffma2_rn(make_float2(x[4 * q + 2], x[4 * q + 3]), c2, mb);
        const float pa0 = ex2_approx(ya.x), pa1 = ex2_approx(ya.y);
        const float pb0 = ex2_approx(yb.x), pb1 = ex2_approx(yb.y);
        acc_a = __fadd2_rn(acc_a, make_float2(pa0, pa1));
        acc_b = __fadd2_rn(acc_b, make_float2(pb0, pb1));
        pk[2 * q] = pack_bf16x2(pa0, pa1);
        pk[2 * q + 1] = pack_bf16x2(pb0, pb1);
      }
      sa = acc_a.x + acc_a.y;
      sb = acc_b.x + acc_b.y;
    };
    // O *= f per row for this warp's lanes (warp-collective TMEM round trip)
    auto rescale_o = [&](float fa, float fb) {
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        uint32_t o[32];
        tmem_ld16x256(t_o + 64 * h, o);
        tmem_wait_ld(o);
#pragma unroll
        for (int e = 0; e < 32; ++e)
          o[e] = __float_as_uint(__uint_as_float(o[e]) * (((e >> 1) & 1) ? fb : fa));
        tmem_st16x256(t_o + 64 * h, o);
      }
    };
    // the rare path: raise the reference of the rows whose shares need it
    // (all rows on the first half of the first tile); returns (fa, fb)
    auto new_reference = [&](const float (&x)[32], bool first_a, bool first_b, float sa, float sb, float& fa,
                             float& fb) {
      const bool na = quad_or(first_a || !(sa <= PART_LIMIT));
      const bool nb = quad_or(first_b || !(sb <= PART_LIMIT));
      float xa = -INFINITY, xb = -INFINITY;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        xa = fmaxf(xa, fmaxf(x[4 * q], x[4 * q + 1]));
        xb = fmaxf(xb, fmaxf(x[4 * q + 2], x[4 * q + 3]));
      }
      xa = quad_max(xa);
      xb = quad_max(xb);
      fa = 1.f;
      fb = 1.f;
      if (na) {
        const float mn = fmaxf(first_a ? -INFINITY : m_a, xa * sl2);
        fa = first_a ? 0.f : ex2_approx(m_a - mn);
        m_a = mn;
        l_a *= fa;
      }
      if (nb) {
        const float mn = fmaxf(first_b ? -INFINITY : m_b, xb * sl2);
        fb = first_b ? 0.f : ex2_approx(m_b - mn);
        m_b = mn;
        l_b *= fb;
      }
    };
    // Publish 64 keys of P (32 TMEM columns at c0 / 2, aliasing S columns
    // already read): every lane's store lands and is fenced, then one arrival.
    auto store_p = [&](int half, const uint32_t (&pk)[16]) {
      __syncwarp();
      tmem_st16x128(t_s + 32 * half, pk);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_p_full(wg, half));
    };

    // Fused RoPE: rotate this tile's Q rows in shared memory, two threads per
    // row (each 8 of the 16 chunks), with the (cos, sin) the rope kernel uses
    // (read from the table) and its rot2 arithmetic, then make the
    // generic-proxy writes visible to the tensor core (async proxy).
    if (fused_rope) {
      if (!warp_wait(bar_q_full(wg), 0, abort_flag, limit, eslot)) ok = false;
      const int tid = (warp & 7) * 32 + lane;
      const int row_in_tile = tid >> 1, part = tid & 1;
      const int row = q_row0 + wg * BM + row_in_tile;
      if (ok && row < p.n_rows) {
        const float4* cs4 = reinterpret_cast<const float4*>(p.rope_cs + (static_cast<long long>(batch) * p.n_rows + row) * 64);
        uint8_t* qrow = gbase + SMEM_Q + wg * TILE_BYTES + row_in_tile * 128;
        const int sw = row_in_tile & 7;           // 128-byte swizzle of this row
        auto chunk = [&](int c) {                 // logical 16-byte chunk c of 16
          return reinterpret_cast<uint4*>(qrow + (c >> 3) * HALF_BYTES + (((c & 7) ^ sw) << 4));
        };
        if (p.rope_layout == 0) {
#pragma unroll 4
          for (int c = 8 * part; c < 8 * part + 8; ++c) {   // pairs 4c .. 4c+3
            const float4 a = __ldg(cs4 + 2 * c), b = __ldg(cs4 + 2 * c + 1);
            const float2 cs[4] = {make_float2(a.x, a.y), make_float2(a.z, a.w), make_float2(b.x, b.y),
                                  make_float2(b.z, b.w)};
            *chunk(c) = rotate_adjacent(*chunk(c), cs);
          }
        } else {
#pragma unroll 2
          for (int c = 4 * part; c < 4 * part + 4; ++c) {   // pairs 8c .. 8c+7
            float2 cs[8];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              const float4 a = __ldg(cs4 + 4 * c + m);
              cs[2 * m] = make_float2(a.x, a.y);
              cs[2 * m + 1] = make_float2(a.z, a.w);
            }
            uint4 a = *chunk(c), b = *chunk(c + 8);
            rotate_half(a, b, cs);
            *chunk(c) = a;
            *chunk(c + 8) = b;
          }
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_q_ready(wg));
    }

    // One key tile, references set (unmasked: from its first half on).  SOME (masked):
    // each row sees all of a half or (bits of `none`: row a, row b of half 0, of half
    // 1) nothing; otherwise all of the tile.
    auto plain_step = [&](auto some, int j, int none) -> bool {
      constexpr bool SOME = decltype(some)::value;
      const bool last = j == nkv - 1;
      if (SOME && __all_sync(0xffffffffu, (none & 3) == 3)) {
        const uint32_t pk[16] = {};
        store_p(0, pk);
      } else {
        // ---- keys 0..63 ----
        uint32_t r[32];
        tmem_ld16x256(t_s, r);
        tmem_wait_ld(r);
        float x[32];
        to_logits(r, 0, last, x);
        uint32_t pk[16];
        float sa, sb;
        const bool na = SOME && (none & 1), nb = SOME && (none & 2);
        exps(x, pk, sa, sb, na, nb);                // speculative against the references
        const bool first = !MASKED && j == 0;
        const bool need = first || !(sa <= PART_LIMIT) || !(sb <= PART_LIMIT);
        if (__any_sync(0xffffffffu, need)) {
          float fa, fb;
          new_reference(x, first, first, sa, sb, fa, fb);
          __syncwarp();
          if (j > 0) rescale_o(fa, fb);   // O holds PV(j-1); PV(j) has not started
          exps(x, pk, sa, sb, na, nb);
        }
        l_a += sa;
        l_b += sb;
        store_p(0, pk);
      }
      if (SOME && __all_sync(0xffffffffu, (none & 12) == 12)) {
        const uint32_t pk[16] = {};
        store_p(1, pk);
      } else {
        // ---- keys 64..127 ----
        uint32_t r[32];
        __syncwarp();
        tmem_ld16x256(t_s + 64, r);
        tmem_wait_ld(r);
        float x[32];
        to_logits(r, 64, last, x);
        uint32_t pk[16];
        float sa, sb;
        const bool na = SOME && (none & 4), nb = SOME && (none & 8);
        exps(x, pk, sa, sb, na, nb);
        const bool need = !(sa <= PART_LIMIT) || !(sb <= PART_LIMIT);
        if (__any_sync(0xffffffffu, need)) {
          // the first half of PV(j) may be in flight: let it land, then rescale
          // O (which now includes it) together with the running sums
          if (!warp_wait(bar_pva_done(wg), j & 1, abort_flag, limit, eslot)) return false;
          tc_fence_after();
          float fa, fb;
          new_reference(x, false, false, sa, sb, fa, fb);
          __syncwarp();
          rescale_o(fa, fb);
          exps(x, pk, sa, sb, na, nb);
        }
        l_a += sa;
        l_b += sb;
        store_p(1, pk);
      }
      return true;
    };
    bool set_a = !MASKED, set_b = !MASKED;         // masked: the rows have a reference (else m is 0, and l)
    int edges = 0;                                 // masked, second run: tiles cleared so far
    // what a row sees of the 64 keys from `key` on
    auto nothing = [](int2 r, int key) { return r.x >= key + 64 || r.y <= key; };
    auto all = [](int2 r, int key) { return r.x <= key && r.y >= key + 64; };
    // masked: the same where an interval ends inside a half, where a row has no
    // reference yet, and in the second run; the halves in a loop, since this code runs a
    // few times per CTA, often from a cold instruction cache
    auto edge_step = [&](int j) -> bool {
      const volatile uint32_t* bad = nullptr;       // second run: the keys that had inf or NaN in V
      if (run == 1 && edge_tile(j)) {
        // all softmax warps clear V(j) together; PV(j) waits for P(j), hence for them
        const int vidx = 2 * j + 1, vs = vidx % KV_STAGES;
        if (!warp_wait(bar_kv_full(vs), (vidx / KV_STAGES) & 1, abort_flag, limit, eslot)) return false;
        const uint2 rows = zero_nonfinite(gbase + SMEM_KV + vs * TILE_BYTES, 8 * warp, 8, lane);
        if (lane == 0)
          reinterpret_cast<volatile uint8_t*>(gbase + SMEM_MISC + 32 + 16 * (edges & 1))[warp] =
              static_cast<uint8_t>(rows.x);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_v_clean);
        if (!warp_wait(bar_v_clean, edges & 1, abort_flag, limit, eslot)) return false;
        bad = unclean + 4 * (edges & 1);            // read before the next arrival: two sets are enough
        ++edges;
      }
      if (!warp_wait(bar_s_full(wg), j & 1, abort_flag, limit, eslot)) return false;
      tc_fence_after();
      const int2 ra = rng[0], rb = rng[8];
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        const int key0 = (tile0 + j) * BN + 64 * h;
        const bool none_a = nothing(ra, key0), none_b = nothing(rb, key0);
        uint32_t pk[16];
        if (__all_sync(0xffffffffu, none_a && none_b)) {
#pragma unroll
          for (int i = 0; i < 16; ++i) pk[i] = 0u;
        } else {
          const bool cut = !(none_a || all(ra, key0)) || !(none_b || all(rb, key0));
          const bool mask = run == 1 || __any_sync(0xffffffffu, cut);   // logit by logit
          uint32_t r[32];
          __syncwarp();
          tmem_ld16x256(t_s + 64 * h, r);
          tmem_wait_ld(r);
          float x[32];
          to_logits(r, 0, false, x);
          if (mask) mask_logits(key0, bad != nullptr ? bad + 2 * h : bad, x);
          float sa, sb;
          exps(x, pk, sa, sb, !mask && none_a, !mask && none_b);
          const bool first_a = !set_a && !none_a, first_b = !set_b && !none_b;
          if (__any_sync(0xffffffffu, first_a || first_b || !(sa <= PART_LIMIT) || !(sb <= PART_LIMIT))) {
            if (h == 1) {
              if (!warp_wait(bar_pva_done(wg), j & 1, abort_flag, limit, eslot)) return false;
              tc_fence_after();
            }
            float fa, fb;
            new_reference(x, first_a, first_b, sa, sb, fa, fb);
            set_a |= first_a;
            set_b |= first_b;
            __syncwarp();
            if (j + h > 0) rescale_o(fa, fb);
            exps(x, pk, sa, sb, !mask && none_a, !mask && none_b);
          }
          l_a += sa;
          l_b += sb;
        }
        store_p(h, pk);
      }
      return true;
    };
    // masked: up to here tiles are seen in full by every row of the CTA, from some tile on
    const int plain_end = MASKED ? min(nkv, full_hi / BN - tile0) : nkv;
    bool refs = !MASKED;                           // masked: all rows of the warp have a reference
    if (MASKED) m_a = m_b = 0.f;
    int j = 0;
    while (ok && j < nkv) {
      if (refs && j < plain_end && !(MASKED && edge_tile(j))) {
        for (; j < plain_end; ++j) {
          if (!warp_wait(bar_s_full(wg), j & 1, abort_flag, limit, eslot)) { ok = false; break; }
          tc_fence_after();
          if (!plain_step(Flag<false>{}, j, 0)) { ok = false; break; }
        }
      } else if constexpr (MASKED) {
        const int key0 = (tile0 + j) * BN;
        const int2 a = rng[0], b = rng[8];
        const int none = (nothing(a, key0) ? 1 : 0) | (nothing(b, key0) ? 2 : 0) | (nothing(a, key0 + 64) ? 4 : 0) |
                         (nothing(b, key0 + 64) ? 8 : 0);
        const bool some = ((none & 1) || (set_a && all(a, key0))) && ((none & 2) || (set_b && all(b, key0))) &&
                          ((none & 4) || (set_a && all(a, key0 + 64))) && ((none & 8) || (set_b && all(b, key0 + 64)));
        if (run == 0 && __all_sync(0xffffffffu, some)) {
          ok = warp_wait(bar_s_full(wg), j & 1, abort_flag, limit, eslot);
          if (ok) {
            tc_fence_after();
            ok = plain_step(Flag<true>{}, j, none);
          }
        } else {
          ok = edge_step(j);
          refs = __all_sync(0xffffffffu, set_a && set_b);
        }
        ++j;
      }
    }

    // epilogue: O / l -> bf16 -> global; optional log-sum-exp
    if (ok && (MASKED ? warp_wait_exact(bar_o_full(wg), 0, abort_flag, limit, eslot)
                      : warp_wait(bar_o_full(wg), 0, abort_flag, limit, eslot))) {
      tc_fence_after();
      // row sums over the four threads of each row
      l_a += __shfl_xor_sync(0xffffffffu, l_a, 1);
      l_a += __shfl_xor_sync(0xffffffffu, l_a, 2);
      l_b += __shfl_xor_sync(0xffffffffu, l_b, 1);
      l_b += __shfl_xor_sync(0xffffffffu, l_b, 2);
      if (MASKED && p.parts > 1) {
        // the parts' rows are joined below
        if (t0 == 0) {
          float2* ml = reinterpret_cast<float2*>(gbase + SMEM_ROW_ML) + wg * BM + lane16 + t1;
          ml[0] = make_float2(set_a ? m_a : -INFINITY, l_a);
          ml[8] = make_float2(set_b ? m_b : -INFINITY, l_b);
        }
#pragma unroll 1
        for (int h = 0; run == 0 && h < 2; ++h) {
          uint32_t o[32];
          __syncwarp();
          tmem_ld16x256(t_o + 64 * h, o);
          tmem_wait_ld(o);
          if (any_nonfinite(o) && (edge_tile(0) || edge_tile(nkv - 1))) *again = 1u;
        }
      } else {
        // masked: a row without keys has l = 0 and O = 0
        const bool empty_a = MASKED && rng[0].x >= rng[0].y, empty_b = MASKED && rng[8].x >= rng[8].y;
        const float inv_a = empty_a ? 0.f : 1.f / l_a, inv_b = empty_b ? 0.f : 1.f / l_b;
        __nv_bfloat16* orow_a = p.o + batch * p.o_batch_stride + static_cast<long long>(row_a) * p.o_row_stride + head * HD;
        __nv_bfloat16* orow_b = orow_a + 8 * p.o_row_stride;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          uint32_t o[32];
          __syncwarp();
          tmem_ld16x256(t_o + 64 * h, o);
          tmem_wait_ld(o);
          if (MASKED && run == 0 && any_nonfinite(o) && (edge_tile(0) || edge_tile(nkv - 1))) *again = 1u;
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const int col = 64 * h + 8 * q + 2 * t0;
            if (row_a < p.n_rows)
              *reinterpret_cast<uint32_t*>(orow_a + col) =
                  pack_bf16x2(__uint_as_float(o[4 * q]) * inv_a, __uint_as_float(o[4 * q + 1]) * inv_a);
            if (row_b < p.n_rows)
              *reinterpret_cast<uint32_t*>(orow_b + col) =
                  pack_bf16x2(__uint_as_float(o[4 * q + 2]) * inv_b, __uint_as_float(o[4 * q + 3]) * inv_b);
          }
        }
        if (p.lse != nullptr && t0 == 0) {
          float* lrow = p.lse + (static_cast<long long>(batch) * p.n_heads + head) * p.n_rows;
          // masked: without keys m = l = 0 and log 0 = -inf
          if (row_a < p.n_rows) lrow[row_a] = (m_a + __log2f(l_a)) * 0.69314718055994530942f;
          if (row_b < p.n_rows) lrow[row_b] = (m_b + __log2f(l_b)) * 0.69314718055994530942f;
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if constexpr (MASKED) {
    if (run == 1 || *again == 0u || *abort_flag != 0u) break;
    // second run: loads, products and waits of the first have ended; the commits
    // that nothing waited for arrive, then the barriers start over
    if (threadIdx.x == 0) {
      volatile uint32_t never = 0u;
      for (int s = 0; s < KV_STAGES; ++s) {
        const int uses = (2 * nkv - s + KV_STAGES - 1) / KV_STAGES;
        if (uses > 0) mbar_wait_bounded(bar_kv_empty(s), (uses - 1) & 1, &never, p.drain_limit_ns, eslot);
      }
      for (int i = 0; i < 2; ++i) mbar_wait_bounded(bar_pva_done(i), (nkv - 1) & 1, &never, p.drain_limit_ns, eslot);
      for (int i = 0; i < NUM_BARS; ++i) mbar_inval(bar0 + 8u * i);
      init_bars();
    }
    __syncthreads();
    tc_fence_after();
  }
  }
  if (MASKED && p.parts > 1) {
    float2* const ml = reinterpret_cast<float2*>(gbase + SMEM_ROW_ML);
    float* const factors = reinterpret_cast<float*>(gbase + SMEM_ROW_F);   // [parts][rows stored here]
    const int per = 2 * BM / p.parts;              // rows that each CTA stores
    if (nkv == 0) {
      for (int i = threadIdx.x; i < 2 * BM; i += THREADS) ml[i] = make_float2(-INFINITY, 0.f);
      if (warp == W_PROD && lane == 0) {           // Q's copies end here: nothing else waited for them
        volatile uint32_t never = 0u;
        for (int i = 0; i < 2; ++i) mbar_wait_bounded(bar_q_full(i), 0, &never, p.drain_limit_ns, eslot);
      }
    } else if (warp < SOFTMAX_WARPS) {
      const int wg = warp >> 3, t0 = lane & 3, t1 = lane >> 2;
      const int lane16 = 32 * (warp & 3) + 16 * ((warp >> 2) & 1);
      float* const to = reinterpret_cast<float*>(gbase) + (wg * BM + lane16 + t1) * MERGE_STRIDE + 2 * t0;
      tc_fence_after();
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        uint32_t o[32];
        __syncwarp();
        tmem_ld16x256(tmem + (static_cast<uint32_t>(lane16) << 16) + TMEM_O0 + wg * 128 + 64 * h, o);
        tmem_wait_ld(o);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          *reinterpret_cast<uint2*>(to + 64 * h + 8 * q) = make_uint2(o[4 * q], o[4 * q + 1]);
          *reinterpret_cast<uint2*>(to + 8 * MERGE_STRIDE + 64 * h + 8 * q) = make_uint2(o[4 * q + 2], o[4 * q + 3]);
        }
      }
      tc_fence_before();
    }
    __syncwarp();
    cluster_sync();                                // every part's O, m and l are there
    if (threadIdx.x < per) {
      const int row = part * per + threadIdx.x;
      float2 v[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = q < p.parts ? ld_dsmem(base + SMEM_ROW_ML + row * 8, q) : make_float2(-INFINITY, 0.f);
      float m = -INFINITY, l = 0.f;
#pragma unroll
      for (int q = 0; q < 8; ++q) m = fmaxf(m, v[q].x);
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (v[q].y != 0.f) l += v[q].y * ex2_approx(v[q].x - m);   // a part that saw no key of the row has l = 0
      const int2 r = reinterpret_cast<const int2*>(gbase + SMEM_RANGES)[row];
      const float inv = r.x >= r.y ? 0.f : 1.f / l;
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (q < p.parts) factors[q * per + threadIdx.x] = v[q].y != 0.f ? inv * ex2_approx(v[q].x - m) : -1.f;
      if (p.lse != nullptr && q_row0 + row < p.n_rows)
        p.lse[(static_cast<long long>(batch) * p.n_heads + head) * p.n_rows + q_row0 + row] =
            (m + __log2f(l)) * 0.69314718055994530942f;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < per * (HD / 4); i += THREADS) {
      const int r = i / (HD / 4), c = 4 * (i % (HD / 4)), row = q_row0 + part * per + r;
      if (row >= p.n_rows) continue;
      const uint32_t at = base + static_cast<uint32_t>(((part * per + r) * MERGE_STRIDE + c) * 4);
      float4 v[8];
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (q < p.parts) v[q] = ld_dsmem4(at, q);
      float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float f = q < p.parts ? factors[q * per + r] : -1.f;
        if (f == -1.f) continue;                   // nothing seen there (an O of zeros, or none at all)
        sum.x = fmaf(v[q].x, f, sum.x);
        sum.y = fmaf(v[q].y, f, sum.y);
        sum.z = fmaf(v[q].z, f, sum.z);
        sum.w = fmaf(v[q].w, f, sum.w);
      }
      *reinterpret_cast<uint2*>(p.o + batch * p.o_batch_stride + static_cast<long long>(row) * p.o_row_stride + head * HD +
                                c) = make_uint2(pack_bf16x2(sum.x, sum.y), pack_bf16x2(sum.z, sum.w));
    }
    __syncwarp();
    cluster_sync();                                // no CTA ends while another reads its rows
  }
  if (warp == W_MMA) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

}  // namespace attn
}  // namespace h3
