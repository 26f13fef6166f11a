// norm.cuh -- layer norm forward and backward, and the backward pass of the
// per-row AdaLN modulation.
//
// Forward, per row of C elements:
//   mean = sum x / C, var = sum (x - mean)^2 / C, rstd = 1 / sqrt(var + eps),
//   xhat = (x - mean) rstd, y = xhat w + b.
// Backward, with g = dy w:
//   dx = rstd (g - mean(g) - xhat mean(g xhat)), dw = sum_rows dy xhat,
//   db = sum_rows dy.
// AdaLN is the same norm with w = 1 + scale[e], b = shift[e] gathered per row,
// so its table gradient is dw, db summed over the rows of each entry e.
//
// All of it is HBM-bound: every row is read once (x, and dy backward) and written once.
// Short rows, and rows that are not 16-byte aligned, are held in registers as they
// were stored (chunks of 8 elements) by a group of G threads: one warp, or 128 to 512
// threads for long rows; thread t holds chunks t, t + G, ...  Aligned rows of 1,025 to
// 11,520 elements pass through rings of rows in shared memory instead (below).
// Statistics and sums are fp32: first the mean, then the squared deviations from it, so
// the variance loses nothing to a large mean.  xhat does: the mean is rounded to fp32, so
// it is off by 2^-24 |mean| / deviation, and the ring kernels, which form xhat as
// x rstd - mean rstd and dx as x B + C, add two or three roundings of that size.
// The column sums of the weight gradient stay in the threads' registers over all rows
// that a group walks and leave once as a partial row; a second kernel adds the
// partials in a fixed order, so results do not depend on scheduling.
//
// Measured at 28,196 x 5,376 bf16 (a copy runs at 6.47 TB/s): forward 105 us, 5.8 TB/s;
// layer norm's gradients 143 us, 6.3 TB/s, and 5 us for the partials; AdaLN's 158 us,
// 5.8 TB/s (4,584 rows 35 us), 9 us for the sorting and 6 us for the partials.
#pragma once

#include <cuda_fp16.h>

#include "adaln.cuh"
#include "common.cuh"

namespace h3 {
namespace norm {

constexpr int THREADS = 256;
constexpr int MAX_HIDDEN = 16384;

// ------------------------------------------------------------- elements ----

// Eight consecutive elements of a row, as stored.
template <typename T>
struct Chunk {
  static constexpr int W = sizeof(T) * 2;   // 32-bit words
  uint32_t w[W];
};

__device__ __forceinline__ float2 unpack2(uint32_t w, const __nv_bfloat16*) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ float2 unpack2(uint32_t w, const __half*) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
__device__ __forceinline__ uint32_t pack2(float2 v, const __nv_bfloat16*) { return pack_bf16x2(v.x, v.y); }
__device__ __forceinline__ uint32_t pack2(float2 v, const __half*) {
  const __half2 h = __floats2half2_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// elements 2 m and 2 m + 1 of a chunk
template <typename T>
__device__ __forceinline__ float2 pair_of(const Chunk<T>& c, int m) {
  if constexpr (sizeof(T) == 4)
    return make_float2(__uint_as_float(c.w[2 * m]), __uint_as_float(c.w[2 * m + 1]));
  else
    return unpack2(c.w[m], static_cast<const T*>(nullptr));
}
template <typename T>
__device__ __forceinline__ void set_pair(Chunk<T>& c, int m, float2 v) {
  if constexpr (sizeof(T) == 4) {
    c.w[2 * m] = __float_as_uint(v.x);
    c.w[2 * m + 1] = __float_as_uint(v.y);
  } else {
    c.w[m] = pack2(v, static_cast<const T*>(nullptr));
  }
}

// Chunk at column `col` of a row.  VEC: the row is 16-byte aligned and its
// length a multiple of 8; otherwise element by element, zero past the end.
template <typename T, bool VEC>
__device__ __forceinline__ Chunk<T> load_chunk(const T* row, int col, int hidden) {
  Chunk<T> c;
  if constexpr (VEC) {
    const uint4* p = reinterpret_cast<const uint4*>(row + col);
#pragma unroll
    for (int i = 0; i < Chunk<T>::W / 4; ++i) {
      const uint4 u = __ldcs(p + i);
      c.w[4 * i] = u.x;
      c.w[4 * i + 1] = u.y;
      c.w[4 * i + 2] = u.z;
      c.w[4 * i + 3] = u.w;
    }
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 8; ++i) c.w[i] = col + i < hidden ? reinterpret_cast<const uint32_t*>(row)[col + i] : 0u;
  } else {
    const uint16_t* p = reinterpret_cast<const uint16_t*>(row);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = col + 2 * i < hidden ? p[col + 2 * i] : 0u;
      const uint32_t hi = col + 2 * i + 1 < hidden ? p[col + 2 * i + 1] : 0u;
      c.w[i] = lo | (hi << 16);
    }
  }
  return c;
}
template <typename T, bool VEC>
__device__ __forceinline__ void store_chunk(T* row, int col, int hidden, const Chunk<T>& c) {
  if constexpr (VEC) {
    uint4* p = reinterpret_cast<uint4*>(row + col);
#pragma unroll
    for (int i = 0; i < Chunk<T>::W / 4; ++i)
      __stcs(p + i, make_uint4(c.w[4 * i], c.w[4 * i + 1], c.w[4 * i + 2], c.w[4 * i + 3]));
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (col + i < hidden) reinterpret_cast<uint32_t*>(row)[col + i] = c.w[i];
  } else {
    uint16_t* p = reinterpret_cast<uint16_t*>(row);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (col + i < hidden) p[col + i] = static_cast<uint16_t>(c.w[i >> 1] >> (16 * (i & 1)));
  }
}

// Parameter elements 8 c .. 8 c + 7 as fp32 pairs (missing: `fill`).  The
// parameters are read again for every row, so they come through the caches.
template <typename P, bool VEC>
__device__ __forceinline__ void load_param(const P* w, int col, int hidden, float fill, float2 (&v)[4]) {
  if (w == nullptr) {
#pragma unroll
    for (int m = 0; m < 4; ++m) v[m] = make_float2(fill, fill);
  } else if constexpr (VEC) {
    Chunk<P> c;
    const uint4* p = reinterpret_cast<const uint4*>(w + col);
#pragma unroll
    for (int i = 0; i < Chunk<P>::W / 4; ++i) {
      const uint4 u = __ldg(p + i);
      c.w[4 * i] = u.x;
      c.w[4 * i + 1] = u.y;
      c.w[4 * i + 2] = u.z;
      c.w[4 * i + 3] = u.w;
    }
#pragma unroll
    for (int m = 0; m < 4; ++m) v[m] = pair_of(c, m);
  } else {
    const Chunk<P> c = load_chunk<P, false>(w, col, hidden);
#pragma unroll
    for (int m = 0; m < 4; ++m) v[m] = pair_of(c, m);
  }
}

template <typename P>
__device__ __forceinline__ P from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }

// ----------------------------------------------------------- reductions ----

// Sum of N values over the G threads of a group.  One warp: shuffles alone.
// Several: the warps' partials meet in shared memory behind one named barrier;
// `buf` alternates between two halves, so that a value still being read is
// never overwritten by the next reduction.
template <int G, int N>
struct GroupSum {
  static constexpr int WARPS = G / 32;
  float (*buf)[N][WARPS];   // [2][N][WARPS] of this group
  int bar;                  // named barrier of this group
  int parity;

  __device__ __forceinline__ void operator()(float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
    if constexpr (WARPS > 1) {
      const int wq = (threadIdx.x % G) >> 5;
      if ((threadIdx.x & 31) == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) buf[parity][i][wq] = v[i];
      }
      asm volatile("bar.sync %0, %1;" ::"r"(bar), "n"(G) : "memory");
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float s = 0.f;
#pragma unroll
        for (int q = 0; q < WARPS; ++q) s += buf[parity][i][q];
        v[i] = s;
      }
      parity ^= 1;
    }
  }
};

template <typename T, int CH>
__device__ __forceinline__ float local_sum(const Chunk<T> (&x)[CH]) {
  float2 s = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < CH; ++i)
#pragma unroll
    for (int m = 0; m < 4; ++m) s = __fadd2_rn(s, pair_of(x[i], m));
  return s.x + s.y;
}

// Squared deviations from `mean` of this thread's elements that are inside the row.
template <typename T, bool VEC, int G, int CH>
__device__ __forceinline__ float local_sq(const Chunk<T> (&x)[CH], float mean, int t, int chunks, int hidden) {
  const float2 nm = make_float2(-mean, -mean);
  float2 s = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = t + G * i;
    if (c >= chunks) continue;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      float2 d = __fadd2_rn(pair_of(x[i], m), nm);
      if constexpr (!VEC) {   // elements past the end were loaded as zeros
        if (8 * c + 2 * m >= hidden) d.x = 0.f;
        if (8 * c + 2 * m + 1 >= hidden) d.y = 0.f;
      }
      s = __ffma2_rn(d, d, s);
    }
  }
  return s.x + s.y;
}

// -------------------------------------------------------------- forward ----

template <typename T, typename P, bool VEC, int G, int CH>
__global__ void __launch_bounds__(G > THREADS ? G : THREADS) layernorm_kernel(
    const T* x, T* y, const P* __restrict__ weight, const P* __restrict__ bias, float* __restrict__ mean_out,
    float* __restrict__ rstd_out, long long n_rows, int hidden, long long x_stride, long long y_stride, float eps) {
  begin_after_predecessor(x, weight, bias);
  constexpr int BLOCK = G > THREADS ? G : THREADS;
  constexpr int GROUPS = BLOCK / G;
  __shared__ float buf[GROUPS][2][1][G / 32];
  const int g = threadIdx.x / G, t = threadIdx.x % G;
  const int chunks = (hidden + 7) / 8;
  const float n = static_cast<float>(hidden);
  GroupSum<G, 1> sum{buf[g], 1 + g, 0};
  for (long long r = static_cast<long long>(blockIdx.x) * GROUPS + g; r < n_rows;
       r += static_cast<long long>(gridDim.x) * GROUPS) {
    const T* xr = x + r * x_stride;
    Chunk<T> u[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if (t + G * i < chunks) {
        u[i] = load_chunk<T, VEC>(xr, 8 * (t + G * i), hidden);
      } else {
#pragma unroll
        for (int k = 0; k < Chunk<T>::W; ++k) u[i].w[k] = 0u;
      }
    }
    float s[1] = {local_sum<T, CH>(u)};
    sum(s);
    const float mean = s[0] / n;
    s[0] = local_sq<T, VEC, G, CH>(u, mean, t, chunks, hidden);
    sum(s);
    const float rstd = 1.f / sqrtf(s[0] / n + eps);
    if (t == 0) {
      if (mean_out != nullptr) mean_out[r] = mean;
      if (rstd_out != nullptr) rstd_out[r] = rstd;
    }
    T* yr = y + r * y_stride;
    const float2 rs = make_float2(rstd, rstd), nm = make_float2(-mean, -mean);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = t + G * i;
      if (c >= chunks) continue;
      float2 w[4], b[4];
      load_param<P, VEC>(weight, 8 * c, hidden, 1.f, w);
      load_param<P, VEC>(bias, 8 * c, hidden, 0.f, b);
      Chunk<T> o;
#pragma unroll
      for (int m = 0; m < 4; ++m)
        set_pair(o, m, __ffma2_rn(__fmul2_rn(__fadd2_rn(pair_of(u[i], m), nm), rs), w[m], b[m]));
      store_chunk<T, VEC>(yr, 8 * c, hidden, o);
    }
  }
}

// ------------------------------------------------------------- backward ----

// One row of the backward pass: from the row's x and dy in registers, its
// statistics and its weight w(c, out), writes dx and adds dy xhat and dy to the
// column sums.
template <typename T, bool VEC, int G, int CH, typename WFn>
__device__ __forceinline__ void backward_row(const Chunk<T> (&ux)[CH], const Chunk<T> (&ud)[CH], float mean, float rstd,
                                             WFn weight, GroupSum<G, 2>& sum, T* dxr, int t, int chunks, int hidden,
                                             float2 (&dw)[CH][4], float2 (&db)[CH][4]) {
  const float2 rs = make_float2(rstd, rstd), nm = make_float2(-mean, -mean);
  float2 a1 = make_float2(0.f, 0.f), a2 = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = t + G * i;
    if (c >= chunks) continue;
    float2 w[4];
    weight(c, w);
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const float2 d = pair_of(ud[i], m);   // zero past the row's end
      const float2 xh = __fmul2_rn(__fadd2_rn(pair_of(ux[i], m), nm), rs);
      const float2 gg = __fmul2_rn(d, w[m]);
      a1 = __fadd2_rn(a1, gg);
      a2 = __ffma2_rn(gg, xh, a2);
      dw[i][m] = __ffma2_rn(d, xh, dw[i][m]);
      db[i][m] = __fadd2_rn(db[i][m], d);
    }
  }
  float s[2] = {a1.x + a1.y, a2.x + a2.y};
  sum(s);
  const float inv_n = 1.f / static_cast<float>(hidden);
  const float2 c1 = make_float2(-s[0] * inv_n, -s[0] * inv_n), c2 = make_float2(-s[1] * inv_n, -s[1] * inv_n);
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = t + G * i;
    if (c >= chunks) continue;
    float2 w[4];
    weight(c, w);
    Chunk<T> o;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const float2 xh = __fmul2_rn(__fadd2_rn(pair_of(ux[i], m), nm), rs);
      const float2 v = __ffma2_rn(xh, c2, __ffma2_rn(pair_of(ud[i], m), w[m], c1));
      set_pair(o, m, __fmul2_rn(v, rs));
    }
    store_chunk<T, VEC>(dxr, 8 * c, hidden, o);
  }
}

template <typename T, bool VEC, int G, int CH>
__device__ __forceinline__ void load_row(const T* row, int t, int chunks, int hidden, Chunk<T> (&u)[CH]) {
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    if (t + G * i < chunks) {
      u[i] = load_chunk<T, VEC>(row, 8 * (t + G * i), hidden);
    } else {
#pragma unroll
      for (int k = 0; k < Chunk<T>::W; ++k) u[i].w[k] = 0u;
    }
  }
}

// Column sums of a group -> one partial row of the workspace, [dw, db][hidden].
template <int G, int CH>
__device__ __forceinline__ void store_partial(float* out, int t, int chunks, int hidden, const float2 (&dw)[CH][4],
                                              const float2 (&db)[CH][4]) {
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = t + G * i;
    if (c >= chunks) continue;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int col = 8 * c + 2 * m;
      if (col < hidden) out[col] = dw[i][m].x, out[hidden + col] = db[i][m].x;
      if (col + 1 < hidden) out[col + 1] = dw[i][m].y, out[hidden + col + 1] = db[i][m].y;
    }
  }
}

// The same for hidden a multiple of 8.
template <int G, int CH>
__device__ __forceinline__ void store_partial_chunks(float* out, int t, int chunks, int hidden, const float2 (&dw)[CH][4],
                                                     const float2 (&db)[CH][4]) {
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = t + G * i;
    if (c >= chunks) continue;
    float4* w = reinterpret_cast<float4*>(out) + 2 * c;
    float4* b = reinterpret_cast<float4*>(out + hidden) + 2 * c;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      w[m] = make_float4(dw[i][2 * m].x, dw[i][2 * m].y, dw[i][2 * m + 1].x, dw[i][2 * m + 1].y);
      b[m] = make_float4(db[i][2 * m].x, db[i][2 * m].y, db[i][2 * m + 1].x, db[i][2 * m + 1].y);
    }
  }
}

// Group (block, g) takes rows group, group + groups, ... and leaves its column
// sums in partial row `group` of `partials` [groups][2][hidden].  dx may be dy or
// x (a group has read its whole row before it writes any of it).
template <typename T, typename P, bool VEC, int G, int CH>
__global__ void __launch_bounds__(G > THREADS ? G : THREADS) layernorm_backward_kernel(
    const T* dy, const T* x, const float* __restrict__ mean, const float* __restrict__ rstd,
    const P* __restrict__ weight, T* dx, float* __restrict__ partials, long long n_rows, int hidden,
    long long dy_stride, long long x_stride, long long dx_stride) {
  begin_after_predecessor(dy, x, mean, rstd, weight);
  constexpr int BLOCK = G > THREADS ? G : THREADS;
  constexpr int GROUPS = BLOCK / G;
  __shared__ float buf[GROUPS][2][2][G / 32];
  const int g = threadIdx.x / G, t = threadIdx.x % G;
  const int chunks = (hidden + 7) / 8;
  GroupSum<G, 2> sum{buf[g], 1 + g, 0};
  float2 dw[CH][4], db[CH][4];
#pragma unroll
  for (int i = 0; i < CH; ++i)
#pragma unroll
    for (int m = 0; m < 4; ++m) dw[i][m] = db[i][m] = make_float2(0.f, 0.f);
  auto weight_of = [&](int c, float2 (&w)[4]) { load_param<P, VEC>(weight, 8 * c, hidden, 1.f, w); };
  const long long group = static_cast<long long>(blockIdx.x) * GROUPS + g;
  for (long long r = group; r < n_rows; r += static_cast<long long>(gridDim.x) * GROUPS) {
    Chunk<T> ux[CH], ud[CH];
    load_row<T, VEC, G, CH>(x + r * x_stride, t, chunks, hidden, ux);
    load_row<T, VEC, G, CH>(dy + r * dy_stride, t, chunks, hidden, ud);
    backward_row<T, VEC, G, CH>(ux, ud, mean[r], rstd[r], weight_of, sum, dx + r * dx_stride, t, chunks, hidden, dw,
                                db);
  }
  if (partials != nullptr) store_partial<G, CH>(partials + group * 2 * hidden, t, chunks, hidden, dw, db);
}

// ------------------------------------------------------- rings of rows ----

// Long aligned rows: a block of G threads with CH chunks of a row each takes R rows
// at a time.  One more warp copies rows into a ring of shared memory (bulk copies),
// so reads from HBM go on while the block reduces and writes, and every pass reads
// the rows from there, so that a thread's registers hold its parameters and column
// sums for all rows.  A block is bound by the latency of its reductions; R rows share
// one reduction, and two blocks per SM hide each other's.
constexpr int MAX_SLOTS = 4;
constexpr unsigned long long RING_DRAIN_NS = 2000000000ull;

struct RingAt {             // slot and phase of a step
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int slots) {
    if (++slot == slots) slot = 0, phase ^= 1u;
  }
};

struct Ring {
  uint32_t full, empty;     // mbarriers, one per slot each
  uint32_t data;            // shared address of slot 0
  uint32_t row_bytes;       // of one row of one tensor
  uint32_t slot_bytes;      // R rows of each tensor: [tensor][R][row]
  int slots;
  volatile uint32_t* abort;
  unsigned long long limit;
  int err_slot;

  __device__ __forceinline__ void init(int consumer_warps) const {
    for (int s = 0; s < slots; ++s) {
      mbar_init(full + 8u * s, 1);
      mbar_init(empty + 8u * s, consumer_warps);
    }
    mbar_fence_init();
  }
  // Consumers: whether the step has landed (bounded wait); its slot is free again.
  __device__ __forceinline__ bool wait(RingAt at) const {
    return mbar_wait_exact(full + 8u * at.slot, at.phase, abort, limit, err_slot);
  }
  __device__ __forceinline__ void release(RingAt at) const {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(empty + 8u * at.slot);
  }
  // Producer thread: steps 0 .. count - 1 of rows(i) rows each; src(tensor, i, r)
  // names row r of step i.  Ends when every copy has landed.
  template <int R, int TENSORS, typename Rows, typename Src>
  __device__ __forceinline__ void produce(int count, Rows rows, Src src) const {
    RingAt at;
    int issued = 0;
    for (; issued < count; ++issued, at.next(slots)) {
      if (issued >= slots && !mbar_wait_exact(empty + 8u * at.slot, at.phase ^ 1u, abort, limit, err_slot)) break;
      const uint32_t bar = full + 8u * at.slot, to = data + at.slot * slot_bytes;
      const int n = rows(issued);
      mbar_arrive_expect_tx(bar, n * TENSORS * row_bytes);
      for (int r = 0; r < n; ++r)
#pragma unroll
        for (int t = 0; t < TENSORS; ++t) bulk_load(to + (t * R + r) * row_bytes, src(t, issued, r), row_bytes, bar);
    }
    volatile uint32_t never = 0u;
    for (int i = issued > slots ? issued - slots : 0; i < issued; ++i)
      mbar_wait_bounded(full + 8u * (i % slots), (i / slots) & 1, &never, RING_DRAIN_NS, err_slot);
  }
};

constexpr int pow2_of(int n) { return n <= 1 ? 1 : 2 * pow2_of((n + 1) / 2); }

// Sums of N values over the G consumer threads; returns whether `fail` holds in any
// of them (all take the same way out).  Each warp halves the number of values a lane
// carries in the first shuffles, so N values take about N + 4 of them, not 5 N; the
// warps' partials meet in `buf` [2][values][warps] (two sets in turn) behind one
// barrier and every warp adds them up with lanes side by side.
template <int G, int N>
struct BlockSum {
  static constexpr int M = pow2_of(N);             // values, padded
  static constexpr int W = G / 32;
  static constexpr int WP = pow2_of(W);            // warps, padded
  static constexpr int PER = 32 / WP;              // values that the lanes add up at once
  static constexpr int SIZE = 2 * M * WP;

  // Where in a set a lane finds its partial of values g PER .. g PER + PER - 1, or -1:
  // with fewer values than lanes to add them up, or a padded number of warps, the
  // others would read beyond the set, into the one that the next sum is written to.
  static __host__ __device__ constexpr int source(int g, int lane) {
    const int value = g * PER + lane / WP, warp = lane % WP;
    return value < N && warp < W ? value * WP + warp : -1;
  }

  static __device__ __forceinline__ bool sum(float (&v)[N], float* buf, int& parity, bool fail) {
    const int lane = threadIdx.x & 31;
    float a[M];
#pragma unroll
    for (int i = 0; i < M; ++i) a[i] = i < N ? v[i] : 0.f;
    int offset = 16;
#pragma unroll
    for (int width = M; width > 1; width /= 2, offset /= 2) {
      const bool upper = (lane & offset) != 0;
#pragma unroll
      for (int i = 0; i < width / 2; ++i) {
        const float send = upper ? a[i] : a[i + width / 2];
        a[i] = (upper ? a[i + width / 2] : a[i]) + __shfl_xor_sync(0xffffffffu, send, offset);
      }
    }
#pragma unroll
    for (; offset > 0; offset /= 2) a[0] += __shfl_xor_sync(0xffffffffu, a[0], offset);
    float* const set = buf + parity * (M * WP);
    if ((lane & (32 / M - 1)) == 0) set[(lane / (32 / M)) * WP + (threadIdx.x >> 5)] = a[0];
    uint32_t any;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(any)
        : "r"(fail ? 1u : 0u), "n"(G)
        : "memory");
#pragma unroll
    for (int g = 0; g < (N + PER - 1) / PER; ++g) {
      const int from = source(g, lane);
      float s = from >= 0 ? set[from] : 0.f;
#pragma unroll
      for (int o = WP / 2; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (g * PER + i < N) v[g * PER + i] = PER == 1 ? s : __shfl_sync(0xffffffffu, s, i * WP);
    }
    parity ^= 1;
    return any != 0u;
  }
};

// Chunk c of a row in shared memory.
template <typename T>
__device__ __forceinline__ Chunk<T> ring_chunk(const uint8_t* row, int c) {
  Chunk<T> u;
#pragma unroll
  for (int k = 0; k < Chunk<T>::W / 4; ++k) {
    const uint4 v = *reinterpret_cast<const uint4*>(row + c * static_cast<int>(sizeof(Chunk<T>)) + 16 * k);
    u.w[4 * k] = v.x;
    u.w[4 * k + 1] = v.y;
    u.w[4 * k + 2] = v.z;
    u.w[4 * k + 3] = v.w;
  }
  return u;
}

// Means of R rows in shared memory.  Returns the verdict on `fail`.
template <typename T, int G, int CH, int R>
__device__ __forceinline__ bool ring_means(const uint8_t* rows, uint32_t row_bytes, int chunks, float inv_n, float* buf,
                                           int& parity, bool fail, float (&mean)[R]) {
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = threadIdx.x + G * i;
      if (c >= chunks) continue;
      const Chunk<T> u = ring_chunk<T>(rows + r * row_bytes, c);
#pragma unroll
      for (int m = 0; m < 4; ++m) s = __fadd2_rn(s, pair_of(u, m));
    }
    mean[r] = s.x + s.y;
  }
  const bool failed = BlockSum<G, R>::sum(mean, buf, parity, fail);
#pragma unroll
  for (int r = 0; r < R; ++r) mean[r] *= inv_n;
  return failed;
}

// Their rstd, from squared deviations.
template <typename T, int G, int CH, int R>
__device__ __forceinline__ void ring_rstds(const uint8_t* rows, uint32_t row_bytes, int chunks, float inv_n, float eps,
                                           float* buf, int& parity, const float (&mean)[R], float (&rstd)[R]) {
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const float2 nm = make_float2(-mean[r], -mean[r]);
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = threadIdx.x + G * i;
      if (c >= chunks) continue;
      const Chunk<T> u = ring_chunk<T>(rows + r * row_bytes, c);
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const float2 d = __fadd2_rn(pair_of(u, m), nm);
        s = __ffma2_rn(d, d, s);
      }
    }
    rstd[r] = s.x + s.y;
  }
  BlockSum<G, R>::sum(rstd, buf, parity, false);
#pragma unroll
  for (int r = 0; r < R; ++r) rstd[r] = rsqrtf(fmaf(rstd[r], inv_n, eps));
}

// The blocks take sets of R rows in turn: set i of this block starts at row(i).
template <int R>
struct RowSets {
  long long n_rows;
  __device__ __forceinline__ int count() const {
    return static_cast<int>(((n_rows + R - 1) / R - blockIdx.x + gridDim.x - 1) / gridDim.x);
  }
  __device__ __forceinline__ long long row(int i) const {
    return (blockIdx.x + static_cast<long long>(i) * gridDim.x) * R;
  }
  __device__ __forceinline__ int rows(int i) const {
    const long long left = n_rows - row(i);
    return left < R ? static_cast<int>(left) : R;
  }
};

template <typename T, typename P, int G, int CH, int R, int MINB>
__global__ void __launch_bounds__(G + 32, MINB) layernorm_ring_kernel(
    const T* x, T* y, const P* __restrict__ weight, const P* __restrict__ bias, float* __restrict__ mean_out,
    float* __restrict__ rstd_out, long long n_rows, int hidden, long long x_stride, long long y_stride, float eps,
    int slots, unsigned long long limit, int err_slot) {
  begin_after_predecessor(x, weight, bias);
  extern __shared__ __align__(128) uint8_t rows[];
  __shared__ uint64_t bars[2 * MAX_SLOTS];
  __shared__ uint32_t abort_word;
  __shared__ float buf[BlockSum<G, R>::SIZE];
  const int t = threadIdx.x, chunks = hidden / 8;
  const uint32_t row_bytes = static_cast<uint32_t>(hidden * sizeof(T));
  const Ring ring{smem_u32(bars), smem_u32(bars + MAX_SLOTS), smem_u32(rows), row_bytes, R * row_bytes, slots,
                  &abort_word, limit, err_slot};
  const RowSets<R> sets{n_rows};
  if (t == 0) {
    abort_word = 0u;
    ring.init(G / 32);
  }
  __syncthreads();
  if (t >= G) {
    if (t == G)
      ring.produce<R, 1>(sets.count(), [&](int i) { return sets.rows(i); },
                         [&](int, int i, int r) { return x + (sets.row(i) + r) * x_stride; });
    return;
  }
  const float inv_n = 1.f / static_cast<float>(hidden);
  float2 w[CH][4], b[CH][4];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    if (t + G * i < chunks) {
      load_param<P, true>(weight, 8 * (t + G * i), hidden, 1.f, w[i]);
      load_param<P, true>(bias, 8 * (t + G * i), hidden, 0.f, b[i]);
    }
  }
  int parity = 0;
  RingAt at;
  for (int i = 0, count = sets.count(); i < count; ++i, at.next(slots)) {
    const bool landed = ring.wait(at);
    const uint8_t* in = rows + at.slot * ring.slot_bytes;
    float mean[R], rstd[R];
    if (ring_means<T, G, CH, R>(in, row_bytes, chunks, inv_n, buf, parity, !landed, mean)) break;
    ring_rstds<T, G, CH, R>(in, row_bytes, chunks, inv_n, eps, buf, parity, mean, rstd);
    const long long r0 = sets.row(i);
    const int n = sets.rows(i);
    T* out = y + r0 * y_stride;
#pragma unroll
    for (int r = 0; r < R; ++r, out += y_stride) {
      if (r >= n) continue;
      if (t == 0) {
        if (mean_out != nullptr) mean_out[r0 + r] = mean[r];
        if (rstd_out != nullptr) rstd_out[r0 + r] = rstd[r];
      }
      const float2 rs = make_float2(rstd[r], rstd[r]), nm = make_float2(-mean[r], -mean[r]);
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const int c = t + G * k;
        if (c >= chunks) continue;
        const Chunk<T> u = ring_chunk<T>(in + r * row_bytes, c);
        Chunk<T> o;
#pragma unroll
        for (int m = 0; m < 4; ++m)
          set_pair(o, m, __ffma2_rn(__fmul2_rn(__fadd2_rn(pair_of(u, m), nm), rs), w[k][m], b[k][m]));
        store_chunk<T, true>(out, 8 * c, hidden, o);
      }
    }
    ring.release(at);
  }
}

// R rows of a backward pass, x and dy in shared memory (`at`, `at_d`): their
// statistics are known and their weight is in registers.  Rows of the bit set
// `active` get their dx (dst(r)) and add to the column sums.  Returns the verdict on
// `fail`.  With xhat = x rstd - mean rstd the row's result is
//   dx = (dy w) rstd + x B + C,  B = -mean(g xhat) rstd^2,  C = -rstd (mean(g) + mean B / rstd).
template <typename T, int G, int CH, int R, typename Dst>
__device__ __forceinline__ bool ring_backward_rows(const uint8_t* at, const uint8_t* at_d, uint32_t row_bytes,
                                                   const float (&mean)[R], const float (&rstd)[R], unsigned active,
                                                   const float2 (&w)[CH][4], float inv_n, float* buf, int& parity,
                                                   bool fail, Dst dst, int chunks, int hidden, float2 (&dw)[CH][4],
                                                   float2 (&db)[CH][4]) {
  const int t = threadIdx.x;
  float s[2 * R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float2 a1 = make_float2(0.f, 0.f), a2 = make_float2(0.f, 0.f);
    if (active >> r & 1u) {
      const float mr = -mean[r] * rstd[r];
      const float2 rs = make_float2(rstd[r], rstd[r]), nm = make_float2(mr, mr);
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int c = t + G * i;
        if (c >= chunks) continue;
        const Chunk<T> ux = ring_chunk<T>(at + r * row_bytes, c), ud = ring_chunk<T>(at_d + r * row_bytes, c);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const float2 d = pair_of(ud, m);
          const float2 xh = __ffma2_rn(pair_of(ux, m), rs, nm);
          const float2 g = __fmul2_rn(d, w[i][m]);
          a1 = __fadd2_rn(a1, g);
          a2 = __ffma2_rn(g, xh, a2);
          dw[i][m] = __ffma2_rn(d, xh, dw[i][m]);
          db[i][m] = __fadd2_rn(db[i][m], d);
        }
      }
    }
    s[2 * r] = a1.x + a1.y;
    s[2 * r + 1] = a2.x + a2.y;
  }
  if (BlockSum<G, 2 * R>::sum(s, buf, parity, fail)) return true;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (!(active >> r & 1u)) continue;
    const float c2 = -s[2 * r + 1] * inv_n * rstd[r], cb = c2 * rstd[r];
    const float cc = fmaf(-mean[r], cb, -s[2 * r] * inv_n * rstd[r]);
    const float2 rs = make_float2(rstd[r], rstd[r]), b2 = make_float2(cb, cb), c = make_float2(cc, cc);
    T* dxr = dst(r);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int ch = t + G * i;
      if (ch >= chunks) continue;
      const Chunk<T> ux = ring_chunk<T>(at + r * row_bytes, ch), ud = ring_chunk<T>(at_d + r * row_bytes, ch);
      Chunk<T> o;
#pragma unroll
      for (int m = 0; m < 4; ++m)
        set_pair(o, m, __ffma2_rn(__fmul2_rn(pair_of(ud, m), w[i][m]), rs, __ffma2_rn(pair_of(ux, m), b2, c)));
      store_chunk<T, true>(dxr, 8 * ch, hidden, o);
    }
  }
  return false;
}

// Layer norm's gradients by rings of (x, dy) rows; partial row blockIdx.
template <typename T, typename P, int G, int CH, int R, int MINB>
__global__ void __launch_bounds__(G + 32, MINB) layernorm_backward_ring_kernel(
    const T* dy, const T* x, const float* __restrict__ mean, const float* __restrict__ rstd,
    const P* __restrict__ weight, T* dx, float* __restrict__ partials, long long n_rows, int hidden,
    long long dy_stride, long long x_stride, long long dx_stride, int slots, unsigned long long limit, int err_slot) {
  begin_after_predecessor(dy, x, mean, rstd, weight);
  extern __shared__ __align__(128) uint8_t rows[];
  __shared__ uint64_t bars[2 * MAX_SLOTS];
  __shared__ uint32_t abort_word;
  __shared__ float buf[BlockSum<G, 2 * R>::SIZE];
  const int t = threadIdx.x, chunks = hidden / 8;
  const uint32_t row_bytes = static_cast<uint32_t>(hidden * sizeof(T));
  const Ring ring{smem_u32(bars), smem_u32(bars + MAX_SLOTS), smem_u32(rows), row_bytes, 2 * R * row_bytes, slots,
                  &abort_word, limit, err_slot};
  const RowSets<R> sets{n_rows};
  if (t == 0) {
    abort_word = 0u;
    ring.init(G / 32);
  }
  __syncthreads();
  if (t >= G) {
    if (t == G)
      ring.produce<R, 2>(sets.count(), [&](int i) { return sets.rows(i); }, [&](int tensor, int i, int r) {
        const long long row = sets.row(i) + r;
        return tensor == 0 ? x + row * x_stride : dy + row * dy_stride;
      });
    return;
  }
  const float inv_n = 1.f / static_cast<float>(hidden);
  float2 w[CH][4], dw[CH][4], db[CH][4];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
#pragma unroll
    for (int m = 0; m < 4; ++m) dw[i][m] = db[i][m] = make_float2(0.f, 0.f);
    if (t + G * i < chunks) load_param<P, true>(weight, 8 * (t + G * i), hidden, 1.f, w[i]);
  }
  int parity = 0;
  RingAt at;
  for (int i = 0, count = sets.count(); i < count; ++i, at.next(slots)) {
    const int n = sets.rows(i);
    const long long r0 = sets.row(i);
    float m[R], s[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      m[r] = r < n ? mean[r0 + r] : 0.f;
      s[r] = r < n ? rstd[r0 + r] : 0.f;
    }
    const bool landed = ring.wait(at);
    const uint8_t* in = rows + at.slot * ring.slot_bytes;
    if (ring_backward_rows<T, G, CH, R>(in, in + R * row_bytes, row_bytes, m, s, (1u << n) - 1u, w, inv_n, buf, parity,
                                        !landed, [&](int r) { return dx + (r0 + r) * dx_stride; }, chunks, hidden, dw,
                                        db))
      break;
    ring.release(at);
  }
  if (partials != nullptr)
    store_partial_chunks<G, CH>(partials + static_cast<long long>(blockIdx.x) * 2 * hidden, t, chunks, hidden, dw, db);
}

// ------------------------------------------------- sums of partial rows ----

// Sums over the partial rows first .. last - 1 of `partials` [..][dw, db][hidden].
// A block takes 64 x W columns: 64 threads side by side, ROWS such rows of threads
// take every ROWS-th partial, in order, and their sums are added in order.  Few
// partials per sum want few rows and W = 4, many want many rows and, where one sum is
// all there is, W = 1 for more blocks.
template <int ROWS, int W, typename Store>
__device__ __forceinline__ void reduce_partials(const float* __restrict__ partials, long long first, long long last,
                                                int half, int hidden, Store store) {
  __shared__ float buf[ROWS][64][W];
  const int lane = threadIdx.x & 63, row = threadIdx.x >> 6;
  const int col = (blockIdx.x * 64 + lane) * W;
  float s[W] = {};
  if (col < hidden) {
    const float* p = partials + half * static_cast<long long>(hidden) + col;
#pragma unroll 4
    for (long long i = first + row; i < last; i += ROWS) {
      if constexpr (W == 4) {
        const float4 v = __ldcs(reinterpret_cast<const float4*>(p + i * 2 * hidden));
        s[0] += v.x;
        s[1] += v.y;
        s[2] += v.z;
        s[3] += v.w;
      } else {
        s[0] += __ldcs(p + i * 2 * hidden);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < W; ++k) buf[row][lane][k] = s[k];
  __syncthreads();
  if (row != 0 || col >= hidden) return;
#pragma unroll
  for (int k = 0; k < W; ++k) {
    float total = s[k];
#pragma unroll
    for (int q = 1; q < ROWS; ++q) total += buf[q][lane][k];
    store(col + k, total);
  }
}

template <typename P>
__global__ void __launch_bounds__(64 * 16) norm_reduce_kernel(const float* __restrict__ partials, int n_partials,
                                                                int hidden, P* dweight, P* dbias) {
  begin_after_predecessor(partials);
  P* out = blockIdx.y == 0 ? dweight : dbias;
  if (out == nullptr) return;
  reduce_partials<16, 1>(partials, 0, n_partials, blockIdx.y, hidden,
                           [&](int col, float v) { out[col] = from_float<P>(v); });
}

// ------------------------------------------- AdaLN backward: row sorting ----

// The table's gradient sums over the rows of each entry, and rows of one entry
// may lie anywhere.  Rows are first put in the order of their entries (stable,
// so sums do not depend on scheduling): blocks of SORT_ROWS rows count their
// entries, then every block finds where its rows of each entry begin and places
// them.  Rows whose entry is out of range go to one more bucket at the end.  Latency
// alone: 2.3 and 6.5 us at 28,196 rows.
constexpr int SORT_ROWS = 1024;
constexpr int MAX_ENTRIES = 8192;      // the counts of one block in shared memory

__device__ __forceinline__ int entry_of(const int32_t* ts, const int32_t* tags, long long r, int n_entries) {
  const long long e = static_cast<long long>(ts[r]) * 3 + tags[r];
  return e < 0 || e >= n_entries ? n_entries : static_cast<int>(e);
}

// hist [blocks][n_entries + 1]
__global__ void __launch_bounds__(SORT_ROWS) adaln_count_kernel(const int32_t* __restrict__ ts,
                                                                const int32_t* __restrict__ tags, int n_entries,
                                                                long long n_rows, int* __restrict__ hist,
                                                                int err_slot) {
  begin_after_predecessor(ts, tags);
  extern __shared__ int counts[];
  for (int e = threadIdx.x; e <= n_entries; e += SORT_ROWS) counts[e] = 0;
  __syncthreads();
  const long long r = static_cast<long long>(blockIdx.x) * SORT_ROWS + threadIdx.x;
  if (r < n_rows) {
    const int e = entry_of(ts, tags, r, n_entries);
    if (e == n_entries) raise_error(err_slot, DEVERR_INPUT);
    atomicAdd(&counts[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e <= n_entries; e += SORT_ROWS)
    hist[static_cast<long long>(blockIdx.x) * (n_entries + 1) + e] = counts[e];
}

// order[position] = (row, entry); starts[e] = first position of entry e (n_entries + 2 values)
__global__ void __launch_bounds__(SORT_ROWS) adaln_place_kernel(const int32_t* __restrict__ ts,
                                                                const int32_t* __restrict__ tags, int n_entries,
                                                                long long n_rows, const int* __restrict__ hist,
                                                                int n_blocks, int2* __restrict__ order,
                                                                int* __restrict__ starts) {
  begin_after_predecessor(ts, tags, hist);
  extern __shared__ int base[];            // [n_entries + 1]: where this block's rows of the entry go
  __shared__ int warp_total[SORT_ROWS / 32];
  __shared__ int carry;
  const int ne = n_entries + 1;
  const int lane = threadIdx.x & 31, wq = threadIdx.x >> 5;
  if (threadIdx.x == 0) carry = 0;
  __syncthreads();
  // exclusive scan over the entries of their totals, 1024 entries at a time
  for (int e0 = 0; e0 < ne; e0 += SORT_ROWS) {
    const int e = e0 + threadIdx.x;
    int total = 0, before = 0;
    if (e < ne)
      for (int b = 0; b < n_blocks; ++b) {
        const int v = hist[static_cast<long long>(b) * ne + e];
        total += v;
        if (b < static_cast<int>(blockIdx.x)) before += v;
      }
    int incl = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) warp_total[wq] = incl;
    __syncthreads();
    int off = carry;
    for (int q = 0; q < wq; ++q) off += warp_total[q];
    const int first = off + incl - total;
    if (e < ne) {
      base[e] = first + before;
      if (blockIdx.x == 0) starts[e] = first;
    }
    __syncthreads();
    if (threadIdx.x == SORT_ROWS - 1) carry = off + incl;
    __syncthreads();
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) starts[ne] = static_cast<int>(n_rows);
  // warps in turn, so that the rows of one entry keep their order
  const long long r = static_cast<long long>(blockIdx.x) * SORT_ROWS + threadIdx.x;
  const int e = r < n_rows ? entry_of(ts, tags, r, n_entries) : -1;
  const unsigned same = __match_any_sync(0xffffffffu, e);
  const int rank = __popc(same & ((1u << lane) - 1u));
  for (int q = 0; q < SORT_ROWS / 32; ++q) {
    if (q == wq && e >= 0) {
      order[base[e] + rank] = make_int2(static_cast<int>(r), e);
    }
    __syncwarp();
    if (q == wq && e >= 0 && rank == 0) base[e] += __popc(same);
    __syncthreads();
  }
}

// ------------------------------------------------- AdaLN backward: rows ----

// Group c takes the sorted positions [c per, (c + 1) per) and, whenever the
// entry changes, leaves the column sums of the rows just passed in partial row
// c + e.  Both c and e only grow along the positions, so c + e names each
// (group, entry) pair once and groups + entries rows hold all of them.  The
// statistics are recomputed from x, which is in registers anyway.
template <int G, int CH>
__global__ void __launch_bounds__(G > THREADS ? G : THREADS) adaln_backward_kernel(
    const __nv_bfloat16* dy, const __nv_bfloat16* x, const float* __restrict__ table, const int2* __restrict__ order,
    __nv_bfloat16* dx, float* __restrict__ partials, int n_entries, long long n_rows, long long per, int hidden,
    long long dy_stride, long long x_stride, long long dx_stride, float eps) {
  begin_after_predecessor(dy, x, table, order);
  using T = __nv_bfloat16;
  constexpr int BLOCK = G > THREADS ? G : THREADS;
  constexpr int GROUPS = BLOCK / G;
  __shared__ float buf1[GROUPS][2][1][G / 32];
  __shared__ float buf2[GROUPS][2][2][G / 32];
  const int g = threadIdx.x / G, t = threadIdx.x % G;
  const int chunks = hidden / 8;
  const float n = static_cast<float>(hidden);
  GroupSum<G, 1> sum1{buf1[g], 1 + g, 0};
  GroupSum<G, 2> sum2{buf2[g], 1 + g, 0};
  float2 dw[CH][4], db[CH][4];
  auto clear = [&] {
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int m = 0; m < 4; ++m) dw[i][m] = db[i][m] = make_float2(0.f, 0.f);
  };
  clear();
  const long long group = static_cast<long long>(blockIdx.x) * GROUPS + g;
  const long long first = group * per, last = first + per < n_rows ? first + per : n_rows;
  int entry = -1;
  for (long long pos = first; pos < last; ++pos) {
    const int2 o = order[pos];
    const long long r = o.x;
    if (o.y != entry) {
      if (entry >= 0 && entry < n_entries)
        store_partial<G, CH>(partials + (group + entry) * 2 * hidden, t, chunks, hidden, dw, db);
      entry = o.y;
      clear();
    }
    T* dxr = dx + r * dx_stride;
    if (entry == n_entries) {              // no such table entry: NaN, as the forward call gives
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const Chunk<T> nan = {{0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u}};
        if (t + G * i < chunks) store_chunk<T, true>(dxr, 8 * (t + G * i), hidden, nan);
      }
      continue;
    }
    Chunk<T> ux[CH], ud[CH];
    load_row<T, true, G, CH>(x + r * x_stride, t, chunks, hidden, ux);
    load_row<T, true, G, CH>(dy + r * dy_stride, t, chunks, hidden, ud);
    float s[1] = {local_sum<T, CH>(ux)};
    sum1(s);
    const float mean = s[0] / n;
    s[0] = local_sq<T, true, G, CH>(ux, mean, t, chunks, hidden);
    sum1(s);
    const float rstd = 1.f / sqrtf(s[0] / n + eps);
    const float* scale = table + (2LL * entry + 1) * hidden;
    auto weight_of = [&](int c, float2 (&w)[4]) {
      load_param<float, true>(scale, 8 * c, hidden, 0.f, w);
#pragma unroll
      for (int m = 0; m < 4; ++m) w[m] = __fadd2_rn(w[m], make_float2(1.f, 1.f));
    };
    backward_row<T, true, G, CH>(ux, ud, mean, rstd, weight_of, sum2, dxr, t, chunks, hidden, dw, db);
  }
  if (entry >= 0 && entry < n_entries)
    store_partial<G, CH>(partials + (group + entry) * 2 * hidden, t, chunks, hidden, dw, db);
}

// Long rows, one block of G + 32 (S + 1) threads per SM and group: a warp copies
// rows of x and dy into a ring of shared memory, S warps each take a whole row there
// and find its statistics, and G threads with CH chunks each turn rows into dx and
// column sums, with the entry's weights in registers while it lasts.  No step needs a
// barrier of the block: a row's statistics are shuffles of one warp, and rows pass
// from warp to warp by one mbarrier each way.  (With the block's barriers instead, as
// in the layer norm above, 28,196 x 5,376 took 218 us and not 158.)  What bounds it is
// how many rows are on their way from memory while S of the ring's rows are read.
constexpr int ADALN_SLOTS = 10;

struct RowTerms {            // dx = (dy w) rstd + x b + c, xhat = x rstd + shift
  float rstd, shift, b, c;
};

// Table entries: read again for every row, to stay in the L1 cache.
__device__ __forceinline__ float4 load_kept(const float* p) {
  float4 v;
  asm volatile("ld.global.nc.L1::evict_last.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "l"(p));
  return v;
}
// Results: not to displace them there (28,196 x 5,376 172 -> 166 us, and room for a
// larger ring).
__device__ __forceinline__ void store_past_l1(__nv_bfloat16* p, const Chunk<__nv_bfloat16>& c) {
  asm volatile("st.global.L1::no_allocate.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(c.w[0]), "r"(c.w[1]),
               "r"(c.w[2]), "r"(c.w[3])
               : "memory");
}

// Terms of a row in shared memory by one warp; lane 0 holds the result.
__device__ __forceinline__ RowTerms adaln_row_terms(const uint8_t* x, const uint8_t* dy, const float* scale, int chunks,
                                                    float inv_n, float eps, int lane) {
  using T = __nv_bfloat16;
  // four sums side by side: a lane has up to 32 chunks of four pairs, and one chain of 128
  // additions would be off by up to that many roundings (mean of 8,192 elements)
  auto add_up = [](const float2 (&v)[4]) {
    const float2 t = __fadd2_rn(__fadd2_rn(v[0], v[1]), __fadd2_rn(v[2], v[3]));
    return t.x + t.y;
  };
  float2 s[4] = {};
#pragma unroll 4
  for (int c = lane; c < chunks; c += 32) {
    const Chunk<T> u = ring_chunk<T>(x, c);
#pragma unroll
    for (int m = 0; m < 4; ++m) s[m] = __fadd2_rn(s[m], pair_of(u, m));
  }
  float mean = add_up(s);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mean += __shfl_xor_sync(0xffffffffu, mean, o);
  mean *= inv_n;
  const float2 nm = make_float2(-mean, -mean);
  float2 a0[4] = {}, a1[4] = {}, a2[4] = {};       // (x - mean)^2, g, g (x - mean)
#pragma unroll 2
  for (int c = lane; c < chunks; c += 32) {
    const Chunk<T> ux = ring_chunk<T>(x, c), ud = ring_chunk<T>(dy, c);
    const float4 w0 = load_kept(scale + 8 * c), w1 = load_kept(scale + 8 * c + 4);
    const float2 w[4] = {{w0.x, w0.y}, {w0.z, w0.w}, {w1.x, w1.y}, {w1.z, w1.w}};
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const float2 xc = __fadd2_rn(pair_of(ux, m), nm), d = pair_of(ud, m);
      const float2 g = __ffma2_rn(d, w[m], d);
      a0[m] = __ffma2_rn(xc, xc, a0[m]);
      a1[m] = __fadd2_rn(a1[m], g);
      a2[m] = __ffma2_rn(g, xc, a2[m]);
    }
  }
  float var = add_up(a0), sg = add_up(a1), sgx = add_up(a2);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    var += __shfl_xor_sync(0xffffffffu, var, o);
    sg += __shfl_xor_sync(0xffffffffu, sg, o);
    sgx += __shfl_xor_sync(0xffffffffu, sgx, o);
  }
  RowTerms r;
  r.rstd = rsqrtf(fmaf(var, inv_n, eps));
  r.shift = -mean * r.rstd;
  r.b = -sgx * inv_n * r.rstd * r.rstd * r.rstd;
  r.c = fmaf(-mean, r.b, -sg * inv_n * r.rstd);
  return r;
}

template <int G, int CH, int S>
__global__ void __launch_bounds__(G + 32 * (S + 1), 1) adaln_backward_ring_kernel(
    const __nv_bfloat16* dy, const __nv_bfloat16* x, const float* __restrict__ table, const int2* __restrict__ order,
    __nv_bfloat16* dx, float* __restrict__ partials, int n_entries, long long n_rows, long long per, int hidden,
    long long dy_stride, long long x_stride, long long dx_stride, float eps, int slots, unsigned long long limit,
    int err_slot) {
  begin_after_predecessor(dy, x, table, order);
  using T = __nv_bfloat16;
  extern __shared__ __align__(128) uint8_t rows[];
  __shared__ uint64_t bars[3 * ADALN_SLOTS];
  __shared__ RowTerms terms[ADALN_SLOTS];
  __shared__ uint32_t abort_word;
  const int t = threadIdx.x, lane = t & 31, chunks = hidden / 8;
  const uint32_t row_bytes = static_cast<uint32_t>(hidden * sizeof(T)), ready = smem_u32(bars + 2 * ADALN_SLOTS);
  const Ring ring{smem_u32(bars), smem_u32(bars + ADALN_SLOTS), smem_u32(rows), row_bytes, 2 * row_bytes, slots,
                  &abort_word, limit, err_slot};
  const long long group = blockIdx.x, first = group * per;
  const long long last = first + per < n_rows ? first + per : n_rows;
  const int count = last > first ? static_cast<int>(last - first) : 0;
  order += first;
  if (t == 0) {
    abort_word = 0u;
    for (int s = 0; s < slots; ++s) mbar_init(ready + 8u * s, 1);
    ring.init(G / 32);
  }
  __syncthreads();
  if (t >= G + 32 * S) {
    if (lane == 0)
      ring.produce<1, 2>(count, [](int) { return 1; }, [&](int tensor, int i, int) {
        const long long row = order[i].x;
        return tensor == 0 ? x + row * x_stride : dy + row * dy_stride;
      });
    return;
  }
  const float inv_n = 1.f / static_cast<float>(hidden);
  if (t >= G) {
    const int warps = S < slots ? S : slots, mine = (t - G) >> 5;
    for (int i = mine; i < count && mine < warps; i += warps) {
      const RingAt at{i % slots, static_cast<uint32_t>(i / slots) & 1u};
      const int e = order[i].y;
      // the step before in this slot has to be over: copies may land out of order, and the
      // wait for a copy tells two phases of its slot apart, not three
      if (i >= slots && !__all_sync(0xffffffffu, mbar_wait_bounded(ring.empty + 8u * at.slot, at.phase ^ 1u, &abort_word,
                                                                   limit, err_slot)))
        break;
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(ring.full + 8u * at.slot, at.phase, &abort_word, limit, err_slot)))
        break;
      const uint8_t* in = rows + at.slot * ring.slot_bytes;
      if (e < n_entries) {
        const RowTerms r =
            adaln_row_terms(in, in + row_bytes, table + (2LL * e + 1) * hidden, chunks, inv_n, eps, lane);
        if (lane == 0) terms[at.slot] = r;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(ready + 8u * at.slot);
    }
    return;
  }
  float2 w[CH][4], dw[CH][4], db[CH][4];
  auto clear = [&] {
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int m = 0; m < 4; ++m) dw[i][m] = db[i][m] = make_float2(0.f, 0.f);
  };
  clear();
  int entry = -1;
  int2 next = count > 0 ? order[0] : make_int2(0, 0);
  RingAt at;
  for (int i = 0; i < count; ++i, at.next(slots)) {
    const int2 here = next;                        // (row, entry)
    if (i + 1 < count) next = order[i + 1];
    if (here.y != entry) {
      if (entry >= 0 && entry < n_entries)
        store_partial_chunks<G, CH>(partials + (group + entry) * 2 * hidden, t, chunks, hidden, dw, db);
      entry = here.y;
      clear();
      if (entry < n_entries) {
#pragma unroll
        for (int k = 0; k < CH; ++k) {
          if (t + G * k >= chunks) continue;
          load_param<float, true>(table + (2LL * entry + 1) * hidden, 8 * (t + G * k), hidden, 0.f, w[k]);
#pragma unroll
          for (int m = 0; m < 4; ++m) w[k][m] = __fadd2_rn(w[k][m], make_float2(1.f, 1.f));
        }
      }
    }
    if (!__all_sync(0xffffffffu, mbar_wait_bounded(ready + 8u * at.slot, at.phase, &abort_word, limit, err_slot)))
      break;
    const uint8_t* in = rows + at.slot * ring.slot_bytes;
    T* out = dx + here.x * dx_stride;
    if (entry == n_entries) {              // no such table entry: NaN, as the forward call gives
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const Chunk<T> nan = {{0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u}};
        if (t + G * k < chunks) store_chunk<T, true>(out, 8 * (t + G * k), hidden, nan);
      }
    } else {
      const RowTerms r = terms[at.slot];
      const float2 rs = make_float2(r.rstd, r.rstd), nm = make_float2(r.shift, r.shift), b2 = make_float2(r.b, r.b);
      const float2 c0 = make_float2(r.c, r.c);
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const int c = t + G * k;
        if (c >= chunks) continue;
        const Chunk<T> ux = ring_chunk<T>(in, c), ud = ring_chunk<T>(in + row_bytes, c);
        Chunk<T> o;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const float2 xv = pair_of(ux, m), d = pair_of(ud, m);
          dw[k][m] = __ffma2_rn(d, __ffma2_rn(xv, rs, nm), dw[k][m]);
          db[k][m] = __fadd2_rn(db[k][m], d);
          set_pair(o, m, __ffma2_rn(__fmul2_rn(d, w[k][m]), rs, __ffma2_rn(xv, b2, c0)));
        }
        store_past_l1(out + 8 * c, o);
      }
    }
    ring.release(at);
  }
  if (entry >= 0 && entry < n_entries)
    store_partial_chunks<G, CH>(partials + (group + entry) * 2 * hidden, t, chunks, hidden, dw, db);
}

// d_table[e][0] = sum of dy (shift), [e][1] = sum of dy xhat (scale)
template <int ROWS>
__global__ void __launch_bounds__(64 * ROWS) adaln_reduce_kernel(const float* __restrict__ partials,
                                                                 const int* __restrict__ starts, long long per,
                                                                 int hidden, float* __restrict__ dtable) {
  begin_after_predecessor(partials, starts);
  const int e = blockIdx.y >> 1, half = blockIdx.y & 1;
  const long long a = starts[e], b = starts[e + 1];
  const long long c0 = a / per, c1 = b > a ? (b - 1) / per + 1 : c0;   // groups with rows of entry e
  float* out = dtable + (2LL * e + (half == 0 ? 1 : 0)) * hidden;
  reduce_partials<ROWS, 4>(partials, c0 + e, c1 + e, half, hidden, [&](int col, float v) { out[col] = v; });
}

}  // namespace norm
}  // namespace h3
