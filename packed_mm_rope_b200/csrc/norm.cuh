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
// All of it is HBM-bound: every row is read once (x, and dy backward), held in
// registers as it was stored (16-byte chunks of 8 elements, two for fp32) and
// written once.  Statistics and sums are fp32, in two passes over the
// registers (mean, then squared deviations), so a large mean costs no digits.
// A row belongs to a group of G threads: one warp for short rows, 128 to 512
// threads for long ones; thread t holds chunks t, t + G, ...  The column sums
// of the weight gradient stay in the threads' registers over all rows that a
// group walks and leave once as a partial row; a second kernel adds the
// partials in a fixed order, so results do not depend on scheduling.
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

// Group (block, g) takes rows group, group + groups, ... and leaves its column
// sums in partial row `group` of `partials` [groups][2][hidden].  dx may be dy or
// x (a group has read its whole row before it writes any of it).
template <typename T, typename P, bool VEC, int G, int CH>
__global__ void __launch_bounds__(G > THREADS ? G : THREADS) layernorm_backward_kernel(
    const T* dy, const T* x, const float* __restrict__ mean, const float* __restrict__ rstd,
    const P* __restrict__ weight, T* dx, float* __restrict__ partials, long long n_rows, int hidden,
    long long dy_stride, long long x_stride, long long dx_stride) {
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

// Sums over the partial rows first, first + 1, ... < last of `partials`
// [..][2][hidden] for column sets of 32: eight thread rows take every eighth
// partial each, in order, and are added in order.  `half` 0: dw, 1: db.
constexpr int REDUCE_ROWS = 8;
__device__ __forceinline__ float reduce_partials(const float* __restrict__ partials, long long first, long long last,
                                                 int half, int hidden, int col, float (*buf)[32]) {
  const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
  float s = 0.f;
  if (col < hidden) {
    const float* p = partials + half * static_cast<long long>(hidden) + col;
#pragma unroll 4
    for (long long i = first + row; i < last; i += REDUCE_ROWS) s += __ldcs(p + i * 2 * hidden);
  }
  buf[row][lane] = s;
  __syncthreads();
  float total = 0.f;
  if (row == 0) {
#pragma unroll
    for (int q = 0; q < REDUCE_ROWS; ++q) total += buf[q][lane];
  }
  return total;
}

template <typename P>
__global__ void __launch_bounds__(32 * REDUCE_ROWS) norm_reduce_kernel(const float* __restrict__ partials,
                                                                       int n_partials, int hidden, P* dweight,
                                                                       P* dbias) {
  __shared__ float buf[REDUCE_ROWS][32];
  const int col = blockIdx.x * 32 + (threadIdx.x & 31);
  P* out = blockIdx.y == 0 ? dweight : dbias;
  if (out == nullptr) return;
  const float s = reduce_partials(partials, 0, n_partials, blockIdx.y, hidden, col, buf);
  if (threadIdx.x < 32 && col < hidden) out[col] = from_float<P>(s);
}

// ------------------------------------------- AdaLN backward: row sorting ----

// The table's gradient sums over the rows of each entry, and rows of one entry
// may lie anywhere.  Rows are first put in the order of their entries (stable,
// so sums do not depend on scheduling): blocks of SORT_ROWS rows count their
// entries, then every block finds where its rows of each entry begin and places
// them.  Rows whose entry is out of range go to one more bucket at the end.
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

// d_table[e][0] = sum of dy (shift), [e][1] = sum of dy xhat (scale)
__global__ void __launch_bounds__(32 * REDUCE_ROWS) adaln_reduce_kernel(const float* __restrict__ partials,
                                                                        const int* __restrict__ starts, long long per,
                                                                        int hidden, float* __restrict__ dtable) {
  __shared__ float buf[REDUCE_ROWS][32];
  const int col = blockIdx.x * 32 + (threadIdx.x & 31);
  const int e = blockIdx.y >> 1, half = blockIdx.y & 1;
  const long long a = starts[e], b = starts[e + 1];
  const long long c0 = a / per, c1 = b > a ? (b - 1) / per + 1 : c0;   // groups with rows of entry e
  const float s = reduce_partials(partials, c0 + e, c1 + e, half, hidden, col, buf);
  if (threadIdx.x < 32 && col < hidden)
    dtable[(2LL * e + (half == 0 ? 1 : 0)) * hidden + col] = s;
}

}  // namespace norm
}  // namespace h3
