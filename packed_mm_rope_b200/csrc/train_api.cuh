// train_api.cuh -- host side of the training-direction calls and of the
// masked attention (declared in include/h3.h): argument checks, workspace
// layout and launches.  Included by h3.cu, whose helpers it uses.
#pragma once

namespace {

// Launches a kernel that begins with begin_after_predecessor(): it may be set up while
// the kernel before it in the stream still runs (about 2 us per launch), and reads and
// writes nothing until that one has ended.
template <typename... P, typename... A>
h3_status launch(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, A... args) {
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cuda_ok(cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...)) ? H3_OK : H3_ERR_CUDA;
}

inline uint64_t up256(uint64_t b) { return (b + 255u) & ~uint64_t(255u); }

inline bool aligned256(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }

int dtype_size(int32_t dtype) { return dtype == H3_DTYPE_F32 ? 4 : 2; }

bool valid_dtype(int32_t dtype) { return dtype == H3_DTYPE_BF16 || dtype == H3_DTYPE_F16 || dtype == H3_DTYPE_F32; }

// Whether rows of `stride` elements starting at p can be read 16 bytes at a time.
bool vector_rows(const void* p, int64_t stride, int32_t dtype) {
  return aligned16(p) && (stride * dtype_size(dtype)) % 16 == 0;
}

// Rows of `width` elements, `stride` elements apart.
struct RowSpan {
  const void* p;
  int64_t rows, stride, width;
  int size;                            // bytes of an element
};

// Whether two tensors share memory.  Columns of one buffer (equal strides) do not;
// overlapping spans with different strides count as shared.
bool overlap(const RowSpan& a, const RowSpan& b) {
  if (a.p == nullptr || b.p == nullptr || a.rows < 1 || b.rows < 1) return false;
  auto end = [](const RowSpan& r) {
    return reinterpret_cast<uintptr_t>(r.p) + static_cast<uint64_t>((r.rows - 1) * r.stride + r.width) * r.size;
  };
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  if (a0 >= end(b) || b0 >= end(a)) return false;
  const int64_t sa = (a.rows == 1 ? b.stride : a.stride) * a.size, sb = (b.rows == 1 ? a.stride : b.stride) * b.size;
  if (sa != sb || sa == 0) return true;
  const int64_t apart =
      a0 <= b0 ? static_cast<int64_t>((b0 - a0) % sa) : (sa - static_cast<int64_t>((a0 - b0) % sa)) % sa;
  return apart < a.width * a.size || sa - apart < b.width * b.size;
}

// For calls that may work in place: `out` is exactly `in`, or apart from it.
bool in_place_or_apart(const RowSpan& out, const RowSpan& in) {
  return (out.p == in.p && (out.stride == in.stride || out.rows == 1)) || !overlap(out, in);
}

template <typename T>
struct TypeTag {
  using type = T;
};
template <int V>
struct IntTag {
  static constexpr int value = V;
};

// Calls f with the types of (x dtype, parameter dtype); the parameters share
// x's type or are fp32.
template <typename F>
h3_status with_types(int32_t dtype, int32_t param_dtype, F f) {
  if (dtype == H3_DTYPE_F32) return f(TypeTag<float>{}, TypeTag<float>{});
  if (dtype == H3_DTYPE_BF16)
    return param_dtype == H3_DTYPE_F32 ? f(TypeTag<__nv_bfloat16>{}, TypeTag<float>{})
                                       : f(TypeTag<__nv_bfloat16>{}, TypeTag<__nv_bfloat16>{});
  return param_dtype == H3_DTYPE_F32 ? f(TypeTag<__half>{}, TypeTag<float>{})
                                     : f(TypeTag<__half>{}, TypeTag<__half>{});
}

// ---- layer norm ----

// Threads per row and chunks of 8 elements per thread, by the row's length.
template <int G_, int CH_>
struct RowShape {
  static constexpr int G = G_, CH = CH_;
  static constexpr int BLOCK = G > h3::norm::THREADS ? G : h3::norm::THREADS;
  static constexpr int GROUPS = BLOCK / G;
  // aligned rows of other lengths go to the ring kernels
  static constexpr bool ALIGNED = G * CH <= 128 || G * CH == 2048;
};

// Forward: a warp per row up to 1,024 elements, else 128 or 256 threads with
// up to 8 chunks each (rows that the ring kernels do not take).
template <typename F>
h3_status with_forward_shape(int hidden, F f) {
  const int chunks = (hidden + 7) / 8;
  if (chunks <= 32) return f(RowShape<32, 1>{});
  if (chunks <= 128) return f(RowShape<32, 4>{});
  if (chunks <= 512) return f(RowShape<128, 4>{});
  if (chunks <= 1024) return f(RowShape<128, 8>{});
  return f(RowShape<256, 8>{});
}

// Backward: a thread also holds 16 fp32 column sums per chunk, hence more
// threads per row with fewer chunks each.
template <typename F>
h3_status with_backward_shape(int hidden, F f) {
  const int chunks = (hidden + 7) / 8;
  if (chunks <= 32) return f(RowShape<32, 1>{});
  if (chunks <= 128) return f(RowShape<32, 4>{});
  if (chunks <= 512) return f(RowShape<256, 2>{});
  if (chunks <= 768) return f(RowShape<256, 3>{});
  if (chunks <= 1024) return f(RowShape<256, 4>{});
  return f(RowShape<512, 4>{});
}

// Ring kernels (aligned rows of more than 1,024 elements): G consumer threads with
// CH chunks each, CTAS blocks per SM.  With the producer warp a block has 256, 288
// or 512 threads: 224 consumers leave a thread 128 registers at two blocks per SM,
// which the backward kernels need (256 consumers spill: 208 against 156 us for layer
// norm's gradients at 28,196 x 5,376 bf16).
template <int G_, int CH_, int CTAS_>
struct RingShape {
  static constexpr int G = G_, CH = CH_, CTAS = CTAS_;
};

template <typename F>
h3_status with_forward_ring(int hidden, F f) {
  const int chunks = hidden / 8;
  if (chunks <= 256) return f(RingShape<256, 1, 2>{});
  if (chunks <= 512) return f(RingShape<256, 2, 2>{});
  if (chunks <= 768) return f(RingShape<256, 3, 2>{});
  if (chunks <= 960) return f(RingShape<480, 2, 1>{});
  return f(RingShape<480, 3, 1>{});
}

template <typename F>
h3_status with_backward_ring(int hidden, F f) {
  const int chunks = hidden / 8;
  if (chunks <= 224) return f(RingShape<224, 1, 2>{});
  if (chunks <= 448) return f(RingShape<224, 2, 2>{});
  if (chunks <= 672) return f(RingShape<224, 3, 2>{});
  if (chunks <= 960) return f(RingShape<480, 2, 1>{});
  return f(RingShape<480, 3, 1>{});
}

bool ring_takes(int hidden) { return hidden > 1024 && hidden <= 8 * 3 * 480; }

constexpr int kRingSms = 148;                    // SMs of a B200: sizes grids, and with them partial rows
constexpr uint64_t kRingSmem = 224u << 10;       // shared memory of an SM that its blocks share

// Rows per step (R) and slots of a ring: the most rows of `choices` with which every
// block gets several steps and two slots fit; `tensors` rows are read per row.
struct RingPlan {
  int rows, slots;
  long long blocks;
  size_t smem;
};

RingPlan ring_plan(int64_t n_rows, size_t row_bytes, int tensors, int ctas, std::initializer_list<int> choices) {
  const uint64_t budget = kRingSmem / ctas - (3u << 10);
  RingPlan p{1, 1, 0, 0};
  for (int r : choices)
    if (n_rows >= 2LL * r * ctas * kRingSms && 2u * r * tensors * row_bytes <= budget) p.rows = std::max(p.rows, r);
  const uint64_t slot = static_cast<uint64_t>(p.rows) * tensors * row_bytes;
  p.slots = static_cast<int>(std::min<uint64_t>(h3::norm::MAX_SLOTS, std::max<uint64_t>(1u, budget / slot)));
  p.smem = static_cast<size_t>(p.slots * slot);
  p.blocks = std::min<long long>(static_cast<long long>(ctas) * kRingSms, (n_rows + p.rows - 1) / p.rows);
  return p;
}

template <auto Kernel, typename... Args>
h3_status launch_ring(const RingPlan& plan, int threads, cudaStream_t s, Args... args) {
  // the opt-in to more than 48 KB of shared memory, once per kernel and device until h3_shutdown
  static std::atomic<uint32_t> done[64];
  int dev = 0;
  if (!cuda_ok(cudaGetDevice(&dev)) || dev < 0 || dev >= 64) return H3_ERR_CUDA;
  const uint32_t epoch = g_attr_epoch.load();
  if (done[dev].load() != epoch) {
    if (!cuda_ok(cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kRingSmem))))
      return H3_ERR_CUDA;
    done[dev].store(epoch);
  }
  return launch(Kernel, dim3(static_cast<unsigned>(plan.blocks)), threads, plan.smem, s, args...);
}

// Blocks of the plain backward row kernels (a partial row per group of each).
constexpr int kBackwardBlocks = 2 * kRingSms;

template <typename S>
long long backward_blocks(int64_t n_rows) {
  return std::min<long long>(kBackwardBlocks, (n_rows + S::GROUPS - 1) / S::GROUPS);
}

// Partial rows that the backward pass over n_rows rows leaves at most, by either kind of kernel.
long long backward_groups(int64_t n_rows, int hidden) {
  long long groups = 0;
  with_backward_shape(hidden, [&](auto shape) {
    using S = decltype(shape);
    groups = backward_blocks<S>(n_rows) * S::GROUPS;
    return H3_OK;
  });
  return ring_takes(hidden) ? std::max<long long>(groups, std::min<long long>(2LL * kRingSms, n_rows)) : groups;
}

// ---- AdaLN backward ----

// Threads that apply the rows' terms (see the kernel) and their chunks of a row.
template <typename F>
h3_status with_adaln_ring(int hidden, F f) {
  const int chunks = hidden / 8;
  if (chunks <= 224) return f(RingShape<224, 1, 1>{});
  if (chunks <= 448) return f(RingShape<224, 2, 1>{});
  if (chunks <= 672) return f(RingShape<224, 3, 1>{});
  return f(RingShape<352, 3, 1>{});
}

// Warps that find the terms of rows, and the ring's size: what it leaves of an SM's 256 KB
// caches the table entry that these warps read.  28,196 x 5,376: 4, 5, 6, 7 warps (with
// 150 KB) 184, 172, 172, 173 us; 6 warps with 129, 150, 172, 194, 215 KB, results stored past
// that cache, 175, 166, 161, 158, 212 us.
constexpr int kAdalnWarps = 6;
constexpr uint64_t kAdalnSmem = 200u << 10;

struct AdalnWork {
  long long groups, per;               // row groups, sorted positions per group
  int blocks;                          // sorting blocks
  uint64_t order, starts, hist, partials, bytes;   // offsets and total size
};

AdalnWork adaln_work(int64_t n_rows, int hidden, int32_t n_entries) {
  AdalnWork w;
  w.groups = std::max<long long>(1, backward_groups(n_rows, hidden));
  if (ring_takes(hidden))              // the rows are always aligned: one group per block of the ring kernel
    w.groups = std::max<long long>(1, std::min<long long>(kRingSms, n_rows));
  w.per = std::max<long long>(1, (n_rows + w.groups - 1) / w.groups);
  w.blocks = static_cast<int>((n_rows + h3::norm::SORT_ROWS - 1) / h3::norm::SORT_ROWS);
  w.order = 0;
  w.starts = up256(static_cast<uint64_t>(n_rows) * 8u);
  w.hist = w.starts + up256((static_cast<uint64_t>(n_entries) + 2u) * 4u);
  w.partials = w.hist + up256(static_cast<uint64_t>(w.blocks) * (static_cast<uint64_t>(n_entries) + 1u) * 4u);
  w.bytes = w.partials + up256((static_cast<uint64_t>(w.groups) + n_entries) * 2u * hidden * 4u);
  return w;
}

// ---- masked attention ----

// Sizes and strides of a masked attention problem; the strides of tensors that
// a call does not take are left out of `strides`.
h3_status check_attention(const h3_attn_shape* a, std::initializer_list<int64_t> q_strides,
                          std::initializer_list<int64_t> kv_strides) {
  if (a == nullptr || a->batch < 1 || a->n_heads < 1 || a->n_kv_heads < 1 || a->n_heads % a->n_kv_heads != 0 ||
      a->n_q < 0 || a->n_k < 0 || a->n_q >= (1ll << 31) || a->n_k >= (1ll << 31) || a->batch > 65535 ||
      a->n_heads > 65535 || !std::isfinite(a->softmax_scale))
    return H3_ERR_INVALID_ARG;
  if (a->head_dim != 128) return H3_ERR_UNSUPPORTED;
  h3_status st = H3_OK;
  auto check = [&](int64_t stride, int32_t heads) {
    if (stride < static_cast<int64_t>(heads) * 128) st = H3_ERR_INVALID_ARG;
    else if (stride % 8 != 0 && st == H3_OK) st = H3_ERR_UNSUPPORTED;
  };
  for (int64_t s : q_strides) check(s, a->n_heads);
  for (int64_t s : kv_strides) check(s, a->n_kv_heads);
  return st;
}

// Workspace of the backward call: (lse, D) per head and row, the rows'
// intervals, the hull of every query tile, each row count padded to tiles, and the
// sums of split walks.
struct AttentionWork {
  int n_qt, n_kt, parts;
  uint64_t rng, hull, partial, bytes;    // offsets and total size; the (lse, D) pairs come first
};

// Walks of key tiles are cut where there are fewer than two per SM (the dq blocks
// behind them fill up what two or more leave): into enough parts for that, of at
// least eight steps if every row sees every key.
constexpr long long kWalkBlocks = 2 * 148;
constexpr long long kWalkSteps = 8;

AttentionWork attention_work(const h3_attn_shape* a) {
  AttentionWork w;
  w.n_qt = static_cast<int>((a->n_q + h3::attn::BM - 1) / h3::attn::BM);
  w.n_kt = static_cast<int>((a->n_k + h3::attn::BN - 1) / h3::attn::BN);
  const long long walks = static_cast<long long>(w.n_kt) * a->n_kv_heads * a->batch;
  const long long steps = static_cast<long long>(w.n_qt) * (a->n_heads / a->n_kv_heads);
  w.parts = walks == 0 || walks >= kWalkBlocks
                ? 1
                : static_cast<int>(std::max(1LL, std::min((kWalkBlocks + walks - 1) / walks, steps / kWalkSteps)));
  const uint64_t rows = static_cast<uint64_t>(w.n_qt) * h3::attn::BM * a->batch;
  w.rng = up256(rows * a->n_heads * 8u);
  w.hull = w.rng + up256(rows * 8u);
  w.partial = w.hull + up256(static_cast<uint64_t>(w.n_qt) * a->batch * 16u);
  w.bytes = w.partial + 256u +
            (w.parts > 1 ? static_cast<uint64_t>(w.parts) * walks * 2u * h3::attn::BN * h3::attn::HD * 4u : 0u);
  return w;
}

// CTAs that share a block's keys (a cluster): where SMs would stay idle, as many as
// still run all at once, if each has two key tiles when every row sees every key.  What
// that gains depends on the walks, shared against not: 18 key tiles x 1 head (8 parts)
// 21.4 / 39.8 us, x 8 heads (2 parts) 30.6 / 40.5; 9 tiles x 1 (4) 19.0 / 24.8, x 8 (2)
// 23.6 / 25.3; 6 tiles x 8 (2) 18.3 / 19.8; 4 tiles x 8 (2) 16.9 / 16.6.  Only n_k is known
// here, so masks may leave less: 95 documents of 80 rows, walks of up to 4 tiles cut in
// four, 18.3 / 21.0; 30 of 256 rows x 2 heads, walks of 2 tiles cut in two, 16.3 / 14.1.
// Halving walks for the sake of balance alone, with one to two blocks per SM, does not
// pay: 7,660 rows in documents x 8 heads 181 against 158 us.
int attention_parts(uint64_t blocks, int64_t n_k) {
  const int64_t tiles = (n_k + h3::attn::BN - 1) / h3::attn::BN;
  int parts = 1;
  while (parts < 8 && blocks * 2 * parts <= 148 && tiles >= 4 * parts) parts *= 2;
  return parts;
}

RowSpan q_rows(const h3_attn_shape* a, const void* p, int64_t stride) {
  return {p, a->batch * a->n_q, stride, a->n_heads * 128LL, 2};
}

RowSpan kv_rows(const h3_attn_shape* a, const void* p, int64_t stride) {
  return {p, a->batch * a->n_k, stride, a->n_kv_heads * 128LL, 2};
}

float attention_scale(const h3_attn_shape* a) {
  return a->softmax_scale > 0.f ? a->softmax_scale : 1.0f / std::sqrt(128.0f);
}

}  // namespace

extern "C" {

h3_status h3_build_key_ranges(const int32_t* d_doc_starts, const int32_t* d_prefix, int32_t n_docs, int64_t n_rows,
                              int32_t mode, int32_t* d_ranges, void* stream) {
  if (n_docs < 0 || n_rows < 0 || n_rows >= (1ll << 31) ||
      (mode != H3_MASK_DOCUMENT && mode != H3_MASK_PREFIX_CAUSAL && mode != H3_MASK_PREFIX_BLOCK))
    return H3_ERR_INVALID_ARG;
  if (!d_doc_starts || (n_rows > 0 && !d_ranges)) return H3_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(d_ranges) & 7u) return H3_ERR_UNSUPPORTED;
  const long long need = (std::max<long long>(n_rows, n_docs + 1LL) + 255) / 256;
  const int grid = static_cast<int>(std::min<long long>(need, 8LL * sm_count()));
  return launch(h3::key_ranges_kernel, dim3(grid), 256, 0, as_stream(stream), d_doc_starts, d_prefix, n_docs,
                static_cast<int>(n_rows), mode, reinterpret_cast<int2*>(d_ranges), error_slot(stream));
}

h3_status h3_masked_attention(const void* d_q, const void* d_k, const void* d_v, void* d_o, float* d_lse,
                              const int32_t* d_ranges, const h3_attn_shape* a, int64_t q_stride, int64_t k_stride,
                              int64_t v_stride, int64_t o_stride, void* stream) {
  const h3_status st = check_attention(a, {q_stride, o_stride}, {k_stride, v_stride});
  if (st != H3_OK || a->n_q == 0) return st;
  if (!d_q || !d_o || !d_ranges || (a->n_k > 0 && (!d_k || !d_v))) return H3_ERR_INVALID_ARG;
  if (!aligned16(d_q) || !aligned16(d_k) || !aligned16(d_v) || !aligned16(d_o) ||
      (reinterpret_cast<uintptr_t>(d_ranges) & 7u))
    return H3_ERR_UNSUPPORTED;
  const RowSpan out = q_rows(a, d_o, o_stride);
  if (overlap(out, q_rows(a, d_q, q_stride)) || overlap(out, kv_rows(a, d_k, k_stride)) ||
      overlap(out, kv_rows(a, d_v, v_stride)))
    return H3_ERR_INVALID_ARG;
  CUtensorMap tq, tk, tv;
  if (!make_qkv_map(&tq, d_q, a->batch, a->n_q, a->n_heads, q_stride, 128)) return H3_ERR_CUDA;
  tk = tv = tq;                          // without keys every row is empty and K, V are never read
  if (a->n_k > 0 && (!make_qkv_map(&tk, d_k, a->batch, a->n_k, a->n_kv_heads, k_stride, 128) ||
                     !make_qkv_map(&tv, d_v, a->batch, a->n_k, a->n_kv_heads, v_stride, 128)))
    return H3_ERR_CUDA;
  if (device_state() == nullptr) return H3_ERR_CUDA;
  h3::attn::Params p{};
  p.n_rows = static_cast<int>(a->n_q);
  p.n_heads = a->n_heads;
  p.n_keys = static_cast<int>(a->n_k);
  p.group = a->n_heads / a->n_kv_heads;
  p.ranges = reinterpret_cast<const int2*>(d_ranges);
  p.scale_log2 = attention_scale(a) * 1.4426950408889634f;
  p.o = static_cast<__nv_bfloat16*>(d_o);
  p.o_row_stride = o_stride;
  p.o_batch_stride = o_stride * a->n_q;
  p.lse = d_lse;
  p.wait_limit_ns = g_wait_limit_ns.load();
  p.drain_limit_ns = kDrainLimitNs;
  p.err_slot = error_slot(stream);
  const uint64_t blocks = static_cast<uint64_t>((a->n_q + 2 * h3::attn::BM - 1) / (2 * h3::attn::BM)) *
                          static_cast<uint64_t>(a->n_heads) * static_cast<uint64_t>(a->batch);
  p.parts = attention_parts(blocks, a->n_k);
  if (blocks * p.parts >= (1ull << 31)) return H3_ERR_INVALID_ARG;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks * p.parts));
  cfg.blockDim = dim3(h3::attn::THREADS);
  cfg.dynamicSmemBytes = h3::attn::MASKED_SMEM_BYTES;
  cfg.stream = as_stream(stream);
  cudaLaunchAttribute attrs[2];
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // as launch()
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim.x = static_cast<unsigned>(p.parts);
  attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
  cfg.attrs = attrs;
  cfg.numAttrs = p.parts > 1 ? 2 : 1;
  return cuda_ok(cudaLaunchKernelEx(&cfg, h3::attn::attention_kernel<true>, tq, tk, tv, p)) ? H3_OK : H3_ERR_CUDA;
}

uint64_t h3_masked_attention_backward_workspace_bytes(const h3_attn_shape* a) {
  if (check_attention(a, {}, {}) != H3_OK) return 0;
  return attention_work(a).bytes;
}

h3_status h3_masked_attention_backward(const void* d_do, const void* d_q, const void* d_k, const void* d_v,
                                       const void* d_o, const float* d_lse, const int32_t* d_ranges, void* d_dq,
                                       void* d_dk, void* d_dv, void* d_work, const h3_attn_shape* a,
                                       const h3_attn_strides* st, void* stream) {
  if (st == nullptr) return H3_ERR_INVALID_ARG;
  const h3_status check = check_attention(a, {st->dout, st->q, st->o, st->dq}, {st->k, st->v, st->dk, st->dv});
  if (check != H3_OK) return check;
  const bool queries = a->n_q > 0, keys = a->n_k > 0;
  if (queries && (!d_do || !d_q || !d_o || !d_lse || !d_ranges || !d_dq)) return H3_ERR_INVALID_ARG;
  if (keys && (!d_k || !d_v || !d_dk || !d_dv)) return H3_ERR_INVALID_ARG;
  if (!d_work || !aligned256(d_work)) return H3_ERR_INVALID_ARG;
  for (const void* ptr : {d_do, d_q, d_k, d_v, d_o, static_cast<const void*>(d_dq), static_cast<const void*>(d_dk),
                          static_cast<const void*>(d_dv)})
    if (!aligned16(ptr)) return H3_ERR_UNSUPPORTED;
  if (reinterpret_cast<uintptr_t>(d_ranges) & 7u) return H3_ERR_UNSUPPORTED;
  const RowSpan ins[] = {q_rows(a, d_do, st->dout), q_rows(a, d_q, st->q), q_rows(a, d_o, st->o),
                         kv_rows(a, d_k, st->k), kv_rows(a, d_v, st->v)};
  const RowSpan outs[] = {q_rows(a, d_dq, st->dq), kv_rows(a, d_dk, st->dk), kv_rows(a, d_dv, st->dv)};
  for (int i = 0; i < 3; ++i) {
    for (const RowSpan& in : ins)
      if (overlap(outs[i], in)) return H3_ERR_INVALID_ARG;
    if (overlap(outs[i], outs[(i + 1) % 3])) return H3_ERR_INVALID_ARG;
  }
  if (!queries && !keys) return H3_OK;
  cudaStream_t s = as_stream(stream);
  if (!queries) {                          // no row reads the keys
    const size_t rows = static_cast<size_t>(a->batch) * a->n_k, width = static_cast<size_t>(a->n_kv_heads) * 256u;
    return cuda_ok(cudaMemset2DAsync(d_dk, static_cast<size_t>(st->dk) * 2u, 0, width, rows, s)) &&
                   cuda_ok(cudaMemset2DAsync(d_dv, static_cast<size_t>(st->dv) * 2u, 0, width, rows, s))
               ? H3_OK
               : H3_ERR_CUDA;
  }
  CUtensorMap tq, tk, tv, tdo;
  if (!make_qkv_map(&tq, d_q, a->batch, a->n_q, a->n_heads, st->q, 128) ||
      !make_qkv_map(&tdo, d_do, a->batch, a->n_q, a->n_heads, st->dout, 128))
    return H3_ERR_CUDA;
  tk = tv = tq;                            // without keys every row is empty and K, V are never read
  if (keys && (!make_qkv_map(&tk, d_k, a->batch, a->n_k, a->n_kv_heads, st->k, 128) ||
               !make_qkv_map(&tv, d_v, a->batch, a->n_k, a->n_kv_heads, st->v, 128)))
    return H3_ERR_CUDA;
  if (device_state() == nullptr) return H3_ERR_CUDA;
  const AttentionWork w = attention_work(a);
  const uint64_t blocks = static_cast<uint64_t>(w.n_kt) * w.parts * a->n_kv_heads * a->batch +
                          static_cast<uint64_t>(w.n_qt) * a->n_heads * a->batch;
  if (blocks >= (1ull << 31)) return H3_ERR_INVALID_ARG;
  uint8_t* base = static_cast<uint8_t*>(d_work);
  h3::attn_bwd::Params p{};
  p.n_q = static_cast<int>(a->n_q);
  p.n_k = static_cast<int>(a->n_k);
  p.n_heads = a->n_heads;
  p.group = a->n_heads / a->n_kv_heads;
  p.n_qt = w.n_qt;
  p.scale = attention_scale(a);
  p.scale_log2 = p.scale * 1.4426950408889634f;
  float2* stat = reinterpret_cast<float2*>(base);
  int2* rng = reinterpret_cast<int2*>(base + w.rng);
  int4* hull = reinterpret_cast<int4*>(base + w.hull);
  p.stat = stat;
  p.rng = rng;
  p.hull = hull;
  p.dq = static_cast<__nv_bfloat16*>(d_dq);
  p.dk = static_cast<__nv_bfloat16*>(d_dk);
  p.dv = static_cast<__nv_bfloat16*>(d_dv);
  p.dq_stride = st->dq;
  p.dk_stride = st->dk;
  p.dv_stride = st->dv;
  p.n_kv_heads = a->n_kv_heads;
  p.n_kt = w.n_kt;
  p.batch = a->batch;
  p.parts = w.parts;
  p.partial = reinterpret_cast<float*>(base + w.partial);
  p.wait_limit_ns = g_wait_limit_ns.load();
  p.drain_limit_ns = kDrainLimitNs;
  p.err_slot = error_slot(stream);
  const unsigned batch = static_cast<unsigned>(a->batch), heads = static_cast<unsigned>(a->n_heads);
  const h3::attn_bwd::PrepInputs in{static_cast<const __nv_bfloat16*>(d_q),
                                    static_cast<const __nv_bfloat16*>(d_k),
                                    static_cast<const __nv_bfloat16*>(d_v),
                                    st->q,
                                    st->k,
                                    st->v,
                                    p.group,
                                    p.scale_log2};
  h3_status rc = launch(h3::attn_bwd::prep_kernel, dim3(w.n_qt, heads, batch), 256, 0, s, in,
                        static_cast<const __nv_bfloat16*>(d_o), static_cast<const __nv_bfloat16*>(d_do), d_lse,
                        reinterpret_cast<const int2*>(d_ranges), p.n_q, p.n_k, p.n_heads, w.n_qt, st->o, st->dout, stat,
                        rng, hull);
  if (rc == H3_OK)
    rc = launch(h3::attn_bwd::backward_kernel, dim3(static_cast<unsigned>(blocks)), h3::attn_bwd::THREADS,
                h3::attn_bwd::SMEM_BYTES, s, tq, tk, tv, tdo, p);
  if (rc == H3_OK && w.parts > 1)
    rc = launch(h3::attn_bwd::sum_parts_kernel, dim3(8 * sm_count()), 256, 0, s, p);
  return rc;
}

h3_status h3_mmrope_rotate(const void* d_q, const void* d_k, void* d_q_out, void* d_k_out, const float* d_coords,
                           int64_t n_rows, int32_t n_heads, int32_t n_kv_heads, int64_t q_stride, int64_t k_stride,
                           int64_t q_out_stride, int64_t k_out_stride, const h3_rope_cfg* cfg, int32_t inverse,
                           void* stream) {
  if (n_rows < 0 || n_heads < 0 || n_kv_heads < 0 || n_heads + static_cast<int64_t>(n_kv_heads) < 1 ||
      n_heads > 65535 || n_kv_heads > 65535 || !valid_rope_cfg(cfg) || (inverse != 0 && inverse != 1))
    return H3_ERR_INVALID_ARG;
  if (cfg->head_dim != 128) return H3_ERR_UNSUPPORTED;
  const int64_t q_row = static_cast<int64_t>(n_heads) * 128, k_row = static_cast<int64_t>(n_kv_heads) * 128;
  if (q_stride < q_row || q_out_stride < q_row || k_stride < k_row || k_out_stride < k_row) return H3_ERR_INVALID_ARG;
  if (n_rows == 0) return H3_OK;
  if ((n_heads > 0 && (!d_q || !d_q_out)) || (n_kv_heads > 0 && (!d_k || !d_k_out)) || !d_coords)
    return H3_ERR_INVALID_ARG;
  if ((q_stride | k_stride | q_out_stride | k_out_stride) % 8 != 0 || !aligned16(d_q) || !aligned16(d_k) ||
      !aligned16(d_q_out) || !aligned16(d_k_out))
    return H3_ERR_UNSUPPORTED;
  const RowSpan qi{d_q, n_rows, q_stride, q_row, 2}, ki{d_k, n_rows, k_stride, k_row, 2};
  const RowSpan qo{n_heads > 0 ? d_q_out : nullptr, n_rows, q_out_stride, q_row, 2};
  const RowSpan ko{n_kv_heads > 0 ? d_k_out : nullptr, n_rows, k_out_stride, k_row, 2};
  if (!in_place_or_apart(qo, qi) || !in_place_or_apart(ko, ki) || overlap(qo, ki) || overlap(ko, qi) ||
      overlap(qo, ko))
    return H3_ERR_INVALID_ARG;
  h3::RopeTable tab = make_rope_table(cfg);
  if (inverse)   // the rotation by -a: cos is even and sin odd, exactly
    for (double& f : tab.inv_freq) f = -f;
  h3::GroupedRope p;
  p.src[0] = static_cast<const uint4*>(d_q);
  p.src[1] = static_cast<const uint4*>(d_k);
  p.dst[0] = static_cast<uint4*>(d_q_out);
  p.dst[1] = static_cast<uint4*>(d_k_out);
  p.src_stride[0] = q_stride / 8;
  p.src_stride[1] = k_stride / 8;
  p.dst_stride[0] = q_out_stride / 8;
  p.dst_stride[1] = k_out_stride / 8;
  p.heads[0] = n_heads;
  p.heads[1] = n_kv_heads;
  const long long warps_per_cta = h3::ROPE_THREADS / 32;
  const long long nblk = (n_rows + warps_per_cta - 1) / warps_per_cta;
  auto go = [&](auto kernel, int ctas) {
    const long long grid = std::min<long long>(nblk, 2LL * ctas * sm_count());
    return launch(kernel, dim3(static_cast<unsigned>(grid)), h3::ROPE_THREADS, 0, as_stream(stream), p, d_coords,
                  n_rows, tab);
  };
  // up to 16 heads a lane has at most 8 chunks of a row
  if (n_heads + n_kv_heads <= 16)
    return cfg->pair_layout == 0 ? go(h3::rope_grouped_kernel<0, 4, 4>, 4) : go(h3::rope_grouped_kernel<1, 2, 4>, 4);
  return cfg->pair_layout == 0 ? go(h3::rope_grouped_kernel<0, 14, h3::ROPE_CTAS_PER_SM>, h3::ROPE_CTAS_PER_SM)
                               : go(h3::rope_grouped_kernel<1, 8, h3::ROPE_CTAS_PER_SM>, h3::ROPE_CTAS_PER_SM);
}

h3_status h3_layernorm(const void* d_x, void* d_y, const void* d_weight, const void* d_bias, float* d_mean,
                       float* d_rstd, int64_t n_rows, int32_t hidden, int64_t x_row_stride, int64_t y_row_stride,
                       int32_t dtype, int32_t param_dtype, float eps, void* stream) {
  if (n_rows < 0 || hidden < 1 || !(eps >= 0.f) || !std::isfinite(eps) || !valid_dtype(dtype) ||
      !valid_dtype(param_dtype))
    return H3_ERR_INVALID_ARG;
  if (x_row_stride < hidden || y_row_stride < hidden) return H3_ERR_INVALID_ARG;
  if (hidden > h3::norm::MAX_HIDDEN || (param_dtype != dtype && param_dtype != H3_DTYPE_F32)) return H3_ERR_UNSUPPORTED;
  if (n_rows == 0) return H3_OK;
  if (!d_x || !d_y) return H3_ERR_INVALID_ARG;
  if (!in_place_or_apart({d_y, n_rows, y_row_stride, hidden, dtype_size(dtype)},
                         {d_x, n_rows, x_row_stride, hidden, dtype_size(dtype)}))
    return H3_ERR_INVALID_ARG;
  const bool vec = hidden % 8 == 0 && vector_rows(d_x, x_row_stride, dtype) && vector_rows(d_y, y_row_stride, dtype) &&
                   aligned16(d_weight) && aligned16(d_bias);
  const int sms = sm_count();
  return with_types(dtype, param_dtype, [&](auto tt, auto pt) {
    using T = typename decltype(tt)::type;
    using P = typename decltype(pt)::type;
    if (vec && ring_takes(hidden))
      return with_forward_ring(hidden, [&](auto shape) {
        using S = decltype(shape);
        const RingPlan plan = ring_plan(n_rows, sizeof(T) * hidden, 1, S::CTAS, {1, 2, 4});
        auto go = [&](auto rows) {
          return launch_ring<h3::norm::layernorm_ring_kernel<T, P, S::G, S::CH, decltype(rows)::value, S::CTAS>>(
              plan, S::G + 32, as_stream(stream), static_cast<const T*>(d_x), static_cast<T*>(d_y),
              static_cast<const P*>(d_weight), static_cast<const P*>(d_bias), d_mean, d_rstd,
              static_cast<long long>(n_rows), hidden, static_cast<long long>(x_row_stride),
              static_cast<long long>(y_row_stride), eps, plan.slots,
              static_cast<unsigned long long>(g_wait_limit_ns.load()), error_slot(stream));
        };
        return plan.rows == 4 ? go(IntTag<4>{}) : plan.rows == 2 ? go(IntTag<2>{}) : go(IntTag<1>{});
      });
    return with_forward_shape(hidden, [&](auto shape) {
      using S = decltype(shape);
      const long long grid = std::min<long long>((n_rows + S::GROUPS - 1) / S::GROUPS, 16LL * sms);
      auto go = [&](auto kernel) {
        return launch(kernel, dim3(static_cast<unsigned>(grid)), S::BLOCK, 0, as_stream(stream),
                      static_cast<const T*>(d_x), static_cast<T*>(d_y), static_cast<const P*>(d_weight),
                      static_cast<const P*>(d_bias), d_mean, d_rstd, n_rows, hidden, x_row_stride, y_row_stride, eps);
      };
      if constexpr (S::ALIGNED)
        if (vec) return go(h3::norm::layernorm_kernel<T, P, true, S::G, S::CH>);
      return go(h3::norm::layernorm_kernel<T, P, false, S::G, S::CH>);
    });
  });
}

uint64_t h3_layernorm_backward_workspace_bytes(int64_t n_rows, int32_t hidden) {
  if (n_rows < 0 || hidden < 1 || hidden > h3::norm::MAX_HIDDEN) return 0;
  return std::max<uint64_t>(256u, up256(static_cast<uint64_t>(backward_groups(n_rows, hidden)) * 2u * hidden * 4u));
}

h3_status h3_layernorm_backward(const void* d_dy, const void* d_x, const float* d_mean, const float* d_rstd,
                                const void* d_weight, void* d_dx, void* d_dweight, void* d_dbias, void* d_work,
                                int64_t n_rows, int32_t hidden, int64_t dy_row_stride, int64_t x_row_stride,
                                int64_t dx_row_stride, int32_t dtype, int32_t param_dtype, void* stream) {
  if (n_rows < 0 || hidden < 1 || !valid_dtype(dtype) || !valid_dtype(param_dtype)) return H3_ERR_INVALID_ARG;
  if (dy_row_stride < hidden || x_row_stride < hidden || dx_row_stride < hidden) return H3_ERR_INVALID_ARG;
  if (hidden > h3::norm::MAX_HIDDEN || (param_dtype != dtype && param_dtype != H3_DTYPE_F32)) return H3_ERR_UNSUPPORTED;
  const bool params = d_dweight != nullptr || d_dbias != nullptr;
  if (params && (d_work == nullptr || !aligned256(d_work))) return H3_ERR_INVALID_ARG;
  if (n_rows > 0 && (!d_dy || !d_x || !d_mean || !d_rstd || !d_dx)) return H3_ERR_INVALID_ARG;
  const RowSpan dx{d_dx, n_rows, dx_row_stride, hidden, dtype_size(dtype)};
  if (!in_place_or_apart(dx, {d_dy, n_rows, dy_row_stride, hidden, dtype_size(dtype)}) ||
      !in_place_or_apart(dx, {d_x, n_rows, x_row_stride, hidden, dtype_size(dtype)}))
    return H3_ERR_INVALID_ARG;
  const bool vec = hidden % 8 == 0 && vector_rows(d_dy, dy_row_stride, dtype) && vector_rows(d_x, x_row_stride, dtype) &&
                   vector_rows(d_dx, dx_row_stride, dtype) && aligned16(d_weight);
  float* partials = params ? static_cast<float*>(d_work) : nullptr;
  return with_types(dtype, param_dtype, [&](auto tt, auto pt) {
    using T = typename decltype(tt)::type;
    using P = typename decltype(pt)::type;
    long long groups = 0;                          // partial rows
    h3_status st = H3_OK;
    if (n_rows > 0 && vec && ring_takes(hidden)) {
      st = with_backward_ring(hidden, [&](auto shape) {
        using S = decltype(shape);
        const RingPlan plan = ring_plan(n_rows, sizeof(T) * hidden, 2, S::CTAS, {1, 2});
        groups = plan.blocks;
        auto go = [&](auto rows) {
          return launch_ring<
              h3::norm::layernorm_backward_ring_kernel<T, P, S::G, S::CH, decltype(rows)::value, S::CTAS>>(
              plan, S::G + 32, as_stream(stream), static_cast<const T*>(d_dy), static_cast<const T*>(d_x), d_mean,
              d_rstd, static_cast<const P*>(d_weight), static_cast<T*>(d_dx), partials, static_cast<long long>(n_rows),
              hidden, static_cast<long long>(dy_row_stride), static_cast<long long>(x_row_stride),
              static_cast<long long>(dx_row_stride), plan.slots,
              static_cast<unsigned long long>(g_wait_limit_ns.load()), error_slot(stream));
        };
        return plan.rows == 2 ? go(IntTag<2>{}) : go(IntTag<1>{});
      });
    } else if (n_rows > 0) {
      st = with_backward_shape(hidden, [&](auto shape) {
        using S = decltype(shape);
        const long long grid = backward_blocks<S>(n_rows);
        groups = grid * S::GROUPS;
        auto go = [&](auto kernel) {
          return launch(kernel, dim3(static_cast<unsigned>(grid)), S::BLOCK, 0, as_stream(stream),
                        static_cast<const T*>(d_dy), static_cast<const T*>(d_x), d_mean, d_rstd,
                        static_cast<const P*>(d_weight), static_cast<T*>(d_dx), partials, n_rows, hidden, dy_row_stride,
                        x_row_stride, dx_row_stride);
        };
        if constexpr (S::ALIGNED)
          if (vec) return go(h3::norm::layernorm_backward_kernel<T, P, true, S::G, S::CH>);
        return go(h3::norm::layernorm_backward_kernel<T, P, false, S::G, S::CH>);
      });
    }
    if (st != H3_OK || !params) return st;
    return launch(h3::norm::norm_reduce_kernel<P>, dim3((hidden + 63) / 64, 2), 64 * 16, 0, as_stream(stream), partials,
                  static_cast<int>(groups), hidden, static_cast<P*>(d_dweight), static_cast<P*>(d_dbias));
  });
}

uint64_t h3_adaln_backward_workspace_bytes(int64_t n_rows, int32_t hidden, int32_t n_entries) {
  if (n_rows < 0 || n_rows >= (1ll << 31) || hidden < 8 || hidden % 8 != 0 || hidden > h3::ADALN_MAX_HIDDEN ||
      n_entries < 1 || n_entries > h3::norm::MAX_ENTRIES)
    return 0;
  return adaln_work(n_rows, hidden, n_entries).bytes;
}

h3_status h3_adaln_modulate_backward(const void* d_dy, const void* d_x, const int32_t* d_timestep_index,
                                     const int32_t* d_token_tag, const float* d_table, void* d_dx, float* d_dtable,
                                     void* d_work, int32_t n_entries, int64_t n_rows, int32_t hidden,
                                     int64_t dy_row_stride, int64_t x_row_stride, int64_t dx_row_stride, float eps,
                                     void* stream) {
  if (n_rows < 0 || n_rows >= (1ll << 31) || hidden < 8 || n_entries < 1 || !(eps >= 0.f) || !std::isfinite(eps))
    return H3_ERR_INVALID_ARG;
  if (hidden % 8 != 0 || hidden > h3::ADALN_MAX_HIDDEN || n_entries > h3::norm::MAX_ENTRIES) return H3_ERR_UNSUPPORTED;
  if (dy_row_stride < hidden || x_row_stride < hidden || dx_row_stride < hidden) return H3_ERR_INVALID_ARG;
  if (!d_dtable || !d_work || !aligned256(d_work)) return H3_ERR_INVALID_ARG;
  if (n_rows > 0 && (!d_dy || !d_x || !d_timestep_index || !d_token_tag || !d_table || !d_dx)) return H3_ERR_INVALID_ARG;
  if (n_rows > 0 && (!vector_rows(d_dy, dy_row_stride, H3_DTYPE_BF16) || !vector_rows(d_x, x_row_stride, H3_DTYPE_BF16) ||
                     !vector_rows(d_dx, dx_row_stride, H3_DTYPE_BF16) || !aligned16(d_table)))
    return H3_ERR_UNSUPPORTED;
  const RowSpan dx{d_dx, n_rows, dx_row_stride, hidden, 2};
  if (!in_place_or_apart(dx, {d_dy, n_rows, dy_row_stride, hidden, 2}) ||
      !in_place_or_apart(dx, {d_x, n_rows, x_row_stride, hidden, 2}))
    return H3_ERR_INVALID_ARG;
  cudaStream_t s = as_stream(stream);
  if (n_rows == 0)
    return cuda_ok(cudaMemsetAsync(d_dtable, 0, static_cast<size_t>(n_entries) * 2u * hidden * 4u, s))
               ? H3_OK
               : H3_ERR_CUDA;
  const AdalnWork w = adaln_work(n_rows, hidden, n_entries);
  uint8_t* base = static_cast<uint8_t*>(d_work);
  int2* order = reinterpret_cast<int2*>(base + w.order);
  int* starts = reinterpret_cast<int*>(base + w.starts);
  int* hist = reinterpret_cast<int*>(base + w.hist);
  float* partials = reinterpret_cast<float*>(base + w.partials);
  const size_t smem = (static_cast<size_t>(n_entries) + 1u) * sizeof(int);
  h3_status st = launch(h3::norm::adaln_count_kernel, dim3(w.blocks), h3::norm::SORT_ROWS, smem, s, d_timestep_index,
                        d_token_tag, n_entries, n_rows, hist, error_slot(stream));
  if (st == H3_OK)
    st = launch(h3::norm::adaln_place_kernel, dim3(w.blocks), h3::norm::SORT_ROWS, smem, s, d_timestep_index,
                d_token_tag, n_entries, n_rows, hist, w.blocks, order, starts);
  if (st != H3_OK) return st;
  if (ring_takes(hidden))
    st = with_adaln_ring(hidden, [&](auto shape) {
      using S = decltype(shape);
      RingPlan plan{1, 0, w.groups, 0};
      plan.slots = static_cast<int>(std::min<uint64_t>(h3::norm::ADALN_SLOTS, kAdalnSmem / (4u * hidden)));
      plan.smem = static_cast<size_t>(plan.slots) * 4u * hidden;
      return launch_ring<h3::norm::adaln_backward_ring_kernel<S::G, S::CH, kAdalnWarps>>(
          plan, S::G + 32 * (kAdalnWarps + 1), s, static_cast<const __nv_bfloat16*>(d_dy),
          static_cast<const __nv_bfloat16*>(d_x), d_table, static_cast<const int2*>(order),
          static_cast<__nv_bfloat16*>(d_dx), partials, n_entries, static_cast<long long>(n_rows), w.per, hidden,
          static_cast<long long>(dy_row_stride), static_cast<long long>(x_row_stride),
          static_cast<long long>(dx_row_stride), eps, plan.slots,
          static_cast<unsigned long long>(g_wait_limit_ns.load()), error_slot(stream));
    });
  else
    st = with_backward_shape(hidden, [&](auto shape) {
      using S = decltype(shape);
      if constexpr (S::G == 32) {            // up to 1,024 elements
        return launch(h3::norm::adaln_backward_kernel<S::G, S::CH>, dim3(static_cast<unsigned>(w.groups / S::GROUPS)),
                      S::BLOCK, 0, s, static_cast<const __nv_bfloat16*>(d_dy), static_cast<const __nv_bfloat16*>(d_x),
                      d_table, order, static_cast<__nv_bfloat16*>(d_dx), partials, n_entries, n_rows, w.per, hidden,
                      dy_row_stride, x_row_stride, dx_row_stride, eps);
      } else {
        return H3_ERR_UNSUPPORTED;
      }
    });
  if (st != H3_OK) return st;
  // many partial rows per entry are added by 16 rows of threads, few by 2
  const dim3 rgrid((hidden + 255) / 256, 2 * n_entries);
  if (w.groups >= 8LL * n_entries)
    return launch(h3::norm::adaln_reduce_kernel<16>, rgrid, 64 * 16, 0, s, partials, starts, w.per, hidden, d_dtable);
  return launch(h3::norm::adaln_reduce_kernel<2>, rgrid, 64 * 2, 0, s, partials, starts, w.per, hidden, d_dtable);
}

}  // extern "C"
