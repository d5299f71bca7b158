// Host-side checks of the paged-KV calls and the attention's work split, shared by
// the sources of the C ABI.  Every refusal records its message for
// spec_verify_last_error.
#pragma once

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include "kv_args.h"
#include "spec_kv.h"

namespace sv {
namespace host {

#if defined(__GNUC__)
__attribute__((format(printf, 2, 3)))
#endif
inline int32_t fail(int32_t code, const char* fmt, ...) {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return record_error(code, buf);
}

inline int32_t device_error(hipError_t e, const char* what) {
  return fail(SV_ERR_DEVICE, "%s: %s", what, hipGetErrorString(e));
}

#define SV_TRY(expr)              \
  do {                            \
    const int32_t _s = (expr);    \
    if (_s != SV_OK) return _s;   \
  } while (0)

inline bool aligned_to(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

inline int32_t check_ptr(const void* p, bool required, uintptr_t align, const char* name) {
  if (!p) return required ? fail(SV_ERR_INVALID_ARG, "%s is NULL", name) : SV_OK;
  if (!aligned_to(p, align))
    return fail(SV_ERR_MISALIGNED, "%s not %d-byte aligned", name, static_cast<int>(align));
  return SV_OK;
}

constexpr int32_t kMaxHeads = 1 << 16;
constexpr int32_t kMaxRowDim = 1 << 12;   // head_dim of a cache append
constexpr int64_t kMaxStride = int64_t{1} << 40;
constexpr int32_t kMaxBatch = 1 << 24;    // sequences of an extension
// Sequences of an attention call: every workgroup passes over all of them to find
// its share, so the time has a part that grows with the square (single tokens over
// 100 positions: B = 1024 0.18 ms, 4096 1.5, 16384 19, 32768 72).
constexpr int32_t kMaxAttendBatch = SV_MAX_ATTEND_BATCH;
constexpr int32_t kMaxRows = 1 << 30;     // rows of an extension's token arrays
constexpr int64_t kMaxThreads = int64_t{1} << 32;

inline int dtype_bytes(int dtype) { return dtype == SV_DTYPE_F32 ? 4 : 2; }

inline int32_t check_dtype(int32_t dtype) {
  if (dtype != SV_DTYPE_F32 && dtype != SV_DTYPE_BF16 && dtype != SV_DTYPE_F16)
    return fail(SV_ERR_UNSUPPORTED, "dtype must be SV_DTYPE_F32, SV_DTYPE_BF16 or SV_DTYPE_F16");
  return SV_OK;
}

// The cache's shape, shared by append and attention; *block_stride gets its value.
inline int32_t check_cache(int32_t kv_heads, int32_t head_dim, int32_t block_size, int32_t num_blocks,
                    int64_t* block_stride) {
  if (kv_heads < 1) return fail(SV_ERR_INVALID_ARG, "kv_heads < 1");
  if (kv_heads > kMaxHeads) return fail(SV_ERR_UNSUPPORTED, "kv_heads > %d", kMaxHeads);
  if (head_dim < 1) return fail(SV_ERR_INVALID_ARG, "head_dim < 1");
  if (head_dim > kMaxRowDim) return fail(SV_ERR_UNSUPPORTED, "head_dim > %d", kMaxRowDim);
  if (block_size < 1) return fail(SV_ERR_INVALID_ARG, "block_size < 1");
  if (num_blocks < 0) return fail(SV_ERR_INVALID_ARG, "num_blocks < 0");
  if (static_cast<int64_t>(num_blocks) * block_size > INT32_MAX)
    return fail(SV_ERR_UNSUPPORTED, "num_blocks * block_size >= 2^31");
  const int64_t dense = static_cast<int64_t>(kv_heads) * block_size * head_dim;
  if (*block_stride == 0) *block_stride = dense;
  if (*block_stride < dense)
    return fail(SV_ERR_INVALID_ARG, "block_stride < kv_heads * block_size * head_dim");
  if (*block_stride > std::max(kMaxStride, dense))
    return fail(SV_ERR_INVALID_ARG, "block_stride too large");
  return SV_OK;
}

inline int32_t check_stride(int64_t* stride, int64_t dense, const char* name) {
  if (*stride == 0) *stride = dense;
  if (*stride < dense) return fail(SV_ERR_INVALID_ARG, "%s smaller than a row", name);
  if (*stride > kMaxStride) return fail(SV_ERR_INVALID_ARG, "%s too large", name);
  return SV_OK;
}

struct AttendPlan {
  sv::AttendShape shape{};
  int64_t q_stride = 0, block_stride = 0;
  int32_t cap = 0, want_items = 0, max_slots = 0, grid_items = 0;
  int64_t max_tiles = 0;
  size_t info_bytes = 0, ml_bytes = 0, o_bytes = 0, ws_bytes = 0;
};

inline size_t pad256(size_t n) { return (n + 255) / 256 * 256; }

// The checks of an attention descriptor and the strides it leaves open; the caller
// picks the shape, then attend_split sizes the launch.
inline int32_t check_attend_desc(const spec_kv_attention_desc* d, AttendPlan* p) {
  if (!d) return fail(SV_ERR_INVALID_ARG, "desc is NULL");
  if (d->reserved != 0 || d->reserved_f != 0.0f)
    return fail(SV_ERR_INVALID_ARG, "reserved fields must be 0");
  if (d->batch < 0) return fail(SV_ERR_INVALID_ARG, "batch < 0");
  if (d->batch > kMaxAttendBatch) return fail(SV_ERR_UNSUPPORTED, "batch > %d", kMaxAttendBatch);
  if (d->tokens < 0) return fail(SV_ERR_INVALID_ARG, "tokens < 0");
  if (d->max_blocks < 0) return fail(SV_ERR_INVALID_ARG, "max_blocks < 0");
  if (d->sliding_window < 0) return fail(SV_ERR_INVALID_ARG, "sliding_window < 0");
  if (d->max_new < 0) return fail(SV_ERR_INVALID_ARG, "max_new < 0");
  SV_TRY(check_dtype(d->dtype));
  p->block_stride = d->block_stride;
  SV_TRY(check_cache(d->kv_heads, d->head_dim, d->block_size, d->num_blocks, &p->block_stride));
  if (d->head_dim % 8 != 0 || d->head_dim > SV_MAX_HEAD_DIM)
    return fail(SV_ERR_UNSUPPORTED, "head_dim must be a multiple of 8 up to %d", SV_MAX_HEAD_DIM);
  if (d->heads < 1) return fail(SV_ERR_INVALID_ARG, "heads < 1");
  if (d->heads > kMaxHeads) return fail(SV_ERR_UNSUPPORTED, "heads > %d", kMaxHeads);
  if (d->heads % d->kv_heads != 0)
    return fail(SV_ERR_INVALID_ARG, "heads is not a multiple of kv_heads");
  if (static_cast<int64_t>(d->tokens) * d->heads > INT32_MAX)
    return fail(SV_ERR_UNSUPPORTED, "tokens * heads >= 2^31");
  // (the kernels hold scores in units of log2: scale * log2 e)
  if (!(d->scale > 0.0f) || !std::isfinite(d->scale * kLog2e))
    return fail(SV_ERR_INVALID_ARG, "scale must be positive and scale * log2(e) finite");
  p->q_stride = d->q_stride;
  SV_TRY(check_stride(&p->q_stride, static_cast<int64_t>(d->heads) * d->head_dim, "q_stride"));
  const int es = dtype_bytes(d->dtype);
  if (p->q_stride * es % 16 != 0 || p->block_stride * es % 16 != 0)
    return fail(SV_ERR_MISALIGNED, "q_stride and block_stride must be multiples of 16 bytes");
  return SV_OK;
}

// The split of the call over workgroups (of `threads` at most) and its workspace,
// for p->shape.
inline int32_t attend_split(const spec_kv_attention_desc* d, AttendPlan* p, int threads = 256) {
  // (without blocks there is no page, and no block 0 for a missing one to read)
  const int64_t cap = d->num_blocks == 0 ? 0
                      : std::min<int64_t>(static_cast<int64_t>(d->max_blocks) * d->block_size,
                                          INT32_MAX);
  p->cap = static_cast<int32_t>(cap);
  // Tiles of all sequences together: sum ceil(n_b * group / mt), sum n_b <= T.
  const int64_t group = d->heads / d->kv_heads, mt = p->shape.mt, kt = p->shape.kt;
  const int64_t tiles = d->tokens * group / mt + std::min(d->batch, d->tokens);
  const int64_t want = std::max<int64_t>(1, p->shape.wgs / d->kv_heads);
  // Most units the rows of a sequence see together: from position 0 on, or, with
  // a window, W + T - 1 positions from anywhere.
  int64_t units = (cap + kt - 1) / kt;
  if (d->sliding_window > 0)
    units = std::min(units, (static_cast<int64_t>(d->sliding_window) + d->tokens) / kt + 2);
  const int64_t splits =
      std::max<int64_t>(1, (units + p->shape.min_units - 1) / p->shape.min_units);
  const int64_t slots = splits > 1 ? std::min(2 * want, tiles * splits) : 0;
  const int64_t items = std::min(want + tiles, tiles * splits);
  // a launch takes fewer than 2^32 threads
  const int64_t most = kMaxThreads / std::max(threads, 256);
  if (items * d->kv_heads >= most || slots * d->kv_heads >= most)
    return fail(SV_ERR_UNSUPPORTED, "batch too large for one call");
  p->want_items = static_cast<int32_t>(want);
  p->max_slots = static_cast<int32_t>(slots);
  p->grid_items = static_cast<int32_t>(items);
  p->max_tiles = tiles;
  if (slots > 0) {
    const size_t rows = static_cast<size_t>(slots) * d->kv_heads * mt;
    p->info_bytes = pad256(static_cast<size_t>(slots) * sizeof(SlotInfo));
    p->ml_bytes = pad256(rows * 2 * sizeof(float));
    p->o_bytes = pad256(rows * d->head_dim * sizeof(float));
    p->ws_bytes = 256 + p->info_bytes + p->ml_bytes + p->o_bytes;
  }
  return SV_OK;
}

// The kernels' argument block of a planned call, but for the caches.
inline AttendArgs attend_args(const spec_kv_attention_desc& d, const AttendPlan& p, const void* q,
                              const int32_t* block_table, const int32_t* seq_lens,
                              const int32_t* cu_tokens, void* out, float* lse, void* workspace) {
  AttendArgs a{};
  a.q = q;
  a.table = block_table;
  a.lens = seq_lens;
  a.cu = cu_tokens;
  a.out = out;
  a.lse = lse;
  a.B = d.batch;
  a.T = d.tokens;
  a.heads = d.heads;
  a.kv_heads = d.kv_heads;
  a.group = d.heads / d.kv_heads;
  a.D = d.head_dim;
  a.block_size = d.block_size;
  a.num_blocks = d.num_blocks;
  a.max_blocks = d.max_blocks;
  a.window = d.sliding_window;
  a.bs = make_fast_div(static_cast<uint32_t>(d.block_size));
  a.grp = make_fast_div(static_cast<uint32_t>(a.group));
  a.q_stride = p.q_stride;
  a.block_stride = p.block_stride;
  a.cap = p.cap;
  a.scale = d.scale;
  a.want_items = p.want_items;
  a.min_units = p.shape.min_units;
  a.max_slots = p.max_slots;
  a.grid_items = p.grid_items;
  a.max_tiles = p.max_tiles;
  if (p.ws_bytes > 0) {
    char* ws = static_cast<char*>(workspace);
    a.slot_count = reinterpret_cast<int32_t*>(ws);
    a.info = reinterpret_cast<SlotInfo*>(ws + 256);
    a.part_ml = reinterpret_cast<float*>(ws + 256 + p.info_bytes);
    a.part_o = reinterpret_cast<float*>(ws + 256 + p.info_bytes + p.ml_bytes);
  }
  return a;
}

// The pointers of an attention call but for the caches'.
inline int32_t check_attend_ptrs(const spec_kv_attention_desc& d, const AttendPlan& p,
                                 const void* q, const int32_t* block_table,
                                 const int32_t* seq_lens, const int32_t* cu_tokens,
                                 const void* out, const float* lse, const void* workspace,
                                 size_t workspace_bytes) {
  const bool any = d.batch > 0 && d.tokens > 0;
  SV_TRY(check_ptr(q, any, 16, "q"));
  SV_TRY(check_ptr(block_table, any && d.max_blocks > 0, 4, "block_table"));
  SV_TRY(check_ptr(seq_lens, any, 4, "seq_lens"));
  SV_TRY(check_ptr(cu_tokens, any, 4, "cu_tokens"));
  SV_TRY(check_ptr(out, any, 16, "out"));
  SV_TRY(check_ptr(lse, false, 4, "lse"));
  if (p.ws_bytes > 0) {
    if (!workspace) return fail(SV_ERR_WORKSPACE, "workspace is NULL");
    if (!aligned_to(workspace, 256)) return fail(SV_ERR_WORKSPACE, "workspace not 256-byte aligned");
    if (workspace_bytes < p.ws_bytes)
      return fail(SV_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", workspace_bytes,
                  p.ws_bytes);
  }
  return SV_OK;
}

}  // namespace host
}  // namespace sv
