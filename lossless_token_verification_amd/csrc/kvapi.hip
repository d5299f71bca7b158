// C ABI of the paged-KV calls: host-side validation, the attention's workspace
// and launch plan.  See include/spec_kv.h for the contract.
#include "kv_host.h"
#include "kvattend.h"

namespace {

using namespace sv::host;

// The kernel for a call: the matrix-core one for 16-bit types (an eighth to a
// thirtieth of the vector units' time at head_dim 40 to 192), with the smallest
// tile that takes the rows of one sequence and key head (rows: the caller's
// max_new, or the batch's mean, times the heads of a group).  Smaller tiles read
// the keys again, larger ones compute rows that are not there (head_dim 128, B =
// 128 over 2300 positions: 36 rows 387 us in tiles of 32, 214 of 64, 237 of 128; 4
// rows 195, 198, 225).  wgs: items to aim at where keys are split, for most shapes
// the workgroups that the chip holds by registers and LDS (2 to 4 a CU; float32 at
// head_dim 128, 512 against 1024: single tokens over 2300 positions at B = 16 65
// against 79 us, B = 64 220 against 237).  Matrix tiles of 32 rows up to head_dim
// 128, and of 64 at head_dim 64, fit 4 to 8 times a CU; fewer and longer splits
// than that measured better (single tokens, head_dim 128, 768 against 1024: B = 64
// over 2300 positions 95 against 101 us, B = 4 over 110000 275 against 277; head_dim
// 64, 1024 against 2048: B = 128 over 2300 96 against 102; 9 tokens there, 1024
// against 1280: B = 16 over 4000 35 against 39).  min_units: a split costs a row 8
// bytes of partial result per element, written and read, a position 4 of cache; 4
// positions per row and 64 at least measured best where splits are that short, on a
// chip that is not full (9 rows x 4 heads over 4000 positions: 26 us with 16
// positions per row, 17 with 4).
sv::AttendShape attend_shape(const spec_kv_attention_desc& d) {
  sv::AttendShape s{};
  const int D = d.head_dim;
  s.matrix = d.dtype != SV_DTYPE_F32;
  if (s.matrix) {
    const int64_t mean = d.batch > 0 ? (static_cast<int64_t>(d.tokens) + d.batch - 1) / d.batch : 1;
    const int64_t n = std::min<int64_t>(d.max_new > 0 ? d.max_new : mean, d.tokens);
    const int64_t rows = n * (d.heads / d.kv_heads);
    s.mt = rows <= 32 ? 32 : rows <= 64 || D > 128 ? 64 : 128;
    s.kt = s.mt == 128 ? 64 : 32;
    s.wgs = D > 128 || (D > 64 && s.mt == 128) ? 512 : D > 64 || s.mt == 128 ? 768 : 1024;
    s.min_units = static_cast<int32_t>(std::max<int64_t>(64, 4 * std::min<int64_t>(rows, s.mt)) /
                                       s.kt);
  } else {
    s.mt = D <= 64 ? sv::kRowsMT64 : D <= 128 ? sv::kRowsMT128 : sv::kRowsMT256;
    s.kt = sv::kRowsKT;
    s.wgs = D > 64 ? 512 : 1024;
    s.min_units = 256 / s.kt;
  }
  return s;
}

int32_t make_attend_plan(const spec_kv_attention_desc* d, AttendPlan* p) {
  SV_TRY(check_attend_desc(d, p));
  p->shape = attend_shape(*d);
  return attend_split(d, p);
}

}  // namespace

extern "C" {

int32_t spec_kv_abi_version(void) { return SPEC_KV_ABI_VERSION; }

int32_t kv_blocktable_extend(int32_t batch, int32_t max_blocks, int32_t block_size,
                             int32_t* block_table, const int32_t* seq_lens,
                             const int32_t* num_new, int32_t* free_blocks,
                             int32_t free_capacity, const int32_t* free_count,
                             const int32_t* freed_blocks, int32_t max_freed,
                             const int32_t* num_freed, int32_t max_tokens, int32_t* new_lens,
                             int32_t* num_taken, int32_t* free_left, int32_t* cu_tokens,
                             int64_t* slot_map, int32_t* positions, void* hip_stream) {
  if (batch < 0) return fail(SV_ERR_INVALID_ARG, "batch < 0");
  if (batch > kMaxBatch) return fail(SV_ERR_UNSUPPORTED, "batch > %d", kMaxBatch);
  if (max_blocks < 0) return fail(SV_ERR_INVALID_ARG, "max_blocks < 0");
  if (block_size < 1) return fail(SV_ERR_INVALID_ARG, "block_size < 1");
  if (free_capacity < 0) return fail(SV_ERR_INVALID_ARG, "free_capacity < 0");
  if (max_freed < 0) return fail(SV_ERR_INVALID_ARG, "max_freed < 0");
  if (max_tokens < 0) return fail(SV_ERR_INVALID_ARG, "max_tokens < 0");
  if (max_tokens > kMaxRows) return fail(SV_ERR_UNSUPPORTED, "max_tokens > %d", kMaxRows);
  const bool any = batch > 0;
  SV_TRY(check_ptr(block_table, any && max_blocks > 0, 4, "block_table"));
  SV_TRY(check_ptr(seq_lens, any, 4, "seq_lens"));
  SV_TRY(check_ptr(num_new, any, 4, "num_new"));
  SV_TRY(check_ptr(free_blocks, free_capacity > 0, 4, "free_blocks"));
  SV_TRY(check_ptr(free_count, true, 4, "free_count"));
  SV_TRY(check_ptr(freed_blocks, false, 4, "freed_blocks"));
  SV_TRY(check_ptr(num_freed, any && freed_blocks, 4, "num_freed"));
  SV_TRY(check_ptr(new_lens, any, 4, "new_lens"));
  SV_TRY(check_ptr(num_taken, any, 4, "num_taken"));
  SV_TRY(check_ptr(free_left, true, 4, "free_left"));
  SV_TRY(check_ptr(cu_tokens, true, 4, "cu_tokens"));
  SV_TRY(check_ptr(slot_map, max_tokens > 0, 8, "slot_map"));
  SV_TRY(check_ptr(positions, false, 4, "positions"));
  sv::ExtendArgs a{};
  a.B = batch;
  a.max_blocks = max_blocks;
  a.block_size = block_size;
  a.free_capacity = free_capacity;
  a.max_freed = freed_blocks ? max_freed : 0;
  a.T = max_tokens;
  a.bs = sv::make_fast_div(static_cast<uint32_t>(block_size));
  a.table = block_table;
  a.lens = seq_lens;
  a.num_new = num_new;
  a.free_blocks = free_blocks;
  a.free_count = free_count;
  a.freed = max_freed > 0 ? freed_blocks : nullptr;
  a.num_freed = num_freed;
  a.new_lens = new_lens;
  a.num_taken = num_taken;
  a.free_left = free_left;
  a.cu = cu_tokens;
  a.slots = slot_map;
  a.positions = positions;
  const hipError_t err = sv::launch_extend(a, static_cast<hipStream_t>(hip_stream));
  if (err != hipSuccess) return device_error(err, "block-table extension launch");
  return SV_OK;
}

int32_t kv_cache_append(const spec_kv_append_desc* desc, const void* k, const void* v,
                        const int64_t* slot_map, void* k_cache, void* v_cache,
                        void* hip_stream) {
  if (!desc) return fail(SV_ERR_INVALID_ARG, "desc is NULL");
  const spec_kv_append_desc& d = *desc;
  if (d.tokens < 0) return fail(SV_ERR_INVALID_ARG, "tokens < 0");
  SV_TRY(check_dtype(d.dtype));
  int64_t block_stride = d.block_stride, k_stride = d.k_stride, v_stride = d.v_stride;
  SV_TRY(check_cache(d.kv_heads, d.head_dim, d.block_size, d.num_blocks, &block_stride));
  const int64_t row = static_cast<int64_t>(d.kv_heads) * d.head_dim;
  SV_TRY(check_stride(&k_stride, row, "k_stride"));
  SV_TRY(check_stride(&v_stride, row, "v_stride"));
  const int es = dtype_bytes(d.dtype);
  const bool any = d.tokens > 0;
  SV_TRY(check_ptr(k, any, es, "k"));
  SV_TRY(check_ptr(v, any, es, "v"));
  SV_TRY(check_ptr(slot_map, any, 8, "slot_map"));
  SV_TRY(check_ptr(k_cache, any && d.num_blocks > 0, es, "k_cache"));
  SV_TRY(check_ptr(v_cache, any && d.num_blocks > 0, es, "v_cache"));
  const bool wide = d.head_dim * es % 16 == 0 && k_stride * es % 16 == 0 &&
                    v_stride * es % 16 == 0 && block_stride * es % 16 == 0 &&
                    aligned_to(k, 16) && aligned_to(v, 16) && aligned_to(k_cache, 16) &&
                    aligned_to(v_cache, 16);
  const int vb = wide ? 16 : es, per = vb / es;
  if (!any || d.num_blocks == 0) return SV_OK;
  sv::AppendArgs a{};
  a.dst[0] = k_cache;
  a.dst[1] = v_cache;
  a.vec_bytes = vb;
  a.row_vecs = static_cast<int32_t>(row / per);
  a.head_vecs = d.head_dim / per;
  a.num_slots = d.num_blocks * d.block_size;
  a.block_size = d.block_size;
  a.bs = sv::make_fast_div(static_cast<uint32_t>(d.block_size));
  a.row = sv::make_fast_div(static_cast<uint32_t>(a.row_vecs));
  a.head = sv::make_fast_div(static_cast<uint32_t>(a.head_vecs));
  a.src_stride[0] = k_stride / per;
  a.src_stride[1] = v_stride / per;
  a.block_stride = block_stride / per;
  // one launch, or as many as keep a launch's vectors below 2^31
  const int64_t step = INT32_MAX / a.row_vecs;
  for (int64_t t = 0; t < d.tokens; t += step) {
    a.src[0] = static_cast<const char*>(k) + t * k_stride * es;
    a.src[1] = static_cast<const char*>(v) + t * v_stride * es;
    a.slots = slot_map + t;
    a.T = static_cast<int32_t>(std::min<int64_t>(step, d.tokens - t));
    const hipError_t err = sv::launch_append(a, static_cast<hipStream_t>(hip_stream));
    if (err != hipSuccess) return device_error(err, "cache append launch");
  }
  return SV_OK;
}

size_t kv_paged_attention_workspace_bytes(const spec_kv_attention_desc* desc) {
  AttendPlan p;
  return make_attend_plan(desc, &p) == SV_OK ? p.ws_bytes : 0;
}

int32_t kv_paged_attention(const spec_kv_attention_desc* desc, const void* q,
                           const void* k_cache, const void* v_cache,
                           const int32_t* block_table, const int32_t* seq_lens,
                           const int32_t* cu_tokens, void* out, float* lse, void* workspace,
                           size_t workspace_bytes, void* hip_stream) {
  AttendPlan p;
  SV_TRY(make_attend_plan(desc, &p));
  const spec_kv_attention_desc& d = *desc;
  const bool any = d.batch > 0 && d.tokens > 0;
  const bool pages = any && d.max_blocks > 0;
  SV_TRY(check_attend_ptrs(d, p, q, block_table, seq_lens, cu_tokens, out, lse, workspace,
                           workspace_bytes));
  SV_TRY(check_ptr(k_cache, pages && d.num_blocks > 0, 16, "k_cache"));
  SV_TRY(check_ptr(v_cache, pages && d.num_blocks > 0, 16, "v_cache"));
  if (!any) return SV_OK;
  sv::AttendArgs a = attend_args(d, p, q, block_table, seq_lens, cu_tokens, out, lse, workspace);
  a.k = k_cache;
  a.v = v_cache;
  hipStream_t st = static_cast<hipStream_t>(hip_stream);
  hipError_t err;
  if (!p.shape.matrix) err = sv::launch_attend_rows(a, st);
  else if (a.D <= 64) err = sv::launch_attend_d64(a, d.dtype, p.shape.mt, st);
  else if (a.D <= 128) err = sv::launch_attend_d128(a, d.dtype, p.shape.mt, st);
  else err = sv::launch_attend_d256(a, d.dtype, p.shape.mt, st);
  if (err != hipSuccess) return device_error(err, "paged attention launch");
  if (p.max_slots > 0) {
    err = sv::launch_attend_join(a, d.dtype, p.shape.mt, st);
    if (err != hipSuccess) return device_error(err, "paged attention join launch");
  }
  return SV_OK;
}

}  // extern "C"
