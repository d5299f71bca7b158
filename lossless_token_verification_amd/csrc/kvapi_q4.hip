// C ABI of the rotated append and of the cache held in 4 bits: host-side validation
// and launch plans.  See include/spec_kv.h for the contract.
#include "kv_host.h"
#include "kvattend_q4.h"

namespace {

using namespace sv::host;

struct RotaryPlan {
  int64_t q_stride, k_stride, v_stride, q_out_stride, block_stride;
};

int32_t check_rotary(const spec_kv_rotary_desc* desc, bool q4, RotaryPlan* p) {
  if (!desc) return fail(SV_ERR_INVALID_ARG, "desc is NULL");
  const spec_kv_rotary_desc& d = *desc;
  if (d.tokens < 0) return fail(SV_ERR_INVALID_ARG, "tokens < 0");
  SV_TRY(check_dtype(d.dtype));
  p->block_stride = d.block_stride;
  SV_TRY(check_cache(d.kv_heads, d.head_dim, d.block_size, d.num_blocks, &p->block_stride));
  if (q4 && d.block_stride != 0)
    return fail(SV_ERR_INVALID_ARG, "block_stride must be 0: a 4-bit cache is dense");
  if (q4 && (d.head_dim % 32 != 0 || d.head_dim > SV_MAX_HEAD_DIM))
    return fail(SV_ERR_UNSUPPORTED, "head_dim must be a multiple of 32 up to %d", SV_MAX_HEAD_DIM);
  if (d.heads < 0) return fail(SV_ERR_INVALID_ARG, "heads < 0");
  if (d.heads > kMaxHeads) return fail(SV_ERR_UNSUPPORTED, "heads > %d", kMaxHeads);
  if (d.rotary_dim < 0 || d.rotary_dim > d.head_dim || d.rotary_dim % 2 != 0)
    return fail(SV_ERR_INVALID_ARG, "rotary_dim must be even, from 0 to head_dim");
  if (d.rotary_dim == 0 && !q4) return fail(SV_ERR_INVALID_ARG, "rotary_dim must not be 0");
  if (d.rotary_dim == 0 && d.heads > 0)
    return fail(SV_ERR_INVALID_ARG, "queries without a rotation (heads must be 0)");
  if (d.interleaved != 0 && d.interleaved != 1)
    return fail(SV_ERR_INVALID_ARG, "interleaved must be 0 or 1");
  if (d.table_rows < 0) return fail(SV_ERR_INVALID_ARG, "table_rows < 0");
  const int64_t row = static_cast<int64_t>(d.kv_heads) * d.head_dim;
  const int64_t q_row = static_cast<int64_t>(d.heads) * d.head_dim;
  p->q_stride = d.q_stride;
  p->k_stride = d.k_stride;
  p->v_stride = d.v_stride;
  p->q_out_stride = d.q_out_stride;
  SV_TRY(check_stride(&p->q_stride, q_row, "q_stride"));
  SV_TRY(check_stride(&p->k_stride, row, "k_stride"));
  SV_TRY(check_stride(&p->v_stride, row, "v_stride"));
  return check_stride(&p->q_out_stride, q_row, "q_out_stride");
}

// Queries are turned in place, row by row, or to rows that do not overlap them (rows of
// two strides from different places on are the caller's).
int32_t check_in_place(const spec_kv_rotary_desc& d, const RotaryPlan& p, const void* q, const void* q_out) {
  const uint64_t from = reinterpret_cast<uintptr_t>(q), to = reinterpret_cast<uintptr_t>(q_out);
  const uint64_t by = from < to ? to - from : from - to, es = dtype_bytes(d.dtype);
  const uint64_t row = static_cast<uint64_t>(d.heads) * d.head_dim * es;
  const bool alike = d.tokens == 1 || p.q_stride == p.q_out_stride;
  if (by == 0)
    return alike ? SV_OK : fail(SV_ERR_INVALID_ARG, "q_out is q with another stride");
  if (!alike) return SV_OK;
  const uint64_t stride = p.q_stride * es, rows = by / stride, rest = by % stride, last = d.tokens - 1;
  if ((rows <= last && rest < row) || (rows < last && stride - rest < row))
    return fail(SV_ERR_INVALID_ARG, "q_out overlaps q");
  return SV_OK;
}

// The rows' part of the pointer checks.
int32_t check_rows(const spec_kv_rotary_desc& d, const RotaryPlan& p, const void* q, const void* k,
                   const void* v, const int32_t* positions, const float* cos_sin,
                   const int64_t* slot_map, const void* q_out) {
  const int es = dtype_bytes(d.dtype);
  const bool any = d.tokens > 0, turn = any && d.rotary_dim > 0;
  SV_TRY(check_ptr(q, any && d.heads > 0, es, "q"));
  SV_TRY(check_ptr(q_out, any && d.heads > 0, es, "q_out"));
  if (any && d.heads > 0) SV_TRY(check_in_place(d, p, q, q_out));
  SV_TRY(check_ptr(k, any, es, "k"));
  SV_TRY(check_ptr(v, any, es, "v"));
  SV_TRY(check_ptr(positions, turn, 4, "positions"));
  SV_TRY(check_ptr(cos_sin, turn && d.table_rows > 0, 4, "cos_sin"));
  return check_ptr(slot_map, any, 8, "slot_map");
}

bool rows16(const void* p, int64_t stride, int es) { return aligned_to(p, 16) && stride * es % 16 == 0; }

// Whether the turned part of a head is whole units of `vec` elements.
bool turns_in(const spec_kv_rotary_desc& d, int vec) {
  return d.rotary_dim % (d.interleaved ? vec : 2 * vec) == 0;
}

// The argument block of rows [t0, t0 + n).  keys: keys and values are among the units.
sv::RotaryArgs rotary_args(const spec_kv_rotary_desc& d, const RotaryPlan& p, bool wide, bool keys) {
  sv::RotaryArgs a{};
  const int vec = wide ? 16 / dtype_bytes(d.dtype) : 1;
  a.heads = d.heads;
  a.kv_heads = d.kv_heads;
  a.dim = d.head_dim;
  a.rot = d.rotary_dim;
  a.pairs = d.interleaved;
  a.table_rows = d.table_rows;
  a.block_size = d.block_size;
  a.num_slots = d.num_blocks * d.block_size;
  a.q_stride = p.q_stride;
  a.k_stride = p.k_stride;
  a.v_stride = p.v_stride;
  a.q_out_stride = p.q_out_stride;
  a.block_stride = p.block_stride;
  a.turn_units = d.interleaved && wide ? d.rotary_dim / vec : d.rotary_dim / 2 / vec;
  a.row_units = a.turn_units + (d.head_dim - d.rotary_dim) / vec;
  a.v_units = d.head_dim / vec;
  a.token_units = d.heads * a.row_units + (keys ? d.kv_heads * (a.row_units + a.v_units) : 0);
  a.bs = sv::make_fast_div(static_cast<uint32_t>(d.block_size));
  a.token = sv::make_fast_div(static_cast<uint32_t>(std::max(a.token_units, 1)));
  a.row = sv::make_fast_div(static_cast<uint32_t>(a.row_units));
  a.vrow = sv::make_fast_div(static_cast<uint32_t>(a.v_units));
  return a;
}

// Row t.  (Unsigned: rows that no memory holds have no address, and wrap.)
const void* at(const void* p, int64_t t, int64_t stride, int es) {
  const uint64_t bytes = static_cast<uint64_t>(t) * static_cast<uint64_t>(stride) * es;
  return p ? reinterpret_cast<const void*>(reinterpret_cast<uintptr_t>(p) + bytes) : nullptr;
}

void set_rows(sv::RotaryArgs* a, const spec_kv_rotary_desc& d, const RotaryPlan& p, int64_t t,
              int64_t n, const void* q, const void* k, const void* v, const int32_t* positions,
              const float* cos_sin, const int64_t* slot_map, void* q_out) {
  const int es = dtype_bytes(d.dtype);
  a->T = static_cast<int32_t>(n);
  a->q = at(q, t, p.q_stride, es);
  a->k = at(k, t, p.k_stride, es);
  a->v = at(v, t, p.v_stride, es);
  a->q_out = const_cast<void*>(at(q_out, t, p.q_out_stride, es));
  a->positions = positions ? positions + t : nullptr;   // (NULL without a rotation)
  a->cos_sin = cos_sin;
  a->slots = slot_map + t;
}

// Lanes of a row, 8 channels each: a power of two.
int32_t lanes_of(int32_t head_dim) {
  int32_t n = 4;
  while (n * 8 < head_dim) n *= 2;
  return n;
}

int32_t check_q4_cache(bool any, const void* k_codes, const void* k_scales, const void* v_codes,
                       const void* v_scales) {
  SV_TRY(check_ptr(k_codes, any, 16, "k_codes"));
  SV_TRY(check_ptr(k_scales, any, 4, "k_scales"));
  SV_TRY(check_ptr(v_codes, any, 16, "v_codes"));
  return check_ptr(v_scales, any, 4, "v_scales");
}

// The kernel for an attention call over 4-bit pages: tiles of 16 rows a wavefront, with
// as many wavefronts as the rows of one sequence and key head need, 4 where they are
// more.  64 sequences of 2000 positions, head_dim 128, in tiles of 16 / 32 / 48 / 64 rows:
//   12 rows each  45 / 51 / 54 / 55 us     24  60 / 49 / 54 / 54     36  97 / 65 / 55 / 55
//   60           106 / 63 / 92 / 54        prompts of 2500 tokens (4)  573 / 310 / 281 / 264
// (head_dim 64, 12 rows: 35 / 45 / 46 / 48; head_dim 256 has no tile of 16, whose wavefront
// would spill: 596 us against 79 for single tokens of 64 sequences of 2300.  Tiles of 96 and
// 128 rows were slower than 64 in an earlier form of the kernel, 633 and 490 us against
// 423.)
// The keys are split until about `wgs` workgroups have work.  One wavefront each: 4
// sequences of 100000 at head_dim 64 and 128 take 94 and 105 us with 512, 70 and 89 with 1024,
// 56 and 99 with 2048.  More wavefronts: 64 sequences of 2300, 9 tokens each, 49 and 59 us with
// 512, 61 and 76 with 1024 (more to join); one sequence of 30000, 40 tokens, 38 and 46 us with
// 512, 46 and 55 with 256.  A split may be a single unit: one token over 1000 positions takes
// 12.4 us, 14.8 with two at least.
sv::AttendShape q4_shape(const spec_kv_attention_desc& d) {
  sv::AttendShape s{};
  const int64_t mean = d.batch > 0 ? (static_cast<int64_t>(d.tokens) + d.batch - 1) / d.batch : 1;
  const int64_t n = std::min<int64_t>(d.max_new > 0 ? d.max_new : mean, d.tokens);
  const int64_t rows = n * (d.heads / d.kv_heads);
  s.matrix = true;
  s.mt = rows <= 16 && d.head_dim <= 128 ? 16 : rows <= 32 ? 32 : rows <= 48 ? 48 : 64;
  s.kt = sv::kQ4KT;
  s.wgs = s.mt == 16 ? 1024 : 512;
  s.min_units = 1;
  return s;
}

int32_t make_q4_plan(const spec_kv_attention_desc* d, AttendPlan* p) {
  SV_TRY(check_attend_desc(d, p));
  if (d->dtype == SV_DTYPE_F32)
    return fail(SV_ERR_UNSUPPORTED, "dtype must be SV_DTYPE_BF16 or SV_DTYPE_F16");
  if (d->head_dim % 32 != 0)
    return fail(SV_ERR_UNSUPPORTED, "head_dim must be a multiple of 32 up to %d", SV_MAX_HEAD_DIM);
  if (d->block_stride != 0)
    return fail(SV_ERR_INVALID_ARG, "block_stride must be 0: a 4-bit cache is dense");
  if (static_cast<int64_t>(d->num_blocks) * d->block_size * d->kv_heads > UINT32_MAX)
    return fail(SV_ERR_UNSUPPORTED, "num_blocks * block_size * kv_heads >= 2^32");
  p->shape = q4_shape(*d);
  return attend_split(d, p, p->shape.mt * 4);
}

}  // namespace

extern "C" {

int32_t kv_cache_append_rotary(const spec_kv_rotary_desc* desc, const void* q, const void* k,
                               const void* v, const int32_t* positions, const float* cos_sin,
                               const int64_t* slot_map, void* q_out, void* k_cache, void* v_cache,
                               void* hip_stream) {
  RotaryPlan p;
  SV_TRY(check_rotary(desc, false, &p));
  const spec_kv_rotary_desc& d = *desc;
  SV_TRY(check_rows(d, p, q, k, v, positions, cos_sin, slot_map, q_out));
  const int es = dtype_bytes(d.dtype), vec = 16 / es;
  SV_TRY(check_ptr(k_cache, d.tokens > 0 && d.num_blocks > 0, es, "k_cache"));
  SV_TRY(check_ptr(v_cache, d.tokens > 0 && d.num_blocks > 0, es, "v_cache"));
  const bool wide = turns_in(d, vec) && d.head_dim % vec == 0 && rows16(q, p.q_stride, es) &&
                    rows16(k, p.k_stride, es) && rows16(v, p.v_stride, es) &&
                    rows16(q_out, p.q_out_stride, es) && rows16(k_cache, p.block_stride, es) &&
                    rows16(v_cache, p.block_stride, es) && aligned_to(cos_sin, 16);
  sv::RotaryArgs a = rotary_args(d, p, wide, d.num_blocks > 0);
  a.dst[0] = k_cache;
  a.dst[1] = v_cache;
  if (a.token_units == 0) return SV_OK;
  // one launch, or as many as keep a launch's units below 2^31
  const int64_t step = INT32_MAX / a.token_units;
  for (int64_t t = 0; t < d.tokens; t += step) {
    set_rows(&a, d, p, t, std::min<int64_t>(step, d.tokens - t), q, k, v, positions, cos_sin,
             slot_map, q_out);
    const hipError_t err = sv::launch_rotary(a, d.dtype, wide, static_cast<hipStream_t>(hip_stream));
    if (err != hipSuccess) return device_error(err, "rotated cache append launch");
  }
  return SV_OK;
}

int32_t kv_cache_append_q4(const spec_kv_rotary_desc* desc, const void* q, const void* k,
                           const void* v, const int32_t* positions, const float* cos_sin,
                           const int64_t* slot_map, void* q_out, void* k_codes, void* k_scales,
                           void* v_codes, float* v_scales, void* hip_stream) {
  RotaryPlan p;
  SV_TRY(check_rotary(desc, true, &p));
  const spec_kv_rotary_desc& d = *desc;
  SV_TRY(check_rows(d, p, q, k, v, positions, cos_sin, slot_map, q_out));
  SV_TRY(check_q4_cache(d.tokens > 0 && d.num_blocks > 0, k_codes, k_scales, v_codes, v_scales));
  const int es = dtype_bytes(d.dtype), vec = 16 / es;
  const bool table16 = d.rotary_dim == 0 || aligned_to(cos_sin, 16);
  const bool wide = turns_in(d, 8) && rows16(k, p.k_stride, es) && rows16(v, p.v_stride, es) && table16;
  const bool q_wide = turns_in(d, vec) && rows16(q, p.q_stride, es) &&
                      rows16(q_out, p.q_out_stride, es) && table16;
  sv::RotaryArgs qa = rotary_args(d, p, q_wide, false);
  sv::Q4RowsArgs a{};
  a.k_codes = static_cast<uint8_t*>(k_codes);
  a.k_scales = static_cast<uint8_t*>(k_scales);
  a.v_codes = static_cast<uint8_t*>(v_codes);
  a.v_scales = v_scales;
  a.kv_heads = d.num_blocks > 0 ? d.kv_heads : 0;   // (without blocks the queries alone)
  a.dim = d.head_dim;
  a.rot = d.rotary_dim;
  a.pairs = d.interleaved;
  a.table_rows = d.table_rows;
  a.block_size = d.block_size;
  a.num_slots = d.num_blocks * d.block_size;
  a.row_lanes = lanes_of(d.head_dim);
  a.k_stride = p.k_stride;
  a.v_stride = p.v_stride;
  a.bs = sv::make_fast_div(static_cast<uint32_t>(d.block_size));
  a.heads = sv::make_fast_div(static_cast<uint32_t>(d.kv_heads));
  a.cos_sin = cos_sin;
  const int64_t token = static_cast<int64_t>(a.kv_heads) * a.row_lanes + qa.token_units;
  if (token == 0) return SV_OK;
  const int64_t step = INT32_MAX / token;    // both parts of a launch below 2^31 threads together
  for (int64_t t = 0; t < d.tokens; t += step) {
    const int64_t n = std::min<int64_t>(step, d.tokens - t);
    set_rows(&qa, d, p, t, n, q, k, v, positions, cos_sin, slot_map, q_out);
    a.T = static_cast<int32_t>(n);
    a.k = qa.k;
    a.v = qa.v;
    a.positions = qa.positions;
    a.slots = qa.slots;
    const hipError_t err =
        sv::launch_q4_append(a, qa, d.dtype, wide, q_wide, static_cast<hipStream_t>(hip_stream));
    if (err != hipSuccess) return device_error(err, "4-bit cache append launch");
  }
  return SV_OK;
}

int32_t kv_cache_read_q4(int32_t tokens, int32_t kv_heads, int32_t head_dim, int32_t block_size,
                         int32_t num_blocks, int32_t dtype, const int64_t* slot_map,
                         const void* k_codes, const void* k_scales, const void* v_codes,
                         const float* v_scales, void* k, void* v, void* hip_stream) {
  if (tokens < 0) return fail(SV_ERR_INVALID_ARG, "tokens < 0");
  SV_TRY(check_dtype(dtype));
  int64_t dense = 0;
  SV_TRY(check_cache(kv_heads, head_dim, block_size, num_blocks, &dense));
  if (head_dim % 32 != 0 || head_dim > SV_MAX_HEAD_DIM)
    return fail(SV_ERR_UNSUPPORTED, "head_dim must be a multiple of 32 up to %d", SV_MAX_HEAD_DIM);
  const bool any = tokens > 0;
  SV_TRY(check_ptr(slot_map, any, 8, "slot_map"));
  SV_TRY(check_q4_cache(any && num_blocks > 0, k_codes, k_scales, v_codes, v_scales));
  SV_TRY(check_ptr(k, any, 16, "k"));
  SV_TRY(check_ptr(v, any, 16, "v"));
  if (!any) return SV_OK;
  sv::Q4RowsArgs a{};
  a.k_codes = static_cast<uint8_t*>(const_cast<void*>(k_codes));
  a.k_scales = static_cast<uint8_t*>(const_cast<void*>(k_scales));
  a.v_codes = static_cast<uint8_t*>(const_cast<void*>(v_codes));
  a.v_scales = const_cast<float*>(v_scales);
  a.kv_heads = kv_heads;
  a.dim = head_dim;
  a.block_size = block_size;
  a.num_slots = num_blocks * block_size;
  a.row_lanes = lanes_of(head_dim);
  a.bs = sv::make_fast_div(static_cast<uint32_t>(block_size));
  a.heads = sv::make_fast_div(static_cast<uint32_t>(kv_heads));
  const int64_t row = static_cast<int64_t>(kv_heads) * head_dim * dtype_bytes(dtype);
  const int64_t step = INT32_MAX / (static_cast<int64_t>(kv_heads) * a.row_lanes);
  for (int64_t t = 0; t < tokens; t += step) {
    a.T = static_cast<int32_t>(std::min<int64_t>(step, tokens - t));
    a.slots = slot_map + t;
    a.k_out = static_cast<char*>(k) + t * row;
    a.v_out = static_cast<char*>(v) + t * row;
    const hipError_t err = sv::launch_q4_read(a, dtype, static_cast<hipStream_t>(hip_stream));
    if (err != hipSuccess) return device_error(err, "4-bit cache read launch");
  }
  return SV_OK;
}

size_t kv_paged_attention_q4_workspace_bytes(const spec_kv_attention_desc* desc) {
  AttendPlan p;
  return make_q4_plan(desc, &p) == SV_OK ? p.ws_bytes : 0;
}

int32_t kv_paged_attention_q4(const spec_kv_attention_desc* desc, const void* q,
                              const void* k_codes, const void* k_scales, const void* v_codes,
                              const float* v_scales, const int32_t* block_table,
                              const int32_t* seq_lens, const int32_t* cu_tokens, void* out,
                              float* lse, void* workspace, size_t workspace_bytes,
                              void* hip_stream) {
  AttendPlan p;
  SV_TRY(make_q4_plan(desc, &p));
  const spec_kv_attention_desc& d = *desc;
  const bool any = d.batch > 0 && d.tokens > 0;
  SV_TRY(check_attend_ptrs(d, p, q, block_table, seq_lens, cu_tokens, out, lse, workspace,
                           workspace_bytes));
  SV_TRY(check_q4_cache(any && d.max_blocks > 0 && d.num_blocks > 0, k_codes, k_scales, v_codes,
                        v_scales));
  if (!any) return SV_OK;
  sv::AttendArgs a = attend_args(d, p, q, block_table, seq_lens, cu_tokens, out, lse, workspace);
  const sv::Q4Cache c{static_cast<const uint8_t*>(k_codes), static_cast<const uint8_t*>(k_scales),
                      static_cast<const uint8_t*>(v_codes), v_scales};
  hipStream_t st = static_cast<hipStream_t>(hip_stream);
  hipError_t err;
  if (a.D <= 64) err = sv::launch_attend_q4_d64(a, c, d.dtype, p.shape.mt, st);
  else if (a.D <= 128) err = sv::launch_attend_q4_d128(a, c, d.dtype, p.shape.mt, st);
  else err = sv::launch_attend_q4_d256(a, c, d.dtype, p.shape.mt, st);
  if (err != hipSuccess) return device_error(err, "4-bit paged attention launch");
  if (p.max_slots > 0) {
    err = sv::launch_attend_join(a, d.dtype, p.shape.mt, st);
    if (err != hipSuccess) return device_error(err, "4-bit paged attention join launch");
  }
  return SV_OK;
}

}  // extern "C"
