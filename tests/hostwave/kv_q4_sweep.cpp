// The host code of the rotated append and of the 4-bit cache's calls on the CPU, its
// launches replaced by checks of what they are handed: extreme descriptors, with
// pointers and without.  Built with the sanitizers by the test.
#include <stdio.h>
#include <stdlib.h>

#include <initializer_list>

#include "kvapi_q4.hip"

namespace {

long g_launches, g_refused, g_planned;
int64_t g_rows, g_next;     // rows of the call that its launches took, and where the next begins

[[noreturn]] void die(const char* what, long long a, long long b) {
  printf("%s (%lld, %lld)\n", what, a, b);
  fflush(stdout);
  exit(1);
}

void take(int64_t n, const void* slots) {
  const int64_t at = reinterpret_cast<int64_t>(slots) - (int64_t{1} << 40);
  if (n < 1 || at != g_next * 8) die("rows out of order", n, at);
  g_next += n;
  g_rows += n;
  ++g_launches;
}

}  // namespace

namespace sv {
int32_t record_error(int32_t code, const char* msg) noexcept {
  if (!msg[0]) die("no message", code, 0);
  ++g_refused;
  return code;
}
hipError_t launch_rotary(const RotaryArgs& a, int, bool, hipStream_t) {
  if (int64_t{a.T} * a.token_units > INT32_MAX) die("too many units", a.T, a.token_units);
  take(a.T, a.slots);
  return hipSuccess;
}
hipError_t launch_q4_append(const Q4RowsArgs& a, const RotaryArgs& q, int, bool, bool, hipStream_t) {
  if (int64_t{a.T} * a.kv_heads * a.row_lanes > INT32_MAX || int64_t{q.T} * q.token_units > INT32_MAX)
    die("too many threads", a.T, a.kv_heads);
  if (a.T != q.T || 256 % a.row_lanes != 0 || a.row_lanes * 8 < a.dim) die("shape", a.T, a.row_lanes);
  take(a.T, a.slots);
  return hipSuccess;
}
hipError_t launch_q4_read(const Q4RowsArgs& a, int, hipStream_t) {
  if (int64_t{a.T} * a.kv_heads * a.row_lanes > INT32_MAX) die("too many threads", a.T, a.kv_heads);
  take(a.T, a.slots);
  return hipSuccess;
}
static hipError_t attend(const AttendArgs& a, int mt) {
  if (a.grid_items < 1 || int64_t{a.grid_items} * a.kv_heads * mt * 4 >= int64_t{1} << 32)
    die("launch", a.grid_items, a.kv_heads);
  if (int64_t{a.num_blocks} * a.block_size * a.kv_heads > UINT32_MAX) die("rows", a.num_blocks, a.kv_heads);
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_attend_q4_d64(const AttendArgs& a, const Q4Cache&, int, int mt, hipStream_t) { return attend(a, mt); }
hipError_t launch_attend_q4_d128(const AttendArgs& a, const Q4Cache&, int, int mt, hipStream_t) { return attend(a, mt); }
hipError_t launch_attend_q4_d256(const AttendArgs& a, const Q4Cache&, int, int mt, hipStream_t) { return attend(a, mt); }
hipError_t launch_attend_join(const AttendArgs&, int, int, hipStream_t) { return hipSuccess; }
}  // namespace sv

int main() {
  const int32_t big = INT32_MAX;
  void* const P = reinterpret_cast<void*>(int64_t{1} << 40);
  int32_t* const I = static_cast<int32_t*>(P);
  float* const F = static_cast<float*>(P);
  int64_t* const L = static_cast<int64_t*>(P);
  long n = 0;
  const int32_t heads_of[][2] = {{1, 1}, {65536, 65536}, {64, 8}, {65536, 1}, {7, 2}, {0, 3}, {-1, 0}};
  struct Form { int32_t dtype, window; int64_t stride; float scale; };
  const Form forms[] = {{1, 0, 0, 1.0f}, {2, big, int64_t{1} << 40, 3e38f}, {2, 1, int64_t{1} << 62, 1e-45f},
                        {1, 5, INT64_MIN, 0.5f}, {2, big, 0, 2.0f}, {0, -1, 0, 1.0f}};
  for (int32_t B : {-1, 0, 1, 65536, big})
    for (int32_t T : {-1, 0, 1, 1 << 20, big})
      for (const auto& h : heads_of)
        for (int32_t dim : {-32, 32, 64, 160, 256, 4096, big})
          for (int32_t bs : {0, 1, 16, big})
            for (int32_t nb : {0, 1, 1 << 20, big})
              for (int32_t width : {0, 1, big})
                for (const Form& f : forms) {
                  spec_kv_attention_desc d{};
                  d.batch = B, d.tokens = T, d.heads = h[0], d.kv_heads = h[1], d.head_dim = dim;
                  d.block_size = bs, d.num_blocks = nb, d.max_blocks = width, d.dtype = f.dtype;
                  d.sliding_window = f.window, d.max_new = f.window ? big : 0, d.q_stride = f.stride;
                  d.scale = f.scale;
                  g_planned += kv_paged_attention_q4_workspace_bytes(&d) > 0;
                  kv_paged_attention_q4(&d, P, P, P, P, F, I, I, I, P, F, P, SIZE_MAX, nullptr);
                  kv_paged_attention_q4(&d, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                                        nullptr, nullptr, nullptr, nullptr, 0, nullptr);
                  ++n;
                  if (B != 1) continue;      // (the rows know no batch)
                  for (int32_t rot : {0, 2, dim, -big}) {
                    spec_kv_rotary_desc r{};
                    r.tokens = T, r.heads = h[0], r.kv_heads = h[1], r.head_dim = dim, r.block_size = bs;
                    r.num_blocks = nb, r.dtype = f.dtype, r.rotary_dim = rot, r.interleaved = f.window & 1;
                    r.table_rows = width, r.q_stride = r.k_stride = r.v_stride = r.q_out_stride = f.stride;
                    // (a call that would take millions of launches is left out)
                    const double units = (h[0] + 2.0 * h[1]) * dim * T;
                    if (units > 4e12) continue;
                    for (bool q4 : {false, true}) {
                      g_rows = g_next = 0;
                      const int32_t s =
                          q4 ? kv_cache_append_q4(&r, P, P, P, I, F, L, P, P, P, P, F, nullptr)
                             : kv_cache_append_rotary(&r, P, P, P, I, F, L, P, P, P, nullptr);
                      if (s == SV_OK ? g_rows != T && (h[0] > 0 || nb > 0) : g_rows != 0)
                        die("rows", s, g_rows);
                    }
                    kv_cache_append_rotary(&r, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                                           nullptr, nullptr, nullptr);
                    kv_cache_append_q4(&r, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                                       nullptr, nullptr, nullptr, nullptr, nullptr);
                  }
                  if (double(h[1]) * dim * T > 4e12) continue;
                  g_rows = g_next = 0;
                  const int32_t s = kv_cache_read_q4(T, h[1], dim, bs, nb, f.dtype, L, P, P, P, F, P, P, nullptr);
                  if (s == SV_OK ? g_rows != T : g_rows != 0) die("rows read", s, g_rows);
                }
  kv_cache_append_rotary(nullptr, P, P, P, I, F, L, P, P, P, nullptr);
  kv_cache_append_q4(nullptr, P, P, P, I, F, L, P, P, P, P, F, nullptr);
  kv_paged_attention_q4(nullptr, P, P, P, P, F, I, I, I, P, F, P, 0, nullptr);
  kv_paged_attention_q4_workspace_bytes(nullptr);
  printf("sweep ok: %ld descriptors, %ld launches, %ld refusals, %ld workspaces\n", n, g_launches,
         g_refused, g_planned);
  return g_launches > 1000 && g_planned > 100 ? 0 : 1;
}
