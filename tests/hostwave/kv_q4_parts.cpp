// Appends and read-backs of so many rows that they are taken in parts, on the CPU: the
// launches replaced by checks of what they are handed, the pointers that a call need not
// have NULL; and queries turned in place, or to rows that overlap them.  Built with the
// sanitizers by the test.
#include <stdio.h>
#include <stdlib.h>

#include "kvapi_q4.hip"

namespace {

int64_t g_rows, g_launches;
bool g_any;      // pointers are not checked

[[noreturn]] void die(const char* what, long long a, long long b) {
  printf("%s (%lld, %lld)\n", what, a, b);
  fflush(stdout);
  exit(1);
}

void take(const void* p, bool there, int64_t row_bytes, const char* what) {
  if (g_any) return;
  const int64_t want = there ? (int64_t{1} << 44) + g_rows * row_bytes : 0;
  if (reinterpret_cast<int64_t>(p) != want) die(what, reinterpret_cast<int64_t>(p), want);
}

bool g_queries, g_turn;

void rows(int64_t T, const int32_t* positions, const int64_t* slots) {
  take(positions, g_turn, 4, "positions");
  take(slots, true, 8, "slots");
  g_rows += T;
  ++g_launches;
}

}  // namespace

namespace sv {
int32_t record_error(int32_t code, const char* msg) noexcept {
  if (!msg[0]) die("no message", code, 0);
  return code;
}
hipError_t launch_rotary(const RotaryArgs& a, int, bool, hipStream_t) {
  take(a.q, g_queries, a.q_stride * 2, "q");
  take(a.k, true, a.k_stride * 2, "k");
  rows(a.T, a.positions, a.slots);
  return hipSuccess;
}
hipError_t launch_q4_append(const Q4RowsArgs& a, const RotaryArgs& q, int, bool, bool, hipStream_t) {
  take(q.q, g_queries, q.q_stride * 2, "q");
  take(a.k, true, a.k_stride * 2, "k");
  // workgroups of 256 threads for the rows, then for the queries, fewer than 2^32 threads
  const int64_t per = 256 / a.row_lanes;
  const int64_t groups = (int64_t{a.T} * a.kv_heads + per - 1) / per + (int64_t{q.T} * q.token_units + 255) / 256;
  if (groups * 256 >= int64_t{1} << 32) die("threads of a launch", groups, a.T);
  rows(a.T, a.positions, a.slots);
  return hipSuccess;
}
hipError_t launch_q4_read(const Q4RowsArgs& a, int, hipStream_t) {
  rows(a.T, nullptr, a.slots);
  return hipSuccess;
}
hipError_t launch_attend_q4_d64(const AttendArgs&, const Q4Cache&, int, int, hipStream_t) { return 1; }
hipError_t launch_attend_q4_d128(const AttendArgs&, const Q4Cache&, int, int, hipStream_t) { return 1; }
hipError_t launch_attend_q4_d256(const AttendArgs&, const Q4Cache&, int, int, hipStream_t) { return 1; }
hipError_t launch_attend_join(const AttendArgs&, int, int, hipStream_t) { return 1; }
}  // namespace sv

int main() {
  char* const P = reinterpret_cast<char*>(int64_t{1} << 44);
  int32_t* const I = reinterpret_cast<int32_t*>(P);
  float* const F = reinterpret_cast<float*>(P);
  int64_t* const L = reinterpret_cast<int64_t*>(P);
  long parts = 0;
  for (int32_t T : {1, 20000000, 33554431, 500000000, INT32_MAX})
    for (int32_t kv : {1, 4, 8, 64})
      for (int32_t heads : {0, 8, 64})
        for (int32_t dim : {32, 128, 256})
          for (int32_t rot : {0, 32, dim})
            for (int32_t nb : {0, 4096}) {
              spec_kv_rotary_desc d{};
              d.tokens = T, d.heads = heads, d.kv_heads = kv, d.head_dim = dim, d.block_size = 16;
              d.num_blocks = nb, d.dtype = SV_DTYPE_BF16, d.rotary_dim = rot, d.table_rows = 100;
              if (rot == 0 && heads > 0) continue;
              g_queries = heads > 0, g_turn = rot > 0;
              void* const q = g_queries ? P : nullptr;
              const int32_t* const pos = g_turn ? I : nullptr;
              const float* const angles = g_turn ? F : nullptr;
              void* const pages = nb ? P : nullptr;
              float* const scales = nb ? F : nullptr;
              g_rows = g_launches = 0;
              int32_t s = kv_cache_append_q4(&d, q, P, P, pos, angles, L, q, pages, pages, pages, scales, nullptr);
              if (s != SV_OK || g_rows != (heads > 0 || nb > 0 ? T : 0)) die("4-bit append", s, g_rows);
              parts += g_launches;
              if (rot > 0) {
                g_rows = 0;
                s = kv_cache_append_rotary(&d, q, P, P, pos, angles, L, q, pages, pages, nullptr);
                if (s != SV_OK || g_rows != (heads > 0 || nb > 0 ? T : 0)) die("append", s, g_rows);
              }
              g_turn = false, g_rows = 0;
              s = kv_cache_read_q4(T, kv, dim, 16, nb, SV_DTYPE_BF16, L, pages, pages, pages, scales, P, P, nullptr);
              if (s != SV_OK || g_rows != T) die("read", s, g_rows);
            }
  // Queries of 2 heads of 64 (256 bytes a row) to rows `by` bytes on.
  struct Place { int32_t T; int64_t stride, out_stride, by; bool fine; };
  const Place places[] = {
      {5, 0, 0, 0, true}, {5, 512, 512, 0, true}, {5, 512, 0, 0, false}, {5, 0, 512, 0, false},
      {1, 512, 0, 0, true}, {1, 0, 0, 128, false}, {1, 0, 0, 256, true}, {1, 0, 0, -254, false},
      {5, 0, 0, 256, false}, {5, 0, 0, 1024, false}, {5, 0, 0, 1278, false}, {5, 0, 0, 1280, true},
      {5, 0, 0, -1278, false}, {5, 0, 0, -1280, true}, {5, 512, 512, 512, true}, {5, 512, 512, 510, true},
      {5, 512, 512, 768, true}, {5, 512, 512, 770, false}, {5, 512, 512, 1024, false},
      {5, 512, 512, -512, true}, {5, 512, 512, -2046, false}, {5, 512, 512, 5118, true}, {5, 512, 1024, 512, true}};
  g_any = true;
  for (const Place& at : places)
    for (bool q4 : {false, true}) {
      spec_kv_rotary_desc d{};
      d.tokens = at.T, d.heads = 2, d.kv_heads = 1, d.head_dim = 64, d.block_size = 16, d.num_blocks = 9;
      d.dtype = SV_DTYPE_BF16, d.rotary_dim = 64, d.table_rows = 9;
      d.q_stride = at.stride, d.q_out_stride = at.out_stride;
      const int32_t s = q4 ? kv_cache_append_q4(&d, P, P, P, I, F, L, P + at.by, P, P, P, F, nullptr)
                           : kv_cache_append_rotary(&d, P, P, P, I, F, L, P + at.by, P, P, nullptr);
      if (s != (at.fine ? SV_OK : SV_ERR_INVALID_ARG)) die("in place", s, at.by);
    }
  printf("parts ok: %ld launches of the 4-bit append\n", parts);
  return parts > 200 ? 0 : 1;
}
