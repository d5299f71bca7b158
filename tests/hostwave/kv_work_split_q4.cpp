// The work search of the attention over a 4-bit cache on the CPU: the checks of
// kv_work_split.cpp on kv_paged_attention_q4's host code and on the search with the
// sequences of a thread held in registers.
#include "kvattend.h"
#include "kvattend_q4.h"
#include "spec_kv.h"

namespace sv {
// (units of kQ4KT positions are the 4-bit kernel's)
template <int MT, int KT, int WAVES>
bool search_of(const AttendArgs& a, int x, bool count_slots, AttendPlanShared<WAVES>& sh, AttendItem& it) {
  return attend_find<MT, KT, WAVES, KT != kQ4KT ? 0 : WAVES < 3 ? 4 : 2>(a, x, count_slots, sh, it);
}
}  // namespace sv

static int32_t q4_call(const spec_kv_attention_desc* d, const void* q, const void*, const void*,
                       const int32_t* table, const int32_t* lens, const int32_t* cu, void* out,
                       float* lse, void* ws, size_t bytes, void* stream) {
  return kv_paged_attention_q4(d, q, q, q, q, static_cast<const float*>(q), table, lens, cu, out,
                               lse, ws, bytes, stream);
}

#define attend_find search_of
#define kv_paged_attention q4_call
#define kv_paged_attention_workspace_bytes kv_paged_attention_q4_workspace_bytes
#define main plain_main
#include "kv_work_split.cpp"
#undef main

namespace sv {
static hipError_t q4(const AttendArgs& a, int mt) {
  if (mt == 16) return search<16, kQ4KT, 1>(a);
  if (mt == 32) return search<32, kQ4KT, 2>(a);
  if (mt == 48) return search<48, kQ4KT, 3>(a);
  return search<64, kQ4KT, 4>(a);
}
hipError_t launch_attend_q4_d64(const AttendArgs& a, const Q4Cache&, int, int mt, hipStream_t) { return q4(a, mt); }
hipError_t launch_attend_q4_d128(const AttendArgs& a, const Q4Cache&, int, int mt, hipStream_t) { return q4(a, mt); }
hipError_t launch_attend_q4_d256(const AttendArgs& a, const Q4Cache&, int, int mt, hipStream_t) {
  return mt == 16 ? hipError_t(1) : q4(a, mt);
}
hipError_t launch_rotary(const RotaryArgs&, int, bool, hipStream_t) { return 1; }
hipError_t launch_q4_append(const Q4RowsArgs&, const RotaryArgs&, int, bool, bool, hipStream_t) { return 1; }
hipError_t launch_q4_read(const Q4RowsArgs&, int, hipStream_t) { return 1; }
}  // namespace sv

int main() {
  const int bf = SV_DTYPE_BF16, hf = SV_DTYPE_F16;
  run("one prompt", {0}, {4096}, 32, 8, 128, bf);
  run("one chunk, wide heads", {2000}, {300}, 128, 128, 256, hf, 100);
  run("one token", {1000}, {1}, 32, 8, 128, bf);
  run("one token", {9000}, {1}, 8, 1, 64, hf);
  run("one token, wide heads", {50000}, {1}, 8, 1, 256, hf);
  run("one window", {30000}, {9}, 32, 8, 128, bf);
  run("nothing cached", {0}, {1}, 4, 4, 64, bf, 0, 0, 8192);
  run("shorter than its tokens", {-5}, {9}, 4, 4, 64, bf, 0, 0, 8192);
  run("of no length", {-9}, {9}, 4, 2, 64, hf, 0, 0, 8192, 3);
  std::mt19937 g(2);
  auto some = [&](int m, int lo, int hi) {
    std::vector<int32_t> v(m);
    for (auto& x : v) x = lo + static_cast<int>(g() % (hi - lo + 1));
    return v;
  };
  run("tokens", some(64, 0, 6000), some(64, 0, 1), 32, 8, 128, bf);
  run("windows of drafts", some(40, 500, 4000), some(40, 9, 9), 32, 8, 128, bf);
  run("prompts", some(4, 0, 0), some(4, 500, 1500), 16, 8, 128, hf, 0, 1500);
  run("mixed, a window", some(20, 0, 2000), some(20, 1, 200), 8, 8, 256, hf, 257, 200);
  // batches at, and past, the sequences that a workgroup's threads hold
  for (int B : {256, 257, 384, 385, 513}) {
    std::vector<int32_t> long_one = some(B, 0, 9), few = some(B, 0, 2);
    long_one[B / 2] = 3000, few[B / 2] = 2;
    run("many short, one long", long_one, few, 8, 2, 64, bf, 0, B == 256 ? 1 : B == 384 ? 9 : B == 385 ? 20 : 6);
    if (B == 257) run("many short, one long", long_one, few, 8, 2, 64, bf, 0, 1);
  }
  for (int i = 0; i < 24; ++i) {
    const int B = 1 + g() % 9, kv = 1 << g() % 7, group = 1 + g() % 8;
    const int hi = 1 + g() % 9000, most = 1 + g() % 60;
    run("drawn", some(B, -3, hi), some(B, i % 2, most), kv * group, kv, 32 << g() % 4, g() % 2 ? bf : hf,
        g() % 2 ? 0 : 1 + g() % 700, g() % 3 ? 0 : 1 + g() % 100, g() % 2 ? 0 : 2048, g() % 3);
  }
  {
    g_case = "overlapping ranges";
    std::vector<int32_t> cu, lens(12, 700);
    for (int i = 0; i < 13; ++i) cu.push_back(i % 2 ? 160 : 0);
    spec_kv_attention_desc d{};
    d.batch = 12, d.tokens = 160, d.heads = 4, d.kv_heads = 2, d.head_dim = 128, d.block_size = 16;
    d.num_blocks = 1 << 16, d.max_blocks = 64, d.dtype = bf, d.max_new = 160, d.scale = 1.0f;
    const size_t bytes = kv_paged_attention_workspace_bytes(&d);
    std::vector<char> ws(bytes + 256);
    void* p = reinterpret_cast<void*>((reinterpret_cast<uintptr_t>(ws.data()) + 255) / 256 * 256);
    void* some_p = reinterpret_cast<void*>(uintptr_t{1} << 20);
    g_nothing = true;
    if (kv_paged_attention(&d, some_p, some_p, some_p, static_cast<int32_t*>(some_p), lens.data(),
                           cu.data(), some_p, nullptr, p, bytes, nullptr) != SV_OK)
      die("status");
  }
  printf("work split ok, most slots %ld\n", g_most_slots);
  return 0;
}
