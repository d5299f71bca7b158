// The work search of the paged attention on the CPU: kv_paged_attention's own
// host code with its launches replaced by a run of attend_find in every
// workgroup, threads in lockstep.  Checks that no barrier or lane exchange is
// left out by a part of the threads, that all threads find the same item, and
// that the items take every key unit of every tile exactly once within the
// launch and the workspace.
#include <stdio.h>
#include <stdlib.h>
#include <string.h>
#include <ucontext.h>

#include <algorithm>
#include <functional>
#include <map>
#include <memory>
#include <random>
#include <string>
#include <vector>

#include "kvattend.h"
#include "spec_kv.h"

hostwave::Index threadIdx;

namespace {

std::string g_case;
[[noreturn]] void die(const char* what, long a = 0, long b = 0) {
  printf("%s: %s (%ld, %ld)\n", g_case.c_str(), what, a, b);
  fflush(stdout);
  exit(1);
}

constexpr size_t kStack = 64 << 10;
struct Fiber {
  ucontext_t ctx;
  std::vector<char> stack = std::vector<char>(kStack);
  bool done = false, workgroup = false;
  int line = 0;
};
std::vector<std::unique_ptr<Fiber>> g_fibers;
std::vector<uint64_t> g_slots;
ucontext_t g_main;
int g_threads = 0, g_now = 0;
std::function<void()> g_body;

void entry() {
  g_body();
  g_fibers[g_now]->done = true;
  swapcontext(&g_fibers[g_now]->ctx, &g_main);
}

void resume(int t) {
  g_now = t;
  threadIdx.x = t;
  swapcontext(&g_main, &g_fibers[t]->ctx);
}

// Runs body in every thread of one workgroup.
void workgroup(int threads, std::function<void()> body) {
  g_threads = threads;
  g_body = body;
  g_slots.assign(threads, 0);
  while (static_cast<int>(g_fibers.size()) < threads) g_fibers.emplace_back(new Fiber);
  for (int t = 0; t < threads; ++t) {
    Fiber& f = *g_fibers[t];
    f.done = false;
    getcontext(&f.ctx);
    f.ctx.uc_stack.ss_sp = f.stack.data();
    f.ctx.uc_stack.ss_size = kStack;
    f.ctx.uc_link = nullptr;
    makecontext(&f.ctx, entry, 0);
  }
  for (int t = 0; t < threads; ++t) resume(t);
  for (;;) {
    // every thread is at a collective or has ended
    int ended = 0, moved = 0;
    for (int w = 0; w < threads; w += hostwave::kLanes) {
      const Fiber& first = *g_fibers[w];
      for (int t = w; t < w + hostwave::kLanes; ++t) {
        const Fiber& f = *g_fibers[t];
        if (f.done != first.done || (!f.done && (f.line != first.line || f.workgroup != first.workgroup)))
          die("lanes of a wavefront part at a collective", first.done ? 0 : first.line, f.done ? 0 : f.line);
      }
      if (first.done) {
        ++ended;
      } else if (!first.workgroup) {
        ++moved;
        for (int t = w; t < w + hostwave::kLanes; ++t) resume(t);
      }
    }
    const int waves = threads / hostwave::kLanes;
    if (ended == waves) return;
    if (moved) continue;
    const int line = g_fibers[0]->line;
    for (int t = 0; t < threads; ++t)
      if (g_fibers[t]->done || g_fibers[t]->line != line)
        die("threads of a workgroup part at a barrier", line, g_fibers[t]->done ? 0 : g_fibers[t]->line);
    for (int t = 0; t < threads; ++t) resume(t);
  }
}

}  // namespace

namespace hostwave {
void meet(bool wg, int line) {
  Fiber& f = *g_fibers[g_now];
  f.workgroup = wg;
  f.line = line;
  const int t = g_now;
  swapcontext(&f.ctx, &g_main);
  g_now = t;
  threadIdx.x = t;
}
uint64_t* slots() { return g_slots.data() + g_now / kLanes * kLanes; }
int lane() { return g_now % kLanes; }
}  // namespace hostwave

namespace {

long g_items, g_split, g_most_slots;
bool g_any_launch, g_nothing;   // g_nothing: the call's offsets ask for no work at all

// Every workgroup's search of one launch (key head 0: the others find the same).
template <int MT, int KT, int WAVES>
hipError_t search(const sv::AttendArgs& a) {
  g_any_launch = true;
  std::vector<int> slot_used(a.max_slots, 0);
  std::map<std::pair<int, int>, std::vector<sv::AttendItem>> tiles;
  const int grid = a.grid_items;
  bool over = false;
  int32_t slots = -1;
  for (int x = 0; x < grid; ++x) {
    if (over && x + 2 < grid && x % 211) continue;   // past the last item: a sample
    sv::AttendPlanShared<WAVES> sh;
    memset(static_cast<void*>(&sh), 0xab, sizeof(sh));
    std::vector<sv::AttendItem> its(WAVES * 64);
    std::vector<char> found(WAVES * 64);
    workgroup(WAVES * 64, [&] {
      const int t = threadIdx.x;
      found[t] = sv::attend_find<MT, KT, WAVES>(a, x, a.max_slots > 0 && x == 0, sh, its[t]);
    });
    for (size_t t = 1; t < found.size(); ++t)
      if (found[t] != found[0] || (found[0] && memcmp(&its[t], &its[0], sizeof(its[0]))))
        die("threads disagree on an item", x, t);
    if (x == 0 && a.max_slots > 0) slots = *a.slot_count;
    if (!found[0]) {
      over = true;
      continue;
    }
    if (over) die("an item behind the last one", x);
    tiles[{its[0].b, its[0].row0}].push_back(its[0]);
    ++g_items;
  }
  if (g_nothing) {
    if (!tiles.empty() || slots > 0) die("work where there is none", tiles.size(), slots);
    return hipSuccess;
  }
  size_t want_tiles = 0;
  long used = 0;
  for (int b = 0; b < a.B; ++b) {
    const long n = a.cu[b + 1] - a.cu[b], rows = n * a.group;
    for (long r0 = 0; r0 < rows; r0 += MT, ++want_tiles) {
      auto it = tiles.find({b, static_cast<int>(r0)});
      if (it == tiles.end()) die("a tile that nobody takes", b, r0);
      auto& v = it->second;
      std::sort(v.begin(), v.end(), [](const sv::AttendItem& p, const sv::AttendItem& q) {
        return p.split < q.split;
      });
      const long last = std::min(rows, r0 + MT) - 1, pos0 = long{a.lens[b]} - n;
      const long cap = std::min(std::max<long>(a.lens[b], 0), long{a.cap});
      const long hi = std::max<long>(std::min(pos0 + last / a.group + 1, cap), 0);
      const long lo = a.window > 0 ? std::max<long>(pos0 + r0 / a.group - a.window + 1, 0) : 0;
      long next = hi > lo ? lo / KT : 0;
      const long end = hi > lo ? (hi - 1) / KT + 1 : next;
      for (size_t s = 0; s < v.size(); ++s) {
        const sv::AttendItem& i = v[s];
        if (i.split != static_cast<int>(s) || i.splits != static_cast<int>(v.size()))
          die("splits", i.split, i.splits);
        if (i.token0 != a.cu[b] || i.rows != last - r0 + 1 || i.pos0 != pos0) die("rows", b, r0);
        if (hi > lo ? i.key_lo != lo || i.key_hi != hi : i.key_lo < i.key_hi) die("keys", b, r0);
        if (i.u1 > i.u0) {
          if (i.u0 != next) die("key units out of order", i.u0, next);
          next = i.u1;
        }
        if (v.size() > 1) {
          if (i.slot < 0 || i.slot >= a.max_slots || slot_used[i.slot]++) die("slot", i.slot);
          if (i.slot - i.split != v[0].slot) die("slots of a tile apart", i.slot, v[0].slot);
          ++used;
        }
      }
      if (hi > lo && next != end) die("key units that nobody takes", next, end);
    }
  }
  if (want_tiles != tiles.size()) die("tiles beside the sequences'", tiles.size(), want_tiles);
  if (a.max_slots > 0 && slots != used) die("slots counted", slots, used);
  g_split += used;
  g_most_slots = std::max(g_most_slots, used);
  return hipSuccess;
}

}  // namespace

namespace sv {
int32_t record_error(int32_t code, const char* msg) noexcept {
  printf("refused: %s\n", msg);
  return code;
}
hipError_t launch_extend(const ExtendArgs&, hipStream_t) { return 1; }
hipError_t launch_append(const AppendArgs&, hipStream_t) { return 1; }
hipError_t launch_attend_rows(const AttendArgs& a, hipStream_t) {
  if (a.D <= 64) return search<kRowsMT64, kRowsKT, 4>(a);
  if (a.D <= 128) return search<kRowsMT128, kRowsKT, 4>(a);
  return search<kRowsMT256, kRowsKT, 4>(a);
}
static hipError_t matrix(const AttendArgs& a, int mt) {
  if (mt == 32) return search<32, 32, 2>(a);
  if (mt == 64) return search<64, 32, 4>(a);
  return search<128, 64, 4>(a);
}
hipError_t launch_attend_d64(const AttendArgs& a, int, int mt, hipStream_t) { return matrix(a, mt); }
hipError_t launch_attend_d128(const AttendArgs& a, int, int mt, hipStream_t) { return matrix(a, mt); }
hipError_t launch_attend_d256(const AttendArgs& a, int, int mt, hipStream_t) { return matrix(a, mt); }
hipError_t launch_attend_join(const AttendArgs&, int, int, hipStream_t) { return hipSuccess; }
}  // namespace sv

namespace {

void run(const char* name, const std::vector<int32_t>& ctx, const std::vector<int32_t>& n, int heads,
         int kv, int dim, int dtype, int window = 0, int hint = 0, int wide = 0, int lead = 0) {
  char text[200];
  snprintf(text, sizeof text, "%s B%zu n%d heads%d-%d d%d type%d w%d hint%d", name, n.size(),
           n.empty() ? 0 : n[0], heads, kv, dim, dtype, window, hint);
  g_case = text;
  std::vector<int32_t> lens, cu = {lead};
  int longest = 1;
  for (size_t b = 0; b < n.size(); ++b) {
    lens.push_back(ctx[b] + n[b]);
    cu.push_back(cu.back() + n[b]);
    longest = std::max(longest, lens.back());
  }
  spec_kv_attention_desc d{};
  d.batch = static_cast<int32_t>(n.size());
  d.tokens = cu.back();
  d.heads = heads;
  d.kv_heads = kv;
  d.head_dim = dim;
  d.block_size = 16;
  d.num_blocks = 1 << 20;
  d.max_blocks = std::max(wide, (longest + 15) / 16);
  d.dtype = dtype;
  d.sliding_window = window;
  d.max_new = hint;
  d.scale = 1.0f;
  const size_t bytes = kv_paged_attention_workspace_bytes(&d);
  std::vector<char> ws(bytes + 256);
  void* p = reinterpret_cast<void*>((reinterpret_cast<uintptr_t>(ws.data()) + 255) / 256 * 256);
  void* some = reinterpret_cast<void*>(uintptr_t{1} << 20);   // addresses that nothing here reads
  g_items = g_split = 0;
  g_any_launch = false;
  const int32_t s = kv_paged_attention(&d, some, some, some, static_cast<int32_t*>(some), lens.data(),
                                       cu.data(), some, nullptr, p, bytes, nullptr);
  if (s != SV_OK) die("status", s);
  if (!g_any_launch) die("no launch");
  printf("%s: %ld items, %ld of them splits\n", text, g_items, g_split);
}

}  // namespace

int main() {
  // one sequence with more tiles than the chip holds workgroups for a key head,
  // on a table wide enough that its keys could be split
  run("one prompt", {0}, {4096}, 32, 8, 128, SV_DTYPE_BF16);
  run("one prompt of short tiles", {300}, {140}, 256, 256, 64, SV_DTYPE_BF16, 0, 1);
  run("one chunk", {300}, {300}, 16, 16, 128, SV_DTYPE_F32);
  run("one chunk, wide heads", {2000}, {300}, 128, 128, 256, SV_DTYPE_F16, 100);
  // one sequence, split
  run("one token", {1000}, {1}, 32, 8, 128, SV_DTYPE_BF16);
  run("one token", {9000}, {1}, 8, 1, 64, SV_DTYPE_F16);
  run("one token", {5000}, {1}, 1, 1, 8, SV_DTYPE_F32);
  run("nothing cached", {0}, {1}, 4, 4, 64, SV_DTYPE_BF16, 0, 0, 8192);
  run("shorter than its tokens", {-5}, {9}, 4, 4, 64, SV_DTYPE_BF16, 0, 0, 8192);
  run("of no length", {-9}, {9}, 4, 2, 64, SV_DTYPE_F32, 0, 0, 8192, 3);
  // batches
  std::mt19937 g(1);
  auto some = [&](int m, int lo, int hi) {
    std::vector<int32_t> v(m);
    for (auto& x : v) x = lo + static_cast<int>(g() % (hi - lo + 1));
    return v;
  };
  run("tokens", some(64, 0, 3000), some(64, 0, 1), 32, 8, 128, SV_DTYPE_BF16);
  run("windows of drafts", some(40, 500, 4000), some(40, 9, 9), 32, 8, 128, SV_DTYPE_BF16);
  run("prompts", some(4, 0, 0), some(4, 500, 1500), 16, 8, 128, SV_DTYPE_F16, 0, 1500);
  run("mixed, a window", some(20, 0, 2000), some(20, 1, 200), 8, 8, 256, SV_DTYPE_F16, 257, 200);
  run("mixed", some(9, 0, 900), some(9, 0, 40), 6, 2, 64, SV_DTYPE_F32, 0, 1, 4096, 7);
  std::vector<int32_t> long_one = some(300, 0, 9), few = some(300, 0, 2);
  long_one[150] = 3000, few[150] = 2;
  run("many short, one long", long_one, few, 2, 1, 64, SV_DTYPE_BF16);
  for (int i = 0; i < 16; ++i) {
    const int B = 1 + g() % 9, kv = 1 << g() % 7, group = 1 + g() % 4, type = g() % 3;
    const int hi = 1 + g() % 5000, most = 1 + g() % 60;
    run("drawn", some(B, -3, hi), some(B, i % 2, most), kv * group, kv, 8 << g() % 6, type,
        g() % 2 ? 0 : 1 + g() % 700, g() % 3 ? 0 : 1 + g() % 100, g() % 2 ? 0 : 2048, g() % 3);
  }
  // offsets that do not ascend ask for more tiles than the launch was sized for
  {
    g_case = "overlapping ranges";
    std::vector<int32_t> cu, lens(12, 700);
    for (int i = 0; i < 13; ++i) cu.push_back(i % 2 ? 160 : 0);
    spec_kv_attention_desc d{};
    d.batch = 12, d.tokens = 160, d.heads = 4, d.kv_heads = 2, d.head_dim = 128, d.block_size = 16;
    d.num_blocks = 1 << 16, d.max_blocks = 64, d.dtype = SV_DTYPE_BF16, d.max_new = 160, d.scale = 1.0f;
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
