// Device code shared by the paged-attention kernels: which (tile, split) of
// which sequence a workgroup takes, and the form of a split's partial result.
#pragma once

#include "kv_args.h"

namespace sv {

// One workgroup's share: query rows [row0, row0 + rows) of a sequence and the
// key units [u0, u1) of its split.
struct AttendItem {
  int32_t token0, row0, rows;
  int32_t pos0;              // position of the sequence's first new token
  int32_t b;
  int32_t key_lo, key_hi;    // positions any row of the tile may see
  int32_t u0, u1;
  int32_t split, splits, slot;   // slot: partial slot (splits > 1)
};

struct AttendSeq {
  int64_t pos0;
  int32_t token0, n, tiles, units, kmax;
};

// A sequence's extent; every value read from the device arrays is limited to
// what the descriptor allows, so that nothing out of range is ever addressed.
// Token ranges that overlap (offsets that do not ascend) can have more tiles
// than the launch and the workspace were sized for: attend_find then takes none.
template <int MT, int KT>
__device__ __forceinline__ AttendSeq attend_seq(const AttendArgs& a, int b) {
  AttendSeq s;
  const int c0 = min(max(a.cu[b], 0), a.T), c1 = min(max(a.cu[b + 1], c0), a.T);
  const int L = max(a.lens[b], 0);
  s.token0 = c0;
  s.n = c1 - c0;
  // (32 bits hold all of it: n * group <= T * heads < 2^31, and L - n >= -2^31 + 1)
  const int pos0 = L - s.n;
  s.pos0 = pos0;
  s.kmax = min(L, a.cap);
  s.tiles = static_cast<int>((static_cast<uint32_t>(s.n) * static_cast<uint32_t>(a.group) + MT - 1) / MT);
  const int lo = a.window > 0 && pos0 >= a.window ? pos0 - a.window + 1 : 0;
  s.units = s.kmax > lo ? static_cast<int>((static_cast<uint32_t>(s.kmax) + KT - 1) / KT) - lo / KT : 0;
  return s;
}

// Inclusive prefix sum over a wavefront.
__device__ __forceinline__ uint64_t wave_prefix(uint64_t v) {
  const int lane = threadIdx.x & (kWave - 1);
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const uint64_t u = __shfl_up(static_cast<unsigned long long>(v), o, kWave);
    if (lane >= o) v += u;
  }
  return v;
}

constexpr int kLengthClasses = 32;

template <int WAVES>
struct AttendPlanShared {
  uint64_t sum[2][WAVES];
  uint64_t cls[kLengthClasses];
  uint64_t items[WAVES];
  int32_t longest[WAVES];
  AttendItem item;
  int32_t found;
};

// Finds item x of the call.  All threads of the workgroup call it; false (for
// all of them) if there are fewer items.
//
// A sequence's keys are cut into splits of about S units, where S is what
// spreads the call's units evenly over want_items workgroups and at least
// min_units: with many tiles nothing is split, with few rows the key axis
// fills the chip: units / want_items if the splits then round up to want_items
// at most (one workgroup too many of equal ones costs a whole round: 461 against
// 322 us at B = 4, 110k positions), else units / (want_items - tiles), which
// sum tiles * ceil(units / S) <= want_items follows from, or units /
// (want_items / 2) where there is no such room.  There are never more than
// want_items + tiles items, which bounds the launch; the sequences that are
// split have units > S, so they use at most 2 want_items partial slots.  Items are
// numbered from the longest class of splits to the shortest, so that the last
// workgroups to start are the short ones (B = 256, 512 to 4096 positions: 474 -> 437
// us).  Every workgroup makes these sums itself, three or four passes over the batch
// from cache, which costs less than the launch that a separate planning kernel
// would be up to some 2000 sequences (single tokens over 1000 positions: 6.0 TB/s
// of pages at 2048 of them, 5.2 at 4096).
//
// kHeld: the sequences of a thread that are read once and held in registers (each
// pass reads them again where the batch has more, or with 0).
template <int MT, int KT, int WAVES, int kHeld = 0>
__device__ __forceinline__ bool attend_find(const AttendArgs& a, int x, bool count_slots,
                                            AttendPlanShared<WAVES>& sh, AttendItem& it) {
  constexpr int NT = WAVES * kWave;
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  if (tid < kLengthClasses) sh.cls[tid] = 0;
  if (tid == 0) sh.found = 0;
  AttendSeq held[kHeld > 0 ? kHeld : 1];
  if constexpr (kHeld > 0) {
    if (a.B > kHeld * NT) return attend_find<MT, KT, WAVES, 0>(a, x, count_slots, sh, it);
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int b = i * NT + tid;
      held[i] = AttendSeq{};
      if (b < a.B) held[i] = attend_seq<MT, KT>(a, b);
    }
  }
  // f(b, sequence b) for this thread's sequences from the first-th on
  auto each = [&](int first, auto f) {
    if constexpr (kHeld > 0) {
#pragma unroll
      for (int i = 0; i < kHeld; ++i)
        if (i * NT + first < a.B) f(i * NT + first, held[i]);
    } else {
      for (int b = first; b < a.B; b += NT) f(b, attend_seq<MT, KT>(a, b));
    }
  };
  // Sums over the sequences, the same in every thread (the branches on them below
  // hold barriers): reduced, or, of one sequence, made by each thread for itself.
  uint64_t units = 0, tiles = 0;
  int longest = 0;
  auto add = [&](int, const AttendSeq& s) {
    tiles += s.tiles;
    units += static_cast<uint64_t>(s.tiles) * s.units;
    if (s.tiles > 0) longest = max(longest, s.units);
  };
  if (a.B == 1) add(0, attend_seq<MT, KT>(a, 0));
  else each(tid, add);
  if (a.B > 1) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
      tiles += __shfl_xor(static_cast<unsigned long long>(tiles), o, kWave);
      units += __shfl_xor(static_cast<unsigned long long>(units), o, kWave);
      longest = max(longest, __shfl_xor(longest, o, kWave));
    }
    if (WAVES > 1) {
      if (lane == 0) {
        sh.sum[0][wave] = units;
        sh.sum[1][wave] = tiles;
        sh.longest[wave] = longest;
      }
      __syncthreads();
      units = tiles = 0;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) {
        units += sh.sum[0][w];
        tiles += sh.sum[1][w];
        longest = max(longest, sh.longest[w]);
      }
    }
    if (tiles > static_cast<uint64_t>(a.max_tiles)) {   // offsets that do not ascend
      if (count_slots && tid == 0) *a.slot_count = 0;
      return false;
    }
  }
  int S = INT32_MAX;
  if (a.max_slots > 0) {
    // a little over units / n, at least it
    auto share = [&](int n) -> int {
      const float f = static_cast<float>(units) * 1.0001f / static_cast<float>(n);
      return max(a.min_units, f < 1e9f ? static_cast<int>(f) + 1 : INT32_MAX);
    };
    const int64_t room = static_cast<int64_t>(a.want_items) - static_cast<int64_t>(tiles);
    const int over = max(static_cast<int>(max(room, static_cast<int64_t>(0))),
                         (a.want_items + 1) / 2);
    S = share(a.want_items);      // if the splits round up to few enough items
    uint64_t items = tiles;
    if (tiles <= static_cast<uint64_t>(a.want_items) && a.B == 1) {
      items = tiles * max((static_cast<uint32_t>(longest) + S - 1) / S, 1u);
    } else if (tiles <= static_cast<uint64_t>(a.want_items)) {
      items = 0;
      each(tid, [&](int, const AttendSeq& s) {
        items += static_cast<uint64_t>(s.tiles) *
                 max((static_cast<uint32_t>(s.units) + S - 1) / S, 1u);
      });
#pragma unroll
      for (int o = 32; o > 0; o >>= 1)
        items += __shfl_xor(static_cast<unsigned long long>(items), o, kWave);
      if (WAVES > 1) {
        if (lane == 0) sh.items[wave] = items;
        __syncthreads();
        items = 0;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) items += sh.items[w];
      }
    }
    if (items > static_cast<uint64_t>(a.want_items)) S = share(over);
  }
  // splits of a sequence, their length's class and its (items << 32) + slots
  const int top = min(longest, S);
  auto shape = [&](const AttendSeq& s, int& splits, int& cls) -> uint64_t {
    splits = s.units > S ? static_cast<int>((static_cast<uint32_t>(s.units) + S - 1) / S) : 1;
    // (any class is right: it only orders the items, the same way in every workgroup)
    const float len = static_cast<float>(s.units) * kLengthClasses /
                      (static_cast<float>(splits) * static_cast<float>(top + 1));
    const int c = static_cast<int>(len);
    cls = kLengthClasses - 1 - min(max(c, 0), kLengthClasses - 1);
    const uint64_t items = static_cast<uint64_t>(s.tiles) * splits;
    return (items << 32) + (splits > 1 ? items : 0);
  };
  int my_cls = 0;
  uint64_t carry = 0, all = 0;   // (items << 32) + slots before this class, of the call
  if (a.B > 1) {
    each(tid, [&](int, const AttendSeq& s) {
      int splits, cls;
      const uint64_t mine = shape(s, splits, cls);
      if (mine) atomicAdd(reinterpret_cast<unsigned long long*>(&sh.cls[cls]),
                          static_cast<unsigned long long>(mine));
    });
    __syncthreads();
    const uint64_t n = lane < kLengthClasses ? sh.cls[lane] : 0;
    const uint64_t to = wave_prefix(n);
    const uint64_t with = __ballot(static_cast<int64_t>(to >> 32) > x);
    all = __shfl(static_cast<unsigned long long>(to), kWave - 1, kWave);
    my_cls = with ? __builtin_ctzll(with) : -1;
    carry = with ? __shfl(static_cast<unsigned long long>(to - n), my_cls, kWave) : 0;
  }
  bool done = my_cls < 0;
  // sequences c .. c + NT - 1, one a thread; all threads agree on `done`
  auto search = [&](int c, const AttendSeq& s) {
    const int b = c + tid;
    int splits = 1;
    uint64_t mine = 0;
    if (b < a.B) {
      int cls;
      mine = shape(s, splits, cls);
      if (a.B == 1) all = mine;
      else if (cls != my_cls) mine = 0;
    }
    const uint64_t v = wave_prefix(mine);
    uint64_t here = 0, before = carry;
    if (WAVES > 1) {
      __syncthreads();
      if (lane == kWave - 1) sh.sum[1][wave] = v;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < WAVES; ++w) {
        if (w < wave) before += sh.sum[1][w];
        here += sh.sum[1][w];
      }
    } else {
      here = __shfl(static_cast<unsigned long long>(v), kWave - 1, kWave);
    }
    before += v - mine;
    carry += here;
    const int64_t y = x - static_cast<int64_t>(before >> 32);
    if (y >= 0 && y < static_cast<int64_t>(mine >> 32)) {
      // the tiles of a sequence from its last (with the most keys) to its first
      const uint32_t q = static_cast<uint32_t>(y) / static_cast<uint32_t>(splits);
      const int split = static_cast<int>(static_cast<uint32_t>(y) - q * splits);
      const int tile = s.tiles - 1 - static_cast<int>(q);
      const int rows_all = s.n * a.group;
      AttendItem r;
      r.b = b;
      r.token0 = s.token0;
      r.row0 = tile * MT;
      r.rows = min(MT, rows_all - r.row0);
      r.pos0 = static_cast<int32_t>(s.pos0);
      const int j0 = fast_div(r.row0, a.grp), j1 = fast_div(r.row0 + r.rows - 1, a.grp);
      const int64_t hi = min(s.pos0 + j1 + 1, static_cast<int64_t>(s.kmax));
      const int64_t lo = a.window > 0 ? max(s.pos0 + j0 - a.window + 1, static_cast<int64_t>(0)) : 0;
      r.key_lo = static_cast<int32_t>(min(lo, max(hi, static_cast<int64_t>(0))));
      r.key_hi = static_cast<int32_t>(max(hi, static_cast<int64_t>(r.key_lo)));
      const int f = r.key_lo / KT;
      const int e = r.key_hi > r.key_lo ? (r.key_hi - 1) / KT + 1 : f;
      const int len = static_cast<int>(static_cast<uint32_t>(e - f + splits - 1) /
                                       static_cast<uint32_t>(splits));
      r.u0 = min(e, f + split * len);
      r.u1 = min(e, r.u0 + len);
      r.split = split;
      r.splits = splits;
      r.slot = static_cast<int32_t>(static_cast<uint32_t>(before)) + tile * splits + split;
      sh.item = r;
      sh.found = 1;
    }
    done = static_cast<int64_t>(carry >> 32) > x;
  };
  if constexpr (kHeld > 0) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (i * NT < a.B && !done) search(i * NT, held[i]);
  } else {
    for (int c = 0; c < a.B && !done; c += NT) {
      AttendSeq s{};
      if (c + tid < a.B) s = attend_seq<MT, KT>(a, c + tid);
      search(c, s);
    }
  }
  if (count_slots && tid == 0)   // (thread 0 has the one sequence where B = 1)
    *a.slot_count = static_cast<int32_t>(min(static_cast<uint32_t>(all),
                                             static_cast<uint32_t>(a.max_slots)));
  __syncthreads();
  if (!sh.found) return false;
  it = sh.item;
  return it.splits == 1 || it.slot < a.max_slots;
}

// What a split leaves for the joining launch: the unnormalised output of each
// row relative to its maximum (in log2 units, -inf where it saw nothing) and
// the sum of its weights.
__device__ __forceinline__ void attend_slot_info(const AttendArgs& a, const AttendItem& it) {
  SlotInfo s{};
  s.split = it.split;
  s.splits = it.splits;
  s.token0 = it.token0;
  s.row0 = it.row0;
  s.rows = it.rows;
  a.info[it.slot] = s;
}

// Row r of a tile: token row and query head.
__device__ __forceinline__ void attend_row(const AttendArgs& a, int token0, int row, int h,
                                           int& token, int& head) {
  const int j = fast_div(row, a.grp);
  token = token0 + j;
  head = h * a.group + (row - j * a.group);
}

hipError_t launch_attend_rows(const AttendArgs& a, hipStream_t st);
hipError_t launch_attend_d64(const AttendArgs& a, int dtype, int mt, hipStream_t st);
hipError_t launch_attend_d128(const AttendArgs& a, int dtype, int mt, hipStream_t st);
hipError_t launch_attend_d256(const AttendArgs& a, int dtype, int mt, hipStream_t st);
hipError_t launch_attend_join(const AttendArgs& a, int dtype, int mt, hipStream_t st);

}  // namespace sv
