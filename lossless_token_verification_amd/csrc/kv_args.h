// Argument blocks and helpers of the paged-KV kernels: block-table extension,
// cache append, paged attention.  The C ABI is include/spec_kv.h.
#pragma once

#include "sv_common.h"

namespace sv {

constexpr float kLn2 = 0.6931471805599453f;

// Records the message of a failing call (spec_verify_last_error); returns code.
int32_t record_error(int32_t code, const char* msg) noexcept;

// Division of n < 2^31 by a constant d >= 1 (the page size): with
// s = ceil(log2 d) and m = floor(2^(31+s) / d) + 1, m * d - 2^(31+s) is in
// (0, 2^s], so floor(n * m / 2^(31+s)) is exact for every n < 2^31.
struct FastDiv {
  uint32_t d, m, s;
};
inline FastDiv make_fast_div(uint32_t d) {
  uint32_t s = 0;
  while (s < 31 && (1u << s) < d) ++s;
  return {d, static_cast<uint32_t>((uint64_t{1} << (31 + s)) / d + 1), 31 + s};
}
__device__ __forceinline__ int fast_div(int n, const FastDiv& f) {
  return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(n)) * f.m) >> f.s);
}

struct ExtendArgs {
  int32_t B, max_blocks, block_size, free_capacity, max_freed, T;
  FastDiv bs;
  int32_t* table;
  const int32_t* lens;
  const int32_t* num_new;
  int32_t* free_blocks;
  const int32_t* free_count;
  const int32_t* freed;      // NULL: nothing to push
  const int32_t* num_freed;
  int32_t* new_lens;
  int32_t* num_taken;
  int32_t* free_left;
  int32_t* cu;
  int64_t* slots;
  int32_t* positions;        // NULL: not wanted
};
hipError_t launch_extend(const ExtendArgs& a, hipStream_t st);

struct AppendArgs {
  const void* src[2];        // k, v
  void* dst[2];              // k_cache, v_cache
  const int64_t* slots;
  int32_t T, vec_bytes;      // T * row_vecs < 2^31; bytes one thread moves: 16, or an element
  int32_t row_vecs;          // vectors of one token row (kv_heads * head_vecs)
  int32_t head_vecs;         // vectors of one head of a row
  int32_t num_slots, block_size;
  FastDiv bs, row, head;     // division by block_size, row_vecs, head_vecs
  int64_t src_stride[2];     // vectors between token rows
  int64_t block_stride;      // vectors between blocks
};
hipError_t launch_append(const AppendArgs& a, hipStream_t st);

// Paged attention.  The query rows of a sequence, token-major with the heads
// that share a key head next to each other (row r: token r / group, head
// h * group + r % group), are cut into tiles of MT rows; the keys of a tile
// may be cut into splits.  One workgroup takes one (tile, split, key head).
struct AttendArgs {
  const void* q;
  const void* k;
  const void* v;
  const int32_t* table;
  const int32_t* lens;
  const int32_t* cu;
  void* out;
  float* lse;
  int32_t B, T, heads, kv_heads, group, D, block_size, num_blocks, max_blocks, window;
  FastDiv bs, grp;
  int64_t q_stride, block_stride;   // elements
  int32_t cap;                      // positions the table can hold (limited to 2^31 - 1)
  float scale;
  // work split (all host-side, from the descriptor)
  int32_t want_items;   // (tile, split) items per key head that fill the chip
  int32_t min_units;    // fewest key units (of the kernel's KT keys) of a split
  int32_t max_slots;    // partial slots per key head in the workspace (0: never split)
  int32_t grid_items;   // launched (tile, split) items per key head
  int64_t max_tiles;    // most tiles of token ranges that do not overlap
  struct SlotInfo* info;   // [max_slots]
  int32_t* slot_count;     // slots in use
  float* part_o;        // [max_slots * kv_heads, MT, D]
  float* part_ml;       // [max_slots * kv_heads, MT, 2]: running maximum and sum
};
// What the joining launch needs to know of a partial slot.
struct SlotInfo {
  int32_t split, splits;   // which split of its tile this slot holds, of how many
  int32_t token0, row0;    // the sequence's first token row, the tile's first query row
  int32_t rows;            // query rows of the tile
};

// Element types, as in the C ABI.
constexpr int kF32 = 0, kBF16 = 1, kF16 = 2;
// Query rows per tile of the vector-unit kernel, by head size.
constexpr int kRowsMT64 = 4, kRowsMT128 = 4, kRowsMT256 = 2, kRowsKT = 32;

// A kernel variant: query rows per tile, keys per unit, workgroups that fill
// the chip, keys a split is worth at least.
struct AttendShape {
  int32_t mt, kt, wgs, min_units;
  bool matrix;   // on the matrix cores
};

}  // namespace sv
