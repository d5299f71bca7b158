// Paged attention over a cache held in 4 bits, on the matrix instructions that take
// 4-bit operands with a power of two per 32 of their terms (head_dim 64, 128, 256,
// and every other multiple of 32 in the next of these, the rest of a row zero).
//
// The codes are never unpacked.  Both products are formed transposed, as in the
// 16-bit kernel (a lane holds one query row throughout):
//     S^T = K Q^T     A = key codes from LDS with their block scales
//     O^T += V^T P^T  A = value codes from LDS, transposed by the read
// and what stands against the codes is split into pieces that the instructions take
// at the 4-bit rate: 6-bit numbers (e2m3: 4 significant bits, magnitudes to 7.5, step
// 1/8 up to 2, 1/4 up to 4, 1/2 above) with a power of two s per 32.  The second piece
// holds what the first leaves over s / 32, and so on.
//   Scaled so that the largest of the 32 is in [2, 4) s, a piece leaves an eighth at
//   most, 4 of the next one's units: n pieces are off by 2^-(5n - 1) of the largest.
//   Queries, as they are: 3 pieces for bfloat16 (2^-14 of the largest of 32 channels;
//   its 8 bits are held whole down to a 128th of that), 4 for float16 (2^-19; 11 bits
//   down to a 512th), and 4 at head_dim 64, where two lie side by side in a step of
//   128 terms.  The scale is applied to their products, in the weights' exponent: the
//   pieces of a query times 24 bits of a scale held none of it whole, and every lse was
//   off by that.
//   Weights times their value's scale: 3 pieces (2^-14 of the largest of the 32
//   positions that a lane holds).  Two would be faster in bfloat16 (256 windows of 9
//   tokens 173 us against 194, four prompts 359 against 405), but end at 2^-11 of the
//   largest: 31 weights just below that were missing from the output, 1.4 % of it, and
//   not from the sum of the weights.  The largest is taken anew for every 32 positions, so
//   that many small weights far from a large one are not lost; the sum of the weights is
//   taken before, in float32.
// The products are exact in the instruction, their sums float32.  Codes hold no
// infinity: a position that a row does not see has weight 0 and value scale 0, and
// needs no more care than that.
//
// A wavefront takes 16 query rows (of the tokens of one sequence and the heads that
// share a key head), a workgroup 1 to 4 of them, so that one load of a unit of 128
// positions (8704 bytes of keys, as many of values, at head_dim 128) serves them all.  Two
// units lie in LDS, loaded directly.  The weights and their split (some 370 vector
// instructions a unit for 16 rows) are what no row shares with another.
// What bounds it, bfloat16, 32 query and 8 key heads of 128 (shares of the cycles by
// the counters; loads: with the arithmetic left out):
//   256 sequences of 512 to 4096 positions, 9 tokens each (719 MB): 185 us, 3.9 TB/s; the
//     loads take 137 (a short sequence fills its buffers anew), vector instructions are
//     issued in 56 % of the cycles, the matrix cores busy in 19 %;
//   4 sequences of 125000, single tokens (553 MB): 106 us, 5.2 TB/s, the loads (102);
//   4 prompts of 2200 to 3800 tokens (332 GFLOP): 395 us; the vector instructions of
//     softmax and splits (74 % of the cycles), then the matrix cores (24 %), not the
//     loads (138).
#pragma once

#include "kvattend_mfma.h"
#include "kvattend_q4.h"

namespace sv {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x6 __attribute__((ext_vector_type(6)));
typedef float f32x32 __attribute__((ext_vector_type(32)));

// Codes (4 bits, A) times pieces (6 bits, B), each with its scale's byte.
template <int kByte = 0>   // of piece_scale: the piece's
__device__ __forceinline__ f32x4 mma_q4(u32x4 codes, int code_scale, u32x6 piece, int piece_scale,
                                        f32x4 c) {
  const i32x8 x = {static_cast<int>(codes[0]), static_cast<int>(codes[1]),
                   static_cast<int>(codes[2]), static_cast<int>(codes[3]), 0, 0, 0, 0};
  const i32x8 y = {static_cast<int>(piece[0]), static_cast<int>(piece[1]),
                   static_cast<int>(piece[2]), static_cast<int>(piece[3]),
                   static_cast<int>(piece[4]), static_cast<int>(piece[5]), 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 4, 2, 0, code_scale, kByte,
                                                          piece_scale);
}

// 32 numbers, even ones in x0 and odd ones in x1, over the power of two s as 6-bit
// numbers (ties to even, at most 7.5), and back.  The instructions write their results
// while they still read, so the two may share no register: the early clobber says so
// (the compiler's own forms of them do not, and it does let them overlap).  A matrix
// instruction may read the result two states later; the compiler, which does not see
// what is in here, would not wait for that.
__device__ __forceinline__ u32x6 to_fp6(f32x16 x0, f32x16 x1, float s) {
  u32x6 y;
  asm("v_cvt_scalef32_2xpk16_fp6_f32 %0, %1, %2, %3\n\ts_nop 1"
      : "=&v"(y) : "v"(x0), "v"(x1), "v"(s));
  return y;
}
__device__ __forceinline__ f32x32 from_fp6(u32x6 x, float s) {
  f32x32 y;
  asm("v_cvt_scalef32_pk32_f32_fp6 %0, %1, %2" : "=&v"(y) : "v"(x), "v"(s));
  return y;
}

// The N pieces of 32 numbers, even ones in x0 and odd ones in x1, the largest of
// magnitude `top` (as bits), scaled so that it is in [2, 4).  Numbers below 2^-102 lose
// bits (the first piece's scale is 2^-103 at least, so that the last one's is a number).
template <int N>
__device__ __forceinline__ void split_pieces(f32x16 x0, f32x16 x1, uint32_t top, u32x6 (&piece)[N],
                                             int (&scale)[N]) {
#pragma clang fp contract(off)
  const int b = max(static_cast<int>(top >> 23) - 1, 24);
#pragma unroll
  for (int p = 0; p < N; ++p) {
    const float s = __uint_as_float(static_cast<uint32_t>(b - 5 * p) << 23);
    piece[p] = to_fp6(x0, x1, s);
    // infinity or NaN among them: NaN
    scale[p] = top >= 0x7f800000u ? 255 : b - 5 * p;
    if (p + 1 < N) {
      const f32x32 y = from_fp6(piece[p], s);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        x0[i] -= y[2 * i];
        x1[i] -= y[2 * i + 1];
      }
    }
  }
}

// Waits for the wavefront's LDS reads, not for its loads under way.
__device__ __forceinline__ void wait_entries() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xc07f);     // vector memory 63, LDS 0
  asm volatile("" ::: "memory");
}

template <typename T_, int D_, bool kPad_, int W_>
struct Q4Cfg {
  using T = T_;
  static constexpr bool kPad = kPad_;
  static constexpr int D = D_, W = W_, KT = kQ4KT, MT = 16 * W;
  static constexpr bool kBf = std::is_same<T, __bf16>::value;
  // pieces; at D = 64 two of a query's lie side by side in one step
  static constexpr int PQ = D == 64 || !kBf ? 4 : 3, PP = 3;
  static constexpr int HALVES = D == 256 ? 2 : 1;          // steps along a row
  static constexpr int QS = D == 64 ? PQ / 2 : PQ;         // steps of a half
  static constexpr int ROW = D / 2;                        // bytes of a row of codes
  static constexpr int NV = D / 32;                        // its 16-byte vectors
  static constexpr int RPL = kWave / NV;                   // rows of one direct load
  static constexpr int LOADS = KT / RPL;                   // of K and of V, per unit
  static constexpr int SW = D == 256 ? 2 : 1;              // words of key scales a row
  static constexpr int kV = KT * ROW, kKS = 2 * kV;        // bytes: V codes, key scales,
  static constexpr int kVS = kKS + SW * KT * 4;            //   value scales
  static constexpr int BYTES = kVS + KT * 4;
  static constexpr int CHUNKS = (LOADS + W - 1) / W;       // loads of a wavefront
  static constexpr int IDS = (CHUNKS * RPL + kWave - 1) / kWave;   // its lookups, per unit
  static constexpr int OT = D / 16;                        // result tiles
  // Sequences of a thread that the work search holds in registers: 256 single tokens over
  // 100 positions take 26.0 us, 28.3 without; over 2300 133 and 138.
  static constexpr int kHeld = W < 3 ? 4 : 2;
  // Nontemporal loads where a sequence's keys are mostly read by one tile: 256 sequences of
  // 2300 positions, single tokens 133 against 142 us, 9 tokens 189 against 194; with more
  // tiles the next one finds keys in the cache (prompts of 2500 270 against 264).
  static constexpr bool kOnce = MT <= 48;
  // Wavefronts to a SIMD, by the registers.  Three, although some values then lie in
  // scratch memory (12 to 40 bytes a lane): 256 sequences of 2300, 9 tokens, head_dim 128
  // bfloat16 190 us against 218 with two, float16 197 against 231, head_dim 64 (512 to
  // 4096 positions) 140 against 185; prompts of 2500 264 and 307, 278 and 317, 222 and 268.
  // Two where three spill in the loop: head_dim 256, prompts 455 against 706 (up to 64
  // bytes with two), or have no more to hide: one wavefront of head_dim 64 73 against 83.
  static constexpr int kPerSimd = D == 256 || W == 1 || (D == 128 && W == 2) ? 2 : 3;
};

// LDS vector permutation of row r: vector v lies at v ^ swz(r), so that the 16 rows
// that 16 lanes read transposed (4 neighbours in each of 4 places, 16 vectors in all)
// fall on different banks.
template <int D>
__device__ __forceinline__ int swz_q4(int r) {
  return D == 64 ? (r >> 3) & 1 : D == 128 ? (r >> 2) & 3 : (r >> 1) & 7;
}

template <class C>
__global__ __launch_bounds__(4 * kWave) __attribute__((amdgpu_waves_per_eu(C::kPerSimd))) void
attend_q4_kernel(AttendArgs a, Q4Cache cache) {
  using T = typename C::T;
  constexpr int D = C::D, KT = C::KT, ROW = C::ROW, NV = C::NV, RPL = C::RPL, OT = C::OT;
  constexpr int IDS = C::IDS, CHUNKS = C::CHUNKS, HALVES = C::HALVES, QS = C::QS, PQ = C::PQ, PP = C::PP;
  // (two LDS objects: a direct load into one is known to leave the other alone)
  __shared__ __attribute__((aligned(1024))) char sb0[C::BYTES], sb1[C::BYTES];
  __shared__ __attribute__((aligned(256))) int32_t sid[C::W * 2 * IDS * kWave];
  __shared__ int32_t missing[8];   // unit + 1 where a page of the unit is missing
  __shared__ AttendPlanShared<C::W> plan;
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int dim = C::kPad ? a.D : D, row_bytes = dim / 2;
  const int x = blockIdx.x / a.kv_heads, h = blockIdx.x - x * a.kv_heads;
  AttendItem it;
  if (!attend_find<C::MT, KT, C::W, C::kHeld>(a, x, a.max_slots > 0 && blockIdx.x == 0, plan, it)) return;
  if (it.splits > 1 && h == 0 && tid == 0) attend_slot_info(a, it);

  // this lane's query row (rows past the tile repeat its last one) and the quarter
  // of a step's 128 terms it holds
  const int g = lane >> 4;
  const int row = wave * 16 + (lane & 15);
  int see_lo;
  uint32_t see_span;     // the positions it sees: see_span of them from see_lo on, and that one
  int q_token, q_head;
  {
    attend_row(a, it.token0, it.row0 + min(row, it.rows - 1), h, q_token, q_head);
    const int pos = it.pos0 + q_token - it.token0;
    const int key_last = min(pos, it.key_hi - 1);
    const int key_first = a.window > 0 && pos >= a.window ? pos - a.window + 1 : 0;
    see_lo = key_last >= key_first ? key_first : INT32_MIN;
    see_span = key_last >= key_first ? key_last - key_first : 0;
  }
  // positions every row of the tile may see: units inside need no mask
  const int all_hi = min(it.pos0 + fast_div(it.row0, a.grp), it.key_hi - 1);
  const int pos_last = it.pos0 + fast_div(it.row0 + it.rows - 1, a.grp);
  const int all_lo = a.window > 0 && pos_last >= a.window ? pos_last - a.window + 1 : 0;

  const int32_t* table = a.table + static_cast<int64_t>(it.b) * a.max_blocks;
  // (rows of the cache are numbered in 32 bits)
  const uint32_t head_rows = static_cast<uint32_t>(h) * a.block_size;
  const uint32_t block_rows = static_cast<uint32_t>(a.kv_heads) * a.block_size;
  // A unit's rows are loaded RPL at a time, CHUNKS loads of neighbouring rows by each
  // wavefront.  Lane l looks up the l-th of its wavefront's rows (and the 64 + l-th): its
  // number in the cache, and whether there is such a page.  Positions outside the
  // item's range read the nearest one inside (and are masked); a missing page reads
  // block 0.
  const int wave_row = wave * (CHUNKS * RPL);
  auto in_unit = [&](int i) { return wave_row + i * kWave + lane; };   // (may be past the unit)
  auto own_row = [&](int i) { return i * kWave + lane < CHUNKS * RPL && in_unit(i) < KT; };
  // (past 2^31 - 1, behind the last unit of the longest sequences, that is key_lo)
  auto nearest = [&](uint32_t key) { return min(max(static_cast<int>(key), it.key_lo), it.key_hi - 1); };
  auto paged = [&](int id) { return id >= 0 && id < a.num_blocks; };
  int32_t* const ids = sid + wave * (2 * IDS * kWave);
  auto look = [&](int slot, uint32_t base) {     // starts the lookups of the unit at position `base`
#pragma unroll
    for (int i = 0; i < IDS; ++i)
      __builtin_amdgcn_global_load_lds((gptr_t)(table + fast_div(nearest(base + in_unit(i)), a.bs)),
                                       (lptr_t)(ids + (slot * IDS + i) * kWave), 4, 0, 0);
  };
  uint32_t off[IDS];
  auto turn = [&](int slot, int n, uint32_t base) {   // the n-th unit, looked up, is the next to load
#pragma unroll
    for (int i = 0; i < IDS; ++i) {
      const int id = ids[(slot * IDS + i) * kWave + lane];
      const int key = nearest(base + in_unit(i));
      off[i] = (paged(id) ? id : 0) * block_rows + head_rows +
               (key - fast_div(key, a.bs) * a.block_size);
      if (__any(!paged(id) && own_row(i))) missing[n & 7] = n + 1;
    }
  };
  // Loads the unit at position `base` into LDS.  Inside the item's range, with whole
  // pages of rows, a load's address is one lane's row plus a lane constant and moves
  // through scalar registers.
  const int lq = lane / NV, lslot = lane & (NV - 1);
  const bool whole_rows = a.block_size % RPL == 0;
  auto load_unit = [&](uint32_t from_key, char* sb) {
    const int base = static_cast<int>(from_key);
    const bool inside = whole_rows && base >= it.key_lo && base <= it.key_hi - KT;
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) {
      const int j = wave * CHUNKS + i;               // which RPL rows
      if (C::LOADS % CHUNKS != 0 || C::W * CHUNKS > C::LOADS)
        if (j >= C::LOADS) break;
      const int from = i * RPL & (kWave - 1);
      const uint32_t rows = off[i * RPL / kWave];
      const int vec = lslot ^ swz_q4<D>(j * RPL + lq);
      if (inside) {
        const uint32_t r = __builtin_amdgcn_readlane(rows, from);
        const int64_t at = static_cast<int64_t>(r) * row_bytes;
        const uint32_t in = fresh(lq * row_bytes + vec * 16);
        if (!C::kPad || vec * 16 < row_bytes) {
          load_lds<C::kOnce>(cache.k_codes + at + in, sb + j * 1024);
          load_lds<C::kOnce>(cache.v_codes + at + in, sb + C::kV + j * 1024);
        }
        asm volatile("; scalar addresses");   // keeps the two forms from being merged
      } else {
        const uint32_t r = __shfl(rows, from + lq, kWave);
        const int64_t at = static_cast<int64_t>(r) * row_bytes + fresh(vec * 16);
        if (!C::kPad || vec * 16 < row_bytes) {
          load_lds<C::kOnce>(cache.k_codes + at, sb + j * 1024);
          load_lds<C::kOnce>(cache.v_codes + at, sb + C::kV + j * 1024);
        }
      }
    }
    // the scales of the same rows (a direct load's place in LDS is one for the
    // wavefront, and 4 bytes on for each lane: neighbouring rows need one load)
#pragma unroll
    for (int i = 0; i < IDS; ++i) {
      if (!own_row(i)) continue;
      const int to = (wave_row + i * kWave) * 4;
#pragma unroll
      for (int w = 0; w < C::SW; ++w)
        __builtin_amdgcn_global_load_lds(
            (gptr_t)(cache.k_scales + static_cast<int64_t>(off[i]) * (4 * C::SW) + w * 4),
            (lptr_t)(sb + C::kKS + w * KT * 4 + to), 4, 0, 0);
      __builtin_amdgcn_global_load_lds((gptr_t)(cache.v_scales + off[i]),
                                       (lptr_t)(sb + C::kVS + to), 4, 0, 0);
    }
  };

  // The queries, the first lookups and loads.
  u32x4 raw[HALVES][4];
  {
    const T* qr = static_cast<const T*>(a.q) + q_token * a.q_stride + static_cast<int64_t>(q_head) * dim;
#pragma unroll
    for (int hf = 0; hf < HALVES; ++hf) {
      const int group = D == 64 ? g & 1 : hf * 4 + g;      // the lane's 32 channels
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        raw[hf][i] = u32x4{0, 0, 0, 0};
        if (!C::kPad || group * 32 < dim) raw[hf][i] = reinterpret_cast<const u32x4*>(qr)[group * 4 + i];
      }
    }
  }
  const int n_units = it.u1 - it.u0;
  auto unit_key = [&](int n) { return static_cast<uint32_t>(it.u0 + n) * KT; };   // of the n-th unit
  if (n_units > 0) {
    look(0, unit_key(0));
    look(1, unit_key(1));
    if (C::kPad) {
      // (vectors that a row does not have are loaded by no one: zero from here on)
      for (int i = tid; i < C::kKS / 16; i += C::W * kWave) {
        reinterpret_cast<u32x4*>(sb0)[i] = u32x4{0, 0, 0, 0};
        reinterpret_cast<u32x4*>(sb1)[i] = u32x4{0, 0, 0, 0};
      }
    }
    if (tid < 8) missing[tid] = 0;
    wait_loads();
    __syncthreads();
    turn(0, 0, unit_key(0));
    load_unit(unit_key(0), sb0);
    turn(1, 1, unit_key(1));
    wait_entries();
    look(0, unit_key(2));
  }
  u32x6 qf[HALVES][QS];
  int qs[HALVES];        // a byte for each step's pieces
  {
#pragma unroll
    for (int hf = 0; hf < HALVES; ++hf) {
      f32x16 x0, x1;
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        typedef T t8 __attribute__((ext_vector_type(8)));
        const t8 v = __builtin_bit_cast(t8, raw[hf][i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x0[i * 4 + j] = static_cast<float>(v[2 * j]);
          x1[i * 4 + j] = static_cast<float>(v[2 * j + 1]);
          top = max(top, __float_as_uint(x0[i * 4 + j]) & 0x7fffffffu);
          top = max(top, __float_as_uint(x1[i * 4 + j]) & 0x7fffffffu);
        }
      }
      u32x6 piece[PQ];
      int scale[PQ];
      split_pieces<PQ>(x0, x1, top, piece, scale);
      qs[hf] = 0;
#pragma unroll
      for (int s = 0; s < QS; ++s) {
        qf[hf][s] = piece[D == 64 ? 2 * s : s];
        int byte = scale[D == 64 ? 2 * s : s];
        if (D == 64 && g >= 2) {
          qf[hf][s] = piece[D == 64 ? 2 * s + 1 : s];
          byte = scale[D == 64 ? 2 * s + 1 : s];
        }
        qs[hf] |= byte << (8 * s);
      }
    }
  }
  // Weights are 2^(factor * product - ref): the reference of a row, in log2 units, lies
  // kSlack above its largest score where it moved last: 2^-kSlack is the largest weight
  // then, and a lane's 32 add up to an eighth at most.
  // It moves again when the weights of one of the row's four lanes add up to more than
  // 1, which takes no maximum over the scores in the other units.  The other rows of the
  // tile have no part in that: theirs stay, and so do their bits.  most: that limit, or -1
  // until the row sees a position (its reference is 0 till then), so that any sum is over it.
  constexpr float kMost = 1.0f;
  const float factor = a.scale * kLog2e;
  f32x4 o[OT];
  float ref = 0.0f, most = -1.0f, l = 0.0f;
#pragma unroll
  for (int t = 0; t < OT; ++t) o[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  // Operand reads.  Keys: lane's row of 16, its 32 channels.  Values: a transposed
  // read gives lane n of 16 channel n of 16 rows, of which lane n fetches the n-th.
  // The pieces of a lane's weights alternate between its 16 results of the lower and
  // of the upper 64 positions (even and odd terms), so the 16 rows of the first read
  // are 4 g + {0 .. 3} + {0, 16} of both halves in turn, of the second 32 further on.
  const int krow = lane & 15;
  const int kgroup = D == 64 ? g & 1 : g;
  const int koff = krow * ROW + ((kgroup ^ swz_q4<D>(krow)) << 4);
  const int ksoff = krow * 4 + kgroup;
  const int n16 = lane & 15;
  const int vkey = 64 * (n16 & 1) + 16 * (n16 >> 3) + 4 * g + ((n16 >> 1) & 3);
  const int voff = vkey * ROW + (swz_q4<D>(vkey) << 4);

  // The products of unit u: st[t][r] of position 16 t + r and the lane's part 4 g, -inf
  // where it is not seen (masked: there may be such; dead: their bits 4 t + r).
  auto scores = [&](const char* sb, int u, int n, f32x4 (&st)[8], bool masked,
                    uint32_t& dead) {
#pragma unroll
    for (int hf = 0; hf < HALVES; ++hf) {
      u32x4 k[8];
      int ks[8];
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        k[t] = *reinterpret_cast<const u32x4*>(sb + (koff ^ (hf << 6)) + t * 16 * ROW);
        ks[t] = static_cast<uint8_t>(sb[C::kKS + hf * KT * 4 + ksoff + t * 64]);
        if (C::kPad && (hf * 4 + kgroup) * 32 >= dim) ks[t] = 0;
      }
#pragma unroll
      for (int t = 0; t < 8; ++t)
        st[t] = mma_q4<0>(k[t], ks[t], qf[hf][0], qs[hf], hf ? st[t] : f32x4{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
      for (int t = 0; t < 8; ++t) st[t] = mma_q4<1>(k[t], ks[t], qf[hf][1], qs[hf], st[t]);
      if constexpr (QS > 2) {
#pragma unroll
        for (int t = 0; t < 8; ++t) st[t] = mma_q4<2>(k[t], ks[t], qf[hf][2], qs[hf], st[t]);
      }
      if constexpr (QS > 3) {
#pragma unroll
        for (int t = 0; t < 8; ++t) st[t] = mma_q4<3>(k[t], ks[t], qf[hf][3], qs[hf], st[t]);
      }
    }
    if (!masked) return;
    // a row that sees nothing has span 0 at a position that is none
    const uint32_t d = static_cast<uint32_t>(u * KT + 4 * g) - static_cast<uint32_t>(see_lo);
    dead = 0;
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        dead |= (d + t * 16 + r > see_span ? 1u : 0u) << (4 * t + r);
    if (missing[n & 7] == n + 1) {
      const int b0 = u * KT + lane;
      const uint64_t page0 = __ballot(paged(table[fast_div(nearest(b0), a.bs)]));
      const uint64_t page1 = __ballot(paged(table[fast_div(nearest(b0 + kWave), a.bs)]));
#pragma unroll
      for (int t = 0; t < 8; ++t)
        dead |= (~static_cast<uint32_t>((t < 4 ? page0 : page1) >> (16 * (t & 3) + 4 * g)) & 15u)
                << (4 * t);
    }
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) st[t][r] = (dead >> (4 * t + r)) & 1 ? -INFINITY : st[t][r];
  };
  // The weights of the lane's positions and their sum; times their scales in x0 (the
  // lower 64 positions) and x1 (the upper).
  auto weigh = [&](const char* sb, const f32x4 (&st)[8], f32x16& x0, f32x16& x1) -> float {
#pragma clang fp contract(off)
    float sum = 0.0f;
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const f32x4 vs = *reinterpret_cast<const f32x4*>(sb + C::kVS + (t * 16 + 4 * g) * 4);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(st[t][r], factor, -ref));
        sum += p;
        if (t < 4) x0[t * 4 + r] = p * vs[r];
        else x1[(t - 4) * 4 + r] = p * vs[r];
      }
    }
    return sum;
  };
  // Moves the references of the rows that are over their limit to these products.
  auto move_up = [&](const f32x4 (&st)[8], bool over) {
    float mx = st[0][0];
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) mx = fmaxf(mx, st[t][r]);
    mx = max_across<16>(mx);
    mx = max_across<32>(mx);
    mx *= factor;
    const bool move = over && mx > -INFINITY;
    const float to = move ? mx + kSlack : ref;
    // (0 where the row has seen nothing before)
    const float f = move && most < 0.0f ? 0.0f : __builtin_amdgcn_exp2f(ref - to);
    most = move ? kMost : most;
    ref = to;
    l *= f;
#pragma unroll
    for (int t = 0; t < OT; ++t) o[t] *= f;
  };
  // Unit u, the n-th of the item; kFirst: n is 0.
  auto compute = [&](auto kFirst, const char* sb, int u, int n) {
    const bool masked = u * KT + KT - 1 > all_hi || u * KT < all_lo || missing[n & 7] == n + 1;
    uint32_t dead = 0;
    f32x4 st[8];
    f32x16 x0, x1;
    scores(sb, u, n, st, masked, dead);
    if (decltype(kFirst)::value) move_up(st, true);
    float sum = weigh(sb, st, x0, x1);
    const uint64_t lanes = decltype(kFirst)::value ? 0 : __ballot(sum > most);
    if (lanes != 0) {
      asm volatile("" ::: "memory");        // (formed again: not held through the other units)
      scores(sb, u, n, st, masked, dead);
      const uint64_t rows = lanes | lanes >> 32;
      move_up(st, ((rows | rows >> 16) >> (lane & 15)) & 1);
      sum = weigh(sb, st, x0, x1);
    }
    asm volatile("" : "+v"(sum));       // formed here: 32 weights need not be held until later
    if (masked) {        // (their scales may be anything)
      const uint32_t gone = fresh(static_cast<int>(dead));
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        x0[i] = (gone >> i) & 1 ? 0.0f : x0[i];
        x1[i] = (gone >> (16 + i)) & 1 ? 0.0f : x1[i];
      }
    }
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) top = max(max(top, __float_as_uint(x0[i])), __float_as_uint(x1[i]));
    l += sum;
    u32x6 piece[PP];
    int scale[PP];
    split_pieces<PP>(x0, x1, top, piece, scale);
    const int vo = fresh(voff);
#pragma unroll
    for (int t0 = 0; t0 < OT; t0 += 4) {
      u32x4 v[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        typedef __attribute__((address_space(3))) i32x2* tr_t;
        const char* p = sb + C::kV + (vo ^ ((t0 + t) * 8));
        const i32x2 y0 = __builtin_amdgcn_ds_read_tr4_b64_v2i32((tr_t)(p));
        const i32x2 y1 = __builtin_amdgcn_ds_read_tr4_b64_v2i32((tr_t)(p + 32 * ROW));
        v[t] = u32x4{static_cast<uint32_t>(y0.x), static_cast<uint32_t>(y0.y),
                     static_cast<uint32_t>(y1.x), static_cast<uint32_t>(y1.y)};
      }
#pragma unroll
      for (int s = 0; s < PP; ++s)
#pragma unroll
        for (int t = 0; t < 4; ++t) o[t0 + t] = mma_q4(v[t], 127, piece[s], scale[s], o[t0 + t]);
    }
  };

  if (n_units > 0) {
    // Step n computes unit n from buffer n % 2 while unit n + 1 is under way; the
    // table entries of unit n + 2 are turned into addresses meanwhile and those of
    // unit n + 3 looked up, into LDS as well.  Loads past the last unit read its
    // nearest position again.
    auto step = [&](auto kFirst, int n, int slot, char* now, char* next) {
      wait_loads();
      __builtin_amdgcn_s_barrier();
      load_unit(unit_key(n + 1), next);
      turn(slot, n + 2, unit_key(n + 2));
      look(1 - slot, unit_key(n + 3));
      if (n < n_units) compute(kFirst, now, it.u0 + n, n);
    };
    step(std::true_type{}, 0, 0, sb0, sb1);
    for (int n = 1; n < n_units; n += 2) {
      step(std::false_type{}, n, 1, sb1, sb0);
      step(std::false_type{}, n + 1, 0, sb0, sb1);
    }
    // no load may still be under way when the workgroup gives its LDS back
    wait_loads();
    __syncthreads();
  }
  l += __shfl_xor(l, 16, kWave);
  l += __shfl_xor(l, 32, kWave);
  if (row < it.rows && g == 0) {
    if (it.splits > 1) {
      const int64_t p = (static_cast<int64_t>(it.slot) * a.kv_heads + h) * C::MT + row;
      a.part_ml[p * 2] = most < 0.0f ? -INFINITY : ref;
      a.part_ml[p * 2 + 1] = l;
    } else if (a.lse) {
      int token, head;
      attend_row(a, it.token0, it.row0 + fresh(row), h, token, head);
      a.lse[static_cast<int64_t>(token) * a.heads + head] =
          l == 0.0f ? -INFINITY : (ref + log2f(l)) * kLn2;
    }
  }
  if (it.splits > 1) {
    if (row < it.rows) {
      const int64_t p = (static_cast<int64_t>(it.slot) * a.kv_heads + h) * C::MT + row;
      float* po = a.part_o + p * dim + 4 * g;
#pragma unroll
      for (int t = 0; t < OT; ++t)
        if (!C::kPad || t * 16 < dim) *reinterpret_cast<f32x4*>(po + t * 16) = o[t];
    }
    return;
  }
  // whole output rows: turned in LDS (each wavefront its 16 rows), then 16 bytes a lane
  static_assert(4 * 16 * D * 2 <= C::BYTES, "the rows of four wavefronts fit a buffer");
  char* const turned = sb0 + wave * 16 * D * 2;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  const bool none = l == 0.0f;
  const int mine = lane & 15;
#pragma unroll
  for (int t = 0; t < OT; ++t) {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    const int e = t * 16 + 4 * g;
    const f32x4 y = none ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : o[t] * inv;
    *reinterpret_cast<u32x2*>(turned + mine * (D * 2) + (((e >> 3) ^ swz_k<D>(mine)) << 4) +
                              (e & 4) * 2) = u32x2{pack2<T>(y[0], y[1]), pack2<T>(y[2], y[3])};
  }
  constexpr int OV = D / 8, PER = kWave / OV;   // vectors of an output row, rows a pass
#pragma unroll
  for (int i = 0; i < 16 / PER; ++i) {
    const int r = i * PER + lane / OV, slot = lane & (OV - 1);
    const u32x4 w = *reinterpret_cast<const u32x4*>(turned + r * (D * 2) + ((slot ^ swz_k<D>(r)) << 4));
    if (wave * 16 + r < it.rows && (!C::kPad || slot * 8 < dim)) {
      int token, head;
      attend_row(a, it.token0, it.row0 + wave * 16 + r, h, token, head);
      T* po = static_cast<T*>(a.out) + (static_cast<int64_t>(token) * a.heads + head) * dim;
      reinterpret_cast<u32x4*>(po)[slot] = w;
    }
  }
}

template <class C>
void launch_q4_cfg(const AttendArgs& a, const Q4Cache& c, hipStream_t st) {
  const unsigned grid = static_cast<unsigned>(a.grid_items) * a.kv_heads;
  hipLaunchKernelGGL(attend_q4_kernel<C>, dim3(grid), dim3(C::W * kWave), 0, st, a, c);
}

template <typename T, int D, bool kPad>
hipError_t launch_q4_rows(const AttendArgs& a, const Q4Cache& c, int mt, hipStream_t st) {
  if constexpr (D < 256) {      // (there one wavefront spills: 16 rows go by 32)
    if (mt == 16) {
      launch_q4_cfg<Q4Cfg<T, D, kPad, 1>>(a, c, st);
      return hipGetLastError();
    }
  }
  switch (mt) {
    case 32: launch_q4_cfg<Q4Cfg<T, D, kPad, 2>>(a, c, st); break;
    case 48: launch_q4_cfg<Q4Cfg<T, D, kPad, 3>>(a, c, st); break;
    case 64: launch_q4_cfg<Q4Cfg<T, D, kPad, 4>>(a, c, st); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

template <int D>
hipError_t launch_q4_width(const AttendArgs& a, const Q4Cache& c, int dtype, int mt, hipStream_t st) {
  if (dtype == kBF16)
    return a.D == D ? launch_q4_rows<__bf16, D, false>(a, c, mt, st)
                    : launch_q4_rows<__bf16, D, true>(a, c, mt, st);
  return a.D == D ? launch_q4_rows<_Float16, D, false>(a, c, mt, st)
                  : launch_q4_rows<_Float16, D, true>(a, c, mt, st);
}

}  // namespace sv
