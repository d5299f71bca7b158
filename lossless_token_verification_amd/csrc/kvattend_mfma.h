// Paged attention on the matrix cores (bf16 / f16 caches; head_dim 64, 128 and
// 256, and every other one in the next of these, the rest of a row zero in LDS).
//
// One workgroup takes up to MT query rows of a sequence and key head (the
// heads of a group and the new tokens side by side, so a key is read once for
// all of them) and a range of key units of KT positions.  Both products are
// formed transposed:
//     S^T = K Q^T     (A = keys from LDS, B = queries in registers)
//     O^T += V^T P^T  (A = values from LDS, read transposed; B = weights)
// so that a lane holds one query row throughout (column n = lane of both
// results): its running maximum, sum, mask limits and rescaling factor are
// plain per-lane scalars, and the weights go from the first product's result
// registers to the second one's B operand with a conversion and no exchange --
// the positions that a result register quadruple holds are taken as that
// operand's k order, and V is read in the same order.
//
// Softmax in one pass: weights are 2^(score - m) in log2 units, and m moves, to
// kShift below the largest score, only when a score exceeds that by more than
// kSlack, so the accumulators are rescaled in the first unit and hardly ever
// after.  The weights are rounded to the type for the second product (half a
// step, 2^-8 of a weight in bf16, 2^-11 in f16: a choice that keeps both products
// at the 16-bit rate); their sum is taken before the rounding, in float32.  bf16
// has float32's exponents: kShift = -kSlack keeps weights at 1 and less, so that
// no sum of values overflows that would not with the exact maximum.  f16
// has 5 exponent bits: at kShift = 7 weights reach 2^15, those of 2^-21 of the
// largest and more keep all their bits, smaller ones lose up to 2^-32 of it each
// (131072 keys far below one dominant key: 2^-15 of the output, against f16's
// own 2^-11; with kShift = 0 the whole share of such keys, 0.4 % of the output).
//
// K and V units go from the pages straight into LDS (16-byte direct loads, no
// register stage), the next unit while one is computed.  Two buffers, and as many
// workgroups to a CU as registers and LDS then allow, hide start-up and memory
// latency better than a deeper ring with fewer workgroups (four buffers, head_dim
// 128, B = 256: single tokens over 500 positions 109 us against 94, windows of 9
// tokens over 512 to 4096 431 against 427; the other way only where the items just
// overflow the chip: B = 128 over 2300 positions 211 against 222).  Rows are
// permuted by 16-byte vectors (swz_k, swz_v) so that the operand reads of either
// product spread over all banks.  A row's page comes from the block table a unit
// before its loads, into LDS like them, so that nothing waits for it alone.
//
// What bounds it and what it measured (bf16, 32 query and 8 key heads of 128):
// up to 64 rows the pages' bandwidth (B = 256 verifications of 9 tokens over 512
// to 4096 positions: 2.60 GB in 426 to 428 us, 6.1 TB/s; B = 4 single tokens over 90000
// to 131071: 2.08 GB in 321 to 324 us, 6.4 to 6.5 TB/s; a plain read of such an amount runs at
// 6.9).  With 128 rows the matrix cores (busy 42 % of the cycles) and the vector
// units (53 %), which a wavefront uses in turn and two to a SIMD do not overlap
// further: 4 prompts of 2048 to 4096 tokens 332 GF in 377 to 397 us, 836 to 881 TF;
// 16384 tokens 1000 TF (head_dim 64: 870).  Head sizes between the three move
// fewer bytes in little less time, since buffers, steps and tiles are the next
// one's (B = 64, 9 tokens over 2300 positions: 80 us at 80, 85 at 96, 98 at 128, 170
// at 192, 220 at 256).
#pragma once

#include <type_traits>

#include "kvattend.h"

namespace sv {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr float kSlack = 8.0f;   // log2 units that a weight may grow before m moves

template <typename T>
struct Mma;
template <>
struct Mma<__bf16> {
  static constexpr uint32_t kExp = 0x7f80u;   // exponent bits: all set = not finite
  static constexpr float kShift = -kSlack;    // log2 of the largest weight where m moves
  __device__ static f32x16 mma32(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
  __device__ static f32x4 mma16(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
};
template <>
struct Mma<_Float16> {
  static constexpr uint32_t kExp = 0x7c00u;
  static constexpr float kShift = 7.0f;
  __device__ static f32x16 mma32(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
  __device__ static f32x4 mma16(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
};

// Two floats rounded to the type, packed.
template <typename T>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  typedef T t2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{x, y}), t2));
}

// Maximum over the lane pairs N apart (16 or 32), by lane swaps on the vector
// unit: the two results of swapping a value with itself hold, in every lane,
// the pair's two values.
template <int N>
__device__ __forceinline__ float max_across(float x) {
  const uint32_t w = __float_as_uint(x);
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  u32x2 p;
  if constexpr (N == 32) {
    const auto q = __builtin_amdgcn_permlane32_swap(w, w, false, false);
    p = u32x2{q[0], q[1]};
  } else {
    const auto q = __builtin_amdgcn_permlane16_swap(w, w, false, false);
    p = u32x2{q[0], q[1]};
  }
  return fmaxf(__uint_as_float(p.x), __uint_as_float(p.y));
}

// LDS vector permutation of row r (D / 8 vectors a row; 256 bytes of LDS span
// all banks: two rows at D = 64): vector v of row r lies at v ^ swz(r).  K: the
// 16 consecutive rows an operand read takes at one vector fall on 16 different
// vectors.  V: the 4 rows x 64 bytes (or 8 x 32) that half a wavefront reads
// transposed fall on different banks.  Both maps are linear over xor and depend
// on the low four bits of r (K) or three (V) alone.
template <int D>
__device__ __forceinline__ int swz_k(int r) {
  return D == 64 ? (r >> 1) & 7 : r & 15;
}
template <int D>
__device__ __forceinline__ int swz_v(int r) {
  return D == 64 ? (((r >> 1) & 1) << 2) | (((r >> 2) & 1) << 1)
                 : ((r & 3) << 2) | (((r >> 2) & 1) << 1);
}

// Hides a lane-constant value from the optimiser: what is derived from it is
// formed where it is used (one xor) instead of being held in registers for
// the whole loop.
__device__ __forceinline__ int fresh(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// RW: query rows per wavefront (16 or 32, the matrix instruction's width), W
// wavefronts with different rows; units of KT positions, two under way in turn.
// kPad: head_dim is less than D.
template <typename T_, int D_, bool kPad_, int RW_, int W_, int KT_>
struct AttendCfg {
  using T = T_;
  static constexpr bool kPad = kPad_;
  static constexpr int D = D_, RW = RW_, W = W_, KT = KT_, NB = 2;
  static constexpr int MT = RW * W;
  static constexpr int NV = D / 8;                 // vectors of a row
  static constexpr int RPL = kWave / NV;           // rows of one direct load
  static constexpr int LOADS = KT / RPL / W;       // of K and of V, per wavefront and unit
  static constexpr int SUPER = KT * NB;            // positions of both buffers, a turn
  static constexpr int IDS = SUPER / kWave;        // table lookups per lane and turn
  static constexpr int QS = RW == 32 ? D / 16 : D / 32;     // steps of the first product
  static constexpr int ST = KT / RW;               // its result tiles
  static constexpr int SR = RW == 32 ? 16 : 4;     // registers of a result tile
  static constexpr int PS = RW == 32 ? KT / 16 : KT / 32;   // steps of the second product
  static constexpr int OT = D / RW;                // its result tiles
  // Nontemporal direct loads where a sequence has one tile, which reads a page
  // once (B = 256 verification 511 -> 474 us; at head_dim 256 sequences of many
  // tiles come with 64 rows too, and lose a tenth by them).
  static constexpr bool kOnce = MT <= (D == 256 ? 32 : 64);
  static constexpr int kPerSimd = D == 64 || (D == 128 && RW == 16) ? 3 : 2;   // wavefronts
  static_assert(KT % (RPL * W) == 0 && KT % 32 == 0 && KT <= kWave && SUPER % kWave == 0,
                "unit shape");
};

typedef const void __attribute__((address_space(1)))* gptr_t;
typedef void __attribute__((address_space(3)))* lptr_t;
// 16 bytes per lane from memory straight into LDS (from `l` on, in lane order).
template <bool kOnce>
__device__ __forceinline__ void load_lds(const void* g, void* l) {
  if constexpr (kOnce) __builtin_amdgcn_global_load_lds((gptr_t)g, (lptr_t)l, 16, 0, 2);
  else __builtin_amdgcn_global_load_lds((gptr_t)g, (lptr_t)l, 16, 0, 0);
}

// Waits until none of the wavefront's vector-memory operations and LDS reads are
// under way.  The builtin (counts in the hardware's fields: vector memory in bits
// 0-3 and 14-15, LDS in bits 8-11) is known to the compiler, which then adds no
// wait of its own for the loads it covers.
__device__ __forceinline__ void wait_loads() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(7 << 4);
  asm volatile("" ::: "memory");
}

// The bounds name four wavefronts for every W, two or three of them to a SIMD, for
// which the compiler keeps to 256 or 168 registers and forms the products in them
// (given more, it moves every accumulator through the other half of the file in
// each unit).
template <class C>
__global__ __launch_bounds__(4 * kWave) __attribute__((amdgpu_waves_per_eu(C::kPerSimd))) void
attend_mfma_kernel(AttendArgs a) {
  using T = typename C::T;
  constexpr int D = C::D, RW = C::RW, KT = C::KT, NB = C::NB, NV = C::NV, RPL = C::RPL;
  constexpr int SR = C::SR, ST = C::ST, OT = C::OT, PS = C::PS, QS = C::QS, IDS = C::IDS;
  typedef typename std::conditional<RW == 32, f32x16, f32x4>::type acc_t;
  // K rows, then V rows of a unit.  Each buffer its own LDS object: the compiler
  // then knows that a direct load into one does not change the others, and does
  // not wait for it.
  constexpr int kV = KT * D;   // where the V rows start
  __shared__ __attribute__((aligned(1024))) uint16_t sb0[2 * kV], sb1[2 * kV];
  // looked-up table entries of the next turn, a copy per wavefront
  __shared__ __attribute__((aligned(256))) int32_t sid[C::W * C::SUPER];
  __shared__ AttendPlanShared<C::W> plan;
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int dim = C::kPad ? a.D : D, nv = dim / 8;   // elements and vectors of a row
  const int x = blockIdx.x / a.kv_heads, h = blockIdx.x - x * a.kv_heads;
  AttendItem it;
  if (!attend_find<C::MT, KT, C::W>(a, x, a.max_slots > 0 && blockIdx.x == 0, plan, it)) return;
  if (it.splits > 1 && h == 0 && tid == 0) attend_slot_info(a, it);

  // this lane's query row; rows past the tile repeat its last one
  const int hi_lane = RW == 32 ? lane >> 5 : lane >> 4;   // which part of k a lane holds
  const int row = wave * RW + (lane & (RW - 1));
  // the positions it sees: see_span of them from see_lo on, and that one
  int see_lo;
  uint32_t see_span;
  u32x4 qf[QS];
  {
    int token, head;
    attend_row(a, it.token0, it.row0 + min(row, it.rows - 1), h, token, head);
    const int pos = it.pos0 + token - it.token0;
    const int key_last = min(pos, it.key_hi - 1);
    const int key_first = a.window > 0 && pos >= a.window ? pos - a.window + 1 : 0;
    see_lo = key_last >= key_first ? key_first : INT32_MAX;
    see_span = key_last >= key_first ? key_last - key_first : 0;
    const T* qr = static_cast<const T*>(a.q) + token * a.q_stride + static_cast<int64_t>(head) * dim;
#pragma unroll
    for (int s = 0; s < QS; ++s) {
      const int v = s * (RW == 32 ? 2 : 4) + hi_lane;
      qf[s] = u32x4{0, 0, 0, 0};
      if (!C::kPad || v < nv) qf[s] = reinterpret_cast<const u32x4*>(qr)[v];
    }
  }
  // positions every row of the tile may see: units inside need no mask
  const int all_hi = min(it.pos0 + fast_div(it.row0, a.grp), it.key_hi - 1);
  const int pos_last = it.pos0 + fast_div(it.row0 + it.rows - 1, a.grp);
  const int all_lo = a.window > 0 && pos_last >= a.window ? pos_last - a.window + 1 : 0;

  const int32_t* table = a.table + static_cast<int64_t>(it.b) * a.max_blocks;
  const int64_t head_off = static_cast<int64_t>(h) * a.block_size;
  // Lane l looks up position base + l: its element offset in the caches, and
  // whether there is such a page.  Positions outside the item's range read the
  // nearest one inside (and are masked); a missing page reads block 0.
  auto nearest = [&](int base) { return min(max(base + lane, it.key_lo), it.key_hi - 1); };
  auto entry = [&](int base) { return table + fast_div(nearest(base), a.bs); };
  auto offset = [&](int base, int id) -> int64_t {
    const int key = nearest(base);
    const int r = key - fast_div(key, a.bs) * a.block_size;
    const int safe = id >= 0 && id < a.num_blocks ? id : 0;
    return safe * a.block_stride + (head_off + r) * dim;
  };
  auto paged = [&](int id) -> uint64_t { return __ballot(id >= 0 && id < a.num_blocks); };

  const T* kb = static_cast<const T*>(a.k);
  const T* vb = static_cast<const T*>(a.v);
  // lane part of a direct load: row q of its RPL rows, vector `slot` of that row
  const int lq = lane / NV, lslot = lane & (NV - 1);
  const bool whole_rows = a.block_size % RPL == 0;   // a load's rows share a page
  // Loads the unit at position `base`; off: offsets of 64 positions, the unit's
  // from lane `from` on.  Inside the item's range, with whole pages of rows, a
  // load's address is one lane's offset plus a lane constant, so the offset
  // moves through scalar registers; otherwise every lane fetches its row's.  Lanes
  // of vectors that a row does not have (kPad) load nothing: those places of a
  // buffer are the same in every unit and hold the zeros they started with.
  auto load_unit = [&](int base, int64_t off, int from, uint16_t* sb) {
    constexpr int kUnroll = C::LOADS > (C::kPad ? 4 : 8) ? 4 : C::LOADS;
    int lk = lslot ^ swz_k<D>(lq), lv = lslot ^ swz_v<D>(lq);
    if (D != 128 || C::LOADS > 4) {   // registers are short: formed at each load
      lk = fresh(lk);
      lv = fresh(lv);
    }
    if (whole_rows && base >= it.key_lo && base + KT <= it.key_hi) {
      const int lo = static_cast<int>(off), hi = static_cast<int>(off >> 32);
      const uint32_t lane_row = lq * dim * 2;
#pragma unroll kUnroll
      for (int i = 0; i < C::LOADS; ++i) {
        const int j = wave + i * C::W;               // which RPL rows
        const uint32_t r0 = __builtin_amdgcn_readlane(lo, from + j * RPL);
        const uint32_t r1 = __builtin_amdgcn_readlane(hi, from + j * RPL);
        const int64_t ro = static_cast<int64_t>((static_cast<uint64_t>(r1) << 32) | r0);
        const uint32_t ko = lane_row + (lk ^ swz_k<D>(j * RPL)) * 16;
        const uint32_t vo = lane_row + (lv ^ swz_v<D>(j * RPL)) * 16;
        if (!C::kPad || (lk ^ swz_k<D>(j * RPL)) < nv)
          load_lds<C::kOnce>(reinterpret_cast<const char*>(kb + ro) + ko, sb + j * 512);
        if (!C::kPad || (lv ^ swz_v<D>(j * RPL)) < nv)
          load_lds<C::kOnce>(reinterpret_cast<const char*>(vb + ro) + vo, sb + kV + j * 512);
      }
      asm volatile("; scalar addresses");   // keeps the two forms from being merged
      return;
    }
#pragma unroll kUnroll
    for (int i = 0; i < C::LOADS; ++i) {
      const int j = wave + i * C::W;
      const int64_t ro = __shfl(static_cast<long long>(off), from + j * RPL + lq, kWave);
      const int vk = lk ^ swz_k<D>(j * RPL), vv = lv ^ swz_v<D>(j * RPL);
      if (!C::kPad || vk < nv) load_lds<C::kOnce>(kb + ro + vk * 8, sb + j * 512);
      if (!C::kPad || vv < nv) load_lds<C::kOnce>(vb + ro + vv * 8, sb + kV + j * 512);
    }
  };

  acc_t o[OT];
  float m, l;
  const float c = a.scale * kLog2e;

  // Operand reads.  Byte offset of the lane's part at step / tile 0; the others
  // differ by an xor inside the row and by whole rows.
  const int krow = lane & (RW - 1);
  const int koff = krow * (D * 2) + ((hi_lane ^ swz_k<D>(krow)) << 4);
  constexpr int kKStep = RW == 32 ? 32 : 64;       // bytes of a row per step
  // V, k order of the operand = positions of the result registers.  32 wide:
  // 4h + i and 8 + 4h + i of 16; 16 wide: 4g + i and 16 + 4g + i of 32.  A
  // transposed read gives lane n of 16 element n of 4 rows; lane n fetches row
  // n / 4, elements 4 (n % 4) ..
  const int vrow = 4 * hi_lane + ((lane & 15) >> 2);
  const int vvec = (RW == 32 ? ((lane >> 4) & 1) * 2 : 0) + ((lane & 3) >> 1);
  const int voff = vrow * (D * 2) + ((vvec ^ swz_v<D>(vrow)) << 4) + (lane & 1) * 8;
  constexpr int kVTile = RW * 2;                    // bytes of a row per result tile
  constexpr int kVSpan = RW == 32 ? 16 : 32;        // positions per step
  auto vread = [&](const uint16_t* sb, int vo, int s, int ot) -> u32x4 {
    typedef __attribute__((address_space(3))) s16x4* tr_t;
    const char* p = reinterpret_cast<const char*>(sb + kV) + (vo ^ (ot * kVTile)) + s * kVSpan * D * 2;
    const s16x4 x0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((tr_t)(p));
    const s16x4 x1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((tr_t)(p + kVSpan * D));
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    const u32x2 y0 = __builtin_bit_cast(u32x2, x0), y1 = __builtin_bit_cast(u32x2, x1);
    return u32x4{y0.x, y0.y, y1.x, y1.y};
  };
  auto mma = [&](u32x4 x, u32x4 y, acc_t z) -> acc_t {
    if constexpr (RW == 32) return Mma<T>::mma32(x, y, z);
    else return Mma<T>::mma16(x, y, z);
  };

  // One unit.  The scores and weights of its positions: pf gets the weights in
  // the second product's operand form, `scale` is called with the factor of the
  // accumulators where the maximum moves.  pages: which positions have a page.
  auto weigh = [&](const uint16_t* sb, int u, uint64_t pages, u32x4 (&pf)[PS], auto always_mask,
                   auto scale) {
    acc_t st[ST];
    const int ko = fresh(koff);
#pragma unroll
    for (int t = 0; t < ST; ++t) {
#pragma unroll
      for (int r = 0; r < SR; ++r) st[t][r] = 0.0f;
#pragma unroll
      for (int s = 0; s < QS; ++s)
        st[t] = mma(*reinterpret_cast<const u32x4*>(reinterpret_cast<const char*>(sb) +
                                                    (ko ^ (s * kKStep)) + t * RW * D * 2),
                    qf[s], st[t]);
    }
    // position of register r of tile t, less the lane's part 4 * hi_lane
    auto at = [&](int t, int r) { return t * RW + (RW == 32 ? (r >> 2) * 8 + (r & 3) : r); };
    constexpr uint64_t kEvery = KT == 64 ? ~uint64_t{0} : (uint64_t{1} << (KT & 63)) - 1;
    pages &= kEvery;
    if (decltype(always_mask)::value || u * KT + KT - 1 > all_hi || u * KT < all_lo) {
      // key_lo <= position <= key_hi as one unsigned comparison; a row that sees
      // nothing has span 0 at a position that is none
      const int d = u * KT + 4 * hi_lane - see_lo;
#pragma unroll
      for (int t = 0; t < ST; ++t)
#pragma unroll
        for (int r = 0; r < SR; ++r)
          st[t][r] = static_cast<uint32_t>(d + at(t, r)) > see_span ? -INFINITY : st[t][r];
    }
    if (pages != kEvery) {
      const uint64_t here = pages >> (4 * hi_lane);
#pragma unroll
      for (int t = 0; t < ST; ++t)
#pragma unroll
        for (int r = 0; r < SR; ++r)
          st[t][r] = (here >> at(t, r)) & 1 ? st[t][r] : -INFINITY;
    }
    float mx = st[0][0];
#pragma unroll
    for (int t = 0; t < ST; ++t)
#pragma unroll
      for (int r = 0; r < SR; ++r) mx = fmaxf(mx, st[t][r]);
    if (RW == 16) mx = max_across<16>(mx);
    mx = max_across<32>(mx);
    constexpr float kShift = Mma<T>::kShift;
    const bool move = mx * c > m + (kSlack + kShift);      // m = -inf: any score moves it
    if (__any(move)) {
      const float mn = move ? mx * c - kShift : m;
      const float f = __builtin_amdgcn_exp2f(m - (mn == -INFINITY ? 0.0f : mn));
      m = mn;
      l *= f;
      scale(f);
    }
    const float ref = m == -INFINITY ? 0.0f : m;
    float sum = 0.0f;
#pragma unroll
    for (int t = 0; t < ST; ++t)
#pragma unroll
      for (int r = 0; r < SR; r += 2) {
        const float p0 = __builtin_amdgcn_exp2f(fmaf(st[t][r], c, -ref));
        const float p1 = __builtin_amdgcn_exp2f(fmaf(st[t][r + 1], c, -ref));
        sum += p0 + p1;
        if (RW == 32) pf[t * 2 + r / 8][(r & 7) / 2] = pack2<T>(p0, p1);
        else pf[t / 2][(t & 1) * 2 + r / 2] = pack2<T>(p0, p1);
      }
    l += sum;
  };
  auto compute = [&](const uint16_t* sb, int u, uint64_t pages) {
    u32x4 pf[PS];
    weigh(sb, u, pages, pf, std::false_type{}, [&](float f) {
#pragma unroll
      for (int t = 0; t < OT; ++t)
#pragma unroll
        for (int r = 0; r < SR; ++r) o[t][r] *= f;
    });
    const int vo = fresh(voff);
#pragma unroll
    for (int s = 0; s < PS; ++s)
#pragma unroll
      for (int t = 0; t < OT; ++t) o[t] = mma(vread(sb, vo, s, t), pf[s], o[t]);
  };
  // One unit's product for the result tile at vt, with values that are not finite
  // reaching only the rows that see their position (0 times infinity is NaN in
  // a product over all positions): they are left out of the product, and each
  // position that has one is multiplied alone, for the rows that see it.
  auto compute_careful = [&](const uint16_t* sb, int u, uint64_t pages, int vt, acc_t& x) {
    u32x4 pf[PS];
    weigh(sb, u, pages, pf, std::true_type{}, [&](float f) {
#pragma unroll
      for (int r = 0; r < SR; ++r) x[r] *= f;
    });
#pragma unroll
    for (int s = 0; s < PS; ++s) {
      const u32x4 vf = vread(sb, vt, s, 0);
      u32x4 clean, rest;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t lo = (vf[i] & Mma<T>::kExp) == Mma<T>::kExp ? 0xffffu : 0u;
        const uint32_t hi = ((vf[i] >> 16) & Mma<T>::kExp) == Mma<T>::kExp ? 0xffff0000u : 0u;
        clean[i] = vf[i] & ~(lo | hi);
        rest[i] = vf[i] & (lo | hi);
      }
      x = mma(clean, pf[s], x);
      if (!__any((rest.x | rest.y | rest.z | rest.w) != 0u)) continue;
      for (int k = 0; k < kVSpan; ++k) {
        // position k of the step: operand part (k >> 2), element el of the lane
        const int part = RW == 32 ? (k >> 2) & 1 : (k >> 2) & 3;
        const int el = (k & 3) + (k >= kVSpan / 2 ? 4 : 0);
        u32x4 one;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          one[i] = part == hi_lane && (el >> 1) == i
                       ? rest[i] & ((el & 1) ? 0xffff0000u : 0xffffu) : 0u;
        if (!__any((one.x | one.y | one.z | one.w) != 0u)) continue;
        acc_t zero;
#pragma unroll
        for (int r = 0; r < SR; ++r) zero[r] = 0.0f;
        const acc_t add = mma(one, pf[s], zero);
        const int in = s * kVSpan + k;
        if (static_cast<uint32_t>(u * KT + in - see_lo) <= see_span && ((pages >> in) & 1)) {
#pragma unroll
          for (int r = 0; r < SR; ++r) x[r] += add[r];
        }
      }
    }
  };
  // The sum of a row's lanes, and the row's results.
  auto row_sum = [&]() {
    if (RW == 16) l += __shfl_xor(l, 16, kWave);
    l += __shfl_xor(l, 32, kWave);
  };
  auto store_tile = [&](const acc_t& x, int t) {
    if (row >= it.rows) return;
    if (it.splits > 1) {
      const int64_t p = (static_cast<int64_t>(it.slot) * a.kv_heads + h) * C::MT + row;
      const int e = t * RW + 4 * hi_lane;       // first element
      float* po = a.part_o + p * dim + e;
#pragma unroll
      for (int r = 0; r < SR; r += 4)
        if (!C::kPad || e + r * 2 < dim)
          *reinterpret_cast<f32x4*>(po + r * 2) = f32x4{x[r], x[r + 1], x[r + 2], x[r + 3]};
      return;
    }
    const float inv = 1.0f / l;
    auto y = [&](int r) { return l == 0.0f ? 0.0f : x[r] * inv; };   // (x may be NaN there)
    int token, head;
    attend_row(a, it.token0, it.row0 + fresh(row), h, token, head);
    const int e = t * RW + 4 * hi_lane;
    T* po = static_cast<T*>(a.out) + (static_cast<int64_t>(token) * a.heads + head) * dim + e;
#pragma unroll
    for (int r = 0; r < SR; r += 4) {
      if (C::kPad && e + r * 2 >= dim) continue;
      typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
      *reinterpret_cast<u32x2*>(po + r * 2) =
          u32x2{pack2<T>(y(r), y(r + 1)), pack2<T>(y(r + 2), y(r + 3))};
    }
  };
  auto store_sums = [&]() {
    if (row >= it.rows || hi_lane != 0) return;
    if (it.splits > 1) {
      const int64_t p = (static_cast<int64_t>(it.slot) * a.kv_heads + h) * C::MT + row;
      a.part_ml[p * 2] = m;
      a.part_ml[p * 2 + 1] = l;
    } else if (a.lse) {
      int token, head;
      attend_row(a, it.token0, it.row0 + fresh(row), h, token, head);
      a.lse[static_cast<int64_t>(token) * a.heads + head] =
          l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
    }
  };
  auto start = [&]() {
    m = -INFINITY;
    l = 0.0f;
#pragma unroll
    for (int t = 0; t < OT; ++t)
#pragma unroll
      for (int r = 0; r < SR; ++r) o[t][r] = 0.0f;
  };
  start();
  const int n_units = it.u1 - it.u0;
  if (n_units > 0) {
    // Step n computes unit n from buffer n % NB while unit n + 1 is under way.
    // Loads past the last unit read its nearest position again (one row).  The
    // table entries of turn q (units q NB ..) are loaded into LDS as well, one turn
    // before their use.
    if (C::kPad) {
      auto clear = [&](uint16_t* sb) {
        for (int i = tid; i < 2 * kV / 8; i += C::W * kWave)
          reinterpret_cast<u32x4*>(sb)[i] = u32x4{0, 0, 0, 0};
      };
      clear(sb0);
      clear(sb1);
      __syncthreads();
    }
    uint16_t* const ring[NB] = {sb0, sb1};
    const int first = it.u0 * KT;
    int32_t* const ids = sid + wave * C::SUPER;
    int64_t off[IDS];
    uint64_t mask[IDS], mask_next[IDS];
    auto look = [&](int q) {          // starts the lookups of turn q
#pragma unroll
      for (int i = 0; i < IDS; ++i)
        __builtin_amdgcn_global_load_lds((gptr_t)entry(first + q * C::SUPER + i * kWave),
                                         (lptr_t)(ids + i * kWave), 4, 0, 0);
    };
    auto turn = [&](int q) {          // turn q, looked up, becomes the one that loads
#pragma unroll
      for (int i = 0; i < IDS; ++i) {
        const int id = ids[i * kWave + lane];
        mask_next[i] = paged(id);
        off[i] = offset(first + q * C::SUPER + i * kWave, id);
      }
    };
    auto load = [&](int n, int s) {   // unit n = unit s of the turn that loads
      load_unit(first + n * KT, off[s * KT / kWave], s * KT % kWave, ring[s]);
    };
    look(0);
    wait_loads();
    turn(0);
    wait_loads();                     // the entries are read before the next overwrite them
    look(1);
#pragma unroll
    for (int s = 0; s < NB - 1; ++s) load(s, s);
    for (int n = 0; n < n_units; n += NB) {
#pragma unroll
      for (int s = 0; s < NB; ++s) {
        wait_loads();
        __builtin_amdgcn_s_barrier();
        if (s == 0) {
#pragma unroll
          for (int i = 0; i < IDS; ++i) mask[i] = mask_next[i];
        }
        if (s == 1) turn(n / NB + 1);
        load(n + s + NB - 1, (s + NB - 1) % NB);
        if (s == 1) look(n / NB + 2);
        if (n + s < n_units)
          compute(ring[s], it.u0 + n + s, mask[s * KT / kWave] >> (s * KT % kWave));
      }
    }
    // no load may still be under way when the workgroup gives its LDS back
    wait_loads();
    // anything not finite: again, a result tile and a unit at a time, carefully
    float z = l * 0.0f;
#pragma unroll
    for (int t = 0; t < OT; ++t)
#pragma unroll
      for (int r = 0; r < SR; ++r) z = fmaf(o[t][r], 0.0f, z);
    if (__syncthreads_or(!(z == 0.0f))) {
      for (int t = 0; t < OT; ++t) {
        start();
        acc_t x = o[0];
        for (int u = it.u0; u < it.u1; ++u) {
          const int page = *entry(u * KT);
          load_unit(u * KT, offset(u * KT, page), 0, sb0);
          wait_loads();
          __syncthreads();
          compute_careful(sb0, u, paged(page), voff ^ (t * kVTile), x);
          __syncthreads();
        }
        row_sum();
        store_tile(x, t);
      }
      store_sums();
      return;
    }
  }
  row_sum();
  store_sums();
  if (it.splits > 1) {
#pragma unroll
    for (int t = 0; t < OT; ++t) store_tile(o[t], t);
    return;
  }
  // whole output rows: turned in LDS (each wavefront its rows, permuted as K's),
  // then 16 bytes a lane (8 bytes a lane straight from the registers touch every
  // row in each store: 1024-token prompts 233 against 219 us)
  static_assert(C::MT <= 2 * KT, "the rows fit the first buffer");
  char* const turned = reinterpret_cast<char*>(sb0) + wave * RW * D * 2;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  const int mine = lane & (RW - 1);
#pragma unroll
  for (int t = 0; t < OT; ++t)
#pragma unroll
    for (int r = 0; r < SR; r += 4) {
      typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
      const int e = t * RW + r * 2 + 4 * hi_lane;     // element of the row
      *reinterpret_cast<u32x2*>(turned + mine * (D * 2) + (((e >> 3) ^ swz_k<D>(mine)) << 4) +
                                (e & 4) * 2) =
          u32x2{pack2<T>(o[t][r] * inv, o[t][r + 1] * inv),
                pack2<T>(o[t][r + 2] * inv, o[t][r + 3] * inv)};
    }
#pragma unroll
  for (int i = 0; i < RW / RPL; ++i) {
    const int r = i * RPL + lq;
    const u32x4 w = *reinterpret_cast<const u32x4*>(turned + r * (D * 2) +
                                                    ((lslot ^ swz_k<D>(r)) << 4));
    if (wave * RW + r < it.rows && (!C::kPad || lslot < nv)) {
      int token, head;
      attend_row(a, it.token0, it.row0 + wave * RW + r, h, token, head);
      T* po = static_cast<T*>(a.out) + (static_cast<int64_t>(token) * a.heads + head) * dim;
      reinterpret_cast<u32x4*>(po)[lslot] = w;
    }
  }
}

template <class C>
void launch_cfg(const AttendArgs& a, hipStream_t st) {
  hipLaunchKernelGGL(attend_mfma_kernel<C>, dim3(static_cast<unsigned>(a.grid_items) * a.kv_heads),
                     dim3(C::W * kWave), 0, st, a);
}

// Tiles of 32, 64 and 128 rows.  Up to 64 rows the cache's bandwidth bounds the
// kernel: short units and 16 rows a wavefront, since more wavefronts start and
// load a unit faster (with four buffers and head_dim 128, 32 rows a wavefront: 36
// rows over 500 positions at B = 256 130 us against 122; a 16-row tile of one
// wavefront: single tokens there 126 us against 107, over 1000 positions at B = 1
// 14.5 against 12.4, over 110000 at B = 4 274 against 282).  128 rows are bound by
// the matrix and vector units: 32 rows a wavefront and units of 64 positions, half
// the operand reads and barriers.  Rows of head_dim 256 leave registers for 16
// query rows a wavefront, 64 a tile.
template <typename T, int D, bool kPad>
hipError_t launch_rows_of(const AttendArgs& a, int mt, hipStream_t st) {
  switch (mt) {
    case 32: launch_cfg<AttendCfg<T, D, kPad, 16, 2, 32>>(a, st); break;
    case 64: launch_cfg<AttendCfg<T, D, kPad, 16, 4, 32>>(a, st); break;
    default:
      if constexpr (D <= 128) launch_cfg<AttendCfg<T, D, kPad, 32, 4, 64>>(a, st);
      else return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

template <int D>
hipError_t launch_width(const AttendArgs& a, int dtype, int mt, hipStream_t st) {
  if (dtype == kBF16)
    return a.D == D ? launch_rows_of<__bf16, D, false>(a, mt, st)
                    : launch_rows_of<__bf16, D, true>(a, mt, st);
  return a.D == D ? launch_rows_of<_Float16, D, false>(a, mt, st)
                  : launch_rows_of<_Float16, D, true>(a, mt, st);
}

}  // namespace sv
