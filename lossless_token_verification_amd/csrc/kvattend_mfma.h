// Paged attention on the matrix cores (bf16 / f16 caches, head_dim 64, 128 or
// 256).
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
// Softmax in one pass: the maximum m moves only when a score exceeds it by
// more than kSlack (log2 units), so the accumulators are rescaled in the first
// unit and hardly ever after; weights stay below 2^kSlack, exactly represented
// relative to their size in both types.
//
// K and V units go from the pages straight into LDS (16-byte direct loads, no
// register stage), one unit ahead in the other of two buffers; rows are
// permuted by 16-byte vectors (swz_k, swz_v) so that the operand reads of
// either product spread over all banks.  A row's page comes from the block
// table one unit before that.
#pragma once

#include <type_traits>

#include "kvattend.h"

namespace sv {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

template <typename T>
struct Mma;
template <>
struct Mma<__bf16> {
  static constexpr uint32_t kExp = 0x7f80u;   // exponent bits: all set = not finite
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

// RW: query rows per wavefront (16 or 32, the matrix instruction's width).  WR
// wavefronts take different rows of a unit, WK different positions.
template <typename T_, int D_, int RW_, int WR_, int WK_, int KT_>
struct AttendCfg {
  using T = T_;
  static constexpr int D = D_, RW = RW_, WR = WR_, WK = WK_, KT = KT_;
  static constexpr int W = WR * WK, MT = RW * WR;
  static constexpr int KW = KT / WK;               // positions per wavefront and unit
  static constexpr int NV = D / 8;                 // vectors of a row
  static constexpr int RPL = kWave / NV;           // rows of one direct load
  static constexpr int LOADS = KT / RPL / W;       // of K and of V, per wavefront
  static constexpr int QS = RW == 32 ? D / 16 : D / 32;     // steps of the first product
  static constexpr int ST = KW / RW;               // its result tiles
  static constexpr int SR = RW == 32 ? 16 : 4;     // registers of a result tile
  static constexpr int PS = RW == 32 ? KW / 16 : KW / 32;   // steps of the second product
  static constexpr int OT = D / RW;                // its result tiles
  static_assert(KT % (RPL * W) == 0 && KW % 32 == 0 && KT <= kWave, "unit shape");
};

constexpr float kSlack = 8.0f;

template <class C>
__global__ __launch_bounds__(C::W * kWave) __attribute__((amdgpu_waves_per_eu(C::W >= 4 && C::D < 256 ? 2 : 1))) void
attend_mfma_kernel(AttendArgs a) {
  using T = typename C::T;
  constexpr int D = C::D, RW = C::RW, KT = C::KT, KW = C::KW, NV = C::NV, RPL = C::RPL;
  constexpr int SR = C::SR, ST = C::ST, OT = C::OT, PS = C::PS, QS = C::QS;
  typedef typename std::conditional<RW == 32, f32x16, f32x4>::type acc_t;
  // each buffer its own LDS object: the compiler then knows that a direct load
  // into one does not change the other, and does not wait for it
  __shared__ __attribute__((aligned(1024))) uint16_t sk0[KT * D], sk1[KT * D];
  __shared__ __attribute__((aligned(1024))) uint16_t sv0[KT * D], sv1[KT * D];
  __shared__ AttendPlanShared<C::W> plan;
  __shared__ float smerge[C::WK > 1 ? 2 * C::WR * RW : 1];
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int wr = wave / C::WK, wk = wave - wr * C::WK;
  const int x = blockIdx.x / a.kv_heads, h = blockIdx.x - x * a.kv_heads;
  AttendItem it;
  if (!attend_find<C::MT, KT, C::W>(a, x, a.max_slots > 0 && blockIdx.x == 0, plan, it)) return;
  if (it.splits > 1 && h == 0 && tid == 0) attend_slot_info(a, it);

  // this lane's query row; rows past the tile repeat its last one
  const int hi_lane = RW == 32 ? lane >> 5 : lane >> 4;   // which part of k a lane holds
  const int row = wr * RW + (lane & (RW - 1));
  int token, head;
  attend_row(a, it.token0, it.row0 + min(row, it.rows - 1), h, token, head);
  const int pos = it.pos0 + token - it.token0;
  const int key_hi = min(pos, it.key_hi - 1);            // last and first position it may see
  const int key_lo = a.window > 0 ? max(pos - a.window + 1, 0) : 0;
  // positions every row of the tile may see: units inside need no mask
  const int all_hi = min(it.pos0 + fast_div(it.row0, a.grp), it.key_hi - 1);
  const int all_lo =
      a.window > 0 ? it.pos0 + fast_div(it.row0 + it.rows - 1, a.grp) - a.window + 1 : 0;

  u32x4 qf[QS];
  {
    const T* qr = static_cast<const T*>(a.q) + token * a.q_stride + static_cast<int64_t>(head) * D;
#pragma unroll
    for (int s = 0; s < QS; ++s)
      qf[s] = reinterpret_cast<const u32x4*>(qr)[s * (RW == 32 ? 2 : 4) + hi_lane];
  }

  const int32_t* table = a.table + static_cast<int64_t>(it.b) * a.max_blocks;
  const int64_t head_off = static_cast<int64_t>(h) * a.block_size;
  // Lane l looks up position l of a unit: its element offset in the caches, and
  // whether there is such a page.  Positions outside the item's range read the
  // nearest one inside (and are masked); a missing page reads block 0.
  auto lookup = [&](int u) -> int {
    const int key = min(max(u * KT + (lane & (KT - 1)), it.key_lo), it.key_hi - 1);
    return table[fast_div(key, a.bs)];
  };
  auto offset = [&](int u, int id) -> int64_t {
    const int key = min(max(u * KT + (lane & (KT - 1)), it.key_lo), it.key_hi - 1);
    const int r = key - fast_div(key, a.bs) * a.block_size;
    const int safe = id >= 0 && id < a.num_blocks ? id : 0;
    return safe * a.block_stride + (head_off + r) * D;
  };
  auto paged = [&](int id) -> uint64_t { return __ballot(id >= 0 && id < a.num_blocks); };

  typedef const void __attribute__((address_space(1)))* gptr_t;
  typedef void __attribute__((address_space(3)))* lptr_t;
  const T* kb = static_cast<const T*>(a.k);
  const T* vb = static_cast<const T*>(a.v);
  // lane part of a direct load: row q of its RPL rows, vector `slot` of that row
  const int lq = lane / NV, lslot = lane & (NV - 1);
  auto load_unit = [&](int64_t off, uint16_t* sk, uint16_t* sv) {
    const int lk = fresh(lslot ^ swz_k<D>(lq)), lv = fresh(lslot ^ swz_v<D>(lq));
#pragma unroll
    for (int i = 0; i < C::LOADS; ++i) {
      const int j = wave + i * C::W;                 // which RPL rows
      const int64_t ro = __shfl(static_cast<long long>(off), j * RPL + lq, kWave);
      __builtin_amdgcn_global_load_lds((gptr_t)(kb + ro + (lk ^ swz_k<D>(j * RPL)) * 8),
                                       (lptr_t)(sk + j * 512), 16, 0, 0);
      __builtin_amdgcn_global_load_lds((gptr_t)(vb + ro + (lv ^ swz_v<D>(j * RPL)) * 8),
                                       (lptr_t)(sv + j * 512), 16, 0, 0);
    }
  };

  acc_t o[OT];
  float m, l;
  const float c = a.scale * kLog2e;

  // Operand reads.  Byte offset of the lane's part at step / tile 0; the others
  // differ by an xor inside the row and by whole rows.
  const int krow = wk * KW + (lane & (RW - 1));
  const int koff = krow * (D * 2) + ((hi_lane ^ swz_k<D>(krow)) << 4);
  constexpr int kKStep = RW == 32 ? 32 : 64;       // bytes of a row per step
  // V, k order of the operand = positions of the result registers.  32 wide:
  // 4h + i and 8 + 4h + i of 16; 16 wide: 4g + i and 16 + 4g + i of 32.  A
  // transposed read gives lane n of 16 element n of 4 rows; lane n fetches row
  // n / 4, elements 4 (n % 4) ..
  const int vrow = wk * KW + 4 * hi_lane + ((lane & 15) >> 2);
  const int vvec = (RW == 32 ? ((lane >> 4) & 1) * 2 : 0) + ((lane & 3) >> 1);
  const int voff = vrow * (D * 2) + ((vvec ^ swz_v<D>(vrow)) << 4) + (lane & 1) * 8;
  constexpr int kVTile = RW * 2;                    // bytes of a row per result tile
  constexpr int kVSpan = RW == 32 ? 16 : 32;        // positions per step
  auto vread = [&](const uint16_t* sv, int vo, int s, int ot) -> u32x4 {
    typedef __attribute__((address_space(3))) s16x4* tr_t;
    const char* p = reinterpret_cast<const char*>(sv) + (vo ^ (ot * kVTile)) + s * kVSpan * D * 2;
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

  // One unit.  CAREFUL: values that are not finite reach only the rows that see
  // their position (0 times infinity is NaN in a product over all positions).
  auto compute = [&](const uint16_t* sk, const uint16_t* sv, int u, uint64_t pages, auto careful) {
    constexpr bool kCareful = decltype(careful)::value;
    acc_t st[ST];
    const int ko = fresh(koff), vo = fresh(voff);
#pragma unroll
    for (int t = 0; t < ST; ++t) {
#pragma unroll
      for (int r = 0; r < SR; ++r) st[t][r] = 0.0f;
#pragma unroll
      for (int s = 0; s < QS; ++s)
        st[t] = mma(*reinterpret_cast<const u32x4*>(reinterpret_cast<const char*>(sk) +
                                                    (ko ^ (s * kKStep)) + t * RW * D * 2),
                    qf[s], st[t]);
    }
    // position of register r of tile t, less the lane's part 4 * hi_lane
    auto at = [&](int t, int r) { return t * RW + (RW == 32 ? (r >> 2) * 8 + (r & 3) : r); };
    const int base = u * KT + wk * KW + 4 * hi_lane;
    const uint64_t every = KT == 64 ? ~uint64_t{0} : (uint64_t{1} << (KT & 63)) - 1;
    const bool masked = u * KT + KT - 1 > all_hi || u * KT < all_lo || (pages & every) != every;
    const uint64_t seen = pages >> (wk * KW + 4 * hi_lane);
    if (masked || kCareful) {
#pragma unroll
      for (int t = 0; t < ST; ++t)
#pragma unroll
        for (int r = 0; r < SR; ++r) {
          const int key = base + at(t, r);
          if (key > key_hi || key < key_lo || !((seen >> at(t, r)) & 1)) st[t][r] = -INFINITY;
        }
    }
    float mx = st[0][0];
#pragma unroll
    for (int t = 0; t < ST; ++t)
#pragma unroll
      for (int r = 0; r < SR; ++r) mx = fmaxf(mx, st[t][r]);
    if (RW == 16) mx = fmaxf(mx, __shfl_xor(mx, 16, kWave));
    mx = fmaxf(mx, __shfl_xor(mx, 32, kWave));
    const bool move = mx * c > m + kSlack;      // m = -inf: any score moves it
    if (__any(move)) {
      const float mn = move ? mx * c : m;
      const float f = __builtin_amdgcn_exp2f(m - (mn == -INFINITY ? 0.0f : mn));
      m = mn;
      l *= f;
#pragma unroll
      for (int t = 0; t < OT; ++t)
#pragma unroll
        for (int r = 0; r < SR; ++r) o[t][r] *= f;
    }
    const float ref = m == -INFINITY ? 0.0f : m;
    u32x4 pf[PS];
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
#pragma unroll
    for (int s = 0; s < PS; ++s)
#pragma unroll
      for (int t = 0; t < OT; ++t) {
        u32x4 vf = vread(sv, vo, s, t);
        if constexpr (!kCareful) {
          o[t] = mma(vf, pf[s], o[t]);
        } else {
          u32x4 clean = vf, rest;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t lo = (vf[i] & Mma<T>::kExp) == Mma<T>::kExp ? 0xffffu : 0u;
            const uint32_t hi = ((vf[i] >> 16) & Mma<T>::kExp) == Mma<T>::kExp ? 0xffff0000u : 0u;
            clean[i] = vf[i] & ~(lo | hi);
            rest[i] = vf[i] & (lo | hi);
          }
          o[t] = mma(clean, pf[s], o[t]);
          if (__any((rest.x | rest.y | rest.z | rest.w) != 0u)) {
            // one position at a time: the product of its values alone, for the
            // rows that see it
            constexpr int kSpan = RW == 32 ? 16 : 32;
            for (int k = 0; k < kSpan; ++k) {
              // operand element of position k: part (k >> 2), register pair
              const int part = RW == 32 ? (k >> 2) & 1 : (k >> 2) & 3;
              const int el = (k & 3) + (k >= kSpan / 2 ? 4 : 0);
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
              const int in = wk * KW + s * kSpan + k, key = u * KT + in;
              if (key <= key_hi && key >= key_lo && ((pages >> in) & 1)) {
#pragma unroll
                for (int r = 0; r < SR; ++r) o[t][r] += add[r];
              }
            }
          }
        }
      }
  };
  // All units of the item.  Unit u computes on buffer (u - u0) % 2 while unit
  // u + 1 is loaded into the other and the pages of unit u + 2 are looked up;
  // the barrier that ends a unit also ends the loads under way.
  auto run = [&](auto careful) {
    m = -INFINITY;
    l = 0.0f;
#pragma unroll
    for (int t = 0; t < OT; ++t)
#pragma unroll
      for (int r = 0; r < SR; ++r) o[t][r] = 0.0f;
    if (it.u0 >= it.u1) return;
    int id = lookup(it.u0);
    uint64_t pages = paged(id), pages_next = 0;
    load_unit(offset(it.u0, id), sk0, sv0);
    if (it.u0 + 1 < it.u1) id = lookup(it.u0 + 1);
    auto step = [&](int u, const uint16_t* sk, const uint16_t* sv, uint16_t* nk, uint16_t* nv) {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();
      if (u + 1 < it.u1) {
        pages_next = paged(id);
        load_unit(offset(u + 1, id), nk, nv);
        if (u + 2 < it.u1) id = lookup(u + 2);
      }
      compute(sk, sv, u, pages, careful);
      pages = pages_next;
    };
    int u = it.u0;
    for (; u + 2 <= it.u1; u += 2) {
      step(u, sk0, sv0, sk1, sv1);
      step(u + 1, sk1, sv1, sk0, sv0);
    }
    if (u < it.u1) step(u, sk0, sv0, sk1, sv1);
  };
  run(std::false_type{});
  {
    // anything not finite: again, carefully
    float z = l * 0.0f;
#pragma unroll
    for (int t = 0; t < OT; ++t)
#pragma unroll
      for (int r = 0; r < SR; ++r) z = fmaf(o[t][r], 0.0f, z);
    if (__syncthreads_or(!(z == 0.0f))) run(std::true_type{});
  }

  // the sums of a row's lanes, then of the wavefronts that shared its positions
  if (RW == 16) l += __shfl_xor(l, 16, kWave);
  l += __shfl_xor(l, 32, kWave);
  if constexpr (C::WK > 1) {
    static_assert(C::WK == 2 && C::WR == 1 && OT * SR * 4 <= KT * D * 2 / kWave, "merge space");
    float* so = reinterpret_cast<float*>(sk0);
    __syncthreads();
    if (wk == 1) {
#pragma unroll
      for (int t = 0; t < OT; ++t)
#pragma unroll
        for (int r = 0; r < SR; ++r) so[(t * SR + r) * kWave + lane] = o[t][r];
      if (hi_lane == 0) {
        smerge[2 * row] = m;
        smerge[2 * row + 1] = l;
      }
    }
    __syncthreads();
    if (wk == 1) return;
    const float m1 = smerge[2 * row], l1 = smerge[2 * row + 1];
    const float mn = fmaxf(m, m1), ref = mn == -INFINITY ? 0.0f : mn;
    const float f0 = __builtin_amdgcn_exp2f(m - ref), f1 = __builtin_amdgcn_exp2f(m1 - ref);
    m = mn;
    l = l * f0 + l1 * f1;
#pragma unroll
    for (int t = 0; t < OT; ++t)
#pragma unroll
      for (int r = 0; r < SR; ++r)
        o[t][r] = o[t][r] * f0 + so[(t * SR + r) * kWave + lane] * f1;
  }
  if (row >= it.rows) return;
  if (it.splits > 1) {
    const int64_t p = (static_cast<int64_t>(it.slot) * a.kv_heads + h) * C::MT + row;
    float* po = a.part_o + p * D;
#pragma unroll
    for (int t = 0; t < OT; ++t)
#pragma unroll
      for (int r = 0; r < SR; r += 4)
        *reinterpret_cast<f32x4*>(po + t * RW + r * 2 + 4 * hi_lane) =
            f32x4{o[t][r], o[t][r + 1], o[t][r + 2], o[t][r + 3]};
    if (hi_lane == 0) {
      a.part_ml[p * 2] = m;
      a.part_ml[p * 2 + 1] = l;
    }
    return;
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  const int64_t out = static_cast<int64_t>(token) * a.heads + head;
  T* po = static_cast<T*>(a.out) + out * D;
#pragma unroll
  for (int t = 0; t < OT; ++t)
#pragma unroll
    for (int r = 0; r < SR; r += 4) {
      typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
      *reinterpret_cast<u32x2*>(po + t * RW + r * 2 + 4 * hi_lane) =
          u32x2{pack2<T>(o[t][r] * inv, o[t][r + 1] * inv),
                pack2<T>(o[t][r + 2] * inv, o[t][r + 3] * inv)};
    }
  if (a.lse && hi_lane == 0) a.lse[out] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
}

template <class C>
void launch_cfg(const AttendArgs& a, hipStream_t st) {
  hipLaunchKernelGGL(attend_mfma_kernel<C>, dim3(static_cast<unsigned>(a.grid_items) * a.kv_heads),
                     dim3(C::W * kWave), 0, st, a);
}

// Tiles of 16, 32, 64 and 128 rows.  Up to 32 rows one set of rows is shared by
// two wavefronts that take half a unit each (one at head_dim 256, whose unit is
// half as long for the same LDS); above that each wavefront has 32 rows.
template <typename T, int D>
hipError_t launch_rows_of(const AttendArgs& a, int mt, hipStream_t st) {
  constexpr int KT = D == 256 ? 32 : 64, WK = D == 256 ? 1 : 2;
  switch (mt) {
    case 16: launch_cfg<AttendCfg<T, D, 16, 1, WK, KT>>(a, st); break;
    case 32: launch_cfg<AttendCfg<T, D, 32, 1, WK, KT>>(a, st); break;
    case 64: launch_cfg<AttendCfg<T, D, 32, 2, 1, KT>>(a, st); break;
    default: launch_cfg<AttendCfg<T, D, 32, 4, 1, KT>>(a, st); break;
  }
  return hipGetLastError();
}

}  // namespace sv
