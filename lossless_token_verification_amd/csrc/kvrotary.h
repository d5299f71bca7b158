// Device code of the rotated rows: (x_i, x_j) -> (x_i cos - x_j sin, x_j cos + x_i
// sin), j = i + rot / 2, or neighbours (pairs).
#pragma once

#include "kv_args.h"

namespace sv {

template <typename T, int N>
struct alignas(sizeof(T) * N) RowVec {
  T e[N];
};

// VEC floats of the table, from 4 * VEC or fewer aligned bytes.
template <int N>
__device__ __forceinline__ void load_angles(const float* p, float (&x)[N]) {
  const RowVec<float, N >= 4 ? 4 : N>* v = reinterpret_cast<const RowVec<float, N >= 4 ? 4 : N>*>(p);
  constexpr int kPer = N >= 4 ? 4 : N;
#pragma unroll
  for (int i = 0; i < N / kPer; ++i) {
    const RowVec<float, kPer> y = v[i];
#pragma unroll
    for (int j = 0; j < kPer; ++j) x[i * kPer + j] = y.e[j];
  }
}

// Unit u of a row: rotated and written from `src` to `dst` (which may be the same
// row: a unit reads and writes the same elements).  The turn is made in float32,
// one product rounded and the sum with the other, and rounded once to the type.
template <typename T, int VEC>
__device__ __forceinline__ void turn_unit(const RotaryArgs& a, const float* angles, int u,
                                          const T* src, T* dst) {
  typedef RowVec<T, VEC> V;
  const int half = a.rot / 2;
  if (u >= a.turn_units) {
    const int e = a.rot + (u - a.turn_units) * VEC;
    *reinterpret_cast<V*>(dst + e) = *reinterpret_cast<const V*>(src + e);
  } else if (a.pairs) {
    // (single elements: the unit is a pair)
    constexpr int N = VEC > 1 ? VEC / 2 : 1;
    typedef RowVec<T, N * 2> P;
    const int e = u * N * 2;
    P x;
    if constexpr (VEC > 1) {
      x = *reinterpret_cast<const P*>(src + e);
    } else {
      x.e[0] = src[e];
      x.e[1] = src[e + 1];
    }
    float c[N], s[N];
    load_angles<N>(angles + u * N, c);
    load_angles<N>(angles + half + u * N, s);
    P y;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float x0 = static_cast<float>(x.e[2 * i]), x1 = static_cast<float>(x.e[2 * i + 1]);
      y.e[2 * i] = static_cast<T>(fmaf(x0, c[i], -(x1 * s[i])));
      y.e[2 * i + 1] = static_cast<T>(fmaf(x1, c[i], x0 * s[i]));
    }
    if constexpr (VEC > 1) {
      *reinterpret_cast<P*>(dst + e) = y;
    } else {
      dst[e] = y.e[0];
      dst[e + 1] = y.e[1];
    }
  } else {
    const int e = u * VEC;
    const V x0 = *reinterpret_cast<const V*>(src + e);
    const V x1 = *reinterpret_cast<const V*>(src + half + e);
    float c[VEC], s[VEC];
    load_angles<VEC>(angles + e, c);
    load_angles<VEC>(angles + half + e, s);
    V y0, y1;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const float f0 = static_cast<float>(x0.e[i]), f1 = static_cast<float>(x1.e[i]);
      y0.e[i] = static_cast<T>(fmaf(f0, c[i], -(f1 * s[i])));
      y1.e[i] = static_cast<T>(fmaf(f1, c[i], f0 * s[i]));
    }
    *reinterpret_cast<V*>(dst + e) = y0;
    *reinterpret_cast<V*>(dst + half + e) = y1;
  }
}

// Unit i of the call: of a query, key or value row of a token.
template <typename T, int VEC>
__device__ __forceinline__ void rotary_unit(const RotaryArgs& a, uint32_t i) {
  const int t = fast_div(static_cast<int>(i), a.token);
  int c = static_cast<int>(i) - t * a.token_units;
  const int pos = a.positions[t];
  if (pos < 0 || pos >= a.table_rows) return;
  const float* angles = a.cos_sin + static_cast<int64_t>(pos) * a.rot;
  const int q_units = a.heads * a.row_units;
  if (c < q_units) {
    const int h = fast_div(c, a.row), u = c - h * a.row_units;
    turn_unit<T, VEC>(a, angles, u,
                      static_cast<const T*>(a.q) + t * a.q_stride + static_cast<int64_t>(h) * a.dim,
                      static_cast<T*>(a.q_out) + t * a.q_out_stride +
                          static_cast<int64_t>(h) * a.dim);
    return;
  }
  c -= q_units;
  const int64_t slot = a.slots[t];
  if (slot < 0 || slot >= a.num_slots) return;
  const int blk = fast_div(static_cast<int>(slot), a.bs);
  const int row = static_cast<int>(slot) - blk * a.block_size;
  const int k_units = a.kv_heads * a.row_units;
  const bool key = c < k_units;
  if (!key) c -= k_units;
  const int h = fast_div(c, key ? a.row : a.vrow), u = c - h * (key ? a.row_units : a.v_units);
  const int64_t at = blk * a.block_stride + (static_cast<int64_t>(h) * a.block_size + row) * a.dim;
  if (key) {
    turn_unit<T, VEC>(a, angles, u,
                      static_cast<const T*>(a.k) + t * a.k_stride + static_cast<int64_t>(h) * a.dim,
                      static_cast<T*>(a.dst[0]) + at);
  } else {
    typedef RowVec<T, VEC> V;
    const T* src = static_cast<const T*>(a.v) + t * a.v_stride + static_cast<int64_t>(h) * a.dim;
    *reinterpret_cast<V*>(static_cast<T*>(a.dst[1]) + at + u * VEC) =
        *reinterpret_cast<const V*>(src + u * VEC);
  }
}

constexpr int kRotaryThreads = 256;

}  // namespace sv
