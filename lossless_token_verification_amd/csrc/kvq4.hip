// Rows to and from the cache held in 4 bits (e2m1 codes: a sign and 0, 0.5, 1, 1.5,
// 2, 3, 4 or 6).  Keys: a power of two for 32 channels, the least 2^e with amax <= 7 *
// 2^e, so that no key is off by more than half a step of its level's binade, as the
// exponent + 127; that is the matrix instructions' own block format, and the
// attention multiplies codes as they lie.  Values: one scale a row, amax / 6 rounded
// to 8 bits, since the attention's sum over positions cannot take a scale that
// changes along channels.
//
// A row is taken by dim / 8 lanes, 8 channels each.  The turn of a key is made in
// float64, where the products of 24-bit numbers are exact, and rounded once to
// float32: a key next to a border between two levels falls on its own side.  From
// there on every step is exact: the code of a key is the conversion of x * 2^-e, that
// of a value counts the borders scale * c below x, products of 8 and 3 bits.
//
// Bound by memory in large calls: 32 + 2 x 8 heads of 128 bfloat16, the queries turned in
// the same launch, 16 100 rows 82 us (348 MB, 4.2 TB/s), 2304 rows 13.2 us, the latter with
// the float64 turns (8 a lane, at half the float32 rate) beside the loads.  The rows
// back from it (16 100, 84 MB) 19 us, 4.4 TB/s.
#include "kvrotary.h"

namespace sv {

namespace {

constexpr int kRowThreads = 256;

template <typename T, bool kWide>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]) {
  if constexpr (kWide) {
    constexpr int N = 16 / sizeof(T);
#pragma unroll
    for (int i = 0; i < 8 / N; ++i) {
      const RowVec<T, N> y = reinterpret_cast<const RowVec<T, N>*>(p)[i];
#pragma unroll
      for (int j = 0; j < N; ++j) x[i * N + j] = static_cast<float>(y.e[j]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = static_cast<float>(p[i]);
  }
}

// Maximum over `lanes` (a power of two) neighbouring lanes.
__device__ __forceinline__ uint32_t max_of_lanes(uint32_t v, int lanes) {
  for (int o = 1; o < lanes; o <<= 1) v = max(v, static_cast<uint32_t>(__shfl_xor(v, o, kWave)));
  return v;
}

// The bits of the largest |x| of 8 (as integers: NaN above infinity above numbers).
__device__ __forceinline__ uint32_t top_bits(const float (&x)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
  return m;
}

constexpr uint32_t kInfBits = 0x7f800000u;

// Eight channels of a key row from channel e on, turned.  Wide: a unit's elements
// have one role, and their partners are a vector too.
template <typename T, bool kWide>
__device__ __forceinline__ void turned8(const Q4RowsArgs& a, const float* angles, const T* src, int e,
                                        float (&x)[8]) {
  load8<T, kWide>(src + e, x);
  const int half = a.rot / 2;
  if (kWide) {
    if (e >= a.rot) return;
    float c[8], s[8], y[8];
    if (a.pairs) {
      float c4[4], s4[4];
      load_angles<4>(angles + e / 2, c4);
      load_angles<4>(angles + half + e / 2, s4);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        c[i] = c4[i / 2];
        s[i] = i & 1 ? s4[i / 2] : -s4[i / 2];
        y[i] = x[i ^ 1];
      }
    } else {
      const bool low = e < half;
      const int at = low ? e : e - half;
      load8<T, kWide>(src + (low ? e + half : at), y);
      load_angles<8>(angles + at, c);
      load_angles<8>(angles + half + at, s);
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = low ? -s[i] : s[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      x[i] = static_cast<float>(fma(static_cast<double>(x[i]), static_cast<double>(c[i]),
                                    static_cast<double>(y[i]) * static_cast<double>(s[i])));
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int j = e + i;
    if (j >= a.rot) break;
    const bool low = a.pairs ? (j & 1) == 0 : j < half;
    const int at = a.pairs ? j >> 1 : low ? j : j - half;
    const int other = a.pairs ? j ^ 1 : low ? j + half : at;
    const double s = static_cast<double>(angles[half + at]);
    x[i] = static_cast<float>(fma(static_cast<double>(x[i]), static_cast<double>(angles[at]),
                                  static_cast<double>(static_cast<float>(src[other])) * (low ? -s : s)));
  }
}

// The code of a value: how many borders of its scale lie below it (ties to the even
// code), and its sign.
__device__ __forceinline__ uint32_t value_code(float x, float s) {
  const float v = fabsf(x);
  const uint32_t n = (v > s * 0.25f) + (v >= s * 0.75f) + (v > s * 1.25f) + (v >= s * 1.75f) +
                     (v > s * 2.5f) + (v >= s * 3.5f) + (v > s * 5.0f);
  return n | ((__float_as_uint(x) >> 28) & 8u);
}

template <typename T, bool kWide, int QV>
__global__ __launch_bounds__(kRowThreads) void q4_append_kernel(Q4RowsArgs a, uint32_t row_groups,
                                                                RotaryArgs q, uint32_t q_total) {
  if (blockIdx.x >= row_groups) {      // the queries' part of the launch
    const uint32_t i = (blockIdx.x - row_groups) * kRowThreads + threadIdx.x;
    if (i < q_total) rotary_unit<T, QV>(q, i);
    return;
  }
  const int per = kRowThreads / a.row_lanes;
  const int lane = threadIdx.x & (a.row_lanes - 1);
  const int64_t r = static_cast<int64_t>(blockIdx.x) * per + threadIdx.x / a.row_lanes;
  if (r >= static_cast<int64_t>(a.T) * a.kv_heads) return;      // (whole rows leave)
  const int t = fast_div(static_cast<int>(r), a.heads), h = static_cast<int>(r) - t * a.kv_heads;
  const int64_t slot = a.slots[t];
  if (slot < 0 || slot >= a.num_slots) return;
  const float* angles = nullptr;
  if (a.rot > 0) {
    const int pos = a.positions[t];
    if (pos < 0 || pos >= a.table_rows) return;
    angles = a.cos_sin + static_cast<int64_t>(pos) * a.rot;
  }
  const int e = lane * 8;
  float x[8] = {}, y[8] = {};
  if (e < a.dim) {
    const T* k = static_cast<const T*>(a.k) + t * a.k_stride + static_cast<int64_t>(h) * a.dim;
    const T* v = static_cast<const T*>(a.v) + t * a.v_stride + static_cast<int64_t>(h) * a.dim;
    load8<T, kWide>(v + e, y);
    if (a.rot > 0) turned8<T, kWide>(a, angles, k, e, x);
    else load8<T, kWide>(k + e, x);
  }
  const int blk = fast_div(static_cast<int>(slot), a.bs);
  const int row = static_cast<int>(slot) - blk * a.block_size;
  const int64_t at = (static_cast<int64_t>(blk) * a.kv_heads + h) * a.block_size + row;
  // keys: top / 2^(E - 127) is in [1, 2); 7 / 4 of it is the border
  const uint32_t top = max_of_lanes(top_bits(x), 4);
  int byte = static_cast<int>(top >> 23) - 2 + ((top & 0x7fffffu) > 0x600000u);
  byte = top >= kInfBits ? 255 : max(byte, 0);
  uint32_t codes = 0;
  if (byte != 255) {
    float z[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = ldexpf(x[i], 127 - byte);
    codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, z[0], z[1], 1.0f, 0);
    codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, z[2], z[3], 1.0f, 1);
    codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, z[4], z[5], 1.0f, 2);
    codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, z[6], z[7], 1.0f, 3);
  }
  // values
  const uint32_t vtop = max_of_lanes(top_bits(y), a.row_lanes);
  const uint32_t sixth = __float_as_uint(__uint_as_float(vtop) / 6.0f);
  float scale = __uint_as_float((sixth + 0x7fffu + ((sixth >> 16) & 1u)) & 0xffff0000u);
  if (vtop >= kInfBits) scale = __uint_as_float(0x7fc00000u);
  uint32_t vcodes = 0;
  if (scale > 0.0f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) vcodes |= value_code(y[i], scale) << (4 * i);
  }
  if (e < a.dim) {
    reinterpret_cast<uint32_t*>(a.k_codes)[at * (a.dim / 8) + lane] = codes;
    reinterpret_cast<uint32_t*>(a.v_codes)[at * (a.dim / 8) + lane] = vcodes;
    if ((lane & 3) == 0) a.k_scales[at * ((a.dim + 127) / 128 * 4) + lane / 4] = byte;
    if (lane == 0) a.v_scales[at] = scale;
  }
}

template <typename T>
__global__ __launch_bounds__(kRowThreads) void q4_read_kernel(Q4RowsArgs a) {
  const int per = kRowThreads / a.row_lanes;
  const int lane = threadIdx.x & (a.row_lanes - 1);
  const int64_t r = static_cast<int64_t>(blockIdx.x) * per + threadIdx.x / a.row_lanes;
  if (r >= static_cast<int64_t>(a.T) * a.kv_heads || lane * 8 >= a.dim) return;
  const int t = fast_div(static_cast<int>(r), a.heads), h = static_cast<int>(r) - t * a.kv_heads;
  const int64_t slot = a.slots[t];
  float x[8] = {}, y[8] = {};
  if (slot >= 0 && slot < a.num_slots) {
    const int blk = fast_div(static_cast<int>(slot), a.bs);
    const int row = static_cast<int>(slot) - blk * a.block_size;
    const int64_t at = (static_cast<int64_t>(blk) * a.kv_heads + h) * a.block_size + row;
    const uint32_t kc = reinterpret_cast<const uint32_t*>(a.k_codes)[at * (a.dim / 8) + lane];
    const uint32_t vc = reinterpret_cast<const uint32_t*>(a.v_codes)[at * (a.dim / 8) + lane];
    const int byte = a.k_scales[at * ((a.dim + 127) / 128 * 4) + lane / 4];
    const float scale = a.v_scales[at];
    typedef float f2 __attribute__((ext_vector_type(2)));
    const f2 k[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(kc, 1.0f, 0),
                     __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(kc, 1.0f, 1),
                     __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(kc, 1.0f, 2),
                     __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(kc, 1.0f, 3)};
    const f2 v[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(vc, 1.0f, 0),
                     __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(vc, 1.0f, 1),
                     __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(vc, 1.0f, 2),
                     __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(vc, 1.0f, 3)};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = byte == 255 ? __uint_as_float(0x7fc00000u) : ldexpf(k[i / 2][i & 1], byte - 127);
      y[i] = v[i / 2][i & 1] * scale;
    }
  }
  constexpr int N = 16 / sizeof(T);
  T* ko = static_cast<T*>(a.k_out) + r * a.dim + lane * 8;
  T* vo = static_cast<T*>(a.v_out) + r * a.dim + lane * 8;
#pragma unroll
  for (int i = 0; i < 8 / N; ++i) {
    RowVec<T, N> p, w;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      p.e[j] = static_cast<T>(x[i * N + j]);
      w.e[j] = static_cast<T>(y[i * N + j]);
    }
    reinterpret_cast<RowVec<T, N>*>(ko)[i] = p;
    reinterpret_cast<RowVec<T, N>*>(vo)[i] = w;
  }
}

template <typename T, int QV>
void launch_append_of(const Q4RowsArgs& a, const RotaryArgs& q, bool wide, hipStream_t st) {
  const int per = kRowThreads / a.row_lanes;
  const uint32_t rows = static_cast<uint32_t>((static_cast<int64_t>(a.T) * a.kv_heads + per - 1) / per);
  const uint32_t q_total = static_cast<uint32_t>(q.T) * q.token_units;
  const dim3 grid(rows + (q_total + kRowThreads - 1) / kRowThreads), block(kRowThreads);
  if (wide) hipLaunchKernelGGL((q4_append_kernel<T, true, QV>), grid, block, 0, st, a, rows, q, q_total);
  else hipLaunchKernelGGL((q4_append_kernel<T, false, QV>), grid, block, 0, st, a, rows, q, q_total);
}

}  // namespace

hipError_t launch_q4_append(const Q4RowsArgs& a, const RotaryArgs& q, int dtype, bool wide,
                            bool q_wide, hipStream_t st) {
  if (dtype == kF32) {
    if (q_wide) launch_append_of<float, 4>(a, q, wide, st);
    else launch_append_of<float, 1>(a, q, wide, st);
  } else if (dtype == kBF16) {
    if (q_wide) launch_append_of<__bf16, 8>(a, q, wide, st);
    else launch_append_of<__bf16, 1>(a, q, wide, st);
  } else {
    if (q_wide) launch_append_of<_Float16, 8>(a, q, wide, st);
    else launch_append_of<_Float16, 1>(a, q, wide, st);
  }
  return hipGetLastError();
}

hipError_t launch_q4_read(const Q4RowsArgs& a, int dtype, hipStream_t st) {
  const int per = kRowThreads / a.row_lanes;
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(a.T) * a.kv_heads + per - 1) / per));
  if (dtype == kF32) hipLaunchKernelGGL(q4_read_kernel<float>, grid, dim3(kRowThreads), 0, st, a);
  else if (dtype == kBF16) hipLaunchKernelGGL(q4_read_kernel<__bf16>, grid, dim3(kRowThreads), 0, st, a);
  else hipLaunchKernelGGL(q4_read_kernel<_Float16>, grid, dim3(kRowThreads), 0, st, a);
  return hipGetLastError();
}

}  // namespace sv
