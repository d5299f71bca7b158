// Paged attention on the vector units (float32 caches), and the launch that joins
// splits.
//
// One workgroup takes a few query rows and a split of their keys; its
// wavefronts take 8 keys a step each, 8 lanes to a key, so that a key's row is
// read in whole 128-byte lines and a dot product needs three exchanges.
// Softmax in one pass: every group of 8 lanes keeps its own reference m, kLead
// above the largest score so far (log2 units), and the sum l and the output
// relative to it; a new one scales both by 2^(m_old - m_new).  The groups' states
// are merged once at the end.  Weights are 2^-kLead at most, so that 256 of the
// largest values add up without overflow.
//
// Single tokens are bound by the pages' bandwidth (B = 64 over 2300 positions, 32
// query and 8 key heads of 128: 1.2 GB in 220 us, 5.5 TB/s), more rows by the
// vector units, which read a key once for 4 rows (2 above head_dim 128, for the
// registers): 9 tokens over the same 1.18 ms, 18 TF.
#include "kvattend.h"

namespace sv {

namespace {

typedef _Float16 half_t;
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kRowWaves = 4;
constexpr int kKeysPerStep = 8;
constexpr float kLead = 8.0f;
static_assert(kRowWaves * kKeysPerStep == kRowsKT, "keys per unit");

// NF: floats of a row each of the 8 lanes of a key holds (8 * NF >= head_dim).
template <int NF, int R>
__global__ __launch_bounds__(kRowWaves * kWave) void attend_rows_kernel(AttendArgs a) {
  constexpr int PV = 4, NV = NF / PV;   // floats of a vector, vectors of a lane
  __shared__ AttendPlanShared<kRowWaves> plan;
  __shared__ float so[kRowWaves][R][8 * NF];
  __shared__ float sm[kRowWaves][R], sl[kRowWaves][R];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const int x = blockIdx.x / a.kv_heads, h = blockIdx.x - x * a.kv_heads;
  AttendItem it;
  if (!attend_find<R, kRowsKT, kRowWaves>(a, x, a.max_slots > 0 && blockIdx.x == 0, plan, it))
    return;
  if (it.splits > 1 && h == 0 && tid == 0) attend_slot_info(a, it);

  const int sub = lane & 7, kg = lane >> 3;
  const int nv = a.D / PV;
  const float c = a.scale * kLog2e;
  float q[R][NF], o[R][NF], m[R], l[R];
  int pos[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    int token, head;
    attend_row(a, it.token0, it.row0 + min(r, it.rows - 1), h, token, head);
    pos[r] = it.pos0 + token - it.token0;
    const float* qr =
        static_cast<const float*>(a.q) + token * a.q_stride + static_cast<int64_t>(head) * a.D;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = sub + 8 * i;
      f32x4 w = {0.0f, 0.0f, 0.0f, 0.0f};
      if (v < nv) w = reinterpret_cast<const f32x4*>(qr)[v];
#pragma unroll
      for (int e = 0; e < PV; ++e) q[r][i * PV + e] = w[e];
    }
    m[r] = -INFINITY;
    l[r] = 0.0f;
#pragma unroll
    for (int i = 0; i < NF; ++i) o[r][i] = 0.0f;
  }

  const int32_t* table = a.table + static_cast<int64_t>(it.b) * a.max_blocks;
  const int64_t head_off = static_cast<int64_t>(h) * a.block_size;
  for (int u = it.u0; u < it.u1; ++u) {
    const int key = u * kRowsKT + wave * kKeysPerStep + kg;
    bool in = key >= it.key_lo && key < it.key_hi;
    int64_t off = 0;
    if (in) {
      const int lb = fast_div(key, a.bs);
      const int id = table[lb];
      in = id >= 0 && id < a.num_blocks;
      off = id * a.block_stride + (head_off + (key - lb * a.block_size)) * a.D;
    }
    f32x4 kw[NV], vw[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = sub + 8 * i;
      kw[i] = vw[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      if (in && v < nv) {
        kw[i] = reinterpret_cast<const f32x4*>(static_cast<const float*>(a.k) + off)[v];
        vw[i] = reinterpret_cast<const f32x4*>(static_cast<const float*>(a.v) + off)[v];
      }
    }
    float s[R];
#pragma unroll
    for (int r = 0; r < R; ++r) s[r] = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int e = 0; e < PV; ++e) s[r] = fmaf(q[r][i * PV + e], kw[i][e], s[r]);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      s[r] += __shfl_xor(s[r], 1, kWave);
      s[r] += __shfl_xor(s[r], 2, kWave);
      s[r] += __shfl_xor(s[r], 4, kWave);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      // a position the row does not see leaves its state alone, whatever it holds
      if (!in || key > pos[r] ||
          (a.window > 0 && static_cast<int64_t>(key) <= static_cast<int64_t>(pos[r]) - a.window))
        continue;
      const float mn = fmaxf(m[r], fmaf(s[r], c, kLead)), ref = mn == -INFINITY ? 0.0f : mn;
      const float f = __builtin_amdgcn_exp2f(m[r] - ref);
      const float p = __builtin_amdgcn_exp2f(fmaf(s[r], c, -ref));
      m[r] = mn;
      l[r] = fmaf(l[r], f, p);
#pragma unroll
      for (int i = 0; i < NF; ++i) o[r][i] = fmaf(p, vw[i / PV][i % PV], o[r][i] * f);
    }
  }

  // merge the wavefront's 8 key groups, then the wavefronts
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float mw = m[r];
#pragma unroll
    for (int b = 8; b < kWave; b <<= 1) mw = fmaxf(mw, __shfl_xor(mw, b, kWave));
    const float f = __builtin_amdgcn_exp2f(m[r] - (mw == -INFINITY ? 0.0f : mw));
    l[r] *= f;
#pragma unroll
    for (int b = 8; b < kWave; b <<= 1) l[r] += __shfl_xor(l[r], b, kWave);
#pragma unroll
    for (int i = 0; i < NF; ++i) {
      float t = o[r][i] * f;
#pragma unroll
      for (int b = 8; b < kWave; b <<= 1) t += __shfl_xor(t, b, kWave);
      if (kg == 0) so[wave][r][(sub + 8 * (i / PV)) * PV + i % PV] = t;
    }
    if (lane == 0) {
      sm[wave][r] = mw;
      sl[wave][r] = l[r];
    }
  }
  __syncthreads();
  for (int i = tid; i < R * a.D; i += kRowWaves * kWave) {
    const int r = i / a.D, d = i - r * a.D;
    if (r >= it.rows) break;
    float mw = sm[0][r];
#pragma unroll
    for (int w = 1; w < kRowWaves; ++w) mw = fmaxf(mw, sm[w][r]);
    const float ref = mw == -INFINITY ? 0.0f : mw;
    float lw = 0.0f, ow = 0.0f;
#pragma unroll
    for (int w = 0; w < kRowWaves; ++w) {
      const float f = __builtin_amdgcn_exp2f(sm[w][r] - ref);
      lw = fmaf(sl[w][r], f, lw);
      ow = fmaf(so[w][r][d], f, ow);
    }
    if (it.splits > 1) {
      const int64_t p = (static_cast<int64_t>(it.slot) * a.kv_heads + h) * R + r;
      a.part_o[p * a.D + d] = ow;
      if (d == 0) {
        a.part_ml[p * 2] = mw;
        a.part_ml[p * 2 + 1] = lw;
      }
    } else {
      int token, head;
      attend_row(a, it.token0, it.row0 + r, h, token, head);
      const int64_t at = static_cast<int64_t>(token) * a.heads + head;
      static_cast<float*>(a.out)[at * a.D + d] = lw == 0.0f ? 0.0f : ow / lw;
      if (a.lse && d == 0) a.lse[at] = lw == 0.0f ? -INFINITY : (mw + log2f(lw)) * kLn2;
    }
  }
}

// Joins the splits of the tiles that were split: out = sum_s 2^(m_s - M) O_s /
// sum_s 2^(m_s - M) l_s.  One workgroup per slot and key head; the slots of a
// tile share its rows.  A row is taken by head_dim / 4 threads, 4 elements
// each; where there are fewer rows than such groups, several groups share a
// row's splits and add up in a fixed order.
template <typename T>
__global__ __launch_bounds__(kRowWaves * kWave) void attend_join_kernel(AttendArgs a, int mt) {
  constexpr int NT = kRowWaves * kWave;
  __shared__ f32x4 so[NT];
  __shared__ float sm[NT], sl[NT];
  const int tid = threadIdx.x;
  const int slot = blockIdx.x / a.kv_heads, h = blockIdx.x - slot * a.kv_heads;
  const SlotInfo s = a.info[slot];
  if (slot >= *a.slot_count) return;
  const int mine = s.split < s.rows ? (s.rows - s.split - 1) / s.splits + 1 : 0;
  if (mine == 0) return;
  const int lanes = a.D / 4, groups = NT / lanes;
  const int parts = mine >= groups ? 1 : min(groups / mine, s.splits);
  const int side = groups / parts;            // rows taken at a time
  const int g = tid / lanes, d = (tid - g * lanes) * 4;
  const int part = g % parts;
  const int64_t step = static_cast<int64_t>(a.kv_heads) * mt;
  const int64_t p00 = (static_cast<int64_t>(slot - s.split) * a.kv_heads + h) * mt;
  // parts > 1 takes every row at once (side >= mine), so its barriers are met by all
  for (int i = g / parts; i < mine || parts > 1; i += side) {
    const bool in = i < mine && g < side * parts;
    const int r = s.split + i * s.splits;
    float mx = -INFINITY, l = 0.0f;
    f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
    if (in) {
      const float* ml = a.part_ml + (p00 + r) * 2;
      const float* po = a.part_o + (p00 + r) * a.D + d;
#pragma unroll 4
      for (int t = part; t < s.splits; t += parts) mx = fmaxf(mx, ml[t * step * 2]);
      const float ref = mx == -INFINITY ? 0.0f : mx;
#pragma unroll 4
      for (int t = part; t < s.splits; t += parts) {
        const float f = __builtin_amdgcn_exp2f(ml[t * step * 2] - ref);
        l = fmaf(ml[t * step * 2 + 1], f, l);
        const f32x4 x = *reinterpret_cast<const f32x4*>(po + t * step * a.D);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = fmaf(x[e], f, o[e]);
      }
    }
    if (parts > 1) {
      so[tid] = o;
      sm[tid] = mx;
      sl[tid] = l;
      __syncthreads();
      if (!in || part != 0) return;
      for (int t = 1; t < parts; ++t) mx = fmaxf(mx, sm[tid + t * lanes]);
      const float ref = mx == -INFINITY ? 0.0f : mx;
      l = 0.0f;
      o = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      for (int t = 0; t < parts; ++t) {
        const float f = __builtin_amdgcn_exp2f(sm[tid + t * lanes] - ref);
        l = fmaf(sl[tid + t * lanes], f, l);
        const f32x4 x = so[tid + t * lanes];
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = fmaf(x[e], f, o[e]);
      }
    }
    if (in) {
      int token, head;
      attend_row(a, s.token0, s.row0 + r, h, token, head);
      const int64_t at = static_cast<int64_t>(token) * a.heads + head;
      const float inv = 1.0f / l;
      typedef T t4 __attribute__((ext_vector_type(4)));
      t4 y;
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = static_cast<T>(l == 0.0f ? 0.0f : o[e] * inv);
      *reinterpret_cast<t4*>(static_cast<T*>(a.out) + at * a.D + d) = y;
      if (a.lse && d == 0) a.lse[at] = l == 0.0f ? -INFINITY : (mx + log2f(l)) * kLn2;
    }
    if (parts > 1) return;
  }
}

}  // namespace

hipError_t launch_attend_rows(const AttendArgs& a, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(a.grid_items) * a.kv_heads), block(kRowWaves * kWave);
  if (a.D <= 64) hipLaunchKernelGGL((attend_rows_kernel<8, kRowsMT64>), grid, block, 0, st, a);
  else if (a.D <= 128)
    hipLaunchKernelGGL((attend_rows_kernel<16, kRowsMT128>), grid, block, 0, st, a);
  else
    hipLaunchKernelGGL((attend_rows_kernel<32, kRowsMT256>), grid, block, 0, st, a);
  return hipGetLastError();
}

hipError_t launch_attend_join(const AttendArgs& a, int dtype, int mt, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(a.max_slots) * a.kv_heads), block(kRowWaves * kWave);
  if (dtype == kF32) hipLaunchKernelGGL(attend_join_kernel<float>, grid, block, 0, st, a, mt);
  else if (dtype == kBF16) hipLaunchKernelGGL(attend_join_kernel<__bf16>, grid, block, 0, st, a, mt);
  else hipLaunchKernelGGL(attend_join_kernel<half_t>, grid, block, 0, st, a, mt);
  return hipGetLastError();
}

}  // namespace sv
