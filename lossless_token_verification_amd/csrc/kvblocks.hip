// Block-table extension: prefix sums over the sequences give every sequence
// its rows in the packed token arrays and its place in the pool's stack; each
// token's slot then follows from its position alone.
//
// With L_b tokens held and n_b new ones (page size s):
//   need_b = ceil((L_b + n_b) / s) - ceil(L_b / s),  off_b = sum_{b' < b} need_b',
//   block i of b = stack[top - 1 - off_b - i],  cu_b = sum_{b' < b} n_b'.
// A new logical block starts at a position >= L_b, which is always a new
// token's, so the token standing there writes the block's table entry, and
// every token computes its slot from the stack without waiting for a table
// write.
//
// The bytes are few (12 per token, a handful per sequence), so what counts is
// the latency of the launches: one workgroup makes the prefix sums and, up to
// kFusedTokens tokens, fills the token arrays itself; beyond that a second
// launch spreads the fill over the chip.  A batch of one thread per sequence
// keeps the sums' results in LDS for the fill and scans by lane moves on the
// vector unit.  One sequence and token takes 2.8 us on the device, B = 256 with 9
// tokens each 6.4, B = 64 prompts of up to 4096 (145000 rows) 4.3 and 7.9 for the
// fill; a call spends 8 to 10 us on the host.  The fill is a launch of its own
// because it reads what the first one wrote (sums, and freed blocks pushed); each
// of its workgroups makes the sums of the taken blocks again.  More sequences than
// threads go in chunks, three scans each: a call takes 20 us at 2048 single tokens,
// 37 at 4096, 0.22 ms at 16384 and 0.85 ms at 65536.
#include "kv_args.h"

namespace sv {

namespace {

constexpr int kScanThreads = 1024;     // most threads of the prefix-sum workgroup
constexpr int kFillThreads = 256;
constexpr int kFillTokens = 1024;      // tokens per workgroup of the fill launch
// Rows that the prefix-sum workgroup fills itself (64 sequences: 8.1 us against
// 9.8 with a second launch at 4096 rows, 10.9 against 9.9 at 8192).
constexpr int kFusedTokens = 6144;

// Exclusive prefix sum over the workgroup's threads; *total gets the sum.
// scratch: one value per wavefront.
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t* scratch, int64_t* total) {
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const int waves = blockDim.x / kWave;
  int64_t v = x;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const int64_t u = __shfl_up(static_cast<long long>(v), o, kWave);
    if (lane >= o) v += u;
  }
  __syncthreads();   // scratch may still be read from the scan before
  if (lane == kWave - 1) scratch[wave] = v;
  __syncthreads();
  int64_t before = 0, all = 0;
  for (int w = 0; w < waves; ++w) {
    if (w < wave) before += scratch[w];
    all += scratch[w];
  }
  *total = all;
  return before + v - x;
}

__device__ __forceinline__ int64_t ceil_blocks(int64_t n, const FastDiv& bs) {
  // n <= 2^31 - 1: the quotient of n - 1 never leaves the exact range
  return n > 0 ? fast_div(static_cast<int>(n - 1), bs) + 1 : 0;
}

// Inclusive prefix sum over a wavefront by lane moves: shifts within rows of 16
// lanes, then the last lane of a row, or of both, added to the rows after it.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t scan_step(uint32_t x) {
  return x + __builtin_amdgcn_update_dpp(0, x, CTRL, ROWS, 0xf, false);
}
__device__ __forceinline__ uint32_t wave_scan(uint32_t x) {
  x = scan_step<0x111, 0xf>(x);
  x = scan_step<0x112, 0xf>(x);
  x = scan_step<0x114, 0xf>(x);
  x = scan_step<0x118, 0xf>(x);
  x = scan_step<0x142, 0xa>(x);
  return scan_step<0x143, 0xc>(x);
}

// Exclusive prefix sums of two values over the workgroup (sums below 2^32); the
// totals in *ta and *tb.  scratch: two values per wavefront, not used since the
// last barrier.
__device__ __forceinline__ void block_scan2(uint32_t& x, uint32_t& y, uint32_t* scratch,
                                            uint32_t* ta, uint32_t* tb) {
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const int waves = blockDim.x / kWave;
  const uint32_t a = wave_scan(x), b = wave_scan(y);
  if (lane == kWave - 1) {
    scratch[2 * wave] = a;
    scratch[2 * wave + 1] = b;
  }
  __syncthreads();
  uint32_t before_a = 0, before_b = 0, all_a = 0, all_b = 0;
  for (int w = 0; w < waves; ++w) {
    const uint32_t p = scratch[2 * w], q = scratch[2 * w + 1];
    if (w < wave) {
      before_a += p;
      before_b += q;
    }
    all_a += p;
    all_b += q;
  }
  *ta = all_a;
  *tb = all_b;
  x = before_a + a - x;
  y = before_b + b - y;
}

// Rows [lo, hi) of the token arrays, all of the m sequences from c on, whose
// first rows (m + 1 of them), lengths before (-1: not served) and stack tops
// are in LDS.  Four rows a thread at a time: their lookups before their stores.
__device__ __forceinline__ void fill_chunk(const ExtendArgs& a, int c, int m, int lo, int hi,
                                           const int32_t* s_cu, const int32_t* s_len,
                                           const int64_t* s_off) {
  constexpr int kSide = 4;
  const int tid = threadIdx.x, nt = blockDim.x;
  const int first = s_cu[0], all = s_cu[m] - first;
  const float rate = all > 0 ? static_cast<float>(m) / static_cast<float>(all) : 0.0f;
  for (int t0 = lo + tid; t0 < hi; t0 += kSide * nt) {
    int pos[kSide], row[kSide], id[kSide];
    int32_t* fresh_entry[kSide];
#pragma unroll
    for (int i = 0; i < kSide; ++i) {
      const int t = t0 + i * nt;
      pos[i] = -1;
      fresh_entry[i] = nullptr;
      if (t >= hi) continue;
      // the last sequence that starts at or before t: where equal shares would
      // have it, or by bisection
      int l = min(static_cast<int>(static_cast<float>(t - first) * rate), m - 1);
      if (s_cu[l] > t || s_cu[l + 1] <= t) {
        l = 0;
        for (int r = m; r - l > 1;) {
          const int mid = (l + r) >> 1;
          if (s_cu[mid] <= t) l = mid; else r = mid;
        }
      }
      const int len = s_len[l];
      if (len < 0) continue;
      pos[i] = len + (t - s_cu[l]);
      const int lb = fast_div(pos[i], a.bs);
      row[i] = pos[i] - lb * a.block_size;
      const int64_t fresh = lb - ceil_blocks(len, a.bs);   // index among the blocks just taken
      int32_t* entry = a.table + static_cast<int64_t>(c + l) * a.max_blocks + lb;
      id[i] = fresh >= 0 ? a.free_blocks[s_off[l] - fresh] : *entry;
      if (fresh >= 0 && row[i] == 0) fresh_entry[i] = entry;
    }
#pragma unroll
    for (int i = 0; i < kSide; ++i) {
      const int t = t0 + i * nt;
      if (t >= hi) break;
      if (fresh_entry[i]) *fresh_entry[i] = id[i];
      a.slots[t] = pos[i] < 0 ? -1 : static_cast<int64_t>(id[i]) * a.block_size + row[i];
      if (a.positions) a.positions[t] = pos[i];
    }
  }
}

// Rows [t0, t1) behind the last token.
__device__ __forceinline__ void fill_rest(const ExtendArgs& a, int t0, int t1) {
  for (int t = t0 + threadIdx.x; t < t1; t += blockDim.x) {
    a.slots[t] = -1;
    if (a.positions) a.positions[t] = -1;
  }
}

// Fills rows [t0, t1) of the token arrays from the plan's outputs (cu,
// new_lens, num_taken, free_left), a chunk of blockDim.x sequences at a time.
__device__ void fill_tokens(const ExtendArgs& a, int t0, int t1, int64_t* scratch, int32_t* s_cu,
                            int32_t* s_len, int64_t* s_off) {
  const int tid = threadIdx.x, nt = blockDim.x;
  fill_rest(a, max(t0, a.cu[a.B]), t1);
  // ids in the stack before any was taken: what is left and what was taken
  int64_t taken_all = 0;
  if (a.B > nt)
    for (int c = 0; c < a.B; c += nt) {
      int64_t sum;
      block_scan(c + tid < a.B ? max(a.num_taken[c + tid], 0) : 0, scratch, &sum);
      taken_all += sum;
    }
  int64_t carry = 0;
  for (int c = 0; c < a.B; c += nt) {
    const int b = c + tid, m = min(nt, a.B - c);
    const int32_t got = b < a.B ? a.num_taken[b] : 0;
    int64_t sum;
    const int64_t off = carry + block_scan(max(got, 0), scratch, &sum);
    if (a.B <= nt) taken_all = sum;
    carry += sum;
    const int64_t top = a.free_left[0] + taken_all;
    if (b < a.B) {
      const int32_t lo = a.cu[b];
      s_cu[tid] = lo;
      if (b == a.B - 1 || tid == nt - 1) s_cu[tid + 1] = a.cu[b + 1];
      s_len[tid] = got >= 0 ? a.new_lens[b] - (a.cu[b + 1] - lo) : -1;   // -1: not served
      s_off[tid] = top - 1 - off;
    }
    __syncthreads();
    fill_chunk(a, c, m, max(t0, s_cu[0]), min(t1, s_cu[m]), s_cu, s_len, s_off);
    __syncthreads();
  }
}

struct FillShared {
  int64_t scratch[kScanThreads / kWave];
  int64_t off[kScanThreads];
  int32_t cu[kScanThreads + 1];
  int32_t len[kScanThreads];
  int32_t given;   // blocks handed out
};

// One thread per sequence (B <= blockDim; B * (T + 1) and B * max_freed below 2^32).
__global__ __launch_bounds__(kScanThreads) void extend_small_kernel(ExtendArgs a, int fused) {
  __shared__ FillShared sh;
  __shared__ uint32_t scratch[2][2 * kScanThreads / kWave];
  const int b = threadIdx.x;
  const bool in = b < a.B;
  const int64_t L = in ? a.lens[b] : 0, n = in ? a.num_new[b] : 0;
  const int m = in && a.freed ? min(max(a.num_freed[b], 0), a.max_freed) : 0;
  const int count = min(max(a.free_count[0], 0), a.free_capacity);
  if (b == 0) sh.given = 0;
  const uint32_t want = static_cast<uint32_t>(
      min(max(n, static_cast<int64_t>(0)), static_cast<int64_t>(a.T) + 1));
  uint32_t at = m, first = want, pushed, rows;
  block_scan2(at, first, scratch[0], &pushed, &rows);
  const int64_t top = min(static_cast<int64_t>(count) + pushed,
                          static_cast<int64_t>(a.free_capacity));
  for (int i = 0; i < m && static_cast<int64_t>(count) + at + i < a.free_capacity; ++i)
    a.free_blocks[static_cast<int64_t>(count) + at + i] =
        a.freed[static_cast<int64_t>(b) * a.max_freed + i];
  const int64_t cap = min(static_cast<int64_t>(a.max_blocks) * a.block_size,
                          static_cast<int64_t>(INT32_MAX));
  const bool good = n >= 0 && L >= 0 && L + n <= cap &&
                    static_cast<int64_t>(first) + want <= a.T;
  const uint32_t need =
      good ? static_cast<uint32_t>(ceil_blocks(L + n, a.bs) - ceil_blocks(L, a.bs)) : 0;
  uint32_t off = need, none = 0, unused_total, all_need;
  block_scan2(off, none, scratch[1], &all_need, &unused_total);
  const bool served = good && (need == 0 || static_cast<int64_t>(off) + need <= top);
  if (in) {
    const int lo = static_cast<int>(min(first, static_cast<uint32_t>(a.T)));
    a.new_lens[b] = static_cast<int32_t>(served ? L + n : L);
    a.num_taken[b] = served ? static_cast<int32_t>(need) : good ? -2 : -1;
    a.cu[b] = lo;
    sh.cu[b] = lo;
    sh.len[b] = served ? static_cast<int32_t>(L) : -1;
    sh.off[b] = top - 1 - off;
    // the served sequences that need blocks are the first ones: the last of them
    // knows how many were taken
    if (served && need > 0 && static_cast<int64_t>(off) + need <= top)
      atomicMax(&sh.given, static_cast<int32_t>(off + need));
  }
  const int used = static_cast<int>(min(rows, static_cast<uint32_t>(a.T)));
  if (b == 0) {
    a.cu[a.B] = used;
    sh.cu[a.B] = used;
  }
  __syncthreads();
  if (b == 0) a.free_left[0] = static_cast<int32_t>(top - sh.given);
  if (!fused) return;
  fill_rest(a, used, a.T);
  if (a.B > 0) fill_chunk(a, 0, a.B, 0, used, sh.cu, sh.len, sh.off);
}

__global__ __launch_bounds__(kScanThreads) void extend_kernel(ExtendArgs a, int fused) {
  __shared__ FillShared sh;
  const int tid = threadIdx.x, nt = blockDim.x;
  int64_t top = min(max(a.free_count[0], 0), a.free_capacity);
  if (a.freed) {
    for (int c = 0; c < a.B; c += nt) {
      const int b = c + tid;
      const int m = b < a.B ? min(max(a.num_freed[b], 0), a.max_freed) : 0;
      int64_t sum;
      const int64_t at = top + block_scan(m, sh.scratch, &sum);
      for (int i = 0; i < m && at + i < a.free_capacity; ++i)
        a.free_blocks[at + i] = a.freed[static_cast<int64_t>(b) * a.max_freed + i];
      top = min(top + sum, static_cast<int64_t>(a.free_capacity));
    }
  }
  const int64_t cap = min(static_cast<int64_t>(a.max_blocks) * a.block_size,
                          static_cast<int64_t>(INT32_MAX));
  int64_t rows = 0, taken = 0;   // tokens and blocks of the chunks before
  int64_t given = 0;             // blocks handed out
  for (int c = 0; c < a.B; c += nt) {
    const int b = c + tid;
    const int64_t L = b < a.B ? a.lens[b] : 0, n = b < a.B ? a.num_new[b] : 0;
    const int64_t want = max(n, static_cast<int64_t>(0));
    int64_t sum;
    const int64_t first = rows + block_scan(want, sh.scratch, &sum);
    rows += sum;
    const bool good = n >= 0 && L >= 0 && L + n <= cap && first + want <= a.T;
    const int64_t need = good ? ceil_blocks(L + n, a.bs) - ceil_blocks(L, a.bs) : 0;
    const int64_t off = taken + block_scan(need, sh.scratch, &sum);
    taken += sum;
    const bool served = good && (need == 0 || off + need <= top);
    if (b < a.B) {
      a.new_lens[b] = static_cast<int32_t>(served ? L + n : L);
      a.num_taken[b] = served ? static_cast<int32_t>(need) : good ? -2 : -1;
      a.cu[b] = static_cast<int32_t>(min(first, static_cast<int64_t>(a.T)));
    }
    block_scan(served ? need : 0, sh.scratch, &sum);
    given += sum;
  }
  if (tid == 0) {
    a.cu[a.B] = static_cast<int32_t>(min(rows, static_cast<int64_t>(a.T)));
    a.free_left[0] = static_cast<int32_t>(top - given);
  }
  if (!fused) return;
  __syncthreads();
  fill_tokens(a, 0, a.T, sh.scratch, sh.cu, sh.len, sh.off);
}

__global__ __launch_bounds__(kFillThreads) void fill_kernel(ExtendArgs a) {
  __shared__ FillShared sh;
  const int t0 = blockIdx.x * kFillTokens;
  fill_tokens(a, t0, min(a.T, t0 + kFillTokens), sh.scratch, sh.cu, sh.len, sh.off);
}

}  // namespace

hipError_t launch_extend(const ExtendArgs& a, hipStream_t st) {
  const int fused = a.T <= kFusedTokens;
  const int work = max(a.B, fused ? min(a.T, kScanThreads) : 0);
  const unsigned threads = static_cast<unsigned>(
      min(kScanThreads, max(kWave, (work + kWave - 1) / kWave * kWave)));
  const bool small = a.B <= static_cast<int>(threads) &&
                     static_cast<int64_t>(a.B) * (max(a.T, a.max_freed) + int64_t{1}) < UINT32_MAX;
  if (small)
    hipLaunchKernelGGL(extend_small_kernel, dim3(1), dim3(threads), 0, st, a, fused);
  else
    hipLaunchKernelGGL(extend_kernel, dim3(1), dim3(threads), 0, st, a, fused);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess || fused) return err;
  hipLaunchKernelGGL(fill_kernel, dim3((a.T + kFillTokens - 1) / kFillTokens), dim3(kFillThreads),
                     0, st, a);
  return hipGetLastError();
}

}  // namespace sv
