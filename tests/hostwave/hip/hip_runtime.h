// The few names of the HIP language that the work search of the paged attention
// uses, for a build on the CPU: every thread of a workgroup is a fiber, and
// barriers and lane exchanges are met in lockstep.  A barrier or an exchange
// that some threads of its workgroup or wavefront do not take ends the program.
#pragma once

#include <math.h>
#include <stdint.h>
#include <stddef.h>

#define __host__
#define __device__
#define __global__
#define __forceinline__ inline

typedef int hipError_t;
typedef void* hipStream_t;
typedef void* hipEvent_t;
constexpr hipError_t hipSuccess = 0;
inline const char* hipGetErrorString(hipError_t) { return "error"; }
struct dim3 {
  unsigned x, y, z;
};

inline float __uint_as_float(uint32_t u) { return __builtin_bit_cast(float, u); }
inline uint32_t __float_as_uint(float f) { return __builtin_bit_cast(uint32_t, f); }
template <typename T>
inline T min(T a, T b) { return b < a ? b : a; }
template <typename T>
inline T max(T a, T b) { return a < b ? b : a; }

namespace hostwave {

constexpr int kLanes = 64;
struct Index {
  unsigned x;
};
// Leaves the running thread at a collective (kind, line); returns when all of
// them are there.
void meet(bool workgroup, int line);
// This wavefront's values of the current exchange.
uint64_t* slots();
int lane();

template <typename T>
inline T exchange(T v, int from, int line) {
  static_assert(sizeof(T) <= 8, "one register pair");
  uint64_t bits = 0;
  __builtin_memcpy(&bits, &v, sizeof(T));
  slots()[lane()] = bits;
  meet(false, line);
  const uint64_t got = slots()[from & (kLanes - 1)];
  meet(false, line);
  T r;
  __builtin_memcpy(&r, &got, sizeof(T));
  return r;
}

}  // namespace hostwave

extern hostwave::Index threadIdx;

template <typename T>
inline T __shfl(T v, int from, int, int line = __builtin_LINE()) {
  return hostwave::exchange(v, from, line);
}
template <typename T>
inline T __shfl_xor(T v, int mask, int, int line = __builtin_LINE()) {
  return hostwave::exchange(v, hostwave::lane() ^ mask, line);
}
template <typename T>
inline T __shfl_up(T v, int by, int, int line = __builtin_LINE()) {
  const int at = hostwave::lane();
  return hostwave::exchange(v, at >= by ? at - by : at, line);
}
inline uint64_t __ballot(bool p, int line = __builtin_LINE()) {
  hostwave::slots()[hostwave::lane()] = p;
  hostwave::meet(false, line);
  uint64_t r = 0;
  for (int i = 0; i < hostwave::kLanes; ++i) r |= (hostwave::slots()[i] & 1) << i;
  hostwave::meet(false, line);
  return r;
}
inline void __syncthreads(int line = __builtin_LINE()) { hostwave::meet(true, line); }
template <typename T>
inline T atomicAdd(T* p, T v) {
  const T old = *p;
  *p = old + v;
  return old;
}
