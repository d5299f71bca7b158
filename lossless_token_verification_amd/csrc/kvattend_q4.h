// Paged attention over a cache held in 4 bits: what the host code needs to know.
#pragma once

#include "kvattend.h"

namespace sv {

constexpr int kQ4KT = 128;   // positions of a key unit

hipError_t launch_attend_q4_d64(const AttendArgs& a, const Q4Cache& c, int dtype, int mt, hipStream_t st);
hipError_t launch_attend_q4_d128(const AttendArgs& a, const Q4Cache& c, int dtype, int mt, hipStream_t st);
hipError_t launch_attend_q4_d256(const AttendArgs& a, const Q4Cache& c, int dtype, int mt, hipStream_t st);

}  // namespace sv
