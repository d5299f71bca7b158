// Attention over 4-bit pages for head sizes above 128 and up to 256.
#include "kvattend_q4_mx.h"

namespace sv {

hipError_t launch_attend_q4_d256(const AttendArgs& a, const Q4Cache& c, int dtype, int mt,
                               hipStream_t st) {
  return launch_q4_width<256>(a, c, dtype, mt, st);
}

}  // namespace sv
