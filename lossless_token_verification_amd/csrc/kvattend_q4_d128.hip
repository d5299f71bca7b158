// Attention over 4-bit pages for head sizes above 64 and up to 128.
#include "kvattend_q4_mx.h"

namespace sv {

hipError_t launch_attend_q4_d128(const AttendArgs& a, const Q4Cache& c, int dtype, int mt,
                               hipStream_t st) {
  return launch_q4_width<128>(a, c, dtype, mt, st);
}

}  // namespace sv
