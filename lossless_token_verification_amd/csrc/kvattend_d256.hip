// Matrix-core paged attention for head sizes above 128 and up to 256.
#include "kvattend_mfma.h"

namespace sv {

hipError_t launch_attend_d256(const AttendArgs& a, int dtype, int mt, hipStream_t st) {
  return launch_width<256>(a, dtype, mt, st);
}

}  // namespace sv
