// Matrix-core paged attention for head sizes above 64 and up to 128.
#include "kvattend_mfma.h"

namespace sv {

hipError_t launch_attend_d128(const AttendArgs& a, int dtype, int mt, hipStream_t st) {
  return launch_width<128>(a, dtype, mt, st);
}

}  // namespace sv
