// Matrix-core paged attention for head sizes up to 64.
#include "kvattend_mfma.h"

namespace sv {

hipError_t launch_attend_d64(const AttendArgs& a, int dtype, int mt, hipStream_t st) {
  return launch_width<64>(a, dtype, mt, st);
}

}  // namespace sv
