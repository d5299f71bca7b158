// Matrix-core paged attention, head_dim 256.
#include "kvattend_mfma.h"

namespace sv {

hipError_t launch_attend_d256(const AttendArgs& a, int dtype, int mt, hipStream_t st) {
  return dtype == kBF16 ? launch_rows_of<__bf16, 256>(a, mt, st)
                        : launch_rows_of<_Float16, 256>(a, mt, st);
}

}  // namespace sv
