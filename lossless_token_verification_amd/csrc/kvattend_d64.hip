// Matrix-core paged attention, head_dim 64.
#include "kvattend_mfma.h"

namespace sv {

hipError_t launch_attend_d64(const AttendArgs& a, int dtype, int mt, hipStream_t st) {
  return dtype == kBF16 ? launch_rows_of<__bf16, 64>(a, mt, st)
                        : launch_rows_of<_Float16, 64>(a, mt, st);
}

}  // namespace sv
