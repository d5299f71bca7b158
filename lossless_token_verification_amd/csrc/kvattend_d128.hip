// Matrix-core paged attention, head_dim 128.
#include "kvattend_mfma.h"

namespace sv {

hipError_t launch_attend_d128(const AttendArgs& a, int dtype, int mt, hipStream_t st) {
  return dtype == kBF16 ? launch_rows_of<__bf16, 128>(a, mt, st)
                        : launch_rows_of<_Float16, 128>(a, mt, st);
}

}  // namespace sv
