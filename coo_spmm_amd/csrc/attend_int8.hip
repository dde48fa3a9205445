// attend_int8.hip -- the attention kernels for caches of 8-bit integers.
#include "attend_kernels.h"

namespace snack {
template snack_status launch_attend<SNACK_INT8>(const AttendArgs&, int, int, unsigned, hipStream_t);
}
