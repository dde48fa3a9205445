// attend_e2m1.hip -- the attention kernels for caches of 4-bit e2m1 numbers.
#include "attend_kernels.h"

namespace snack {
template snack_status launch_attend<SNACK_E2M1>(const AttendArgs&, int, int, unsigned, hipStream_t);
}
