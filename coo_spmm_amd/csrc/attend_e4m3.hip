// attend_e4m3.hip -- the attention kernels for caches of e4m3 numbers.
#include "attend_kernels.h"

namespace snack {
template snack_status launch_attend<SNACK_E4M3>(const AttendArgs&, int, int, unsigned, hipStream_t);
}
