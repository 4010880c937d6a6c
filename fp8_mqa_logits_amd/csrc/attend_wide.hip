// Attention over ranges, 128 or 256 columns a tile.
#include "attend_wide.h"

template void mqa::attend_wide<mqa::kRange>(const AttendParams&, dim3, hipStream_t);
