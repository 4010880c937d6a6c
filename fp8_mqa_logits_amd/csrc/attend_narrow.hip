// Attention over ranges, up to 64 columns a tile.
#include "attend_narrow.h"

template void mqa::attend_narrow<mqa::kRange>(const AttendParams&, dim3, hipStream_t);
