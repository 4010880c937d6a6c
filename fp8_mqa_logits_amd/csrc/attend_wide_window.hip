// Attention through a window with sinks, 128 or 256 columns a tile.
#include "attend_wide.h"

template void mqa::attend_wide<mqa::kWindow>(const AttendParams&, dim3, hipStream_t);
