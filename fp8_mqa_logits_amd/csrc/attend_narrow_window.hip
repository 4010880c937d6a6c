// Attention through a window with sinks, up to 64 columns a tile.
#include "attend_narrow.h"

template void mqa::attend_narrow<mqa::kWindow>(const AttendParams&, dim3, hipStream_t);
