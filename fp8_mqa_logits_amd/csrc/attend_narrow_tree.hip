// Attention over trees of drafts, up to 64 columns a tile.
#include "attend_narrow.h"

template void mqa::attend_narrow<mqa::kTree>(const AttendParams&, dim3, hipStream_t);
