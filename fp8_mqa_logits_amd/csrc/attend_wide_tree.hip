// Attention over trees of drafts, 128 or 256 columns a tile.
#include "attend_wide.h"

template void mqa::attend_wide<mqa::kTree>(const AttendParams&, dim3, hipStream_t);
