// The launches of lookup.hip (arguments checked by the caller) and what they take of sort.hip.
#pragma once

#include "matrix.h"

namespace gsk {

// index: int32, or int64 where wide.
hipError_t launch_lookup_fwd(const MatArg& table, const void* index, bool wide, float scale, const MatArg& y, int64_t rows,
                             int64_t entries, int cols, hipStream_t s);
size_t lookup_bwd_ws_bytes(int64_t rows, int cols, int64_t entries);
hipError_t launch_lookup_bwd(const MatArg& dy, const void* index, bool wide, float scale, const MatArg& dtable, int64_t rows,
                             int64_t entries, int cols, void* ws, hipStream_t s);

// ---- sort.hip: the places 0 .. count - 1 in the order of their entries (index as above; outside
// [0, entries): behind all others, as entry `entries`), equal ones in their own order.  keys, vals:
// count values each, count > 0.  marks: a byte for each entry, in whole 16 bytes, cleared on the way.
size_t sort_index_ws_bytes(int64_t count);
hipError_t launch_sort_index(const void* index, bool wide, uint32_t count, uint32_t entries, uint32_t* keys, uint32_t* vals,
                             uint8_t* marks, void* ws, hipStream_t s);

}  // namespace gsk
