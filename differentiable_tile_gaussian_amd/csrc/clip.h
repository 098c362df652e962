// The launches of clip.hip (arguments checked by the caller).
#pragma once

#include "gs_internal.h"

namespace gsk {

size_t clip_ws_bytes();
// out nullable: only the norm.
hipError_t launch_clip_grads(const gs_matrix* grads, const gs_matrix* out, int count, double max_norm, float* norm, void* ws,
                             hipStream_t s);

}  // namespace gsk
