// What the linear layers' kernels share: the forward's epilogue and the launches of the
// variants, among which linear.hip chooses.
#pragma once

#include "matrix.h"

namespace gsk {

// ------------------------------------------------------------- epilogue of the forward

struct Epilogue {
  const float* bias;   // nullable
  int act;
  MatArg r, z, y;      // residual and kept pre-activation nullable
};

// 16 columns of a row to memory; for MX8 the lanes 16 apart hold the two halves of a
// 32-column block (all lanes active).  n: columns of the 16 that exist (<= 0: none); the
// others' values are zero where m is MX8.
__device__ inline void store16(const MatArg& m, int64_t row, int col, const float v[16], int n) {
  if (m.type == GS_MAT_MX8) {
    const uint32_t byte = mx8_scale_byte(max_across16(finite_top<16>(v)));
    const float scale = mx8_scale(byte);
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = mx8_encode4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3], scale);
    char* p = m.p + row * m.ld + col;
    if (n >= 16) {
      __builtin_memcpy(p, &w, 16);
    } else if (n > 0) {
      store_bytes8(p, w[0], w[1], n);
      if (n > 8) store_bytes8(p + 8, w[2], w[3], n - 8);
    }
    if (n > 0 && (col & 31) == 0) m.s[row * m.lds + (col >> 5)] = uint8_t(byte);
    return;
  }
  if (n > 0) store8(m, row, col, v, n);
  if (n > 8) store8(m, row, col + 8, v + 8, n - 8);
}

// v: x W^T for 16 columns of a row.
__device__ inline void finish16(const Epilogue& e, int64_t row, int col, float v[16], int n) {
  if (e.bias) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] += i < n ? e.bias[col + i] : 0.0f;
  }
  if (e.z.p) store16(e.z, row, col, v, n);
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = activate(v[i], e.act);
  if (e.r.p) {
    float r[16];
    raw8_to_float(load_raw8(e.r, row, col, n), e.r.type, r);
    raw8_to_float(load_raw8(e.r, row, col + 8, n - 8), e.r.type, r + 8);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] += r[i];
  }
  store16(e.y, row, col, v, n);
}

// ---- linear_rows.hip: narrow layers over many rows, the weight kept in LDS
bool rows_fwd_takes(int k, int n);
hipError_t launch_rows_fwd(const MatArg& x, const MatArg& w, const Epilogue& e, int64_t rows, int k, int n,
                           hipStream_t s);

// ---- linear_rows_bwd.hip: the gradients of the narrowest of them in one pass
bool rows_bwd_takes(int k, int n);
size_t rows_bwd_ws_bytes(int64_t rows, int k, int n);
hipError_t launch_rows_bwd(const MatArg& dy, const MatArg& z, int act, const MatArg& x, const MatArg& w,
                           const MatArg& dx, const MatArg& dw, float* dbias, int64_t rows, int k, int n, void* ws,
                           hipStream_t s);

}  // namespace gsk
