// Row-major matrices in MX4 on the device (gs.h has the format): a row is whole blocks of 32
// columns, 16 bytes each, two elements to a byte with the even column in the low half; byte b
// of a row's scales belongs to its block b.  Every value is exact in bfloat16 (two significant
// bits, from 2^-126 on), so products read decoded elements without another rounding.
#pragma once

#include "matrix.h"

namespace gsk {

// Bytes between the rows of an MX4 matrix.
__host__ __device__ inline int64_t mx4_pitch(const MatArg& m) { return m.ld / 2; }

// The matrix's rows from `row` on.
inline MatArg mx4_rows_from(MatArg m, int64_t row) {
  m.p += row * mx4_pitch(m);
  m.s += row * m.lds;
  return m;
}

// The scale byte for a block whose largest magnitude has these bits: the exponent field of
// the smallest 2^e with magnitude <= 1.5 2^(e + 2) (the addition carries into the exponent exactly
// when the mantissa is above 1.5's).  e2m1 has no NaN: an infinity or a NaN makes the whole
// block NaN by its scale.
__device__ inline uint32_t mx4_scale_byte(uint32_t top) {
  const int e = int((top + 0x3fffffu) >> 23) - 2;
  return top >= 0x7f800000u ? 255u : uint32_t(e < 1 ? 1 : e);
}

// The largest |v| of N values' bits, NaN above all.
template <int N>
__device__ inline uint32_t top_bits(const float* v) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t u = __float_as_uint(v[i]) & 0x7fffffffu;
    top = u > top ? u : top;
  }
  return top;
}

// Eight values of a block, divided by its scale, to e2m1 (nearest, ties to even).
__device__ inline uint32_t mx4_encode8(const float v[8], float scale) {
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], scale, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], scale, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], scale, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], scale, 3);
}

__device__ inline void mx4_decode8(uint32_t w, float scale, float v[8]) {
  const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 1);
  const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 3);
  v[0] = a[0], v[1] = a[1], v[2] = b[0], v[3] = b[1], v[4] = c[0], v[5] = c[1], v[6] = d[0], v[7] = d[1];
}

// Eight elements as bfloat16, exactly.
__device__ inline bf16x8 mx4_to_bf16x8(uint32_t w, float scale) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Of eight elements, or of a block's 32, the first n are kept (n from 8, 32 on: all; n <= 0: none).
__device__ inline uint32_t mx4_keep8(uint32_t w, int n) {
  return w & (n >= 8 ? ~0u : n <= 0 ? 0u : (1u << (4 * n)) - 1u);
}

__device__ inline u32x4 mx4_keep(u32x4 q, int n) {
#pragma unroll
  for (int j = 0; j < 4; ++j) q[j] = mx4_keep8(q[j], n - 8 * j);
  return q;
}

// ---- mx4.hip, linear_mx4.hip: the calls' launches (arguments checked by the caller)
hipError_t launch_mx4_pack(const MatArg& x, const MatArg& q, int64_t rows, int cols, hipStream_t s);
hipError_t launch_mx4_unpack(const MatArg& q, const MatArg& x, int64_t rows, int cols, hipStream_t s);
hipError_t launch_linear_mx4(const MatArg& x, const MatArg& w, const float* bias, int act, const MatArg& r,
                             const MatArg& y, int64_t rows, int k, int n, hipStream_t s);

}  // namespace gsk
