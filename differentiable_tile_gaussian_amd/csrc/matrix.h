// Row-major matrices of the network operators on the device: 8-column chunks loaded from
// float32, bfloat16 or MX8 storage, and the MX8 encoding.
//
// MX8 (the microscaling format with e4m3 elements): the 32-column block b of a row holds
// v = q 2^(scale byte - 127), with the smallest scale exponent >= -126 for which the
// block's largest finite magnitude is at most 448 2^e (448 is e4m3's largest value).  A
// power-of-two scale makes the decoded value exact in bfloat16 (4 significant bits; from 2^-126
// on, where its full precision ends), so the matrix products read the decoded values without
// another rounding.
#pragma once

#include "gs_internal.h"

namespace gsk {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// A matrix argument of a kernel (gs_matrix without its sizes).  p == nullptr: absent.
struct MatArg {
  char* p;
  uint8_t* s;
  int64_t ld, lds;
  int32_t type;
};

inline MatArg mat_arg(const gs_matrix* m) {
  if (!m) return MatArg{nullptr, nullptr, 0, 0, GS_MAT_F32};
  return MatArg{static_cast<char*>(m->data), m->scales, m->ld, m->scales_ld, m->type};
}

// 8 columns as loaded: float32 uses both halves, bfloat16 lo, MX8 the first two words of lo
// and the scale byte.
struct Raw8 {
  u32x4 lo, hi;
  uint32_t scale;
};

// Columns col .. col + 7 of a row, of which the first n exist (n >= 8: all; the others
// read as zero).  col is a multiple of 8.  The addresses need only the element's own
// alignment: the copies compile to wide loads in the unaligned access mode, which is the
// amdhsa default.
__device__ inline Raw8 load_raw8(const MatArg& m, int64_t row, int col, int n) {
  Raw8 r;
  r.lo = u32x4{0, 0, 0, 0};
  r.hi = u32x4{0, 0, 0, 0};
  r.scale = 0;
  if (m.type == GS_MAT_BF16) {
    const char* p = m.p + (row * m.ld + col) * 2;
    if (n >= 8) {
      __builtin_memcpy(&r.lo, __builtin_assume_aligned(p, 2), 16);
    } else {
      const uint16_t* e = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) r.lo[i / 2] |= uint32_t(e[i]) << (16 * (i & 1));
    }
  } else if (m.type == GS_MAT_F32) {
    const char* p = m.p + (row * m.ld + col) * 4;
    if (n >= 8) {
      __builtin_memcpy(&r.lo, __builtin_assume_aligned(p, 4), 16);
      __builtin_memcpy(&r.hi, __builtin_assume_aligned(p + 16, 4), 16);
    } else {
      const uint32_t* e = reinterpret_cast<const uint32_t*>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i < n) r.lo[i] = e[i];
        if (i + 4 < n) r.hi[i] = e[i + 4];
      }
    }
  } else {
    const char* p = m.p + row * m.ld + col;
    if (n > 0) r.scale = m.s[row * m.lds + (col >> 5)];
    if (n >= 8) {
      u32x2 v;
      __builtin_memcpy(&v, p, 8);
      r.lo[0] = v[0];
      r.lo[1] = v[1];
    } else {
      const uint8_t* e = reinterpret_cast<const uint8_t*>(p);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) r.lo[i / 4] |= uint32_t(e[i]) << (8 * (i & 3));
    }
  }
  return r;
}

__device__ inline float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ inline float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// A scale byte as the float whose exponent the scaled conversions read (2^-127 for byte
// 0, NaN for byte 255).
__device__ inline float mx8_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

__device__ inline void raw8_to_float(const Raw8& r, int type, float v[8]) {
  if (type == GS_MAT_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_lo(r.lo[i]);
      v[2 * i + 1] = bf16_hi(r.lo[i]);
    }
  } else if (type == GS_MAT_F32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = __uint_as_float(r.lo[i]);
      v[4 + i] = __uint_as_float(r.hi[i]);
    }
  } else {
    const float s = mx8_scale(r.scale);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(r.lo[i], s, false);
      const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(r.lo[i], s, true);
      v[4 * i] = a[0];
      v[4 * i + 1] = a[1];
      v[4 * i + 2] = b[0];
      v[4 * i + 3] = b[1];
    }
  }
}

// Four e4m3 values as bfloat16, exactly.
__device__ inline u32x2 mx8_to_bf16x4(uint32_t w, float scale) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, true);
  return u32x2{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b)};
}

// Two floats rounded to bfloat16 (nearest even).
__device__ inline uint32_t pack_bf16(float a, float b) {
  const bf16x2 v{(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, v);
}

// ---- rows of at least 8 columns, 8 to a lane, without branches
//
// A row is held by neighbouring lanes, lane l's chunk starting at column 8 l.  A chunk that
// would pass the row's end is held from column cols - 8 instead: its first `skip` values are
// columns that the lane before it holds too (from 8 on: the whole chunk is another's).  So
// every load is a full one, inside the row.  Sums leave the repeated values out; float32 and
// bfloat16 results are written from where they are held, the repeated ones twice with the
// same bits; MX8 results, whose blocks have their places, are moved down first.
struct Held {
  int at, skip;
};

__device__ inline Held held_at(int col, int cols) {
  const int at = col < cols - 8 ? col : cols - 8;
  return {at, col - at};
}

// The chunk's columns at .. at + 7 (any alignment).  MX8: a chunk at a block's end takes two
// scales, in the low and the second byte.
__device__ inline Raw8 load_held(const MatArg& m, int64_t row, const Held& c) {
  Raw8 r;
  r.hi = u32x4{0, 0, 0, 0};
  r.scale = 0;
  if (m.type == GS_MAT_BF16) {
    __builtin_memcpy(&r.lo, __builtin_assume_aligned(m.p + (row * m.ld + c.at) * 2, 2), 16);
  } else if (m.type == GS_MAT_F32) {
    const char* p = m.p + (row * m.ld + c.at) * 4;
    __builtin_memcpy(&r.lo, __builtin_assume_aligned(p, 4), 16);
    __builtin_memcpy(&r.hi, __builtin_assume_aligned(p + 16, 4), 16);
  } else {
    u32x2 v;
    __builtin_memcpy(&v, m.p + row * m.ld + c.at, 8);
    r.lo = u32x4{v[0], v[1], 0, 0};
    const uint8_t* s = m.s + row * m.lds;
    r.scale = s[c.at >> 5] | uint32_t(s[(c.at + 7) >> 5]) << 8;
  }
  return r;
}

__device__ inline void held_to_float(const Raw8& r, int type, const Held& c, float v[8]) {
  if (type != GS_MAT_MX8) {
    raw8_to_float(r, type, v);
    return;
  }
  Raw8 one = r;
  one.scale = r.scale & 255u;
  raw8_to_float(one, type, v);
  if (c.skip > 0) {   // only such a chunk can lie across a block's end
    one.scale = r.scale >> 8;
    float w[8];
    raw8_to_float(one, type, w);
    const int left = 32 - (c.at & 31);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < left ? v[i] : w[i];
  }
}

// Moves a held chunk's own values to its front, zeros behind them.
__device__ inline void move_down(const Held& c, float v[8]) {
#pragma unroll
  for (int b = 4; b > 0; b /= 2)
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c.skip & b ? (i + b < 8 ? v[i + b] : 0.0f) : v[i];
  if (c.skip >= 8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
  }
}

// ---- 16 columns of a row of any width and alignment, without branches
//
// A piece that would pass the row's end is loaded from column cols - 16 instead and moved
// down when it is used; what is behind the row's end, and an absent row, reads as zero.
// NARROW: for rows of fewer than 16 columns, loaded one by one (a kernel of its own: the other
// loads would wait where the two ways join).
template <int TYPE, bool NARROW>
struct Raw16 {
  static constexpr int kWords = TYPE == GS_MAT_F32 ? 16 : TYPE == GS_MAT_BF16 ? 8 : 4;
  uint32_t w[kWords];
  uint32_t scale, skip;

  // row: a row of the matrix, also where the piece is absent (live false).
  __device__ void load(const MatArg& m, int64_t row, int col, int cols, bool live) {
    constexpr int kE = 4 * kWords / 16;
    if constexpr (!NARROW) {
      const int at = col < cols - 16 ? col : cols - 16;
      const char* p = m.p + (row * m.ld + at) * kE;
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        u32x4 v;
        __builtin_memcpy(&v, __builtin_assume_aligned(p + 16 * i, kE), 16);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[4 * i + j] = v[j];
      }
      if constexpr (TYPE == GS_MAT_MX8) scale = m.s[row * m.lds + ((col < cols ? col : cols - 1) >> 5)];
      skip = live ? (col - at < 16 ? col - at : 16) : 16;
    } else {
      const int n = live ? cols - col : 0;
      const Raw8 lo = load_raw8(m, row, col, n), hi = load_raw8(m, row, col + 8, n - 8);
#pragma unroll
      for (int i = 0; i < kWords / 2; ++i) {
        w[i] = i < 4 ? lo.lo[i] : lo.hi[i % 4];
        w[kWords / 2 + i] = i < 4 ? hi.lo[i] : hi.hi[i % 4];
      }
      scale = lo.scale;
      skip = 0;
    }
  }
  // For a piece that lies within the row: zeros if its row is absent.
  __device__ void settle_whole() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = skip >= 16 ? 0u : w[i];
  }
  // Moves the piece's own columns to its front, zeros behind them.
  __device__ void settle() {
    constexpr int kE = 4 * kWords / 16;
    const uint32_t bytes = skip * kE;
#pragma unroll
    for (int b = kWords; b > 0; b /= 2)
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = bytes & (4 * b) ? (i + b < kWords ? w[i + b] : 0u) : w[i];
    if constexpr (kE < 4) {
#pragma unroll
      for (int i = 0; i < kWords; ++i)
        w[i] = __builtin_amdgcn_alignbyte(i + 1 < kWords ? w[i + 1] : 0u, w[i], bytes & 3);
    }
  }
};

// ---- buffer access
//
// The row kernels' fast paths load and store through buffer descriptors, whose range check
// stands in for branches: an absent row or piece gets the offset kAbsent, past the
// descriptor's range, and then reads as zero or is not written.  Without branches the number
// of memory operations in flight is known at compile time, and a wait for one turn's loads
// does not also wait for the stores issued since.
typedef __amdgpu_buffer_rsrc_t Buffer;
constexpr uint32_t kAbsent = 0x80000000u;

// p is the same in all lanes (and said to be, so that the descriptor is in scalar registers).
__device__ inline Buffer buffer_at(const void* p) {
  const uint64_t u = reinterpret_cast<uint64_t>(p);
  const uint64_t lo = uint32_t(__builtin_amdgcn_readfirstlane(int(u)));
  const uint64_t hi = uint32_t(__builtin_amdgcn_readfirstlane(int(u >> 32)));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(lo | hi << 32), 0, 0x7fffffff, 0x00020000);
}
__device__ inline u32x4 buffer_load16(Buffer b, uint32_t off) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(b, int(off), 0, 0));
}
__device__ inline uint32_t buffer_load1(Buffer b, uint32_t off) {
  return uint32_t(uint8_t(__builtin_amdgcn_raw_buffer_load_b8(b, int(off), 0, 0)));
}
__device__ inline void buffer_store16(Buffer b, uint32_t off, u32x4 v) {
  __builtin_amdgcn_raw_buffer_store_b128(v, b, int(off), 0, 0);
}
__device__ inline void buffer_store1(Buffer b, uint32_t off, uint32_t v) {
  __builtin_amdgcn_raw_buffer_store_b8(uint8_t(v), b, int(off), 0, 0);
}

// Bytes of an element, and of n of them.
__host__ __device__ constexpr uint32_t element_bytes(int type) {
  return type == GS_MAT_F32 ? 4 : type == GS_MAT_BF16 ? 2 : 1;
}

// The matrix's rows from `row` on.
inline MatArg rows_from(MatArg m, int64_t row) {
  if (m.p) m.p += row * m.ld * element_bytes(m.type);
  if (m.s) m.s += row * m.lds;
  return m;
}

// A launch has fewer than 2^32 threads along x: the most blocks of 256, beyond which the rows
// are taken by several launches.
constexpr int64_t kMaxBlocks = (int64_t(1) << 24) - 1;

// launch(first, count, blocks) for parts of the rows, per_block of them to a block.
template <class Launch>
inline void for_row_parts(int64_t rows, int64_t per_block, Launch launch) {
  const int64_t most = kMaxBlocks * per_block;
  for (int64_t first = 0; first < rows; first += most) {
    const int64_t count = rows - first < most ? rows - first : most;
    launch(first, count, div_up(count, per_block));
  }
}

// Whether a matrix can be taken through buffers: rows start at multiples of 4 bytes, and 256
// rows (at most what a block spans from its base) stay within the descriptor's range.
inline bool buffer_ok(const MatArg& m) {
  if (!m.p) return true;
  const int64_t pitch = m.ld * element_bytes(m.type);
  return reinterpret_cast<uintptr_t>(m.p) % 4 == 0 && pitch % 4 == 0 && pitch < (int64_t(1) << 22) &&
         (m.type != GS_MAT_MX8 || m.lds < (int64_t(1) << 22));
}

// ---- encoding

// The largest finite |v| of N values' bits.  The float maximum passes over NaN; only when an
// infinity is among them are the finite ones gone through one by one.
template <int N>
__device__ inline uint32_t finite_top(const float* v) {
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < N; i += 2) top = fmaxf(fmaxf(fabsf(v[i]), fabsf(v[i + 1])), top);
  uint32_t bits = __float_as_uint(top);
  if (bits >= 0x7f800000u) {
    bits = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t u = __float_as_uint(v[i]) & 0x7fffffffu;
      bits = u < 0x7f800000u && u > bits ? u : bits;
    }
  }
  return bits;
}

// The scale byte for a block whose largest finite magnitude has these bits: the exponent
// field of the smallest 2^e with magnitude <= 1.75 2^(e + 8) (the addition carries into
// the exponent exactly when the mantissa is above 1.75's).
__device__ inline uint32_t mx8_scale_byte(uint32_t top) {
  const int e = int((top + 0x1fffffu) >> 23) - 8;
  return uint32_t(e < 1 ? 1 : e);
}

// Four values of a block, divided by its scale, to e4m3 (nearest even; infinities and NaN
// become NaN).
__device__ inline uint32_t mx8_encode4(float a, float b, float c, float d, float scale) {
  typedef short s16x2 __attribute__((ext_vector_type(2)));
  s16x2 w{0, 0};
  w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, a, b, scale, false);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, c, d, scale, true);
  return __builtin_bit_cast(uint32_t, w);
}

// The larger of x and the same value of the lane 16 or 32 away.
__device__ inline uint32_t max_across16(uint32_t x) {
  const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
  return r[0] > r[1] ? r[0] : r[1];
}

// ---- stores of 8 (or the first n) columns

__device__ inline void store_f32x8(float* p, const float v[8], int n) {
  if (n >= 8) {
    const f32x4 a{v[0], v[1], v[2], v[3]}, b{v[4], v[5], v[6], v[7]};
    __builtin_memcpy(__builtin_assume_aligned(p, 4), &a, 16);
    __builtin_memcpy(__builtin_assume_aligned(p + 4, 4), &b, 16);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = v[i];
  }
}

__device__ inline void store_bf16x8(char* p, const float v[8], int n) {
  const u32x4 w{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
  if (n >= 8) {
    __builtin_memcpy(__builtin_assume_aligned(p, 2), &w, 16);
  } else {
    uint16_t* e = reinterpret_cast<uint16_t*>(p);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) e[i] = uint16_t(w[i / 2] >> (16 * (i & 1)));
  }
}

__device__ inline void store_bytes8(char* p, uint32_t a, uint32_t b, int n) {
  if (n >= 8) {
    const u32x2 w{a, b};
    __builtin_memcpy(p, &w, 8);
  } else {
    uint8_t* e = reinterpret_cast<uint8_t*>(p);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) e[i] = uint8_t((i < 4 ? a : b) >> (8 * (i & 3)));
  }
}

// float32 or bfloat16 (the other types are the callers').
__device__ inline void store8(const MatArg& m, int64_t row, int col, const float v[8], int n) {
  if (m.type == GS_MAT_F32)
    store_f32x8(reinterpret_cast<float*>(m.p) + row * m.ld + col, v, n);
  else
    store_bf16x8(m.p + (row * m.ld + col) * 2, v, n);
}

// The largest magnitude over the four neighbouring lanes that hold a 32-column block.
__device__ inline uint32_t max_over_quad(uint32_t x) {
  uint32_t y = uint32_t(__builtin_amdgcn_mov_dpp(int(x), 0xb1, 0xf, 0xf, true));  // lanes 1 0 3 2
  x = x > y ? x : y;
  y = uint32_t(__builtin_amdgcn_mov_dpp(int(x), 0x4e, 0xf, 0xf, true));           // lanes 2 3 0 1
  return x > y ? x : y;
}

// A chunk of 8 columns to MX8, where four neighbouring lanes (all active) hold the four
// chunks of one block; values of absent columns are zero.
__device__ inline void store_mx8_quad(const MatArg& m, int64_t row, int col, const float v[8], int n) {
  const uint32_t byte = mx8_scale_byte(max_over_quad(finite_top<8>(v)));
  const float scale = mx8_scale(byte);
  const uint32_t a = mx8_encode4(v[0], v[1], v[2], v[3], scale), b = mx8_encode4(v[4], v[5], v[6], v[7], scale);
  if (n > 0) {
    store_bytes8(m.p + row * m.ld + col, a, b, n);
    if ((col & 31) == 0) m.s[row * m.lds + (col >> 5)] = uint8_t(byte);
  }
}

// ---- activations (GS_ACT_*)

// exp2 and the reciprocal are the hardware's (1 unit in the last place each); the exponential
// overflows to infinity and the reciprocal of that is zero.
__device__ inline float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.4426950408889634f));
}

constexpr float kGelu = 1.5957691216057308f;   // 2 sqrt(2 / pi)

__device__ inline float activate(float z, int act) {
  if (act == GS_ACT_RELU) return z < 0.0f ? 0.0f : z;   // NaN passes
  if (act == GS_ACT_SILU) return z * sigmoid(z);
  if (act == GS_ACT_GELU) return z * sigmoid(kGelu * z * (1.0f + 0.044715f * z * z));
  return z;
}

// act'(z).  With g the sigmoid of u, the slope is g + z u' g (1 - g).  Where g (1 - g)
// underflows the second term's limit is zero, so its z may be bounded (an infinity would
// make NaN of zero); a NaN in z comes through g.
__device__ inline float act_slope(float z, int act) {
  if (act == GS_ACT_RELU) return z > 0.0f ? 1.0f : 0.0f;
  if (act == GS_ACT_SILU) {
    const float g = sigmoid(z);
    return g + __builtin_amdgcn_fmed3f(z, -128.0f, 128.0f) * (g * (1.0f - g));
  }
  if (act == GS_ACT_GELU) {
    const float g = sigmoid(kGelu * z * (1.0f + 0.044715f * z * z)), b = __builtin_amdgcn_fmed3f(z, -32.0f, 32.0f);
    return g + b * (kGelu + 0.134145f * kGelu * b * b) * (g * (1.0f - g));
  }
  return 1.0f;
}

// An operand of a 16x16x32 product whose contraction runs down the rows of an LDS tile: lane
// l names the row l % 16 / 4 and the four columns (l % 4) * 4 of its eight rows (8 (l / 16)
// on), and receives column l % 16 of those eight rows.
__device__ inline bf16x8 read_transposed(const uint8_t* p, int pitch) {
  typedef short s16x4 __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) s16x4* Lds;
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(p));
  const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(p + 4 * pitch));
  const short __attribute__((ext_vector_type(8))) v{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  return __builtin_bit_cast(bf16x8, v);
}

// ---- partial sums of `size` entries each (part p at part + p size): entries below split go
// to the matrix out (its rows have cols entries; absent: not wanted), the others to tail
// (nullable).  The order of the additions depends on the number of parts alone.
hipError_t launch_sum_parts(const float* part, int parts, int64_t size, int64_t split, int cols, const MatArg& out,
                            float* tail, hipStream_t s);

// ---- mx8.hip, rmsnorm.hip, linear.hip: the calls' launches (arguments checked by the caller)
hipError_t launch_mx8_pack(const MatArg& x, const MatArg& q, int64_t rows, int cols, hipStream_t s);
hipError_t launch_mx8_unpack(const MatArg& q, const MatArg& x, int64_t rows, int cols, hipStream_t s);
hipError_t launch_rmsnorm_fwd(const MatArg& x, const MatArg& r, const float* w, float eps, const MatArg& h,
                              const MatArg& ckpt, const MatArg& y, float* rstd, int64_t rows, int cols,
                              hipStream_t s);
size_t rmsnorm_bwd_ws_bytes(int64_t rows, int cols);
hipError_t launch_rmsnorm_bwd(const MatArg& dy, const MatArg& h, const float* w, const float* rstd,
                              const MatArg& dres, const MatArg& dh, float* dweight, int64_t rows, int cols, void* ws,
                              hipStream_t s);
hipError_t launch_linear_fwd(const MatArg& x, const MatArg& w, const float* bias, int act, const MatArg& r,
                             const MatArg& z, const MatArg& y, int64_t rows, int k, int n, hipStream_t s);
size_t linear_bwd_ws_bytes(int64_t rows, int k, int n);
hipError_t launch_linear_bwd(const MatArg& dy, const MatArg& z, int act, const MatArg& x, const MatArg& w,
                             const MatArg& dx, const MatArg& dw, float* dbias, int64_t rows, int k, int n, void* ws,
                             hipStream_t s);

}  // namespace gsk
