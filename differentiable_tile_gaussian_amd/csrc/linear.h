// What the linear layers' kernels share: the forward's epilogue and the launches of the
// variants, among which linear.hip chooses.
#pragma once

#include <atomic>

#include "matrix.h"

namespace gsk {

// A kernel's leave to take more than the default of dynamic LDS, which belongs to a device: asked
// for on each device that launches the kernel, and again after a refusal.
class LdsLimit {
 public:
  template <class Kernel>
  hipError_t allow(Kernel* kernel, size_t bytes) {
    int device = 0;
    hipError_t e = hipGetDevice(&device);
    if (e != hipSuccess) return e;
    const uint64_t bit = device < 64 ? uint64_t(1) << device : 0;
    if (given_.load(std::memory_order_acquire) & bit) return hipSuccess;
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize,
                            int(bytes));
    if (e == hipSuccess)
      given_.fetch_or(bit, std::memory_order_release);
    else
      (void)hipGetLastError();   // returned here, and not to be found by the next launch
    return e;
  }

 private:
  std::atomic<uint64_t> given_{0};
};

// ------------------------------------------------------------- epilogue of the forward

struct Epilogue {
  const float* bias;   // nullable
  int act;
  MatArg r, z, y;      // residual and kept pre-activation nullable
};

constexpr int kAny = -1;    // a matrix type that the arguments tell
constexpr int kNone = -2;   // no such matrix

// How a kernel reaches its operands: through buffers in whole 16-column pieces, or pieces held
// within the row or one by one (matrix.h's Raw16).
enum Reach { kWhole, kHeldIn, kNarrow };

// 16 columns of a row in MX8; the lanes 16 apart hold the two halves of a 32-column block
// (all lanes active).  Values of absent columns are zero.
struct Mx8x16 {
  u32x4 q;
  uint32_t byte;
};

__device__ inline Mx8x16 encode16(const float v[16]) {
  Mx8x16 o;
  o.byte = mx8_scale_byte(max_across16(finite_top<16>(v)));
  const float scale = mx8_scale(o.byte);
#pragma unroll
  for (int i = 0; i < 4; ++i) o.q[i] = mx8_encode4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3], scale);
  return o;
}

// n: columns of the 16 that exist (<= 0: none).  WHOLE: all or none of the 16 exist.
template <bool WHOLE>
__device__ inline void store_mx8x16(const MatArg& m, int64_t row, int col, const Mx8x16& o, int n) {
  if (n <= 0) return;
  char* p = m.p + row * m.ld + col;
  if (WHOLE || n >= 16) {
    __builtin_memcpy(p, &o.q, 16);
  } else {
    store_bytes8(p, o.q[0], o.q[1], n);
    if (n > 8) store_bytes8(p + 8, o.q[2], o.q[3], n - 8);
  }
  if ((col & 31) == 0) m.s[row * m.lds + (col >> 5)] = uint8_t(o.byte);
}

// 16 columns of a row to memory (all lanes active for MX8).
template <bool WHOLE>
__device__ inline void store16(const MatArg& m, int type, int64_t row, int col, const float v[16], int n) {
  if (type == GS_MAT_MX8) {
    store_mx8x16<WHOLE>(m, row, col, encode16(v), n);
    return;
  }
  if (n <= 0) return;
  if (type == GS_MAT_F32) {
    float* p = reinterpret_cast<float*>(m.p) + row * m.ld + col;
    store_f32x8(p, v, WHOLE ? 8 : n);
    if (WHOLE || n > 8) store_f32x8(p + 8, v + 8, WHOLE ? 8 : n - 8);
  } else {
    char* p = m.p + (row * m.ld + col) * 2;
    store_bf16x8(p, v, WHOLE ? 8 : n);
    if (WHOLE || n > 8) store_bf16x8(p + 16, v + 8, WHOLE ? 8 : n - 8);
  }
}

template <int ACT>
__device__ inline void activate16(float v[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = activate(v[i], ACT);
}

// v: x W^T (with the bias) for 16 columns of a row.  Z, Y: the types of z and y, or kAny,
// or kNone for z.
template <bool WHOLE, int Z, int Y>
__device__ inline void finish16(const Epilogue& e, int64_t row, int col, float v[16], int n) {
  if (Z != kNone && (Z != kAny || e.z.p)) store16<WHOLE>(e.z, Z == kAny ? e.z.type : Z, row, col, v, n);
  if (e.act == GS_ACT_SILU)
    activate16<GS_ACT_SILU>(v);
  else if (e.act == GS_ACT_GELU)
    activate16<GS_ACT_GELU>(v);
  else if (e.act == GS_ACT_RELU)
    activate16<GS_ACT_RELU>(v);
  if (e.r.p && n > 0) {
    float r[16];
    raw8_to_float(load_raw8(e.r, row, col, WHOLE ? 8 : n), e.r.type, r);
    raw8_to_float(load_raw8(e.r, row, col + 8, WHOLE ? 8 : n - 8), e.r.type, r + 8);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] += r[i];
  }
  store16<WHOLE>(e.y, Y == kAny ? e.y.type : Y, row, col, v, n);
}

// ---- linear_rows.hip: narrow layers over many rows, the weight kept in LDS
bool rows_fwd_takes(int k, int n);
hipError_t launch_rows_fwd(const MatArg& x, const MatArg& w, const Epilogue& e, int64_t rows, int k, int n,
                           hipStream_t s);

// ---- linear_rows_bwd.hip: the gradients of the narrowest of them in one pass
bool rows_bwd_takes(int k, int n);   // by the widths alone
bool rows_bwd_runs(const MatArg& dy, const MatArg& z, int act, const MatArg& x, const MatArg& dx, int k, int n);
size_t rows_bwd_ws_bytes(int64_t rows, int k, int n);
hipError_t launch_rows_bwd(const MatArg& dy, const MatArg& z, int act, const MatArg& x, const MatArg& w,
                           const MatArg& dx, const MatArg& dw, float* dbias, int64_t rows, int k, int n, void* ws,
                           hipStream_t s);

// ---- linear_tiles.hip: products bounded by the matrix cores, in 128-column tiles
// out(q, p) = sum_k Q(q, k) P(p, k), finished as a forward's result
hipError_t launch_tile_nt(const MatArg& P, const MatArg& Q, int np, int64_t nq, int nk, const Epilogue& e,
                          hipStream_t s);
// out(q, p) = sum_m Q(m, q) P(m, p) in `slices` parts of the rows m (part: [slices][nq][np]
// where there are several)
int tile_tn_slices(int64_t rows, int np, int nq);
hipError_t launch_tile_tn(const MatArg& P, const MatArg& Q, int np, int nq, int64_t rows, int slices, float* part,
                          const MatArg& out, hipStream_t s);

// ---- linear_split.hip: the same product where it has too few tiles to fill the card
bool split_nt_takes(const MatArg& P, const MatArg& Q, int np, int64_t nq);
hipError_t launch_split_nt(const MatArg& P, const MatArg& Q, int np, int64_t nq, int nk, const Epilogue& e,
                           hipStream_t s);

}  // namespace gsk
