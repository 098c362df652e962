// gs_linear_fwd with the weight in MX4: y = act(x W^T + b) + r.
//
// Operands are taken in steps of 128 k: lane l holds, of row l % 16, the block of 32 k that
// starts at 32 (l / 16), which is 16 bytes of MX4 and its scale byte.  With x in MX4 too a step is one
// 16x16x128 product of scaled 4-bit elements, whose sums are exact to float32's (4096 k of random
// codes: 5e-8 of the result, a float32 chain 8e-8).  x in bfloat16 or MX8 and the decoded weight
// are exact in bfloat16 and take four 16x16x32 products.  (The matrix cores' product of 8-bit
// with 4-bit elements is twice as fast, but it drops the low bits of what it adds: 4.5e-5 of the
// result, which an MX8 or float32 y would show.)
#include "linear.h"
#include "mx4.h"
#include "profile.h"

namespace gsk {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

__device__ inline i32x8 operand4(u32x4 q) {
  return i32x8{int(q[0]), int(q[1]), int(q[2]), int(q[3]), 0, 0, 0, 0};
}

__device__ inline f32x4 product4(u32x4 a, uint32_t a_scale, u32x4 b, uint32_t b_scale, f32x4 c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand4(a), operand4(b), c, 4, 4, 0, int(a_scale), 0, int(b_scale));
}

// A block of 32 k of a row in MX4.
struct Block4 {
  u32x4 q;
  uint32_t scale;
  // in: the row exists; n: how many of the block's k exist.  What does not exist is zero.
  __device__ void load(Buffer data, Buffer scales, uint32_t row, uint32_t pitch, uint32_t lds, bool in, int block, int n) {
    const bool there = in && n > 0;
    q = buffer_load16(data, there ? row * pitch + block * 16 : kAbsent);
    scale = buffer_load1(scales, there ? row * lds + block : kAbsent);
  }
  __device__ void keep(int n) { q = mx4_keep(q, n); }
  __device__ void operands(bf16x8 (&o)[4]) const {
    const float s = mx8_scale(scale);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = mx4_to_bf16x8(q[i], s);
  }
};

// The same of x: MX4, or two pieces of 16 k (matrix.h's Raw16).
template <int XT, bool NARROW>
struct BlockX {
  Raw16<XT, NARROW> a, b;
  __device__ void load(const MatArg& m, int64_t row, int k, int nk, bool live) {
    a.load(m, row, k, nk, live);
    if constexpr (NARROW)
      b = Raw16<XT, NARROW>{};
    else
      b.load(m, row, k + 16, nk, live);
  }
  __device__ void settle() {
    a.settle();
    if constexpr (!NARROW) b.settle();
  }
  __device__ static void half(const Raw16<XT, NARROW>& r, bf16x8& p, bf16x8& q) {
    if constexpr (XT == GS_MAT_MX8) {
      const float s = mx8_scale(r.scale);
      const u32x2 w0 = mx8_to_bf16x4(r.w[0], s), w1 = mx8_to_bf16x4(r.w[1], s);
      const u32x2 w2 = mx8_to_bf16x4(r.w[2], s), w3 = mx8_to_bf16x4(r.w[3], s);
      p = __builtin_bit_cast(bf16x8, u32x4{w0[0], w0[1], w1[0], w1[1]});
      q = __builtin_bit_cast(bf16x8, u32x4{w2[0], w2[1], w3[0], w3[1]});
    } else {
      p = __builtin_bit_cast(bf16x8, u32x4{r.w[0], r.w[1], r.w[2], r.w[3]});
      q = __builtin_bit_cast(bf16x8, u32x4{r.w[4], r.w[5], r.w[6], r.w[7]});
    }
  }
  __device__ void operands(bf16x8 (&o)[4]) const {
    half(a, o[0], o[1]);
    half(b, o[2], o[3]);
  }
};

// Any size and type.  A block of four waves takes 64 columns by 16 QT rows, the waves sharing
// the contraction; their sums are joined through LDS in order.
constexpr int kWaves = 4;

template <int XT, int QT, bool NARROW>
__global__ void __launch_bounds__(kWaves * 64) linear_mx4_kernel(MatArg W, MatArg X, int np, int64_t nq, int nk, Epilogue e) {
  constexpr bool kX4 = XT == GS_MAT_MX4;
  __shared__ f32x4 sums[kWaves * QT * 4 * 64];   // [wave][QT][tile][lane]
  const int lane = threadIdx.x % 64, g = lane / 16, r = lane % 16;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int p0 = blockIdx.y * 64;
  const int64_t q0 = int64_t(blockIdx.x) * (16 * QT);
  const uint32_t wp = uint32_t(mx4_pitch(W)), xp = kX4 ? uint32_t(mx4_pitch(X)) : 0u;
  const Buffer wb = buffer_at(W.p + int64_t(p0) * wp), ws = buffer_at(W.s + int64_t(p0) * W.lds);
  const Buffer xb = buffer_at(kX4 ? X.p + q0 * xp : nullptr), xs = buffer_at(kX4 ? X.s + q0 * X.lds : nullptr);
  f32x4 acc[QT][4];
#pragma unroll
  for (int i = 0; i < QT; ++i)
#pragma unroll
    for (int t = 0; t < 4; ++t) acc[i][t] = f32x4{0, 0, 0, 0};
  const int steps = (nk + 127) / 128;
  for (int s = wave; s < steps; s += kWaves) {
    const int block = s * 4 + g, left = nk - block * 32;
    Block4 w[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int row = r / 4 * 16 + t * 4 + r % 4;   // a lane's tiles: 16 consecutive columns
      w[t].load(wb, ws, row, wp, uint32_t(W.lds), p0 + row < np, block, left);
    }
    if constexpr (kX4) {
      Block4 x[QT];
#pragma unroll
      for (int i = 0; i < QT; ++i) {
        x[i].load(xb, xs, i * 16 + r, xp, uint32_t(X.lds), q0 + i * 16 + r < nq, block, left);
        x[i].keep(left);
      }
#pragma unroll
      for (int i = 0; i < QT; ++i)
#pragma unroll
        for (int t = 0; t < 4; ++t) acc[i][t] = product4(w[t].q, w[t].scale, x[i].q, x[i].scale, acc[i][t]);
    } else {
      bf16x8 wo[4][4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        w[t].keep(left);
        w[t].operands(wo[t]);
      }
#pragma unroll
      for (int i = 0; i < QT; ++i) {
        const int64_t row = q0 + i * 16 + r;
        BlockX<XT, NARROW> x;
        x.load(X, row < nq ? row : nq - 1, block * 32, nk, row < nq);
        x.settle();
        bf16x8 xo[4];
        x.operands(xo);
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int h = 0; h < 4; ++h) acc[i][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wo[t][h], xo[h], acc[i][t], 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < QT; ++i)
#pragma unroll
    for (int t = 0; t < 4; ++t) sums[((wave * QT + i) * 4 + t) * 64 + lane] = acc[i][t];
  __syncthreads();
  if (wave >= QT) return;
  const int64_t row = q0 + wave * 16 + r;
  const int col = p0 + g * 16, n = np - col < 16 ? np - col : 16;
  float v[16];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    f32x4 total = sums[(wave * 4 + t) * 64 + lane];
    for (int o = 1; o < kWaves; ++o) total += sums[((o * QT + wave) * 4 + t) * 64 + lane];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[4 * t + i] = total[i];
  }
#pragma unroll
  for (int j = 0; j < 16; ++j) v[j] += e.bias && j < n ? e.bias[col + j] : 0.0f;
  finish16<false, kNone, kAny>(e, row, col, v, row < nq ? n : 0);
}

template <int XT, bool NARROW>
hipError_t go(const MatArg& x, const MatArg& w, const Epilogue& e, int64_t rows, int k, int n, hipStream_t s) {
  const int64_t most = kMaxBlocks * 64;   // rows of one launch
  for (int64_t first = 0; first < rows; first += most) {
    const int64_t count = rows - first < most ? rows - first : most;
    Epilogue part = e;
    part.r = rows_from(e.r, first);
    part.y = rows_from(e.y, first);
    const MatArg xp = XT == GS_MAT_MX4 ? mx4_rows_from(x, first) : rows_from(x, first);
    linear_mx4_kernel<XT, 4, NARROW><<<dim3(div_up(count, 64), div_up(n, 64)), kWaves * 64, 0, s>>>(w, xp, n, count, k, part);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_mx4(const MatArg& x, const MatArg& w, const float* bias, int act, const MatArg& r,
                             const MatArg& y, int64_t rows, int k, int n, hipStream_t s) {
  const Epilogue e{bias, act, r, MatArg{nullptr, nullptr, 0, 0, GS_MAT_F32}, y};
  GSK_PROF("linear_mx4", s);
  if (x.type == GS_MAT_MX4) return go<GS_MAT_MX4, false>(x, w, e, rows, k, n, s);
  if (x.type == GS_MAT_MX8) return k < 16 ? go<GS_MAT_MX8, true>(x, w, e, rows, k, n, s) : go<GS_MAT_MX8, false>(x, w, e, rows, k, n, s);
  return k < 16 ? go<GS_MAT_BF16, true>(x, w, e, rows, k, n, s) : go<GS_MAT_BF16, false>(x, w, e, rows, k, n, s);
}

}  // namespace gsk
