// Linear layers of narrow width over many rows (Gaussians): K and N of at most a few
// hundred, where a row's input and output are a few hundred bytes and the weight fits a
// compute unit's LDS.  Bounded by HBM (and, with an activation, closely by the vector ALU),
// so each row's operands go from memory straight into matrix-core operands in registers
// and each result from the accumulators to memory.
#include "linear.h"
#include "profile.h"

namespace gsk {
namespace {

constexpr int kThreads = 256;

// Both operands are taken in pieces of 64 k in which lane group g = lane / 16 holds
// k = 16 g .. 16 g + 15 (two 16x16x32 products): 32 contiguous bytes of bfloat16 or 16 of MX8
// a lane, 128 or 64 a row.  The sum's order over k is the matrix core's.

// Piece kc of a row: as loaded, and as two operands.
template <bool MX>
struct Piece;

template <>
struct Piece<false> {
  u32x4 a, b;
  template <bool FULL>
  __device__ void load(const MatArg& x, int64_t row, int k, int cols) {
    if (FULL) {
      const char* p = x.p + (row * x.ld + k) * 2;
      __builtin_memcpy(&a, __builtin_assume_aligned(p, 2), 16);
      __builtin_memcpy(&b, __builtin_assume_aligned(p + 16, 2), 16);
    } else {
      a = load_raw8(x, row, k, cols - k).lo;
      b = load_raw8(x, row, k + 8, cols - k - 8).lo;
    }
  }
  __device__ void operands(bf16x8& p, bf16x8& q) const {
    p = __builtin_bit_cast(bf16x8, a);
    q = __builtin_bit_cast(bf16x8, b);
  }
};

template <>
struct Piece<true> {
  u32x4 a;
  uint32_t scale;
  template <bool FULL>
  __device__ void load(const MatArg& x, int64_t row, int k, int cols) {
    if (FULL) {
      __builtin_memcpy(&a, x.p + row * x.ld + k, 16);
      scale = x.s[row * x.lds + (k >> 5)];
    } else {
      const Raw8 lo = load_raw8(x, row, k, cols - k), hi = load_raw8(x, row, k + 8, cols - k - 8);
      a = u32x4{lo.lo[0], lo.lo[1], hi.lo[0], hi.lo[1]};
      scale = lo.scale;
    }
  }
  __device__ void operands(bf16x8& p, bf16x8& q) const {
    const float s = mx8_scale(scale);
    const u32x2 w0 = mx8_to_bf16x4(a[0], s), w1 = mx8_to_bf16x4(a[1], s);
    const u32x2 w2 = mx8_to_bf16x4(a[2], s), w3 = mx8_to_bf16x4(a[3], s);
    p = __builtin_bit_cast(bf16x8, u32x4{w0[0], w0[1], w1[0], w1[1]});
    q = __builtin_bit_cast(bf16x8, u32x4{w2[0], w2[1], w3[0], w3[1]});
  }
};

// y for 64 columns at a time: tile t of a group of 64 holds the columns 16 g + 4 t + i, so a
// lane's four tiles are 16 consecutive columns of one row.
//
// The block's part of W (groups of 64 columns c0 .. c0 + nc) lies in LDS as operands,
// 1 KiB for each (column group, tile, piece, half): a read is 64 consecutive 16-byte words.
// Wave w of the grid takes rows in turns of 16 MT; the next turn's rows are loaded before
// the present one is computed.
template <int KC, bool MX, bool FULL, int MT>
__global__ void __launch_bounds__(kThreads) rows_fwd_kernel(MatArg x, MatArg w, Epilogue e, int64_t rows, int k, int n,
                                                             int groups) {
  extern __shared__ __align__(16) uint8_t lds[];
  const int c0 = blockIdx.y * groups;
  const int nc = (n + 63) / 64 - c0 < groups ? (n + 63) / 64 - c0 : groups;
  const int lane = threadIdx.x % 64, g = lane / 16, r = lane % 16;
  const uint8_t* wl = lds + lane * 16;
  float* bias = reinterpret_cast<float*>(lds + size_t(groups) * KC * 8192);
  for (int f = threadIdx.x; f < nc * KC * 512; f += kThreads) {
    const int l = f % 64, frag = f / 64, half = frag % 2, kc = frag / 2 % KC, t = frag / (2 * KC) % 4;
    const int c = frag / (8 * KC);
    const int row = (c0 + c) * 64 + l % 16 / 4 * 16 + t * 4 + l % 4, col = kc * 64 + l / 16 * 16 + half * 8;
    *reinterpret_cast<u32x4*>(lds + size_t(f) * 16) = load_raw8(w, row, col, row < n ? k - col : 0).lo;
  }
  for (int j = threadIdx.x; j < nc * 64; j += kThreads)
    bias[j] = e.bias && c0 * 64 + j < n ? e.bias[c0 * 64 + j] : 0.0f;
  e.bias = nullptr;   // the sums start from it
  __syncthreads();
  const int64_t step = int64_t(gridDim.x) * (kThreads / 64) * (16 * MT);
  int64_t row0 = (int64_t(blockIdx.x) * (kThreads / 64) + threadIdx.x / 64) * (16 * MT);
  if (row0 >= rows) return;
  Piece<MX> next[MT][KC];
  auto fetch = [&](int64_t from) {
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int64_t row = from + m * 16 + r < rows ? from + m * 16 + r : rows - 1;   // past the end: not used
#pragma unroll
      for (int kc = 0; kc < KC; ++kc) next[m][kc].template load<FULL>(x, row, kc * 64 + g * 16, k);
    }
  };
  fetch(row0);
  for (; row0 < rows; row0 += step) {
    bf16x8 xf[MT][KC][2];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int kc = 0; kc < KC; ++kc) next[m][kc].operands(xf[m][kc][0], xf[m][kc][1]);
    if (row0 + step < rows) fetch(row0 + step);
    for (int c = 0; c < nc; ++c) {
      f32x4 acc[MT][4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const f32x4 b = *reinterpret_cast<const f32x4*>(bias + c * 64 + g * 16 + t * 4);
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[m][t] = b;
      }
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int kc = 0; kc < KC; ++kc)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const bf16x8 wf =
                *reinterpret_cast<const bf16x8*>(wl + (((c * 4 + t) * KC + kc) * 2 + h) * 1024);
#pragma unroll
            for (int m = 0; m < MT; ++m)
              acc[m][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf, xf[m][kc][h], acc[m][t], 0, 0, 0);
          }
      const int col = (c0 + c) * 64 + g * 16;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int64_t row = row0 + m * 16 + r;
        float v[16];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) v[4 * t + i] = acc[m][t][i];
        finish16(e, row, col, v, row < rows ? (n - col < 16 ? n - col : 16) : 0);
      }
    }
  }
}

constexpr int kMaxLds = 128 << 10;

size_t lds_bytes(int kc, int groups) { return size_t(groups) * (kc * 8192 + 256); }

template <int KC, bool MX, bool FULL>
hipError_t go(const MatArg& x, const MatArg& w, const Epilogue& e, int64_t rows, int k, int n, hipStream_t s) {
  constexpr int MT = KC <= 2 ? 2 : 1;
  const int all = (n + 63) / 64;
  const int64_t turns = div_up(rows, 16 * MT * (kThreads / 64));
  // few rows: the column groups go to blocks of their own
  const int split = turns * all <= 512 ? all : 1;
  const int groups = (all + split - 1) / split;
  const size_t lds = lds_bytes(KC, groups);
  static const hipError_t allowed = hipFuncSetAttribute(
      reinterpret_cast<const void*>(&rows_fwd_kernel<KC, MX, FULL, MT>), hipFuncAttributeMaxDynamicSharedMemorySize,
      kMaxLds);
  if (allowed != hipSuccess) return allowed;
  const int resident = int((160 << 10) / lds) < 4 ? int((160 << 10) / lds) : 4;
  const int64_t blocks = turns < 256 * resident ? turns : 256 * resident;
  GSK_PROF("linear_rows_fwd", s);
  rows_fwd_kernel<KC, MX, FULL, MT><<<dim3(unsigned(blocks), split), kThreads, lds, s>>>(x, w, e, rows, k, n, groups);
  return hipGetLastError();
}

template <int KC>
hipError_t by_type(const MatArg& x, const MatArg& w, const Epilogue& e, int64_t rows, int k, int n, hipStream_t s) {
  const bool full = k == KC * 64;
  if (x.type == GS_MAT_MX8)
    return full ? go<KC, true, true>(x, w, e, rows, k, n, s) : go<KC, true, false>(x, w, e, rows, k, n, s);
  return full ? go<KC, false, true>(x, w, e, rows, k, n, s) : go<KC, false, false>(x, w, e, rows, k, n, s);
}

}  // namespace

bool rows_fwd_takes(int k, int n) {
  return k <= 256 && lds_bytes((k + 63) / 64, (n + 63) / 64) <= kMaxLds;
}

hipError_t launch_rows_fwd(const MatArg& x, const MatArg& w, const Epilogue& e, int64_t rows, int k, int n,
                           hipStream_t s) {
  switch ((k + 63) / 64) {
    case 1: return by_type<1>(x, w, e, rows, k, n, s);
    case 2: return by_type<2>(x, w, e, rows, k, n, s);
    case 3: return by_type<3>(x, w, e, rows, k, n, s);
    default: return by_type<4>(x, w, e, rows, k, n, s);
  }
}

}  // namespace gsk
