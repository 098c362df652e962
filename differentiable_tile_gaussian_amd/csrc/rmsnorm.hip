// gs_rmsnorm_fwd and gs_rmsnorm_bwd: h = x + r, y = h rstd w with rstd = (mean h^2 + eps)^-1/2,
// and its gradients dh = rstd (u - xhat mean(u xhat)) + dres, dw = sum_rows dy xhat, where
// u = dy w and xhat = h rstd.
//
// Streams bounded by HBM.  A row is held by 4 to 256 lanes, 8 columns a lane at a time (so an
// MX8 block is four neighbouring lanes), in registers from its load to its store: each input
// is read once and each output written once, up to kMaxHeld columns.  Wider rows are walked
// twice by one wave, the second time from the caches.
//
// Forward, 3M rows of 128 with a residual and an 8-bit output and checkpoint: 550 us (3.11 GB,
// 5.65 TB/s, a copy's rate); one row's latency sets small calls (1024 rows of 64: 4 us).
// Backward, 1M rows of 128: 160 us (900 MB, 5.6 TB/s) and 5 us for joining dw's sums; 8160
// rows of 1000: 16 and 4 us.  Rows that are not held are for the range, not for speed: a wave has one
// load of each input in flight (8160 rows of 8192: forward 223 us, 2.6 times its bytes at a
// copy's rate, backward 324, 3.3 times; one row of 2^20 columns 4.9 and 5.3 ms).
#include "matrix.h"
#include "profile.h"

namespace gsk {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxHeld = 4096;   // 256 lanes x 2 chunks x 8 columns

// The sum over a row's lanes; LANES == 256: over the block's waves in order, with `turn` (how
// many sums came before) alternating two places, so that one barrier a sum is enough.
template <int LANES>
__device__ inline float row_sum(float v, int turn = 0) {
#pragma unroll
  for (int o = (LANES < 64 ? LANES : 64) / 2; o > 0; o /= 2) v += __shfl_xor(v, o);
  if constexpr (LANES == 256) {
    __shared__ float sums[2][4];
    if (threadIdx.x % 64 == 0) sums[turn & 1][threadIdx.x / 64] = v;
    __syncthreads();
    v = sums[turn & 1][0] + sums[turn & 1][1] + sums[turn & 1][2] + sums[turn & 1][3];
  }
  return v;
}

struct NormFwdArgs {
  MatArg x, r, h, ckpt, y;
  const float* w;
  float* rstd;
  float eps, inv_cols;
  int64_t rows;
  int cols;
};

__device__ inline void load_weight(const float* w, int col, int n, float v[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = i < n ? w[col + i] : 0.0f;
}

__device__ inline void store_chunk(const MatArg& m, int64_t row, int col, const float v[8], int n) {
  if (m.type == GS_MAT_MX8)
    store_mx8_quad(m, row, col, v, n);
  else if (n > 0)
    store8(m, row, col, v, n);
}

// A lane's chunk of a row: held inside it (matrix.h), or for rows of fewer than 8 columns
// (NARROW) what there is of them in the first lane.
template <bool NARROW>
__device__ inline Held chunk_at(int col, int cols) {
  return NARROW ? Held{col, col < cols ? 0 : 8} : held_at(col, cols);
}
template <bool NARROW>
__device__ inline Raw8 load_chunk(const MatArg& m, int64_t row, const Held& c, int cols) {
  return NARROW ? load_raw8(m, row, c.at, cols - c.at) : load_held(m, row, c);
}

// LANES lanes hold a row, CHUNKS chunks each, and take ROWS rows side by side: their loads are
// all issued before the first is used.
template <int LANES, int CHUNKS, int ROWS, bool NARROW>
__global__ void __launch_bounds__(kThreads) rmsnorm_fwd_kernel(NormFwdArgs a) {
  constexpr int kPer = kThreads / LANES;
  const int lane = threadIdx.x % LANES;
  const int64_t first = int64_t(blockIdx.x) * (kPer * ROWS) + threadIdx.x / LANES;
  Raw8 xr[ROWS][CHUNKS], rr[ROWS][CHUNKS];
#pragma unroll
  for (int u = 0; u < ROWS; ++u) {
    const int64_t row = first + u * kPer < a.rows ? first + u * kPer : a.rows - 1;
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) xr[u][c] = load_chunk<NARROW>(a.x, row, chunk_at<NARROW>((c * LANES + lane) * 8, a.cols), a.cols);
  }
  if (a.r.p) {
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
      const int64_t row = first + u * kPer < a.rows ? first + u * kPer : a.rows - 1;
#pragma unroll
      for (int c = 0; c < CHUNKS; ++c) rr[u][c] = load_chunk<NARROW>(a.r, row, chunk_at<NARROW>((c * LANES + lane) * 8, a.cols), a.cols);
    }
  }
  float w[CHUNKS][8];
#pragma unroll
  for (int c = 0; c < CHUNKS; ++c) {
    const Held t = chunk_at<NARROW>((c * LANES + lane) * 8, a.cols);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[c][i] = NARROW && t.at + i >= a.cols ? 0.0f : a.w[t.at + i];
  }
#pragma unroll
  for (int u = 0; u < ROWS; ++u) {
    const int64_t row = first + u * kPer;
    float h[CHUNKS][8], sum = 0.0f;
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
      const Held t = chunk_at<NARROW>((c * LANES + lane) * 8, a.cols);
      raw8_to_float(xr[u][c], a.x.type, h[c]);
      if (a.r.p) {
        float r[8];
        raw8_to_float(rr[u][c], a.r.type, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[c][i] += r[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += i >= t.skip ? h[c][i] * h[c][i] : 0.0f;
    }
    sum = row_sum<LANES>(sum, u);
    const float rstd = 1.0f / sqrtf(sum * a.inv_cols + a.eps);
    const bool in = row < a.rows;
    if (in && lane == 0 && a.rstd) a.rstd[row] = rstd;
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
      const int col = (c * LANES + lane) * 8;
      const Held t = chunk_at<NARROW>(col, a.cols);
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = h[c][i] * rstd * w[c][i];
      const bool mine = in && t.skip < 8;
      if (a.h.p && mine) store8(a.h, row, t.at, h[c], NARROW ? a.cols : 8);
      if (a.y.type == GS_MAT_MX8) {
        if (!NARROW) move_down(t, y);
        store_mx8_quad(a.y, row, col, y, in ? a.cols - col : 0);
      } else if (mine) {
        store8(a.y, row, t.at, y, NARROW ? a.cols : 8);
      }
      if (a.ckpt.p) {
        if (!NARROW) move_down(t, h[c]);
        store_mx8_quad(a.ckpt, row, col, h[c], in ? a.cols - col : 0);
      }
    }
  }
}

// Rows of more than kMaxHeld columns: a wave a row, walked twice.
__global__ void __launch_bounds__(kThreads) rmsnorm_fwd_wide_kernel(NormFwdArgs a) {
  const int lane = threadIdx.x % 64;
  const int64_t row = int64_t(blockIdx.x) * (kThreads / 64) + threadIdx.x / 64;
  if (row >= a.rows) return;
  float sum = 0.0f;
  for (int pass = 0; pass < 2; ++pass) {
    const float rstd = 1.0f / sqrtf(sum * a.inv_cols + a.eps);
    for (int c0 = 0; c0 < a.cols; c0 += 512) {
      const int col = c0 + lane * 8, n = a.cols - col;
      float h[8];
      raw8_to_float(load_raw8(a.x, row, col, n), a.x.type, h);
      if (a.r.p) {
        float t[8];
        raw8_to_float(load_raw8(a.r, row, col, n), a.r.type, t);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] += t[i];
      }
      if (pass == 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += h[i] * h[i];
      } else {
        if (a.h.p) store_chunk(a.h, row, col, h, n);
        if (a.ckpt.p) store_mx8_quad(a.ckpt, row, col, h, n);
        float w[8], y[8];
        load_weight(a.w, col, n, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = h[i] * rstd * w[i];
        store_chunk(a.y, row, col, y, n);
      }
    }
    if (pass == 0) {
      sum = row_sum<64>(sum);
    } else if (lane == 0 && a.rstd) {
      a.rstd[row] = rstd;
    }
  }
}

struct NormBwdArgs {
  MatArg dy, h, dres, dh;
  const float *w, *rstd;
  float* part;   // [gridDim.x][cols] sums of dy xhat, nullptr: not wanted
  float inv_cols;
  int64_t rows;
  int cols;
};

template <int LANES, int CHUNKS, bool NARROW>
__global__ void __launch_bounds__(kThreads) rmsnorm_bwd_kernel(NormBwdArgs a) {
  constexpr int kPer = kThreads / LANES;
  const int lane = threadIdx.x % LANES;
  float w[CHUNKS][8], acc[CHUNKS][8];
#pragma unroll
  for (int c = 0; c < CHUNKS; ++c) {
    const Held t = chunk_at<NARROW>((c * LANES + lane) * 8, a.cols);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w[c][i] = NARROW && t.at + i >= a.cols ? 0.0f : a.w[t.at + i];
      acc[c][i] = 0.0f;
    }
  }
  int turn = 0;
  for (int64_t row0 = int64_t(blockIdx.x) * kPer; row0 < a.rows; row0 += int64_t(gridDim.x) * kPer) {
    const int64_t own = row0 + threadIdx.x / LANES, row = own < a.rows ? own : a.rows - 1;
    const bool in = own < a.rows;
    Raw8 dr[CHUNKS], hr[CHUNKS], rr[CHUNKS];
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
      const Held t = chunk_at<NARROW>((c * LANES + lane) * 8, a.cols);
      dr[c] = load_chunk<NARROW>(a.dy, row, t, a.cols);
      hr[c] = load_chunk<NARROW>(a.h, row, t, a.cols);
    }
    if (a.dres.p) {
#pragma unroll
      for (int c = 0; c < CHUNKS; ++c) rr[c] = load_chunk<NARROW>(a.dres, row, chunk_at<NARROW>((c * LANES + lane) * 8, a.cols), a.cols);
    }
    const float rstd = a.rstd[row];
    float dy[CHUNKS][8], xh[CHUNKS][8], dot = 0.0f;
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
      const Held t = chunk_at<NARROW>((c * LANES + lane) * 8, a.cols);
      const int skip = in ? t.skip : 8;
      raw8_to_float(dr[c], a.dy.type, dy[c]);
      if (NARROW)
        raw8_to_float(hr[c], a.h.type, xh[c]);
      else
        held_to_float(hr[c], a.h.type, t, xh[c]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        xh[c][i] *= rstd;
        const float p = i >= skip ? dy[c][i] * xh[c][i] : 0.0f;
        acc[c][i] += p;
        dot += p * w[c][i];
      }
    }
    const float mean = row_sum<LANES>(dot, turn++) * a.inv_cols;
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
      const Held t = chunk_at<NARROW>((c * LANES + lane) * 8, a.cols);
      float o[8];
      if (a.dres.p) {
        raw8_to_float(rr[c], a.dres.type, o);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] += rstd * (dy[c][i] * w[c][i] - xh[c][i] * mean);
      if (in && t.skip < 8) store8(a.dh, row, t.at, o, NARROW ? a.cols : 8);
    }
  }
  if (!a.part) return;
  // the block's sum of each column, in the order of its row slots
  __shared__ float sums[kThreads * 8];   // one chunk of every thread at a time
  float* out = a.part + int64_t(blockIdx.x) * a.cols;
#pragma unroll
  for (int c = 0; c < CHUNKS; ++c) {
    if (!NARROW) move_down(held_at((c * LANES + lane) * 8, a.cols), acc[c]);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) sums[threadIdx.x * 8 + i] = acc[c][i];
    __syncthreads();
    for (int j = threadIdx.x; j < LANES * 8; j += kThreads) {
      float t = 0.0f;
      for (int k = 0; k < kPer; ++k) t += sums[k * LANES * 8 + j];
      const int col = c * LANES * 8 + j;
      if (col < a.cols) out[col] = t;
    }
  }
}

// Rows of more than kMaxHeld columns: a wave a row, walked twice; the weight's gradient has
// its own kernel.
__global__ void __launch_bounds__(kThreads) rmsnorm_bwd_wide_kernel(NormBwdArgs a) {
  const int lane = threadIdx.x % 64;
  const int64_t row = int64_t(blockIdx.x) * (kThreads / 64) + threadIdx.x / 64;
  if (row >= a.rows) return;
  const float rstd = a.rstd[row];
  float dot = 0.0f;
  for (int pass = 0; pass < 2; ++pass) {
    const float mean = dot * a.inv_cols;
    for (int c0 = 0; c0 < a.cols; c0 += 512) {
      const int col = c0 + lane * 8, n = a.cols - col;
      float dy[8], xh[8], w[8];
      raw8_to_float(load_raw8(a.dy, row, col, n), a.dy.type, dy);
      raw8_to_float(load_raw8(a.h, row, col, n), a.h.type, xh);
      load_weight(a.w, col, n, w);
      if (pass == 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) dot += dy[i] * (xh[i] * rstd) * w[i];
      } else {
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = 0.0f;
        if (a.dres.p) raw8_to_float(load_raw8(a.dres, row, col, n), a.dres.type, o);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] += rstd * (dy[i] * w[i] - (xh[i] * rstd) * mean);
        if (n > 0) store8(a.dh, row, col, o, n);
      }
    }
    if (pass == 0) dot = row_sum<64>(dot);
  }
}

// part[b][col] = sum over the b-th slice of the rows of dy xhat: a block takes 512 columns
// (a wave's width) of its slice, its four waves every fourth row.
__global__ void __launch_bounds__(kThreads) rmsnorm_dw_wide_kernel(NormBwdArgs a, int slices) {
  const int wave = threadIdx.x / 64, lane = threadIdx.x % 64;
  const int col = blockIdx.y * 512 + lane * 8, n = a.cols - col;
  const int64_t per = (a.rows + slices - 1) / slices, first = per * blockIdx.x;
  const int64_t last = first + per < a.rows ? first + per : a.rows;
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
  for (int64_t row = first + wave; row < last; row += kThreads / 64) {
    const float rstd = a.rstd[row];
    float dy[8], xh[8];
    raw8_to_float(load_raw8(a.dy, row, col, n), a.dy.type, dy);
    raw8_to_float(load_raw8(a.h, row, col, n), a.h.type, xh);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] += dy[i] * (xh[i] * rstd);
  }
  __shared__ float sums[kThreads * 8];
#pragma unroll
  for (int i = 0; i < 8; ++i) sums[threadIdx.x * 8 + i] = acc[i];
  __syncthreads();
  for (int j = threadIdx.x; j < 512; j += kThreads) {
    float t = 0.0f;
    for (int k = 0; k < kThreads / 64; ++k) t += sums[k * 512 + j];
    if (blockIdx.y * 512 + j < a.cols) a.part[int64_t(blockIdx.x) * a.cols + blockIdx.y * 512 + j] = t;
  }
}

// Lanes of a row: the smallest power of two that holds it in one chunk up to a wave, a wave
// with two chunks, and the whole block beyond (8160 rows of 4096 columns by one wave each, eight
// chunks in its registers: forward 57 us and backward 85, by the block 47 and 46).
int lanes_for(int cols) {
  int lanes = 4;
  while (lanes < 64 && lanes * 8 < cols) lanes *= 2;
  return cols > 1024 ? 256 : lanes;
}

// Whether the kernels that do not hold a row take it.
bool wide(int cols) { return cols > kMaxHeld; }

// Blocks of the backward: as many as the kernel's registers let reside at once (five waves a
// SIMD; 1M rows of 128: 161 us, with 1024 blocks 178, with 2048 183).
int bwd_blocks(int64_t rows, int cols) {
  if (wide(cols)) return int(rows < 256 ? (rows < 1 ? 1 : rows) : 256);
  const int64_t per = kThreads / lanes_for(cols);
  const int64_t want = (rows + per - 1) / per;
  return int(want < 1 ? 1 : (want > 1280 ? 1280 : want));
}

template <template <int, int, bool> class Launch, typename Args>
void by_width(int cols, const Args& a, unsigned blocks, hipStream_t s) {
  if (cols < 8) {
    Launch<4, 1, true>::go(a, blocks, s);
    return;
  }
  switch (lanes_for(cols)) {
    case 4: Launch<4, 1, false>::go(a, blocks, s); break;
    case 8: Launch<8, 1, false>::go(a, blocks, s); break;
    case 16: Launch<16, 1, false>::go(a, blocks, s); break;
    case 32: Launch<32, 1, false>::go(a, blocks, s); break;
    case 64:
      if (cols <= 512) Launch<64, 1, false>::go(a, blocks, s);
      else Launch<64, 2, false>::go(a, blocks, s);
      break;
    default:
      if (cols <= 2048) Launch<256, 1, false>::go(a, blocks, s);
      else Launch<256, 2, false>::go(a, blocks, s);
  }
}

template <class Kernel>
void launch_fwd(Kernel* kernel, int64_t per_block, const NormFwdArgs& a, hipStream_t s) {
  for_row_parts(a.rows, per_block, [&](int64_t first, int64_t count, unsigned blocks) {
    NormFwdArgs p = a;
    for (MatArg NormFwdArgs::*m : {&NormFwdArgs::x, &NormFwdArgs::r, &NormFwdArgs::h, &NormFwdArgs::ckpt, &NormFwdArgs::y})
      p.*m = rows_from(a.*m, first);
    if (a.rstd) p.rstd = a.rstd + first;
    p.rows = count;
    kernel<<<blocks, kThreads, 0, s>>>(p);
  });
}

template <int L, int C, bool NARROW>
struct Fwd {
  static void go(const NormFwdArgs& a, unsigned, hipStream_t s) {
    constexpr int kRows = C == 1 ? 2 : 1;
    launch_fwd(&rmsnorm_fwd_kernel<L, C, kRows, NARROW>, kThreads / L * kRows, a, s);
  }
};
template <int L, int C, bool NARROW>
struct Bwd {
  static void go(const NormBwdArgs& a, unsigned blocks, hipStream_t s) {
    rmsnorm_bwd_kernel<L, C, NARROW><<<blocks, kThreads, 0, s>>>(a);
  }
};

// A block sums 16 entries: 64 groups of parts side by side, then the groups in order.
__global__ void __launch_bounds__(1024) sum_parts_kernel(const float* __restrict__ part, int parts, int64_t size,
                                                          int64_t first, int64_t last, int64_t split, int cols,
                                                          MatArg out, float* tail) {
  const int j = threadIdx.x % 16, g = threadIdx.x / 16;
  const int64_t c = first + int64_t(blockIdx.x) * 16 + j;
  float t = 0.0f;
  if (c < last) {
#pragma unroll 4
    for (int p = g; p < parts; p += 64) t += part[p * size + c];
  }
  __shared__ float sums[64][17];
  sums[g][j] = t;
  __syncthreads();
  if (g == 0 && c < last) {
#pragma unroll 8
    for (int k = 1; k < 64; ++k) t += sums[k][j];
    if (c >= split) {
      tail[c - split] = t;
      return;
    }
    const int64_t at = (c / cols) * out.ld + c % cols;
    if (out.type == GS_MAT_F32)
      reinterpret_cast<float*>(out.p)[at] = t;
    else
      reinterpret_cast<uint16_t*>(out.p)[at] = uint16_t(pack_bf16(t, 0.0f));
  }
}

// Few parts of many entries: a thread sums 4 entries over the parts in order.
__global__ void __launch_bounds__(kThreads) sum_few_parts_kernel(const float* __restrict__ part, int parts,
                                                                  int64_t size, int64_t first, int64_t last,
                                                                  int64_t split, int cols, MatArg out, float* tail) {
  const int64_t c0 = first + (int64_t(blockIdx.x) * kThreads + threadIdx.x) * 4;
  if (c0 >= last) return;
  const int n = last - c0 < 4 ? int(last - c0) : 4;
  float t[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (n == 4) {
#pragma unroll 4
    for (int p = 0; p < parts; ++p) {
      f32x4 v;
      __builtin_memcpy(&v, __builtin_assume_aligned(part + p * size + c0, 4), 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) t[i] += v[i];
    }
  } else {
    for (int p = 0; p < parts; ++p)
      for (int i = 0; i < n; ++i) t[i] += part[p * size + c0 + i];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t c = c0 + i;
    if (i >= n) break;
    if (c >= split) {
      tail[c - split] = t[i];
    } else {
      const int64_t at = (c / cols) * out.ld + c % cols;
      if (out.type == GS_MAT_F32)
        reinterpret_cast<float*>(out.p)[at] = t[i];
      else
        reinterpret_cast<uint16_t*>(out.p)[at] = uint16_t(pack_bf16(t[i], 0.0f));
    }
  }
}

}  // namespace

hipError_t launch_sum_parts(const float* part, int parts, int64_t size, int64_t split, int cols, const MatArg& out,
                            float* tail, hipStream_t s) {
  const int64_t first = out.p ? 0 : split, last = tail ? size : split;
  GSK_PROF("sum_parts", s);
  if (parts <= 32 && last - first >= 16384) {
    sum_few_parts_kernel<<<div_up(last - first, kThreads * 4), kThreads, 0, s>>>(part, parts, size, first, last, split,
                                                                                cols, out, tail);
    return hipGetLastError();
  }
  sum_parts_kernel<<<div_up(last - first, 16), 1024, 0, s>>>(part, parts, size, first, last, split, cols, out, tail);
  return hipGetLastError();
}

hipError_t launch_rmsnorm_fwd(const MatArg& x, const MatArg& r, const float* w, float eps, const MatArg& h,
                              const MatArg& ckpt, const MatArg& y, float* rstd, int64_t rows, int cols,
                              hipStream_t s) {
  const NormFwdArgs a{x, r, h, ckpt, y, w, rstd, eps, 1.0f / float(cols), rows, cols};
  GSK_PROF("rmsnorm_fwd", s);
  if (wide(cols)) {
    launch_fwd(&rmsnorm_fwd_wide_kernel, kThreads / 64, a, s);
  } else {
    by_width<Fwd>(cols, a, 0, s);
  }
  return hipGetLastError();
}

size_t rmsnorm_bwd_ws_bytes(int64_t rows, int cols) {
  return (size_t(bwd_blocks(rows, cols)) * size_t(cols) * 4 + 255) & ~size_t(255);
}

hipError_t launch_rmsnorm_bwd(const MatArg& dy, const MatArg& h, const float* w, const float* rstd,
                              const MatArg& dres, const MatArg& dh, float* dweight, int64_t rows, int cols, void* ws,
                              hipStream_t s) {
  const int blocks = bwd_blocks(rows, cols);
  float* part = dweight ? static_cast<float*>(ws) : nullptr;
  const NormBwdArgs a{dy, h, dres, dh, w, rstd, part, 1.0f / float(cols), rows, cols};
  if (wide(cols)) {
    if (rows > 0) {
      GSK_PROF("rmsnorm_bwd", s);
      for_row_parts(rows, kThreads / 64, [&](int64_t first, int64_t count, unsigned n) {
        NormBwdArgs p = a;
        for (MatArg NormBwdArgs::*m : {&NormBwdArgs::dy, &NormBwdArgs::h, &NormBwdArgs::dres, &NormBwdArgs::dh})
          p.*m = rows_from(a.*m, first);
        p.rstd = a.rstd + first;
        p.rows = count;
        rmsnorm_bwd_wide_kernel<<<n, kThreads, 0, s>>>(p);
      });
    }
    if (dweight) {
      GSK_PROF("rmsnorm_dw", s);
      rmsnorm_dw_wide_kernel<<<dim3(blocks, div_up(cols, 512)), kThreads, 0, s>>>(a, blocks);
    }
  } else {
    GSK_PROF("rmsnorm_bwd", s);
    by_width<Bwd>(cols, a, unsigned(blocks), s);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !dweight) return e;
  return launch_sum_parts(part, blocks, cols, 0, 1, MatArg{}, dweight, s);
}

}  // namespace gsk
