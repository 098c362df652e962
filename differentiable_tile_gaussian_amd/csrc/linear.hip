// gs_linear_fwd and gs_linear_bwd: y = act(x W^T + b) + r and its gradients.  With
// z = x W^T + b and dz = dy act'(z):  dx = dz W,  dW = dz^T x,  db = sum of the rows of dz.
//
// Every product runs on the matrix cores (16x16x32, bfloat16 operands, float32 sums):
// bfloat16 and MX8 operands are exact there, float32 ones (and dz) are rounded to bfloat16.
#include "linear.h"
#include "profile.h"

namespace gsk {
namespace {

constexpr int kThreads = 256;

// ------------------------------------------------- tiled product, contraction contiguous

// out(q, p) = sum_k Q(q, k) P(p, k) on tiles of 64 WP columns p by 16 QT WQ rows q, a wave
// taking 64 columns by 16 QT rows.  Both operands' tiles of 64 k are staged through
// registers (converting to bfloat16) into LDS; the 16-byte pieces of a 128-byte row are
// permuted by the row's number so that the 16 rows a fragment read covers fall into
// different banks.  P's rows are stored so that a lane's four result tiles are 16
// consecutive columns of one output row: wide stores, and half an MX8 block.
template <int WP, int WQ, int QT>
__global__ void __launch_bounds__(WP* WQ * 64) gemm_nt_kernel(MatArg P, MatArg Q, int64_t np, int64_t nq, int nk,
                                                               Epilogue e) {
  constexpr int kT = WP * WQ * 64, BP = 64 * WP, BQ = 16 * QT * WQ, kLoads = (BP + BQ) * 8 / kT;
  __shared__ __align__(16) uint8_t lds[(BP + BQ) * 128];
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, wp = wave % WP, wq = wave / WP;
  const int64_t p0 = int64_t(blockIdx.y) * BP, q0 = int64_t(blockIdx.x) * BQ;
  f32x4 acc[QT][4];
#pragma unroll
  for (int i = 0; i < QT; ++i)
#pragma unroll
    for (int t = 0; t < 4; ++t) acc[i][t] = f32x4{0, 0, 0, 0};
  for (int k0 = 0; k0 < nk; k0 += 64) {
    Raw8 raw[kLoads];
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const int i = u * kT + threadIdx.x, row = i / 8, k = k0 + i % 8 * 8;
      if (row < BP)
        raw[u] = load_raw8(P, p0 + row, k, p0 + row < np ? nk - k : 0);
      else
        raw[u] = load_raw8(Q, q0 + row - BP, k, q0 + row - BP < nq ? nk - k : 0);
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const int i = u * kT + threadIdx.x;
      int row = i / 8;
      const int type = row < BP ? P.type : Q.type;
      if (row < BP) row = (row & ~63) | ((row & 12) << 2) | ((row & 48) >> 2) | (row & 3);
      *reinterpret_cast<u32x4*>(lds + row * 128 + ((i % 8) ^ ((row >> 1) & 7)) * 16) = raw8_to_bf16(raw[u], type);
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      const int piece = kk * 4 + lane / 16;
      bf16x8 pf[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int row = wp * 64 + t * 16 + lane % 16;
        pf[t] = *reinterpret_cast<const bf16x8*>(lds + row * 128 + (piece ^ ((row >> 1) & 7)) * 16);
      }
#pragma unroll
      for (int i = 0; i < QT; ++i) {
        const int row = BP + (wq * QT + i) * 16 + lane % 16;
        const bf16x8 qf = *reinterpret_cast<const bf16x8*>(lds + row * 128 + (piece ^ ((row >> 1) & 7)) * 16);
#pragma unroll
        for (int t = 0; t < 4; ++t) acc[i][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(pf[t], qf, acc[i][t], 0, 0, 0);
      }
    }
  }
  const int64_t col = p0 + wp * 64 + lane / 16 * 16;
#pragma unroll
  for (int i = 0; i < QT; ++i) {
    const int64_t row = q0 + (wq * QT + i) * 16 + lane % 16;
    float v[16];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) v[4 * t + j] = acc[i][t][j];
    if (e.bias) {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] += col + i < np ? e.bias[col + i] : 0.0f;
    }
    finish16<false, kAny, kAny>(e, row, int(col), v, row < nq ? int(np - col < 16 ? np - col : 16) : 0);
  }
}

// ------------------------------------------------- tiled product, contraction over rows

// out(q, p) = sum_m Q(m, q) P(m, p) for m in the block's slice of the rows: the weight's
// gradient (Q = dz, P = x).  Tiles of 64 rows are kept in LDS as they are in memory (plus
// 32 bytes a row, so that eight rows fall into different banks) and read transposed
// (ds_read_b64_tr_b16: four rows of 16 columns, a column's four values to a lane).
template <int WP, int WQ, int QT>
__global__ void __launch_bounds__(WP* WQ * 64) gemm_tn_kernel(MatArg P, MatArg Q, int np, int nq, int64_t rows,
                                                               int64_t per_slice, float* part, MatArg out) {
  constexpr int kT = WP * WQ * 64, BP = 64 * WP, BQ = 16 * QT * WQ, BM = 64;
  constexpr int kPitchP = BP * 2 + 32, kPitchQ = BQ * 2 + 32, kLoads = BM * (BP + BQ) / 8 / kT;
  __shared__ __align__(16) uint8_t lds[BM * (kPitchP + kPitchQ)];
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, wp = wave % WP, wq = wave / WP;
  const int p0 = blockIdx.x * BP, q0 = blockIdx.y * BQ;
  const int64_t first = int64_t(blockIdx.z) * per_slice;
  const int64_t last = first + per_slice < rows ? first + per_slice : rows;
  f32x4 acc[QT][4];
#pragma unroll
  for (int i = 0; i < QT; ++i)
#pragma unroll
    for (int t = 0; t < 4; ++t) acc[i][t] = f32x4{0, 0, 0, 0};
  for (int64_t m0 = first; m0 < last; m0 += BM) {
    Raw8 raw[kLoads];
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const int i = u * kT + threadIdx.x, m = i / ((BP + BQ) / 8), c = i % ((BP + BQ) / 8) * 8;
      const bool in = m0 + m < last;
      if (c < BP)
        raw[u] = load_raw8(P, m0 + m, p0 + c, in ? np - p0 - c : 0);
      else
        raw[u] = load_raw8(Q, m0 + m, q0 + c - BP, in ? nq - q0 - (c - BP) : 0);
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const int i = u * kT + threadIdx.x, m = i / ((BP + BQ) / 8), c = i % ((BP + BQ) / 8) * 8;
      if (c < BP)
        *reinterpret_cast<u32x4*>(lds + m * kPitchP + c * 2) = raw8_to_bf16(raw[u], P.type);
      else
        *reinterpret_cast<u32x4*>(lds + BM * kPitchP + m * kPitchQ + (c - BP) * 2) = raw8_to_bf16(raw[u], Q.type);
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < BM / 32; ++kk) {
      const int m = kk * 32 + lane / 16 * 8 + lane % 16 / 4, c = lane % 4 * 4;
      bf16x8 pf[4];
#pragma unroll
      for (int t = 0; t < 4; ++t)
        pf[t] = read_transposed(lds + m * kPitchP + (wp * 64 + t * 16 + c) * 2, kPitchP);
#pragma unroll
      for (int i = 0; i < QT; ++i) {
        const bf16x8 qf =
            read_transposed(lds + BM * kPitchP + m * kPitchQ + ((wq * QT + i) * 16 + c) * 2, kPitchQ);
#pragma unroll
        for (int t = 0; t < 4; ++t) acc[i][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(pf[t], qf, acc[i][t], 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < QT; ++i) {
    const int q = q0 + (wq * QT + i) * 16 + lane % 16;
    if (q >= nq) continue;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int p = p0 + wp * 64 + t * 16 + lane / 16 * 4;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (p + j >= np) continue;
        if (part) {
          part[(int64_t(blockIdx.z) * nq + q) * np + p + j] = acc[i][t][j];
        } else if (out.type == GS_MAT_F32) {
          reinterpret_cast<float*>(out.p)[int64_t(q) * out.ld + p + j] = acc[i][t][j];
        } else {
          reinterpret_cast<uint16_t*>(out.p)[int64_t(q) * out.ld + p + j] = uint16_t(pack_bf16(acc[i][t][j], 0.0f));
        }
      }
    }
  }
}

// ------------------------------------------------------------- dz, db and W^T

// dz = dy act'(z) to bfloat16 (unless dz is absent) and part[slice] = the column sums of dz
// before its rounding.  lanes (a power of two in [4, 64]) take 8 columns each of a row (held as
// matrix.h has it; NARROW: fewer than 8 columns), kRows rows at a time.
constexpr int kRows = 2;

template <bool NARROW>
__global__ void __launch_bounds__(kThreads) dz_kernel(MatArg dy, MatArg z, int act, MatArg dz, float* part,
                                                       int64_t rows, int cols, int64_t per_slice, int lanes) {
  const int lane = threadIdx.x & (lanes - 1), slot = threadIdx.x / lanes, per = kThreads / lanes;
  const int col = (int(blockIdx.y) * lanes + lane) * 8;
  const Held c = held_at(col, cols);
  const int64_t first = int64_t(blockIdx.x) * per_slice;
  const int64_t last = first + per_slice < rows ? first + per_slice : rows;
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
  for (int64_t row0 = first + slot; row0 < last; row0 += per * kRows) {
    Raw8 a[kRows], b[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int64_t row = row0 + u * per < last ? row0 + u * per : last - 1;
      a[u] = NARROW ? load_raw8(dy, row, col, cols - col) : load_held(dy, row, c);
    }
    if (act != GS_ACT_NONE) {
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        const int64_t row = row0 + u * per < last ? row0 + u * per : last - 1;
        b[u] = NARROW ? load_raw8(z, row, col, cols - col) : load_held(z, row, c);
      }
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int64_t row = row0 + u * per;
      float v[8];
      raw8_to_float(a[u], dy.type, v);
      if (act != GS_ACT_NONE) {
        float t[8];
        if (NARROW)
          raw8_to_float(b[u], z.type, t);
        else
          held_to_float(b[u], z.type, c, t);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= act_slope(t[i], act);
      }
      const bool in = row < last;
      if (dz.p && in && c.skip < 8)
        store_bf16x8(dz.p + (row * dz.ld + (NARROW ? col : c.at)) * 2, v, NARROW ? cols - col : 8);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] += in && (NARROW || i >= c.skip) ? v[i] : 0.0f;
    }
  }
  if (!NARROW) move_down(c, acc);
  if (!part) return;
  __shared__ float sums[kThreads * 8];
#pragma unroll
  for (int i = 0; i < 8; ++i) sums[threadIdx.x * 8 + i] = acc[i];
  __syncthreads();
  for (int j = threadIdx.x; j < lanes * 8; j += kThreads) {
    float t = 0.0f;
    for (int k = 0; k < per; ++k) t += sums[k * lanes * 8 + j];
    const int c = int(blockIdx.y) * lanes * 8 + j;
    if (c < cols) part[int64_t(blockIdx.x) * cols + c] = t;
  }
}

// wt[k][n] = w[n][k], tiles of 64 x 64, 8 values to a thread on both sides (wt's rows are
// padded to multiples of 8).
__global__ void __launch_bounds__(kThreads) transpose_kernel(MatArg w, MatArg wt, int n, int k) {
  __shared__ uint16_t tile[64][66];   // [k][n]
  const int k0 = blockIdx.x * 64, n0 = blockIdx.y * 64;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int r = threadIdx.x / 8 + u * 32, c = threadIdx.x % 8 * 8;
    const u32x4 v = load_raw8(w, n0 + r, k0 + c, n0 + r < n ? k - k0 - c : 0).lo;
#pragma unroll
    for (int i = 0; i < 8; ++i) tile[c + i][r] = uint16_t(v[i / 2] >> (16 * (i & 1)));
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int r = threadIdx.x / 8 + u * 32, c = threadIdx.x % 8 * 8;
    if (k0 + r >= k || n0 + c >= n) continue;
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const uint32_t*>(&tile[r][c + 2 * i]);
    *reinterpret_cast<u32x4*>(wt.p + (int64_t(k0 + r) * wt.ld + n0 + c) * 2) = v;
  }
}

// out(q, p) = sum_k Q(q, k) P(p, k) by the kernel that fits: few tiles share the contraction
// among waves, many go by tiles; the plain kernel takes widths and alignments that neither does.
hipError_t launch_nt(const char* name, const MatArg& P, const MatArg& Q, int np, int64_t nq, int nk, const Epilogue& e,
                     hipStream_t s) {
  GSK_PROF(name, s);
  if (split_nt_takes(P, Q, np, nq)) return launch_split_nt(P, Q, np, nq, nk, e, s);
  if (tile_nt_takes(P, Q, nk)) return launch_tile_nt(P, Q, np, nq, nk, e, s);
  gemm_nt_kernel<1, 4, 1><<<dim3(div_up(nq, 64), div_up(np, 64)), kThreads, 0, s>>>(P, Q, np, nq, nk, e);
  return hipGetLastError();
}

inline size_t align256(size_t b) { return (b + 255) & ~size_t(255); }
inline int64_t min64(int64_t a, int64_t b) { return a < b ? a : b; }

// How the backward's row loops are split: slices of the rows whose partial sums are joined
// in order.
int dz_slices(int64_t rows) { return int(min64(rows < 64 ? 1 : rows / 64, 1024)); }

int dw_slices(int64_t rows, int k, int n) {
  const int64_t tiles = int64_t(div_up(k, 64)) * div_up(n, 64);
  const int64_t want = tiles >= 512 ? 1 : 512 / tiles;
  return int(min64(want, rows < 256 ? 1 : rows / 256));
}

struct BwdWs {
  char *dz, *wt;
  float *db, *dw;
  int64_t dz_ld, wt_ld;
  size_t bytes;
};

BwdWs carve_bwd(void* ws, int64_t rows, int k, int n) {
  BwdWs w;
  char* p = static_cast<char*>(ws);
  size_t at = 0;
  w.dz_ld = w.wt_ld = (n + 7) & ~7;
  w.dz = p + at;
  at += align256(size_t(rows) * w.dz_ld * 2);
  w.wt = p + at;
  at += align256(size_t(k) * w.wt_ld * 2);
  w.db = reinterpret_cast<float*>(p + at);
  at += align256(size_t(dz_slices(rows)) * n * 4);
  w.dw = reinterpret_cast<float*>(p + at);
  const int a = dw_slices(rows, k, n), c = tile_tn_slices(rows, k, n);
  at += align256(size_t(a > c ? a : c) * n * k * 4);
  w.bytes = at;
  return w;
}

}  // namespace

hipError_t launch_linear_fwd(const MatArg& x, const MatArg& w, const float* bias, int act, const MatArg& r,
                             const MatArg& z, const MatArg& y, int64_t rows, int k, int n, hipStream_t s) {
  const Epilogue e{bias, act, r, z, y};
  if (rows_fwd_takes(k, n)) return launch_rows_fwd(x, w, e, rows, k, n, s);
  return launch_nt("linear_fwd", w, x, n, rows, k, e, s);
}

size_t linear_bwd_ws_bytes(int64_t rows, int k, int n) {
  return rows_bwd_takes(k, n) ? rows_bwd_ws_bytes(rows, k, n) : carve_bwd(nullptr, rows, k, n).bytes;
}

hipError_t launch_linear_bwd(const MatArg& dy, const MatArg& z, int act, const MatArg& x, const MatArg& w,
                             const MatArg& dx, const MatArg& dw, float* dbias, int64_t rows, int k, int n, void* ws,
                             hipStream_t s) {
  if (rows_bwd_takes(k, n)) return launch_rows_bwd(dy, z, act, x, w, dx, dw, dbias, rows, k, n, ws, s);
  const BwdWs b = carve_bwd(ws, rows, k, n);
  // dz in memory: as the activation makes it, or a float32 dy rounded once for both products
  const bool own_dz = (act != GS_ACT_NONE || dy.type == GS_MAT_F32) && (dx.p || dw.p);
  const MatArg dz = own_dz ? MatArg{b.dz, nullptr, b.dz_ld, 0, GS_MAT_BF16} : dy;
  const MatArg none{nullptr, nullptr, 0, 0, GS_MAT_F32};
  hipError_t e;
  if (own_dz || dbias) {
    int lanes = 4;
    while (lanes < 64 && lanes * 8 < n) lanes *= 2;
    const int slices = dz_slices(rows);
    const int64_t per = (rows + slices - 1) / slices;
    {
      GSK_PROF("linear_dz", s);
      const dim3 grid(slices, div_up(n, lanes * 8));
      float* part = dbias ? b.db : nullptr;
      if (n < 8)
        dz_kernel<true><<<grid, kThreads, 0, s>>>(dy, z, act, own_dz ? dz : none, part, rows, n, per, lanes);
      else
        dz_kernel<false><<<grid, kThreads, 0, s>>>(dy, z, act, own_dz ? dz : none, part, rows, n, per, lanes);
    }
    if (dbias) {
      if ((e = launch_sum_parts(b.db, slices, n, 0, 1, MatArg{}, dbias, s)) != hipSuccess) return e;
    }
  }
  if (dx.p && rows > 0) {
    const MatArg wt{b.wt, nullptr, b.wt_ld, 0, GS_MAT_BF16};
    {
      GSK_PROF("linear_wt", s);
      transpose_kernel<<<dim3(div_up(k, 64), div_up(n, 64)), kThreads, 0, s>>>(w, wt, n, k);
    }
    const Epilogue out{nullptr, GS_ACT_NONE, none, none, dx};
    if ((e = launch_nt("linear_dx", wt, dz, k, rows, n, out, s)) != hipSuccess) return e;
  }
  if (dw.p && tile_tn_takes(x, dz, k, n)) {
    const int slices = tile_tn_slices(rows, k, n);
    {
      GSK_PROF("linear_dw", s);
      if ((e = launch_tile_tn(x, dz, k, n, rows, slices, b.dw, dw, s)) != hipSuccess) return e;
    }
    const int64_t size = int64_t(n) * k;
    if (slices > 1 && (e = launch_sum_parts(b.dw, slices, size, size, k, dw, nullptr, s)) != hipSuccess) return e;
  } else if (dw.p) {
    const int slices = dw_slices(rows, k, n);
    const int64_t per = ((rows + slices - 1) / slices + 63) / 64 * 64;
    float* part = slices > 1 ? b.dw : nullptr;
    {
      GSK_PROF("linear_dw", s);
      gemm_tn_kernel<1, 4, 1><<<dim3(div_up(k, 64), div_up(n, 64), slices), kThreads, 0, s>>>(x, dz, k, n, rows, per,
                                                                                              part, dw);
    }
    if (part && (e = launch_sum_parts(part, slices, int64_t(n) * k, int64_t(n) * k, k, dw, nullptr, s)) != hipSuccess)
      return e;
  }
  return hipGetLastError();
}

}  // namespace gsk
