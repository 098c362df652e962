// gs_linear_fwd and gs_linear_bwd: y = act(x W^T + b) + r and its gradients.  With
// z = x W^T + b and dz = dy act'(z):  dx = dz W,  dW = dz^T x,  db = sum of the rows of dz.
//
// Every product runs on the matrix cores (16x16x32, bfloat16 operands, float32 sums):
// bfloat16 and MX8 operands are exact there, float32 ones (and dz) are rounded to bfloat16
// (the matrix cores' float32 products run at a sixteenth of the rate, and dz's rounding is
// that of the bfloat16 gradients it is made from).
//
// The backward's general path is four kernels: dz with db's partial sums, W^T, and the two
// products, dx by launch_nt and dW by launch_tile_tn; and one or two joins of partial sums.  dz is bounded by the slopes' vector
// work (8160 rows of 4096, gelu, z in 8 bits: 41 us; without an activation, only summing
// columns, 18 us); W^T (4096 x 1024) takes 6 us.  Few rows are bounded by the five launches (1 row
// 1024 to 1024 with silu: 22 us a call, 64 rows 27; by one pass 1 row 128 to 128 15, 1000 rows 17).
#include "linear.h"
#include "profile.h"

namespace gsk {
namespace {

constexpr int kThreads = 256;

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

// out(q, p) = sum_k Q(q, k) P(p, k) by the kernel that fits: narrow products with the
// weight in LDS, few tiles with the contraction shared among waves, many by tiles.
hipError_t launch_nt(const char* name, const MatArg& P, const MatArg& Q, int np, int64_t nq, int nk, const Epilogue& e,
                     hipStream_t s) {
  if (rows_fwd_takes(nk, np)) return launch_rows_fwd(Q, P, e, nq, nk, np, s);
  GSK_PROF(name, s);
  if (split_nt_takes(P, Q, np, nq)) return launch_split_nt(P, Q, np, nq, nk, e, s);
  return launch_tile_nt(P, Q, np, nq, nk, e, s);
}

inline size_t align256(size_t b) { return (b + 255) & ~size_t(255); }
inline int64_t min64(int64_t a, int64_t b) { return a < b ? a : b; }

// How the backward's row loops are split: slices of the rows whose partial sums are joined
// in order.
int dz_lanes(int n) {
  int lanes = 4;
  while (lanes < 64 && lanes * 8 < n) lanes *= 2;
  return lanes;
}

int dz_slices(int64_t rows, int n) {
  const int64_t turn = kThreads / dz_lanes(n) * kRows, most = (rows + turn - 1) / turn;
  const int64_t want = 1280 / div_up(n, dz_lanes(n) * 8);   // 5 blocks a compute unit
  return int(min64(most < 1 ? 1 : most, want < 1 ? 1 : want));
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
  w.dz_ld = w.wt_ld = (n + 7) & ~7;   // rows at multiples of 16 bytes
  w.dz = p + at;
  at += align256(size_t(rows) * w.dz_ld * 2);
  w.wt = p + at;
  at += align256(size_t(k) * w.wt_ld * 2);
  w.db = reinterpret_cast<float*>(p + at);
  at += align256(size_t(dz_slices(rows, n)) * n * 4);
  w.dw = reinterpret_cast<float*>(p + at);
  at += align256(size_t(tile_tn_slices(rows, k, n)) * n * k * 4);
  w.bytes = at;
  return w;
}

}  // namespace

hipError_t launch_linear_fwd(const MatArg& x, const MatArg& w, const float* bias, int act, const MatArg& r,
                             const MatArg& z, const MatArg& y, int64_t rows, int k, int n, hipStream_t s) {
  const Epilogue e{bias, act, r, z, y};
  return launch_nt("linear_fwd", w, x, n, rows, k, e, s);
}

// Where the types and addresses decide between the two ways, for either.
size_t linear_bwd_ws_bytes(int64_t rows, int k, int n) {
  const size_t one = rows_bwd_takes(k, n) ? rows_bwd_ws_bytes(rows, k, n) : 0;
  if (one && n <= 128) return one;
  const size_t steps = carve_bwd(nullptr, rows, k, n).bytes;
  return one > steps ? one : steps;
}

hipError_t launch_linear_bwd(const MatArg& dy, const MatArg& z, int act, const MatArg& x, const MatArg& w,
                             const MatArg& dx, const MatArg& dw, float* dbias, int64_t rows, int k, int n, void* ws,
                             hipStream_t s) {
  if (rows_bwd_runs(dy, z, act, x, dx, k, n))
    return launch_rows_bwd(dy, z, act, x, w, dx, dw, dbias, rows, k, n, ws, s);
  const BwdWs b = carve_bwd(ws, rows, k, n);
  // dz in memory: as the activation makes it, or a float32 dy rounded once for both products
  const bool own_dz = (act != GS_ACT_NONE || dy.type == GS_MAT_F32) && (dx.p || dw.p);
  const MatArg dz = own_dz ? MatArg{b.dz, nullptr, b.dz_ld, 0, GS_MAT_BF16} : dy;
  const MatArg none{nullptr, nullptr, 0, 0, GS_MAT_F32};
  hipError_t e;
  if (own_dz || dbias) {
    const int slices = dz_slices(rows, n), lanes = dz_lanes(n);
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
  if (dw.p) {
    const int slices = tile_tn_slices(rows, k, n);
    {
      GSK_PROF("linear_dw", s);
      if ((e = launch_tile_tn(x, dz, k, n, rows, slices, b.dw, dw, s)) != hipSuccess) return e;
    }
    const int64_t size = int64_t(n) * k;
    if (slices > 1 && (e = launch_sum_parts(b.dw, slices, size, size, k, dw, nullptr, s)) != hipSuccess) return e;
  }
  return hipGetLastError();
}

}  // namespace gsk
