// gs_mx8_pack and gs_mx8_unpack: a matrix to and from MX8 (matrix.h has the format).
//
// Both are streams bounded by HBM: pack reads 2 or 4 bytes an element and writes 1 + 1/32,
// unpack the reverse.  A thread takes 8 columns (one 16-byte load of bfloat16, two of
// float32), so a block of 32 columns is four neighbouring lanes and its largest magnitude
// two lane exchanges; 4 to 64 lanes take a row (the smallest power of two that covers it,
// so narrow rows leave few lanes idle), and each keeps kRows rows in flight.
//
// 1M rows of 59 float32 columns: pack 59 us (5.0 TB/s), unpack to bfloat16 29 us (its input
// still in the last-level cache in part); 8160 rows of 4096 bfloat16: 23 and 18 us (4.4 and
// 5.5 TB/s).  A copy of 256 MB reaches 5.4 TB/s.
#include "matrix.h"
#include "profile.h"

namespace gsk {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 2;

// lanes: lanes per row, a power of two in [4, 64].  NARROW: fewer than 8 columns.
template <bool NARROW>
__global__ void __launch_bounds__(kThreads) mx8_pack_kernel(MatArg x, MatArg q, int64_t rows, int cols, int lanes) {
  const int lane = threadIdx.x & (lanes - 1);
  const int per = kThreads / lanes;   // rows a block takes at a time
  const int64_t row0 = int64_t(blockIdx.x) * (per * kRows) + threadIdx.x / lanes;
  const int col = (int(blockIdx.y) * lanes + lane) * 8;
  const Held c = held_at(col, cols);
  Raw8 raw[kRows];
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    const int64_t row = row0 + int64_t(u) * per;
    raw[u] = NARROW ? load_raw8(x, row, col, row < rows ? cols - col : 0)
                    : load_held(x, row < rows ? row : rows - 1, c);
  }
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    const int64_t row = row0 + int64_t(u) * per;
    float v[8];
    raw8_to_float(raw[u], x.type, v);
    if (!NARROW) move_down(c, v);
    store_mx8_quad(q, row, col, v, row < rows ? cols - col : 0);
  }
}

template <bool NARROW>
__global__ void __launch_bounds__(kThreads) mx8_unpack_kernel(MatArg q, MatArg x, int64_t rows, int cols, int lanes) {
  const int lane = threadIdx.x & (lanes - 1);
  const int per = kThreads / lanes;
  const int64_t row0 = int64_t(blockIdx.x) * (per * kRows) + threadIdx.x / lanes;
  const int col = (int(blockIdx.y) * lanes + lane) * 8;
  const Held c = held_at(col, cols);
  Raw8 raw[kRows];
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    const int64_t row = row0 + int64_t(u) * per;
    raw[u] = NARROW ? load_raw8(q, row, col, row < rows ? cols - col : 0)
                    : load_held(q, row < rows ? row : rows - 1, c);
  }
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    const int64_t row = row0 + int64_t(u) * per;
    float v[8];
    if (NARROW)
      raw8_to_float(raw[u], GS_MAT_MX8, v);
    else
      held_to_float(raw[u], GS_MAT_MX8, c, v);
    if (row < rows && c.skip < 8) store8(x, row, NARROW ? col : c.at, v, NARROW ? cols - col : 8);
  }
}

int lanes_for(int cols) {
  int lanes = 4;
  while (lanes < 64 && lanes * 8 < cols) lanes *= 2;
  return lanes;
}

}  // namespace

hipError_t launch_mx8_pack(const MatArg& x, const MatArg& q, int64_t rows, int cols, hipStream_t s) {
  const int lanes = lanes_for(cols);
  GSK_PROF("mx8_pack", s);
  for_row_parts(rows, kThreads / lanes * kRows, [&](int64_t first, int64_t count, unsigned blocks) {
    const auto kernel = cols < 8 ? &mx8_pack_kernel<true> : &mx8_pack_kernel<false>;
    kernel<<<dim3(blocks, div_up(cols, lanes * 8)), kThreads, 0, s>>>(rows_from(x, first), rows_from(q, first), count, cols,
                                                                     lanes);
  });
  return hipGetLastError();
}

hipError_t launch_mx8_unpack(const MatArg& q, const MatArg& x, int64_t rows, int cols, hipStream_t s) {
  const int lanes = lanes_for(cols);
  GSK_PROF("mx8_unpack", s);
  for_row_parts(rows, kThreads / lanes * kRows, [&](int64_t first, int64_t count, unsigned blocks) {
    const auto kernel = cols < 8 ? &mx8_unpack_kernel<true> : &mx8_unpack_kernel<false>;
    kernel<<<dim3(blocks, div_up(cols, lanes * 8)), kThreads, 0, s>>>(rows_from(q, first), rows_from(x, first), count, cols,
                                                                     lanes);
  });
  return hipGetLastError();
}

}  // namespace gsk
