// gs_mx4_pack and gs_mx4_unpack: a matrix to and from MX4 (mx4.h has the layout).
//
// Both are streams bounded by HBM: pack reads 2 or 4 bytes an element and writes 17/32, unpack
// the reverse.  A thread takes 8 columns (one 16-byte load of bfloat16, two of float32), so a
// block of 32 is four neighbouring lanes and its largest magnitude two lane exchanges; 4 to 64
// lanes take a row (the smallest power of two that covers it), and each keeps kRows rows in
// flight.  Unpacked rows are stored past the caches.  1,000,003 rows of 128 bfloat16 to MX4 and
// back: 63 and 45 us (5.1 and 7.2 TB/s, the 4-bit matrix coming from the cache); 1024 rows of 4096
// float32: 5.7 and 3.9 us.
#include "mx4.h"
#include "profile.h"

namespace gsk {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 2;

// lanes: lanes per row, a power of two in [4, 64].  NARROW: fewer than 8 columns.
template <bool NARROW>
__global__ void __launch_bounds__(kThreads) mx4_pack_kernel(MatArg x, MatArg q, int64_t rows, int cols, int lanes) {
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
    const uint32_t byte = mx4_scale_byte(max_over_quad(top_bits<8>(v)));
    const uint32_t w = byte == 255u ? 0u : mx4_encode8(v, mx8_scale(byte));
    if (row < rows && (col & ~31) < cols) {   // the last block whole, zeros behind the last column
      *reinterpret_cast<uint32_t*>(q.p + row * mx4_pitch(q) + col / 2) = w;
      if ((col & 31) == 0) q.s[row * q.lds + (col >> 5)] = uint8_t(byte);
    }
  }
}

template <bool NARROW>
__global__ void __launch_bounds__(kThreads) mx4_unpack_kernel(MatArg q, MatArg x, int64_t rows, int cols, int lanes) {
  const int lane = threadIdx.x & (lanes - 1);
  const int per = kThreads / lanes;
  const int64_t row0 = int64_t(blockIdx.x) * (per * kRows) + threadIdx.x / lanes;
  const int col = (int(blockIdx.y) * lanes + lane) * 8;
  uint32_t w[kRows], byte[kRows];
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    const int64_t row = row0 + int64_t(u) * per;
    const bool in = row < rows && col < cols;
    w[u] = in ? *reinterpret_cast<const uint32_t*>(q.p + row * mx4_pitch(q) + col / 2) : 0u;
    byte[u] = in ? q.s[row * q.lds + (col >> 5)] : 0u;
  }
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    const int64_t row = row0 + int64_t(u) * per;
    float v[8];
    mx4_decode8(w[u], mx8_scale(byte[u]), v);
    if (row < rows && col < cols) store8_once(x, row, col, v, NARROW || cols - col < 8 ? cols - col : 8);
  }
}

int lanes_for(int cols) {
  int lanes = 4;
  while (lanes < 64 && lanes * 8 < cols) lanes *= 2;
  return lanes;
}

}  // namespace

hipError_t launch_mx4_pack(const MatArg& x, const MatArg& q, int64_t rows, int cols, hipStream_t s) {
  const int lanes = lanes_for(cols);
  GSK_PROF("mx4_pack", s);
  for_row_parts(rows, kThreads / lanes * kRows, [&](int64_t first, int64_t count, unsigned blocks) {
    const auto kernel = cols < 8 ? &mx4_pack_kernel<true> : &mx4_pack_kernel<false>;
    kernel<<<dim3(blocks, div_up(cols, lanes * 8)), kThreads, 0, s>>>(rows_from(x, first), mx4_rows_from(q, first), count,
                                                                     cols, lanes);
  });
  return hipGetLastError();
}

hipError_t launch_mx4_unpack(const MatArg& q, const MatArg& x, int64_t rows, int cols, hipStream_t s) {
  const int lanes = lanes_for(cols);
  GSK_PROF("mx4_unpack", s);
  for_row_parts(rows, kThreads / lanes * kRows, [&](int64_t first, int64_t count, unsigned blocks) {
    const auto kernel = cols < 8 ? &mx4_unpack_kernel<true> : &mx4_unpack_kernel<false>;
    kernel<<<dim3(blocks, div_up(cols, lanes * 8)), kThreads, 0, s>>>(mx4_rows_from(q, first), rows_from(x, first), count,
                                                                     cols, lanes);
  });
  return hipGetLastError();
}

}  // namespace gsk
