// gs_clip_grads: the Euclidean norm n of many matrices together, and each times
// min(1, max_norm / n).
//
// Two passes over the data, bounded by HBM.  The first leaves one sum of squares a block, in
// double: a square of a float32 is exact there and neither overflows nor vanishes (gradients of
// a mean over an image are small), and the vector units do float64 at float32's rate.  In the second every
// block adds those sums itself, in the same order, instead of waiting for a kernel between.
// Matrices are cut into pieces of 16384 elements; a matrix whose rows are adjacent is one row.
#include "clip.h"
#include "matrix.h"
#include "profile.h"

namespace gsk {
namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 8;                       // 8 elements each, of a thread and piece
constexpr int kPiece = kThreads * kUnits;       // units of a piece
constexpr int kParts = 32;                      // matrices of a launch (their descriptions are its arguments)
constexpr int kMaxSums = 2048;                  // eight blocks a compute unit

struct Part {
  MatArg in, out;
  int64_t rows, cols;
};

struct List {
  Part part[kParts];
  int64_t piece[kParts + 1];   // a part's first piece; behind the last one their number
  int count;
};

__device__ inline int64_t units_a_row(const Part& p) { return (p.cols + 7) / 8; }

// f(part, row, column, elements) for this thread's units of the pieces of the block.
template <class F>
__device__ inline void for_units(const List& l, bool backwards, F f) {
  const int64_t pieces = l.piece[l.count];
  for (int64_t b = blockIdx.x; b < pieces; b += gridDim.x) {
    const int64_t piece = backwards ? pieces - 1 - b : b;
    int i = 0;
    while (i + 1 < l.count && piece >= l.piece[i + 1]) ++i;
    const Part& p = l.part[i];
    const int64_t a_row = units_a_row(p), first = (piece - l.piece[i]) * kPiece;
    const int64_t row0 = p.rows == 1 ? 0 : first / a_row, unit0 = first - row0 * a_row;
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      int64_t row = row0, unit = unit0 + threadIdx.x + u * kThreads;
      if (p.rows > 1) {   // rows of at most 2^17 units
        const uint32_t more = uint32_t(unit) / uint32_t(a_row);
        row += more;
        unit -= int64_t(more) * a_row;
      }
      const int64_t left = row < p.rows ? p.cols - unit * 8 : 0;
      if (left > 0) f(p, row, unit * 8, left > 8 ? 8 : int(left));
    }
  }
}

__device__ inline void load_unit(const MatArg& m, int64_t row, int64_t col, int n, float v[8]) {
  MatArg at = m;
  at.p += (row * m.ld + col) * element_bytes(m.type);
  raw8_to_float(load_raw8(at, 0, 0, n), m.type, v);
}

// The sum over the block of one double a thread, in all of them.
__device__ inline double block_sum(double x) {
  __shared__ double sums[kThreads];
  sums[threadIdx.x] = x;
  __syncthreads();
#pragma unroll
  for (int d = kThreads / 2; d > 0; d /= 2) {
    if (int(threadIdx.x) < d) sums[threadIdx.x] += sums[threadIdx.x + d];
    __syncthreads();
  }
  return sums[0];
}

__global__ void __launch_bounds__(kThreads) squares_kernel(List l, double* sums) {
  double sum = 0.0;
  for_units(l, false, [&](const Part& p, int64_t row, int64_t col, int n) {
    float v[8];
    load_unit(p.in, row, col, n, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += double(v[i]) * double(v[i]);   // absent elements are zero
  });
  sum = block_sum(sum);
  if (threadIdx.x == 0) sums[blockIdx.x] = sum;
}

// l without parts: only the norm.
__global__ void __launch_bounds__(kThreads) clip_kernel(List l, const double* sums, int count, double max_norm, float* norm) {
  double sum = 0.0;
  for (int i = threadIdx.x; i < count; i += kThreads) sum += sums[i];
  const double n = sqrt(block_sum(sum));
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = float(n);
  const float factor = float(n <= max_norm ? 1.0 : max_norm / n);   // NaN where n is
  for_units(l, true, [&](const Part& p, int64_t row, int64_t col, int k) {
    if (factor == 1.0f && p.in.p == p.out.p) return;
    float v[8];
    load_unit(p.in, row, col, k, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= factor;
    MatArg at = p.out;
    at.p += (row * p.out.ld + col) * element_bytes(p.out.type);
    store8(at, 0, 0, v, k);
  });
}

// The next matrices of the list, from `from` on, as a launch's arguments; returns where it ended.
int take(const gs_matrix* grads, const gs_matrix* out, int count, int from, List* l) {
  l->count = 0;
  l->piece[0] = 0;
  int i = from;
  for (; i < count && l->count < kParts; ++i) {
    if (grads[i].rows == 0) continue;
    Part p{mat_arg(&grads[i]), mat_arg(out ? &out[i] : &grads[i]), grads[i].rows, grads[i].cols};
    if (p.rows == 1 || (p.in.ld == p.cols && p.out.ld == p.cols)) {
      p.cols *= p.rows;
      p.rows = 1;
    }
    const int64_t units = p.rows * ((p.cols + 7) / 8);
    l->part[l->count++] = p;
    l->piece[l->count] = l->piece[l->count - 1] + (units + kPiece - 1) / kPiece;
  }
  return i;
}

}  // namespace

size_t clip_ws_bytes() { return size_t(kMaxSums) * sizeof(double); }

hipError_t launch_clip_grads(const gs_matrix* grads, const gs_matrix* out, int count, double max_norm, float* norm, void* ws,
                             hipStream_t s) {
  double* sums = static_cast<double*>(ws);
  const int launches = int(div_up(count, kParts)), share = kMaxSums / (launches > 0 ? launches : 1);
  int blocks = 0;
  List l;
  for (int from = 0; from < count;) {
    from = take(grads, nullptr, count, from, &l);
    const int64_t pieces = l.piece[l.count];
    const int grid = int(pieces < share ? pieces : share);
    if (grid == 0) continue;
    GSK_PROF("clip_squares", s);
    squares_kernel<<<grid, kThreads, 0, s>>>(l, sums + blocks);
    blocks += grid;
  }
  if (!out) count = 0;
  int from = 0;
  bool first = true;
  do {
    from = take(grads, out, count, from, &l);
    const int64_t pieces = l.piece[l.count];
    if (pieces == 0 && !first) continue;
    GSK_PROF("clip_scale", s);
    clip_kernel<<<unsigned(pieces < 1 ? 1 : pieces < kMaxSums ? pieces : kMaxSums), kThreads, 0, s>>>(
        l, sums, blocks, max_norm, first ? norm : nullptr);
    first = false;
  } while (from < count);
  return hipGetLastError();
}

}  // namespace gsk
