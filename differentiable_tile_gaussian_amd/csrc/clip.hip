// gs_clip_grads: the Euclidean norm n of many matrices together, and each times
// min(1, max_norm / n).
//
// Two passes over the data, bounded by HBM.  The first leaves one sum of squares a block, in
// double: a square of a float32 is exact there and neither overflows nor vanishes (gradients of
// a mean over an image are small), and the vector units do float64 at float32's rate.  In the second every
// block adds those sums itself, in the same order, instead of waiting for a kernel between.
// Matrices are cut into pieces of 16384 elements; a matrix whose rows are adjacent is one row.
// 708 MB of gradients (3M Gaussians and a decoder): 126 us for the norm (5.6 TB/s), 270 to clip
// them (5.3); the gradients of a small network, 1 MB: 5.3 and 4.9 us, latency (6.5 and 6.2 where a block finds
// its part by a loop over them).  A launch takes 32 matrices, and the norm's launches share its 2048 sums
// evenly, so that long lists leave it few blocks at a time: 708 MB in 320 matrices 408 us for the norm,
// in 1024 598 (1.2 TB/s).
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

// Piece number `piece` of the list: its part and the thread's first unit there; whole: it is all full
// units of one row, and what comes out is of the same type.
struct Piece {
  Part p;
  int64_t row, unit;
  bool whole;
};

__device__ __forceinline__ Piece piece_of(const List& l, int64_t piece) {
  // the parts behind the first that begin at or before it, counted by the lanes
  const int lane = __lane_id();
  const int64_t begin = l.piece[lane < kParts ? lane : kParts];
  const int i = __popcll(__ballot(lane > 0 && lane < l.count && piece >= begin));
  Piece x;
  x.p = l.part[i];
  const int64_t a_row = (x.p.cols + 7) / 8, first = (piece - l.piece[i]) * kPiece;
  x.row = x.p.rows == 1 ? 0 : first / a_row;
  x.unit = first - x.row * a_row;
  x.whole = x.p.rows == 1 && (first + kPiece) * 8 <= x.p.cols && x.p.in.type == x.p.out.type;
  return x;
}

// A whole piece is taken in words of 16 bytes, a wave's next to each other, all in flight together:
// the thread's first, and how many it has.
__device__ __forceinline__ char* words_at(const MatArg& m, const Piece& x) {
  return m.p + x.unit * 8 * element_bytes(m.type) + threadIdx.x * 16;
}
constexpr int words_of(int type) { return type == GS_MAT_F32 ? 2 * kUnits : kUnits; }

template <int TYPE>
struct Words {
  static constexpr int N = words_of(TYPE), kEach = TYPE == GS_MAT_F32 ? 4 : 8;
  u32x4 w[N];
  __device__ __forceinline__ void load(const char* p) {
#pragma unroll
    for (int j = 0; j < N; ++j) __builtin_memcpy(&w[j], __builtin_assume_aligned(p + j * (kThreads * 16), 2), 16);
  }
  __device__ __forceinline__ void values(int j, float (&v)[8]) const { raw8_to_float(Raw8{w[j], w[j], 0}, TYPE, v); }
};

// Any piece, unit by unit: f(row, column, elements) for those that the thread has.
template <class F>
__device__ __forceinline__ void for_units(const Piece& x, F f) {
  const uint32_t a_row = uint32_t((x.p.cols + 7) / 8);
#pragma unroll 2
  for (int u = 0; u < kUnits; ++u) {
    int64_t row = x.row, unit = x.unit + threadIdx.x + u * kThreads;
    if (x.p.rows > 1) {   // rows of at most 2^17 units
      const uint32_t more = uint32_t(unit) / a_row;
      row += more;
      unit -= int64_t(more) * a_row;
    }
    const int64_t left = row < x.p.rows ? x.p.cols - unit * 8 : 0;
    if (left > 0) f(row, unit * 8, left > 8 ? 8 : int(left));
  }
}

__device__ __forceinline__ MatArg from(MatArg m, int64_t row, int64_t col) {
  m.p += (row * m.ld + col) * element_bytes(m.type);
  return m;
}

// The sum over the block of one double a thread, in all of them (once in a kernel).
__device__ inline double block_sum(double x) {
  __shared__ double sums[kThreads / 64];
#pragma unroll
  for (int d = 32; d > 0; d /= 2) x += __shfl_xor(x, d, 64);
  if (threadIdx.x % 64 == 0) sums[threadIdx.x / 64] = x;
  __syncthreads();
  return (sums[0] + sums[1]) + (sums[2] + sums[3]);
}

template <int TYPE>
__device__ __forceinline__ double squares_of(const Piece& x) {
  Words<TYPE> all;
  all.load(words_at(x.p.in, x));
  double sum = 0.0;
#pragma unroll
  for (int j = 0; j < all.N; ++j) {
    float v[8];
    all.values(j, v);
#pragma unroll
    for (int i = 0; i < all.kEach; ++i) sum += double(v[i]) * double(v[i]);
  }
  return sum;
}

__global__ void __launch_bounds__(kThreads) squares_kernel(List l, double* sums) {
  double sum = 0.0;
  for (int64_t b = blockIdx.x; b < l.piece[l.count]; b += gridDim.x) {
    const Piece x = piece_of(l, b);
    if (x.whole) {
      sum += x.p.in.type == GS_MAT_F32 ? squares_of<GS_MAT_F32>(x) : squares_of<GS_MAT_BF16>(x);
    } else {
      for_units(x, [&](int64_t row, int64_t col, int n) {
        float v[8];
        raw8_to_float(load_raw8(from(x.p.in, row, col), 0, 0, n), x.p.in.type, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += double(v[i]) * double(v[i]);   // absent elements are zero
      });
    }
  }
  sum = block_sum(sum);
  if (threadIdx.x == 0) sums[blockIdx.x] = sum;
}

template <int TYPE, class Factor>
__device__ __forceinline__ void clip_whole(const Piece& x, Factor factor_of) {
  Words<TYPE> all;
  all.load(words_at(x.p.in, x));
  const float factor = factor_of();   // behind the loads
  char* to = words_at(x.p.out, x);
  if (factor == 1.0f && x.p.in.p == x.p.out.p) return;
#pragma unroll
  for (int j = 0; j < all.N; ++j) {
    float v[8];
    all.values(j, v);
#pragma unroll
    for (int i = 0; i < all.kEach; ++i) v[i] *= factor;
    // past the caches: they keep what is still to be read
    typedef u32x4 Any16 __attribute__((aligned(2)));
    const u32x4 o = TYPE == GS_MAT_F32 ? __builtin_bit_cast(u32x4, f32x4{v[0], v[1], v[2], v[3]})
                                       : u32x4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
    __builtin_nontemporal_store(o, reinterpret_cast<Any16*>(to + j * (kThreads * 16)));
  }
}

// l without parts: only the norm.  The pieces are taken from the list's end, which the first pass read last.
__global__ void __launch_bounds__(kThreads) clip_kernel(List l, const double* sums, int count, double max_norm, float* norm) {
  const int64_t pieces = l.piece[l.count];
  float factor = 1.0f;
  bool known = false;
  auto know = [&]() {
    if (known) return factor;
    double sum = 0.0;
    for (int i = threadIdx.x; i < count; i += kThreads) sum += sums[i];
    const double n = sqrt(block_sum(sum));
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = float(n);
    known = true;
    return factor = float(n <= max_norm ? 1.0 : max_norm / n);   // NaN where n is
  };
  for (int64_t b = blockIdx.x; b < pieces; b += gridDim.x) {
    const Piece x = piece_of(l, pieces - 1 - b);
    if (x.whole) {
      if (x.p.in.type == GS_MAT_F32)
        clip_whole<GS_MAT_F32>(x, know);
      else
        clip_whole<GS_MAT_BF16>(x, know);
      continue;
    }
    know();
    if (factor == 1.0f && x.p.in.p == x.p.out.p) continue;
    for_units(x, [&](int64_t row, int64_t col, int n) {
      float v[8];
      raw8_to_float(load_raw8(from(x.p.in, row, col), 0, 0, n), x.p.in.type, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= factor;
      store8(from(x.p.out, row, col), 0, 0, v, n);
    });
  }
  know();
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
