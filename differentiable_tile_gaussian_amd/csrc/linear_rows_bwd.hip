// Gradients of a narrow linear layer over many rows (widths as rows_bwd_takes says): one
// pass over the rows for dz, dx, dW and db.  Bounded by HBM: dy, z and x are read once and
// dx written once; dz exists only in registers and LDS.
//
// A block of eight waves takes 128 rows a turn, 16 to a wave.  A lane loads the 16 columns
// of its row that it will hold as an operand, forms dz there, adds it to its column sums
// (db, before the rounding) and rounds it: that is the operand of dx = dz W, whose other
// operand W^T lies in LDS.  dz and x also go to LDS as rows, where the contraction over the
// rows, dW += dz^T x, reads them transposed; the eight waves share dW's tiles, whose sums stay
// in registers over all of the block's turns.  The next turn's loads are issued before the
// products of the present one.  Each block writes its sums of dW and db once; they are joined
// in order by launch_sum_parts.
//
// 1M rows 128 to 128, z and x in 8 bits, silu: 185-190 us (776 MB, 4.1 TB/s) and 8 us for the sums;
// without an activation, x in bfloat16, 141 us; 100k rows 64 to 48 with a float32 dy: 15 and
// 4 us.  What is left is the vector work of silu's slope and of the 8-bit decodes, in turns with
// the two products: a block's registers and LDS leave room for one block a compute unit.
#include "linear.h"
#include "profile.h"

namespace gsk {
namespace {

constexpr int kThreads = 512;
constexpr int kRows = 128;

// 16 columns of a row as loaded, of any type.
struct Piece {
  u32x4 v[4];
  uint32_t scale, skip;
};

// Columns col .. col + 15 of a row of any matrix, as matrix.h's Raw16 holds them until they
// are settled.
template <int TYPE, bool NARROW>
__device__ inline void load_piece_as(Piece& p, const MatArg& m, int64_t row, int col, int cols, bool live) {
  Raw16<TYPE, NARROW> r;
  r.load(m, row, col, cols, live);
#pragma unroll
  for (int i = 0; i < r.kWords; ++i) p.v[i / 4][i % 4] = r.w[i];
  p.scale = TYPE == GS_MAT_MX8 ? r.scale : 0;
  p.skip = r.skip;
}

template <int TYPE, bool NARROW>
__device__ inline void load_piece_any(Piece& p, const MatArg& m, int64_t row, int col, int cols, bool live) {
  if (TYPE == GS_MAT_MX8 || (TYPE == kAny && m.type == GS_MAT_MX8))
    load_piece_as<GS_MAT_MX8, NARROW>(p, m, row, col, cols, live);
  else if (TYPE == GS_MAT_BF16 || (TYPE == kAny && m.type == GS_MAT_BF16))
    load_piece_as<GS_MAT_BF16, NARROW>(p, m, row, col, cols, live);
  else
    load_piece_as<GS_MAT_F32, NARROW>(p, m, row, col, cols, live);
}

// last: this may be the row's last piece, which may have to move.
template <int TYPE>
__device__ inline void settle_piece_as(Piece& p, bool last) {
  Raw16<TYPE, false> r;
#pragma unroll
  for (int i = 0; i < r.kWords; ++i) r.w[i] = p.v[i / 4][i % 4];
  r.skip = p.skip;
  if (last)
    r.settle();
  else
    r.settle_whole();
#pragma unroll
  for (int i = 0; i < r.kWords; ++i) p.v[i / 4][i % 4] = r.w[i];
}

// TYPE: the matrix's, or kAny.
template <int TYPE>
__device__ inline void settle_piece(Piece& p, int type, bool last) {
  if (TYPE == GS_MAT_MX8 || (TYPE == kAny && type == GS_MAT_MX8))
    settle_piece_as<GS_MAT_MX8>(p, last);
  else if (TYPE == GS_MAT_BF16 || (TYPE == kAny && type == GS_MAT_BF16))
    settle_piece_as<GS_MAT_BF16>(p, last);
  else
    settle_piece_as<GS_MAT_F32>(p, last);
}

// The pieces of a lane's row through buffers: rows row0 + row, columns 64 c + 16 g.
template <int TYPE, int C>
__device__ inline void load_pieces(Piece (&p)[C], const MatArg& m, int64_t row0, int row, bool in, int g, int cols) {
  constexpr uint32_t kE = element_bytes(TYPE);
  const Buffer data = buffer_at(m.p + row0 * m.ld * kE);
  const Buffer scales = buffer_at(TYPE == GS_MAT_MX8 ? m.s + row0 * m.lds : nullptr);
  const uint32_t off = (row * uint32_t(m.ld) + g * 16) * kE, soff = row * uint32_t(m.lds) + g / 2;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const bool there = in && c * 64 + g * 16 < cols;
#pragma unroll
    for (int i = 0; i < int(kE); ++i) p[c].v[i] = buffer_load16(data, there ? off + c * 64 * kE + i * 16 : kAbsent);
    p[c].scale = TYPE == GS_MAT_MX8 ? buffer_load1(scales, there ? soff + c * 2 : kAbsent) : 0;
  }
}

__device__ inline void piece_to_float(const Piece& p, int type, float v[16]) {
  if (type == GS_MAT_MX8) {
    const float s = mx8_scale(p.scale);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(p.v[0][i], s, false);
      const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(p.v[0][i], s, true);
      v[4 * i] = a[0];
      v[4 * i + 1] = a[1];
      v[4 * i + 2] = b[0];
      v[4 * i + 3] = b[1];
    }
  } else if (type == GS_MAT_BF16) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[2 * i] = bf16_lo(p.v[i / 4][i % 4]);
      v[2 * i + 1] = bf16_hi(p.v[i / 4][i % 4]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(p.v[i / 4][i % 4]);
  }
}

__device__ inline void piece_to_bf16(const Piece& p, int type, u32x4& a, u32x4& b) {
  if (type == GS_MAT_MX8) {
    const float s = mx8_scale(p.scale);
    const u32x2 w0 = mx8_to_bf16x4(p.v[0][0], s), w1 = mx8_to_bf16x4(p.v[0][1], s);
    const u32x2 w2 = mx8_to_bf16x4(p.v[0][2], s), w3 = mx8_to_bf16x4(p.v[0][3], s);
    a = u32x4{w0[0], w0[1], w1[0], w1[1]};
    b = u32x4{w2[0], w2[1], w3[0], w3[1]};
  } else {
    a = p.v[0];
    b = p.v[1];
  }
}

template <int ROTATION>
__device__ inline float add_rotated(float v) {
  return v + __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x120 + ROTATION, 0xf, 0xf, true));
}
// The sum over the 16 lanes of a row of the wave, by rotations within it.
__device__ inline float sum_over16(float v) {
  return add_rotated<1>(add_rotated<2>(add_rotated<4>(add_rotated<8>(v))));
}

// Orders LDS accesses around a barrier; global loads stay in flight across it.
__device__ inline void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

struct RowsBwdArgs {
  MatArg dy, z, x, w, dx;
  float* part;      // a part's sums of dW [n][k], then of db [n]; the parts part_size apart
  int64_t part_size;
  bool want_dw, want_db;
  int64_t rows;
  int act, k, n;
};

// How the eight waves share dW: kWP groups of 64 columns (k), kWQ groups of 16 kQT rows (n),
// and kMS shares of a turn's rows (each a part of its own).
template <int NC, int KC>
struct Share {
  static constexpr int kQT = NC * KC == 4 ? 2 : 1, kWP = KC, kWQ = NC * 4 / kQT, kMS = 8 / (kWP * kWQ);
};

// NC, KC: groups of 64 columns of dz and of x.  DY, Z, X: the types of dy, z (kNone: no
// activation) and x, or all kAny.
template <int NC, int KC, int DY, int Z, int X, Reach HOW>
__global__ void __launch_bounds__(kThreads, 2) rows_bwd_kernel(RowsBwdArgs a) {
  using S = Share<NC, KC>;
  constexpr bool kFew = HOW == kNarrow;
  const int dyt = DY == kAny ? a.dy.type : DY, zt_ = Z == kAny ? a.z.type : Z, xt_ = X == kAny ? a.x.type : X;
  const int act = Z == kNone ? GS_ACT_NONE : a.act;
  constexpr int kPitchQ = NC * 128 + 32, kPitchP = KC * 128 + 32;
  extern __shared__ __align__(16) uint8_t lds[];
  uint8_t* wt = lds;                                  // NC KC 8 KiB of operands
  uint8_t* zt = lds + NC * KC * 8192;                 // dz rows
  uint8_t* xt = zt + kRows * kPitchQ;                 // x rows
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, g = lane / 16, r = lane % 16;
  const int wp = wave % S::kWP, wq = wave / S::kWP % S::kWQ, ms = wave / (S::kWP * S::kWQ);

  float db[NC][16];
  f32x4 dw[S::kQT][4];
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int i = 0; i < 16; ++i) db[c][i] = 0.0f;
#pragma unroll
  for (int q = 0; q < S::kQT; ++q)
#pragma unroll
    for (int t = 0; t < 4; ++t) dw[q][t] = f32x4{0, 0, 0, 0};

  Piece dy[NC], z[NC], x[KC];
  auto fetch = [&](int turn) {
    const int64_t row0 = int64_t(turn) * kRows;
    const int row = wave * 16 + r;
    const bool in = row < a.rows - row0;
    if constexpr (HOW == kWhole) {
      load_pieces<DY>(dy, a.dy, row0, row, in, g, a.n);
      if constexpr (Z != kNone) load_pieces<Z>(z, a.z, row0, row, in, g, a.n);
      load_pieces<X>(x, a.x, row0, row, in, g, a.k);
    } else {
      const int64_t at = in ? row0 + row : a.rows - 1;
#pragma unroll
      for (int c = 0; c < NC; ++c) load_piece_any<DY, kFew>(dy[c], a.dy, at, c * 64 + g * 16, a.n, in);
      if (act != GS_ACT_NONE) {
#pragma unroll
        for (int c = 0; c < NC; ++c) load_piece_any<Z, kFew>(z[c], a.z, at, c * 64 + g * 16, a.n, in);
      }
#pragma unroll
      for (int c = 0; c < KC; ++c) load_piece_any<X, kFew>(x[c], a.x, at, c * 64 + g * 16, a.k, in);
    }
  };
  u32x4 dz[NC][2], xb[KC][2];
  auto convert = [&]() {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      float v[16];
      if constexpr (HOW != kWhole) settle_piece<DY>(dy[c], dyt, c * 2 + 2 > NC);
      piece_to_float(dy[c], dyt, v);
      if (act != GS_ACT_NONE) {
        float t[16];
        if constexpr (HOW != kWhole) settle_piece<Z>(z[c], zt_, c * 2 + 2 > NC);
        piece_to_float(z[c], zt_, t);
        if (act == GS_ACT_SILU) {
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] *= act_slope(t[i], GS_ACT_SILU);
        } else if (act == GS_ACT_GELU) {
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] *= act_slope(t[i], GS_ACT_GELU);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] *= act_slope(t[i], GS_ACT_RELU);
        }
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) db[c][i] += v[i];
#pragma unroll
      for (int i = 0; i < 8; ++i) dz[c][i / 4][i % 4] = pack_bf16(v[2 * i], v[2 * i + 1]);
    }
#pragma unroll
    for (int c = 0; c < KC; ++c) {
      if constexpr (HOW != kWhole) settle_piece<X>(x[c], xt_, c * 2 + 2 > KC);
      piece_to_bf16(x[c], xt_, xb[c][0], xb[c][1]);
    }
  };
  const int turns = int((a.rows + kRows - 1) / kRows);
  const bool any = int64_t(blockIdx.x) < turns;
  if (any) fetch(blockIdx.x);
  // W^T as operands of tile (kc, t), piece (nc, half): lane (g, r) holds rows n = 64 nc + 16 g
  // + 8 half .. + 7 of column k = 64 kc + 16 (r / 4) + 4 t + r % 4.
  constexpr int kChunks = NC * KC;   // of 8 k, for each thread
  u32x4 wr[kChunks];
#pragma unroll
  for (int u = 0; u < kChunks; ++u) {
    const int i = u * kThreads + threadIdx.x, n = i / (KC * 8), k = i % (KC * 8) * 8;
    wr[u] = load_raw8(a.w, n, k, n < a.n ? a.k - k : 0).lo;
  }
#pragma unroll
  for (int u = 0; u < kChunks; ++u) {
    const int i = u * kThreads + threadIdx.x, n = i / (KC * 8), k0 = i % (KC * 8) * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int k = k0 + j, frag = ((k / 64 * 4 + k / 4 % 4) * NC + n / 64) * 2 + n / 8 % 2;
      const int l = n / 16 % 4 * 16 + k / 16 % 4 * 4 + k % 4;
      *reinterpret_cast<uint16_t*>(wt + frag * 1024 + l * 16 + n % 8 * 2) = uint16_t(wr[u][j / 2] >> (16 * (j & 1)));
    }
  }
  if (any) convert();
  for (int turn = blockIdx.x; turn < turns; turn += gridDim.x) {
    lds_barrier();   // the last turn's readers are done (and, at first, W^T is written)
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      uint8_t* p = zt + (wave * 16 + r) * kPitchQ + (c * 64 + g * 16) * 2;
      *reinterpret_cast<u32x4*>(p) = dz[c][0];
      *reinterpret_cast<u32x4*>(p + 16) = dz[c][1];
    }
#pragma unroll
    for (int c = 0; c < KC; ++c) {
      uint8_t* p = xt + (wave * 16 + r) * kPitchP + (c * 64 + g * 16) * 2;
      *reinterpret_cast<u32x4*>(p) = xb[c][0];
      *reinterpret_cast<u32x4*>(p + 16) = xb[c][1];
    }
    fetch(turn + gridDim.x);   // past the last row: all absent
    lds_barrier();
    f32x4 acc[KC][4];
    if (a.dx.p) {
      int at = lane * 16;
      asm volatile("" : "+v"(at));   // W^T stays in LDS: the compiler may not keep it in registers
#pragma unroll
      for (int kc = 0; kc < KC; ++kc)
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          acc[kc][t] = f32x4{0, 0, 0, 0};
#pragma unroll
          for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const bf16x8 wf = *reinterpret_cast<const bf16x8*>(wt + (((kc * 4 + t) * NC + c) * 2 + h) * 1024 + at);
              acc[kc][t] =
                  __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf, __builtin_bit_cast(bf16x8, dz[c][h]), acc[kc][t], 0, 0, 0);
            }
        }
    }
    if (a.want_dw) {
#pragma unroll
      for (int kk = 0; kk < kRows / 32 / S::kMS; ++kk) {
        const int m = (kk * S::kMS + ms) * 32 + g * 8 + r / 4, c = lane % 4 * 4;
        bf16x8 pf[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) pf[t] = read_transposed(xt + m * kPitchP + (wp * 64 + t * 16 + c) * 2, kPitchP);
#pragma unroll
        for (int q = 0; q < S::kQT; ++q) {
          const bf16x8 qf = read_transposed(zt + m * kPitchQ + ((wq * S::kQT + q) * 16 + c) * 2, kPitchQ);
#pragma unroll
          for (int t = 0; t < 4; ++t) dw[q][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(pf[t], qf, dw[q][t], 0, 0, 0);
        }
      }
    }
    convert();   // waits for the next turn's loads; this turn's stores come after, and drain meanwhile
    if (a.dx.p) {
      const int64_t row0 = int64_t(turn) * kRows;
      const int row = wave * 16 + r;
      const bool in = row < a.rows - row0;
      const uint32_t e = element_bytes(a.dx.type);
      const Buffer out = buffer_at(a.dx.p + row0 * a.dx.ld * e);
#pragma unroll
      for (int kc = 0; kc < KC; ++kc) {
        const int col = kc * 64 + g * 16;
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = acc[kc][i / 4][i % 4];
        if constexpr (HOW == kWhole) {
          const uint32_t off = in && col < a.k ? (row * uint32_t(a.dx.ld) + col) * e : kAbsent;
          if (a.dx.type == GS_MAT_F32) {
#pragma unroll
            for (int i = 0; i < 4; ++i) buffer_store16(out, off + i * 16, __builtin_bit_cast(u32x4, acc[kc][i]));
          } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float* o = v + 8 * i;
              buffer_store16(out, off + i * 16, u32x4{pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]),
                                                      pack_bf16(o[4], o[5]), pack_bf16(o[6], o[7])});
            }
          }
        } else if (in && col < a.k) {
          store8(a.dx, row0 + row, col, v, a.k - col);
          if (col + 8 < a.k) store8(a.dx, row0 + row, col + 8, v + 8, a.k - col - 8);
        }
      }
    }
  }

  if (a.want_dw) {
    float* out = a.part + (int64_t(blockIdx.x) * S::kMS + ms) * a.part_size;
#pragma unroll
    for (int q = 0; q < S::kQT; ++q) {
      const int n = (wq * S::kQT + q) * 16 + r;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int k = wp * 64 + t * 16 + g * 4;
        if (n >= a.n || k >= a.k) continue;
        float* o = out + n * a.k + k;
        if (k + 4 <= a.k) {
          __builtin_memcpy(__builtin_assume_aligned(o, 4), &dw[q][t], 16);
        } else {
          for (int i = 0; k + i < a.k; ++i) o[i] = dw[q][t][i];
        }
      }
    }
  }
  if (a.want_db) {
    // over the wave's 16 rows, then over the waves in order
    float* sums = reinterpret_cast<float*>(zt);   // [8][NC 64]
    __syncthreads();
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float t = sum_over16(db[c][i]);
        if (r == 0) sums[wave * NC * 64 + c * 64 + g * 16 + i] = t;
      }
    __syncthreads();
    for (int j = threadIdx.x; j < a.n; j += kThreads) {
      float t = 0.0f;
      for (int w = 0; w < 8; ++w) t += sums[w * NC * 64 + j];
      // the block's first part takes the sum, the others nothing
      float* out = a.part + int64_t(blockIdx.x) * S::kMS * a.part_size + int64_t(a.n) * a.k + j;
      for (int p = 0; p < S::kMS; ++p) out[p * a.part_size] = p ? 0.0f : t;
    }
  }
}

template <int NC, int KC, int DY, int Z, int X, Reach HOW>
hipError_t go(const RowsBwdArgs& a, int blocks, hipStream_t s) {
  constexpr size_t kLds = NC * KC * 8192 + size_t(kRows) * ((NC + KC) * 128 + 64);
  const auto kernel = &rows_bwd_kernel<NC, KC, DY, Z, X, HOW>;
  static LdsLimit limit;
  if (const hipError_t no = limit.allow(kernel, kLds); no != hipSuccess) return no;
  GSK_PROF("linear_rows_bwd", s);
  kernel<<<blocks, kThreads, kLds, s>>>(a);
  return hipGetLastError();
}

template <int NC, int KC, int DY, int Z, Reach HOW>
hipError_t by_x(const RowsBwdArgs& a, int blocks, hipStream_t s) {
  return a.x.type == GS_MAT_MX8 ? go<NC, KC, DY, Z, GS_MAT_MX8, HOW>(a, blocks, s)
                                : go<NC, KC, DY, Z, GS_MAT_BF16, HOW>(a, blocks, s);
}

template <int NC, int KC, int DY, Reach HOW>
hipError_t by_z(const RowsBwdArgs& a, int blocks, hipStream_t s) {
  if (a.act == GS_ACT_NONE) return by_x<NC, KC, DY, kNone, HOW>(a, blocks, s);
  return a.z.type == GS_MAT_MX8 ? by_x<NC, KC, DY, GS_MAT_MX8, HOW>(a, blocks, s)
                                : by_x<NC, KC, DY, GS_MAT_BF16, HOW>(a, blocks, s);
}

// Whole 16-column pieces in buffers' reach.
bool whole(const MatArg& dy, const MatArg& z, int act, const MatArg& x, const MatArg& dx, int k, int n) {
  return k % 16 == 0 && n % 16 == 0 && buffer_ok(dy) && buffer_ok(x) && buffer_ok(dx) &&
         (act == GS_ACT_NONE || buffer_ok(z));
}

// The types are compiled in, but for widths below 16, which take one kernel that reads them
// from the arguments; whole pieces have kernels of their own (500k rows 99 to 113 by the kernel
// for any type: 407 us, with the types compiled in 144; 128 to 128 with a float32 z 257 and 166).
template <int NC, int KC>
hipError_t by_type(const RowsBwdArgs& a, int blocks, hipStream_t s) {
  const bool f32 = a.dy.type == GS_MAT_F32;
  if (whole(a.dy, a.z, a.act, a.x, a.dx, a.k, a.n) && (a.act == GS_ACT_NONE || a.z.type != GS_MAT_F32))
    return f32 ? by_z<NC, KC, GS_MAT_F32, kWhole>(a, blocks, s) : by_z<NC, KC, GS_MAT_BF16, kWhole>(a, blocks, s);
  if constexpr (NC == 4) {   // without an activation, as rows_bwd_runs has it
    return f32 ? by_x<NC, KC, GS_MAT_F32, kNone, kHeldIn>(a, blocks, s)
               : by_x<NC, KC, GS_MAT_BF16, kNone, kHeldIn>(a, blocks, s);
  } else {
    if constexpr (NC == 1 || KC == 1) {
      if (a.k < 16 || a.n < 16) return go<NC, KC, kAny, kAny, kAny, kNarrow>(a, blocks, s);
    }
    if (a.act != GS_ACT_NONE && a.z.type == GS_MAT_F32)
      return f32 ? by_x<NC, KC, GS_MAT_F32, GS_MAT_F32, kHeldIn>(a, blocks, s)
                 : by_x<NC, KC, GS_MAT_BF16, GS_MAT_F32, kHeldIn>(a, blocks, s);
    return f32 ? by_z<NC, KC, GS_MAT_F32, kHeldIn>(a, blocks, s) : by_z<NC, KC, GS_MAT_BF16, kHeldIn>(a, blocks, s);
  }
}

// Blocks: one a turn with few rows; else as many as stay resident at once, each of at least
// two turns (a block's sums of dW cost about as much traffic as a turn).
int blocks_for(int64_t rows, int k, int n) {
  const int resident = k <= 64 && n <= 64 ? 512 : 256;
  const int64_t turns = (rows + kRows - 1) / kRows;
  const int64_t want = turns <= 128 ? turns : turns < 2 * resident ? (turns + 1) / 2 : resident;
  return int(want < 1 ? 1 : want);
}

int shares(int k, int n) { return k <= 64 && n <= 64 ? 2 : 1; }

}  // namespace

// Up to four tiles of 64 x 64 of dW (500k rows 256 to 64: 135 us without an activation, by dz, dx
// and dW in turn 170; 64 to 256: 96 and 167).  Inputs below 16 columns take the kernel for any
// type, whose registers do not hold four groups of dz (5 to 200: 618 us and 300).
bool rows_bwd_takes(int k, int n) {
  return (k <= 128 && n <= 128) || (k <= 256 && n <= 64) || (k >= 16 && k <= 64 && n <= 256);
}

// Four groups of dz with an activation beside dW's tiles are more than the registers hold.  In
// whole pieces with z in 8 or 16 bits the spills cost less than dz's way through memory (500k rows 64
// to 256, silu: 167-198 us, by dz, dx and dW in turn 263-291), moved pieces and a float32 z more
// (45 to 201: 302-354 us and 261-292; 64 to 256 with a float32 z 660 and 348).
bool rows_bwd_runs(const MatArg& dy, const MatArg& z, int act, const MatArg& x, const MatArg& dx, int k, int n) {
  return rows_bwd_takes(k, n) &&
         (n <= 128 || act == GS_ACT_NONE || (z.type != GS_MAT_F32 && whole(dy, z, act, x, dx, k, n)));
}

// No less than fewer rows take: the blocks are up to 128 for 128 turns and fall to 65 for one more.
size_t rows_bwd_ws_bytes(int64_t rows, int k, int n) {
  const int most = rows > 128 * kRows ? 128 : 0, blocks = blocks_for(rows, k, n);
  return size_t(blocks > most ? blocks : most) * shares(k, n) * (size_t(n) * k + n) * 4;
}

hipError_t launch_rows_bwd(const MatArg& dy, const MatArg& z, int act, const MatArg& x, const MatArg& w,
                           const MatArg& dx, const MatArg& dw, float* dbias, int64_t rows, int k, int n, void* ws,
                           hipStream_t s) {
  const int blocks = blocks_for(rows, k, n);
  const int64_t size = int64_t(n) * k + n;
  float* part = static_cast<float*>(ws);
  const RowsBwdArgs a{dy, z, x, w, dx, part, size, dw.p != nullptr, dbias != nullptr, rows, act, k, n};
  hipError_t e;
  if (n <= 64)
    e = k <= 64    ? by_type<1, 1>(a, blocks, s)
        : k <= 128 ? by_type<1, 2>(a, blocks, s)
                   : by_type<1, 4>(a, blocks, s);
  else if (n <= 128)
    e = k <= 64 ? by_type<2, 1>(a, blocks, s) : by_type<2, 2>(a, blocks, s);
  else
    e = by_type<4, 1>(a, blocks, s);
  if (e != hipSuccess || (!dw.p && !dbias)) return e;
  return launch_sum_parts(part, blocks * shares(k, n), size, int64_t(n) * k, k, dw, dbias, s);
}

}  // namespace gsk
