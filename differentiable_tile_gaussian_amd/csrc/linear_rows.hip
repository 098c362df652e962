// Linear layers of narrow width over many rows (Gaussians): widths of at most 256, where a
// row's input and output are a few hundred bytes and the weight fits a compute unit's LDS.
// Bounded by HBM, so each row's operands go from memory straight into matrix-core operands
// in registers and each result from the accumulators to memory.
//
// Both operands are taken in pieces of 64 k in which lane group g = lane / 16 holds
// k = 16 g .. 16 g + 15 (two 16x16x32 products): 32 contiguous bytes of bfloat16 or 16 of MX8
// a lane, 128 or 64 a row.  The results come in groups of 64 columns, tile t holding the
// columns 16 g + 4 t + i, so that a lane's four tiles are 16 consecutive columns of one row:
// wide stores, and half an MX8 block.
//
// 1M rows 128 to 128 from MX8, silu, z kept in MX8: 116-132 us over runs (520 MB, 3.9-4.5
// TB/s; the same reads and writes alone 105 us: two write streams and a read stream, where a
// copy has one of each).
#include "linear.h"
#include "profile.h"

namespace gsk {
namespace {

// Piece kc of a row as loaded, and as two operands.
template <bool MX>
struct Piece;

template <>
struct Piece<false> {
  u32x4 a, b;
  __device__ void load(Buffer data, Buffer, uint32_t off, uint32_t, int kc) {
    a = buffer_load16(data, off + kc * 128);
    b = buffer_load16(data, off + kc * 128 + 16);
  }
  template <class R>
  __device__ void set(const R& r) {
    a = u32x4{r.w[0], r.w[1], r.w[2], r.w[3]};
    b = u32x4{r.w[4], r.w[5], r.w[6], r.w[7]};
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
  __device__ void load(Buffer data, Buffer scales, uint32_t off, uint32_t soff, int kc) {
    a = buffer_load16(data, off + kc * 64);
    scale = buffer_load1(scales, soff + kc * 2);
  }
  template <class R>
  __device__ void set(const R& r) {
    a = u32x4{r.w[0], r.w[1], r.w[2], r.w[3]};
    scale = r.scale;
  }
  __device__ void operands(bf16x8& p, bf16x8& q) const {
    const float s = mx8_scale(scale);
    const u32x2 w0 = mx8_to_bf16x4(a[0], s), w1 = mx8_to_bf16x4(a[1], s);
    const u32x2 w2 = mx8_to_bf16x4(a[2], s), w3 = mx8_to_bf16x4(a[3], s);
    p = __builtin_bit_cast(bf16x8, u32x4{w0[0], w0[1], w1[0], w1[1]});
    q = __builtin_bit_cast(bf16x8, u32x4{w2[0], w2[1], w3[0], w3[1]});
  }
};

// The block's part of W (nc groups of 64 columns from group c0) as operands, 1 KiB for each
// (column group, tile, piece, half), so that a read is 64 consecutive 16-byte words; and the
// bias.
// held: the last 16-column piece is taken from inside the row (as matrix.h's Raw16), so that
// its lanes compute, and write, 16 columns like all others.
template <int KC, int NC, int THREADS, bool NARROW>
__device__ inline void stage_weight(const MatArg& w, const float* bias, int k, int n, int c0, int nc, uint8_t* wl,
                                    float* bl, bool held) {
  // a unit: the 16 k of a lane's two operands; four of a thread's units in flight
  constexpr int kUnits = NC * KC * 256 / THREADS, kBatch = kUnits < 4 ? kUnits : 4;
  for (int f0 = threadIdx.x; f0 < nc * KC * 256; f0 += THREADS * kBatch) {
    Raw16<GS_MAT_BF16, NARROW> raw[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int f = f0 + u * THREADS, l = f % 64, kc = f / 64 % KC, t = f / (64 * KC) % 4, c = f / (256 * KC);
      int first = (c0 + c) * 64 + l % 16 / 4 * 16;
      if (held && first > n - 16) first = n - 16;
      const int row = first + t * 4 + l % 4;
      raw[u].load(w, row < n ? row : n - 1, kc * 64 + l / 16 * 16, k, row < n);
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int f = f0 + u * THREADS, l = f % 64, kc = f / 64 % KC, t = f / (64 * KC) % 4, c = f / (256 * KC);
      if (f >= nc * KC * 256) break;
      raw[u].settle();
      uint8_t* at = wl + (((c * 4 + t) * KC + kc) * 2) * 1024 + l * 16;
      const uint32_t* v = raw[u].w;
      *reinterpret_cast<u32x4*>(at) = u32x4{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<u32x4*>(at + 1024) = u32x4{v[4], v[5], v[6], v[7]};
    }
  }
  for (int j = threadIdx.x; j < nc * 64; j += blockDim.x) {
    int first = (c0 * 64 + j) / 16 * 16;
    if (held && first > n - 16) first = n - 16;
    bl[j] = bias && first + j % 16 < n ? bias[first + j % 16] : 0.0f;
  }
}

// One column group's sums for 16 MT rows.  The bias is added behind the products: sums that start
// from it lose its low bits in the matrix cores (400k rows 128 to 128: 1.6 times the error in small
// z, three times as many wrong roundings of z to 8 bits).  A tile's is added behind the next
// tile's products, which hide the wait for its own (1M rows 99 to 113: 142 us, behind its own
// products 167, all four at the end 146).  The weight does not change from turn
// to turn; the compiler must not see that, or it keeps all of it in registers it does not have
// (KEEP: it may).
template <int KC, int MT, bool KEEP>
__device__ inline void products(const uint8_t* wl, const float* bl, int c, int lane, const bf16x8 (&xf)[MT][KC][2],
                                f32x4 (&acc)[MT][4]) {
  if (!KEEP) asm volatile("" : "+v"(lane));
  auto add_bias = [&](int t) {
    const f32x4 b = *reinterpret_cast<const f32x4*>(bl + c * 64 + lane / 16 * 16 + t * 4);
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[m][t] += b;
  };
#pragma unroll
  for (int t = 0; t < 4; ++t) {
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[m][t] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int kc = 0; kc < KC; ++kc)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bf16x8 wf = *reinterpret_cast<const bf16x8*>(wl + (((c * 4 + t) * KC + kc) * 2 + h) * 1024 + lane * 16);
#pragma unroll
        for (int m = 0; m < MT; ++m)
          acc[m][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf, xf[m][kc][h], acc[m][t], 0, 0, 0);
      }
    if (t > 0) add_bias(t - 1);
  }
  add_bias(3);
}

__device__ inline void activate_any(float v[16], int act) {
  if (act == GS_ACT_SILU)
    activate16<GS_ACT_SILU>(v);
  else if (act == GS_ACT_GELU)
    activate16<GS_ACT_GELU>(v);
  else if (act == GS_ACT_RELU)
    activate16<GS_ACT_RELU>(v);
}

// Rows from row0 on, as far as a turn looks.
__device__ inline int rows_left(int64_t rows, int64_t row0) {
  const int64_t left = rows - row0;
  return left > 1024 ? 1024 : left < 0 ? 0 : int(left);
}

struct RowsArgs {
  MatArg x, w;
  Epilogue e;
  int64_t rows;
  int k, n;
};

// Rows taken in turns of 16 MT by each wave of the grid; a turn's loads are issued before the
// turn in front of it is computed.  The widths are multiples of 16 and every access goes
// through buffers (matrix.h): no branch is taken between a load and its use, so the waits are
// for the loads alone and the stores drain behind them.
// KC, NC: pieces of k and groups of columns.  MX: x is MX8.  Z: MX8 or kNone.  R: the
// residual's type or kNone.
template <int KC_, int NC_, bool MX_, int Z_, int Y_, int R_>
struct Shape {
  static constexpr int KC = KC_, NC = NC_, Z = Z_, Y = Y_, R = R_;
  static constexpr bool MX = MX_;
  static constexpr int kMT = KC <= 2 && KC * NC <= 4 && R == kNone ? 2 : 1;
  static constexpr int kThreads = KC * NC <= 4 ? 256 : KC * NC <= 8 ? 384 : 512;
  static constexpr int kWaves = KC * NC <= 8 ? 3 : 2;   // per SIMD
  static constexpr size_t kLds = NC * (KC * 8192 + 256);
};

template <class S>
__global__ void __launch_bounds__(S::kThreads, S::kWaves) rows_fwd_kernel(RowsArgs a) {
  constexpr int KC = S::KC, NC = S::NC, Z = S::Z, Y = S::Y, R = S::R, MT = S::kMT;
  constexpr bool MX = S::MX;
  extern __shared__ __align__(16) uint8_t lds[];
  float* bl = reinterpret_cast<float*>(lds + NC * KC * 8192);
  const int c0 = blockIdx.y * NC, col0 = c0 * 64;
  const int nc = (a.n + 63) / 64 - c0 < NC ? (a.n + 63) / 64 - c0 : NC;
  const int lane = threadIdx.x % 64, g = lane / 16, r = lane % 16;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int turns = int((a.rows + 16 * MT - 1) / (16 * MT)), step = gridDim.x * (S::kThreads / 64);
  int turn = blockIdx.x * (S::kThreads / 64) + wave;

  const uint32_t xp = uint32_t(a.x.ld) * (MX ? 1 : 2), xs = uint32_t(a.x.lds);
  Piece<MX> next[MT][KC];
  auto fetch = [&](int t) {
    const int64_t from = int64_t(__builtin_amdgcn_readfirstlane(t)) * (16 * MT);
    const Buffer data = buffer_at(a.x.p + from * xp), scales = buffer_at(MX ? a.x.s + from * xs : nullptr);
    const int left = rows_left(a.rows, from);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const bool in = m * 16 + r < left;
      const uint32_t off = (m * 16 + r) * xp + g * (MX ? 16 : 32), soff = (m * 16 + r) * xs + g / 2;
#pragma unroll
      for (int kc = 0; kc < KC; ++kc) {
        // the row ends in the last group of 64, or with four groups the one before it
        const bool there = in && (kc < KC / 2 || kc * 64 + g * 16 < a.k);
        next[m][kc].load(data, scales, there ? off : kAbsent, there ? soff : kAbsent, kc);
      }
    }
  };
  fetch(turn);
  stage_weight<KC, NC, S::kThreads, false>(a.w, a.e.bias, a.k, a.n, c0, nc, lds, bl, false);
  __syncthreads();
  bf16x8 xf[MT][KC][2];
  auto convert = [&]() {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int kc = 0; kc < KC; ++kc) next[m][kc].operands(xf[m][kc][0], xf[m][kc][1]);
  };
  convert();
  for (; turn < turns; turn += step) {
    const int64_t row0 = int64_t(__builtin_amdgcn_readfirstlane(turn)) * (16 * MT);
    const int left = rows_left(a.rows, row0);
    // where this turn's rows of the outputs lie; absent rows have no place
    constexpr int kY = element_bytes(Y), kR = R == kNone ? 1 : element_bytes(R);
    const Buffer yb = buffer_at(a.e.y.p + (row0 * a.e.y.ld + col0) * kY);
    const Buffer zb = buffer_at(Z == kNone ? nullptr : a.e.z.p + row0 * a.e.z.ld + col0);
    const Buffer sb = buffer_at(Z == kNone ? nullptr : a.e.z.s + row0 * a.e.z.lds + col0 / 32);
    const Buffer rb = buffer_at(R == kNone ? nullptr : a.e.r.p + (row0 * a.e.r.ld + col0) * kR);
    u32x4 res[MT][NC][R == GS_MAT_F32 ? 4 : 2];
    if (R != kNone) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const bool there = m * 16 + r < left && col0 + c * 64 + g * 16 < a.n;
          const uint32_t off = ((m * 16 + r) * uint32_t(a.e.r.ld) + c * 64 + g * 16) * kR;
#pragma unroll
          for (int i = 0; i < (R == GS_MAT_F32 ? 4 : 2); ++i)
            res[m][c][i] = buffer_load16(rb, there ? off + i * 16 : kAbsent);
        }
    }
    fetch(turn + step);   // past the last row: all absent
    // MX8 z of two column groups, written together: the halves of a 128-byte line written
    // microseconds apart leave the L2 one by one (1M rows of 128 with silu: 148 us, written
    // together 135)
    Mx8x16 zz[MT][2];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      f32x4 acc[MT][4];
      products<KC, MT, KC * NC == 1>(lds, bl, c, lane, xf, acc);
      const int col = c * 64 + g * 16;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const bool there = m * 16 + r < left && col0 + col < a.n;
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = acc[m][i / 4][i % 4];
        if (Z == GS_MAT_MX8) {
          zz[m][c % 2] = encode16(v);
          if (c % 2 || c == NC - 1) {
#pragma unroll
            for (int h = 0; h <= c % 2; ++h) {
              const int zc = (c - c % 2 + h) * 64 + g * 16;
              const bool at = m * 16 + r < left && col0 + zc < a.n;
              buffer_store16(zb, at ? (m * 16 + r) * uint32_t(a.e.z.ld) + zc : kAbsent, zz[m][h].q);
              buffer_store1(sb, at && g % 2 == 0 ? (m * 16 + r) * uint32_t(a.e.z.lds) + zc / 32 : kAbsent, zz[m][h].byte);
            }
          }
        }
        activate_any(v, a.e.act);
        if (R == GS_MAT_F32) {
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] += __uint_as_float(res[m][c][i / 4][i % 4]);
        } else if (R == GS_MAT_BF16) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            v[2 * i] += bf16_lo(res[m][c][i / 4][i % 4]);
            v[2 * i + 1] += bf16_hi(res[m][c][i / 4][i % 4]);
          }
        }
        const uint32_t off = ((m * 16 + r) * uint32_t(a.e.y.ld) + col) * kY;
        if (Y == GS_MAT_F32) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const f32x4 o{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
            buffer_store16(yb, there ? off + i * 16 : kAbsent, __builtin_bit_cast(u32x4, o));
          }
        } else {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float* o = v + 8 * i;
            buffer_store16(yb, there ? off + i * 16 : kAbsent,
                           u32x4{pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]), pack_bf16(o[4], o[5]),
                                 pack_bf16(o[6], o[7])});
          }
        }
      }
    }
    convert();   // the wait for the next turn's loads, behind this turn's stores
  }
}

// Any width, alignment and types: the same products, the pieces moved into place and the
// stores piece by piece.  1M rows 99 to 113 from bfloat16: 142 us (3.0 TB/s; from MX8 with silu
// and an MX8 z 203, 2.2 TB/s), 35 to 59 with a float32 y 120, 7 to 64 85, 300k rows 201 to 255
// 122: bounded by the vector work of moving pieces and by short stores that do not fill lines.
constexpr int kAnyThreads = 256;

template <int KC, bool MX, bool NARROW>
__global__ void __launch_bounds__(kAnyThreads) rows_fwd_any_kernel(RowsArgs a, int groups) {
  extern __shared__ __align__(16) uint8_t lds[];
  float* bl = reinterpret_cast<float*>(lds + size_t(groups) * KC * 8192);
  const int c0 = blockIdx.y * groups;
  const int nc = (a.n + 63) / 64 - c0 < groups ? (a.n + 63) / 64 - c0 : groups;
  // (not where y replaces the residual: a repeated column's residual would be gone)
  const bool held = a.n >= 16 && !(a.e.r.p && a.e.r.p == a.e.y.p);
  const int lane = threadIdx.x % 64, g = lane / 16, r = lane % 16;
  const int64_t step = int64_t(gridDim.x) * (kAnyThreads / 64) * 16;
  int64_t row0 = (int64_t(blockIdx.x) * (kAnyThreads / 64) + threadIdx.x / 64) * 16;
  Raw16<MX ? GS_MAT_MX8 : GS_MAT_BF16, NARROW> next[KC];
  auto fetch = [&](int64_t from) {
    const int64_t row = from + r;
#pragma unroll
    for (int kc = 0; kc < KC; ++kc)
      next[kc].load(a.x, row < a.rows ? row : a.rows - 1, kc * 64 + g * 16, a.k, row < a.rows);
  };
  fetch(row0);
  stage_weight<KC, 4, kAnyThreads, NARROW>(a.w, a.e.bias, a.k, a.n, c0, nc, lds, bl, held);
  __syncthreads();
  for (; row0 < a.rows; row0 += step) {
    const int64_t row = row0 + r;
    bf16x8 xf[1][KC][2];
#pragma unroll
    for (int kc = 0; kc < KC; ++kc) {
      Piece<MX> piece;
      // the row ends in the last group of 64, or with four groups the one before it; absent
      // rows' results go nowhere
      if (kc == KC - 1 || (KC == 4 && kc == 2)) next[kc].settle();
      piece.set(next[kc]);
      piece.operands(xf[0][kc][0], xf[0][kc][1]);
    }
    fetch(row0 + step);
    for (int c = 0; c < nc; ++c) {
      f32x4 acc[1][4];
      products<KC, 1, false>(lds, bl, c, lane, xf, acc);
      float v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = acc[0][i / 4][i % 4];
      const int col = (c0 + c) * 64 + g * 16, n = row < a.rows ? (a.n - col < 16 ? a.n - col : 16) : 0;
      if (!held) {
        finish16<false, kAny, kAny>(a.e, row, col, v, n);
        continue;
      }
      const int at = col < a.n - 16 ? col : a.n - 16, skip = col - at;
      if (a.e.z.p && a.e.z.type == GS_MAT_MX8) {
        // a block's columns have their places: the piece's own to its front
        float z[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) z[i] = v[i];
#pragma unroll
        for (int b = 8; b > 0; b /= 2)
#pragma unroll
          for (int i = 0; i < 16; ++i) z[i] = skip & b ? (i + b < 16 ? z[i + b] : 0.0f) : z[i];
        if (skip >= 16) {
#pragma unroll
          for (int i = 0; i < 16; ++i) z[i] = 0.0f;
        }
        store_mx8x16<false>(a.e.z, row, col, encode16(z), n);
      } else if (a.e.z.p && n > 0) {
        store16<true>(a.e.z, a.e.z.type, row, at, v, 16);
      }
      finish16<true, kNone, kAny>(a.e, row, at, v, n > 0 ? 16 : 0);
    }
  }
}

constexpr int kMaxLds = 132 << 10;

// Column groups per block: with few rows they go to blocks of their own.
int split_for(int64_t turns, int groups) { return turns * groups <= 512 ? groups : 1; }

int64_t blocks_for(int64_t turns, size_t lds, int most) {
  const int fit = int((160 << 10) / lds), resident = fit < most ? fit : most;
  return turns < 256 * resident ? turns : 256 * resident;
}

template <int KC, int NC, bool MX, int Z, int Y, int R>
hipError_t go(const RowsArgs& a, hipStream_t s) {
  using S = Shape<KC, NC, MX, Z, Y, R>;
  const auto kernel = &rows_fwd_kernel<S>;
  static LdsLimit limit;
  if (const hipError_t no = limit.allow(kernel, kMaxLds); no != hipSuccess) return no;
  const int64_t turns = div_up(a.rows, 16 * S::kMT * (S::kThreads / 64));
  GSK_PROF("linear_rows_fwd", s);
  kernel<<<dim3(unsigned(blocks_for(turns, S::kLds, S::kWaves * 256 / S::kThreads)), div_up(a.n, NC * 64)), S::kThreads,
           S::kLds, s>>>(a);
  return hipGetLastError();
}

template <int KC, int NC, bool MX>
hipError_t by_output(const RowsArgs& a, hipStream_t s) {
  const bool f32 = a.e.y.type == GS_MAT_F32;
  if (a.e.z.p) return go<KC, NC, MX, GS_MAT_MX8, GS_MAT_BF16, kNone>(a, s);
  if (a.e.r.p)
    return f32 ? go<KC, NC, MX, kNone, GS_MAT_F32, GS_MAT_F32>(a, s) : go<KC, NC, MX, kNone, GS_MAT_BF16, GS_MAT_BF16>(a, s);
  return f32 ? go<KC, NC, MX, kNone, GS_MAT_F32, kNone>(a, s) : go<KC, NC, MX, kNone, GS_MAT_BF16, kNone>(a, s);
}

template <int KC, int NC>
hipError_t by_input(const RowsArgs& a, hipStream_t s) {
  return a.x.type == GS_MAT_MX8 ? by_output<KC, NC, true>(a, s) : by_output<KC, NC, false>(a, s);
}

template <int KC>
hipError_t by_columns(const RowsArgs& a, hipStream_t s) {
  const int groups = (a.n + 63) / 64;
  if (split_for(div_up(a.rows, 128), groups) == groups) return by_input<KC, 1>(a, s);
  return groups <= 2 ? by_input<KC, 2>(a, s) : by_input<KC, 4>(a, s);
}

template <int KC, bool MX, bool NARROW>
hipError_t go_any(const RowsArgs& a, hipStream_t s) {
  static LdsLimit limit;
  if (const hipError_t no = limit.allow(&rows_fwd_any_kernel<KC, MX, NARROW>, kMaxLds); no != hipSuccess) return no;
  const int all = (a.n + 63) / 64;
  const int64_t turns = div_up(a.rows, 16 * (kAnyThreads / 64));
  const int split = split_for(turns, all), groups = (all + split - 1) / split;
  const size_t lds = size_t(groups) * (KC * 8192 + 256);
  GSK_PROF("linear_rows_fwd_any", s);
  rows_fwd_any_kernel<KC, MX, NARROW>
      <<<dim3(unsigned(blocks_for(turns, lds, 4)), split), kAnyThreads, lds, s>>>(a, groups);
  return hipGetLastError();
}

// The fast kernel's conditions: whole 16-column pieces, buffers, and one of the combinations
// of outputs that a network makes (a kept MX8 z, or a residual of y's type, or neither; by the
// kernel for any width 1M rows 128 to 128 take 167 us for 134, 199 for 143 and 119 for 106; 300k
// rows 256 to 256 100 for 80).  The others go to that kernel: each would be 18 more kernels, and
// takes 1.3 to 2.1 times its bytes at a copy's rate (a bfloat16 z 169 us and 119, an MX8 z and a
// residual 242 and 144, an MX8 z and a float32 y 303 and 144, a float32 residual and a bfloat16 y 246
// and 190).
bool fast(const RowsArgs& a) {
  const Epilogue& e = a.e;
  if (a.k % 16 || a.n % 16 || !buffer_ok(a.x) || !buffer_ok(e.y) || !buffer_ok(e.z) || !buffer_ok(e.r)) return false;
  if (e.z.p) return e.z.type == GS_MAT_MX8 && e.y.type == GS_MAT_BF16 && !e.r.p;
  return !e.r.p || e.r.type == e.y.type;
}

}  // namespace

bool rows_fwd_takes(int k, int n) { return k <= 256 && n <= 256; }

hipError_t launch_rows_fwd(const MatArg& x, const MatArg& w, const Epilogue& e, int64_t rows, int k, int n,
                           hipStream_t s) {
  const RowsArgs a{x, w, e, rows, k, n};
  const bool mx = x.type == GS_MAT_MX8;
  if (fast(a)) return k <= 64 ? by_columns<1>(a, s) : k <= 128 ? by_columns<2>(a, s) : by_columns<4>(a, s);
  if (k < 16) return mx ? go_any<1, true, true>(a, s) : go_any<1, false, true>(a, s);
  switch ((k + 63) / 64) {
    case 1: return mx ? go_any<1, true, false>(a, s) : go_any<1, false, false>(a, s);
    case 2: return mx ? go_any<2, true, false>(a, s) : go_any<2, false, false>(a, s);
    default: return mx ? go_any<4, true, false>(a, s) : go_any<4, false, false>(a, s);
  }
}

}  // namespace gsk
