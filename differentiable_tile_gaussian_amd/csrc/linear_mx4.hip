// gs_linear_fwd with the weight in MX4: y = act(x W^T + b) + r.
//
// Operands are taken in steps of 128 k: lane l holds, of row l % 16, the block of 32 k that
// starts at 32 (l / 16), which is 16 bytes of MX4 and its scale byte.  With x in MX4 too a step is one
// 16x16x128 product of scaled 4-bit elements, whose sums are exact to float32's (4096 k of random
// codes: 5e-8 of the result, a float32 chain 8e-8).  x in bfloat16 or MX8 and the decoded weight
// are exact in bfloat16 and take four 16x16x32 products.  (The matrix cores' product of 8-bit
// with 4-bit elements is twice as fast, but it drops the low bits of what it adds: 4.5e-5 of the
// result, which an MX8 or float32 y would show.)
#include "linear.h"
#include "mx4.h"
#include "profile.h"

namespace gsk {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

__device__ inline i32x8 operand4(u32x4 q) {
  return i32x8{int(q[0]), int(q[1]), int(q[2]), int(q[3]), 0, 0, 0, 0};
}

__device__ inline f32x4 product4(u32x4 a, uint32_t a_scale, u32x4 b, uint32_t b_scale, f32x4 c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand4(a), operand4(b), c, 4, 4, 0, int(a_scale), 0, int(b_scale));
}

// A block of 32 k of a row in MX4.
struct Block4 {
  u32x4 q;
  uint32_t scale;
  // in: the row exists; n: how many of the block's k exist.  What does not exist is zero.
  __device__ void load(Buffer data, Buffer scales, uint32_t row, uint32_t pitch, uint32_t lds, bool in, int block, int n) {
    const bool there = in && n > 0;
    q = buffer_load16(data, there ? row * pitch + block * 16 : kAbsent);
    scale = buffer_load1(scales, there ? row * lds + block : kAbsent);
  }
  __device__ void keep(int n) { q = mx4_keep(q, n); }
  __device__ void operands(bf16x8 (&o)[4]) const {
    const float s = mx8_scale(scale);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = mx4_to_bf16x8(q[i], s);
  }
};

// The same of x: MX4, or two pieces of 16 k (matrix.h's Raw16).
template <int XT, bool NARROW>
struct BlockX {
  Raw16<XT, NARROW> a, b;
  __device__ void load(const MatArg& m, int64_t row, int k, int nk, bool live) {
    a.load(m, row, k, nk, live);
    if constexpr (NARROW)
      b = Raw16<XT, NARROW>{};
    else
      b.load(m, row, k + 16, nk, live);
  }
  __device__ void settle() {
    a.settle();
    if constexpr (!NARROW) b.settle();
  }
  __device__ static void half(const Raw16<XT, NARROW>& r, bf16x8& p, bf16x8& q) {
    if constexpr (XT == GS_MAT_MX8) {
      const float s = mx8_scale(r.scale);
      const u32x2 w0 = mx8_to_bf16x4(r.w[0], s), w1 = mx8_to_bf16x4(r.w[1], s);
      const u32x2 w2 = mx8_to_bf16x4(r.w[2], s), w3 = mx8_to_bf16x4(r.w[3], s);
      p = __builtin_bit_cast(bf16x8, u32x4{w0[0], w0[1], w1[0], w1[1]});
      q = __builtin_bit_cast(bf16x8, u32x4{w2[0], w2[1], w3[0], w3[1]});
    } else {
      p = __builtin_bit_cast(bf16x8, u32x4{r.w[0], r.w[1], r.w[2], r.w[3]});
      q = __builtin_bit_cast(bf16x8, u32x4{r.w[4], r.w[5], r.w[6], r.w[7]});
    }
  }
  __device__ void operands(bf16x8 (&o)[4]) const {
    half(a, o[0], o[1]);
    half(b, o[2], o[3]);
  }
};

// Any size and type.  A block of four waves takes 64 columns by 16 QT rows, the waves sharing
// the contraction; their sums are joined through LDS in order.
constexpr int kWaves = 4;

template <int XT, int QT, bool NARROW>
__global__ void __launch_bounds__(kWaves * 64) linear_mx4_kernel(MatArg W, MatArg X, int np, int64_t nq, int nk, Epilogue e) {
  constexpr bool kX4 = XT == GS_MAT_MX4;
  __shared__ f32x4 sums[kWaves * QT * 4 * 64];   // [wave][QT][tile][lane]
  const int lane = threadIdx.x % 64, g = lane / 16, r = lane % 16;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int p0 = blockIdx.y * 64;
  const int64_t q0 = int64_t(blockIdx.x) * (16 * QT);
  const uint32_t wp = uint32_t(mx4_pitch(W)), xp = kX4 ? uint32_t(mx4_pitch(X)) : 0u;
  const Buffer wb = buffer_at(W.p + int64_t(p0) * wp), ws = buffer_at(W.s + int64_t(p0) * W.lds);
  const Buffer xb = buffer_at(kX4 ? X.p + q0 * xp : nullptr), xs = buffer_at(kX4 ? X.s + q0 * X.lds : nullptr);
  f32x4 acc[QT][4];
#pragma unroll
  for (int i = 0; i < QT; ++i)
#pragma unroll
    for (int t = 0; t < 4; ++t) acc[i][t] = f32x4{0, 0, 0, 0};
  const int steps = (nk + 127) / 128;
  for (int s = wave; s < steps; s += kWaves) {
    const int block = s * 4 + g, left = nk - block * 32;
    Block4 w[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int row = r / 4 * 16 + t * 4 + r % 4;   // a lane's tiles: 16 consecutive columns
      w[t].load(wb, ws, row, wp, uint32_t(W.lds), p0 + row < np, block, left);
    }
    if constexpr (kX4) {
      Block4 x[QT];
#pragma unroll
      for (int i = 0; i < QT; ++i) {
        x[i].load(xb, xs, i * 16 + r, xp, uint32_t(X.lds), q0 + i * 16 + r < nq, block, left);
        x[i].keep(left);
      }
#pragma unroll
      for (int i = 0; i < QT; ++i)
#pragma unroll
        for (int t = 0; t < 4; ++t) acc[i][t] = product4(w[t].q, w[t].scale, x[i].q, x[i].scale, acc[i][t]);
    } else {
      bf16x8 wo[4][4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        w[t].keep(left);
        w[t].operands(wo[t]);
      }
#pragma unroll
      for (int i = 0; i < QT; ++i) {
        const int64_t row = q0 + i * 16 + r;
        BlockX<XT, NARROW> x;
        x.load(X, row < nq ? row : nq - 1, block * 32, nk, row < nq);
        x.settle();
        bf16x8 xo[4];
        x.operands(xo);
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int h = 0; h < 4; ++h) acc[i][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wo[t][h], xo[h], acc[i][t], 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < QT; ++i)
#pragma unroll
    for (int t = 0; t < 4; ++t) sums[((wave * QT + i) * 4 + t) * 64 + lane] = acc[i][t];
  __syncthreads();
  if (wave >= QT) return;
  const int64_t row = q0 + wave * 16 + r;
  const int col = p0 + g * 16, n = np - col < 16 ? np - col : 16;
  float v[16];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    f32x4 total = sums[(wave * 4 + t) * 64 + lane];
    for (int o = 1; o < kWaves; ++o) total += sums[((o * QT + wave) * 4 + t) * 64 + lane];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[4 * t + i] = total[i];
  }
#pragma unroll
  for (int j = 0; j < 16; ++j) v[j] += e.bias && j < n ? e.bias[col + j] : 0.0f;
  finish16<false, kNone, kAny>(e, row, col, v, row < nq ? n : 0);
}

template <int XT, bool NARROW>
hipError_t go(const MatArg& x, const MatArg& w, const Epilogue& e, int64_t rows, int k, int n, hipStream_t s) {
  const int64_t most = kMaxBlocks * 64;   // rows of one launch
  for (int64_t first = 0; first < rows; first += most) {
    const int64_t count = rows - first < most ? rows - first : most;
    Epilogue part = e;
    part.r = rows_from(e.r, first);
    part.y = rows_from(e.y, first);
    const MatArg xp = XT == GS_MAT_MX4 ? mx4_rows_from(x, first) : rows_from(x, first);
    linear_mx4_kernel<XT, 4, NARROW><<<dim3(div_up(count, 64), div_up(n, 64)), kWaves * 64, 0, s>>>(w, xp, n, count, k, part);
  }
  return hipGetLastError();
}

// ------------------------------------------------------------- both operands in MX4, by tiles

// Tiles of 128 columns by 32 QT rows, 64 x 16 QT for each of four waves, in steps of 128 k.  LDS holds
// the operands as the matrix cores take them: a fragment (16 rows, 128 k) is 1 KiB, 16 bytes a lane
// in the lanes' order, which is how a wave's load writes LDS without passing through registers.
// kStages steps are in LDS or on their way, so that a step's loads have two others' time; one
// barrier a step.  The scales of 16 steps are held beside them, four bytes a row and step, of which
// a lane reads its own.
constexpr int kTileThreads = 256, kStages = 4, kSegment = 16;

template <int QT>
struct TileLds {
  static constexpr int kP = 8, kQ = 2 * QT, kRows = 16 * (kP + kQ);
  uint8_t stage[kStages][(kP + kQ) * 1024];
  uint32_t scales[kSegment][kRows];
};

// A load of 16 bytes a lane from memory to LDS, at `to` (the same in all lanes) and 16 lane on.
__device__ inline void load_to_lds(Buffer from, uint32_t off, uint8_t* to) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (__attribute__((address_space(3))) void*)to, 16, int(off), 0, 0, 0);
}

// Waits until at most N of the wave's loads are on their way and its LDS operations are done, and
// for the other waves to have come as far.  (A fence would wait for all loads to LDS.)
template <int N>
__device__ inline void wait_loads_and_waves() {
  static_assert(N < 64, "six bits");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | (N >> 4) << 14 | 0x0070);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

template <int QT>
__global__ void __launch_bounds__(kTileThreads, 2) tile_mx4_kernel(MatArg W, MatArg X, int np, int64_t nq, int nk, Epilogue e,
                                                                    int ptiles, int tiles) {
  using Lds = TileLds<QT>;
  constexpr int BP = 128, BQ = 32 * QT, kP = Lds::kP, kQ = Lds::kQ, kLoads = (kP + kQ) / 4;
  extern __shared__ __align__(16) uint8_t lds_bytes[];
  Lds& lds = *reinterpret_cast<Lds*>(lds_bytes);
  const int tile = tile_of(blockIdx.x, tiles);
  if (tile >= tiles) return;
  const int p0 = tile % ptiles * BP;
  const int64_t q0 = int64_t(tile / ptiles) * BQ;
  const int lane = threadIdx.x % 64, g = lane / 16, r = lane % 16;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), wp = wave % 2, wq = wave / 2;
  const int blocks = (nk + 31) / 32, steps = (blocks + 3) / 4;
  const uint32_t wpitch = uint32_t(mx4_pitch(W)), xpitch = uint32_t(mx4_pitch(X));
  const Buffer wb = buffer_at(W.p + int64_t(p0) * wpitch), xb = buffer_at(X.p + q0 * xpitch);
  // a lane's four result tiles are 16 consecutive columns
  auto wrow = [](int f, int r) { return f / 4 * 64 + r / 4 * 16 + f % 4 * 4 + r % 4; };
  uint32_t off[kLoads];
#pragma unroll
  for (int u = 0; u < kLoads; ++u) {
    const int f = wave + 4 * u, row = f < kP ? wrow(f, r) : (f - kP) * 16 + r;
    const bool there = f < kP ? p0 + row < np : q0 + row < nq;
    off[u] = there ? row * (f < kP ? wpitch : xpitch) + g * 16 : kAbsent;
  }
  auto issue = [&](int s, int stage) {
    const bool in = s * 4 + g < blocks;
#pragma unroll
    for (int u = 0; u < kLoads; ++u)
      load_to_lds(u < kP / 4 ? wb : xb, in ? off[u] + s * 64 : kAbsent, lds.stage[stage] + (wave + 4 * u) * 1024);
  };
  // The thread's row of scales, 16 bytes (four steps) at a time.  Absent ones are zero, and 2^-127 takes
  // with it whatever LDS holds there.
  const int sf = threadIdx.x / 16, srow = sf < kP ? wrow(sf, r) : (sf - kP) * 16 + r;
  const bool has_scales = sf < kP ? p0 + srow < np : sf < kP + kQ && q0 + srow < nq;
  const uint8_t* scale_row = sf < kP ? W.s + (has_scales ? p0 + srow : 0) * W.lds : X.s + (has_scales ? q0 + srow : 0) * X.lds;
  u32x4 sr[kSegment / 4];
  auto load_scales = [&](int s0) {
#pragma unroll
    for (int j = 0; j < kSegment / 4; ++j) {
      const int at = (s0 + j * 4) * 4, n = blocks - at;
      sr[j] = u32x4{0, 0, 0, 0};
      if (n >= 16) {
        __builtin_memcpy(&sr[j], scale_row + at, 16);
      } else if (n > 0) {
        uint8_t byte[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) byte[i] = scale_row[at + (i < n ? i : 0)];
#pragma unroll
        for (int i = 0; i < 16; ++i) sr[j][i / 4] |= (i < n ? uint32_t(byte[i]) : 0u) << (8 * (i % 4));
      }
      if (!has_scales) sr[j] = u32x4{0, 0, 0, 0};
    }
  };
  auto put_scales = [&]() {
    if (sf < kP + kQ) {
#pragma unroll
      for (int j = 0; j < kSegment; ++j) lds.scales[j][threadIdx.x] = sr[j / 4][j % 4];
    }
  };
  f32x4 acc[QT][4];
#pragma unroll
  for (int i = 0; i < QT; ++i)
#pragma unroll
    for (int t = 0; t < 4; ++t) acc[i][t] = f32x4{0, 0, 0, 0};
  load_scales(0);
#pragma unroll
  for (int d = 0; d < kStages - 1; ++d) issue(d, d);
  put_scales();
  for (int s0 = 0; s0 < steps; s0 += kStages) {
    if (s0 > 0 && s0 % kSegment == 0) {   // the next steps' scales, when all waves are done with the others
      load_scales(s0);
      step_barrier();
      put_scales();
    }
#pragma unroll
    for (int d = 0; d < kStages; ++d) {
      const int s = s0 + d;
      if (s >= steps) break;
      wait_loads_and_waves<(kStages - 2) * kLoads>();
      const uint8_t* data = lds.stage[d] + lane * 16;
      const uint8_t* scales = reinterpret_cast<const uint8_t*>(lds.scales[s % kSegment]) + r * 4 + g;
      u32x4 wf[4], xf[QT];
      uint32_t wsc[4], xsc[QT];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        wf[t] = *reinterpret_cast<const u32x4*>(data + (wp * 4 + t) * 1024);
        wsc[t] = scales[(wp * 4 + t) * 64];
      }
#pragma unroll
      for (int i = 0; i < QT; ++i) {
        xf[i] = *reinterpret_cast<const u32x4*>(data + (kP + wq * QT + i) * 1024);
        xsc[i] = scales[(kP + wq * QT + i) * 64];
      }
      issue(s + kStages - 1, (d + kStages - 1) % kStages);   // always, so that the waits' count holds
      if (nk % 32 && s == steps - 1) {   // x ends inside a block (what the weight holds behind it meets zeros)
#pragma unroll
        for (int i = 0; i < QT; ++i) xf[i] = mx4_keep(xf[i], nk - (s * 4 + g) * 32);
      }
#pragma unroll
      for (int i = 0; i < QT; ++i)
#pragma unroll
        for (int t = 0; t < 4; ++t) acc[i][t] = product4(wf[t], wsc[t], xf[i], xsc[i], acc[i][t]);
    }
  }
  const int col = p0 + wp * 64 + g * 16, n = np - col < 16 ? np - col : 16;
  float bias[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) bias[j] = e.bias && j < n ? e.bias[col + j] : 0.0f;
#pragma unroll
  for (int i = 0; i < QT; ++i) {
    const int64_t row = q0 + (wq * QT + i) * 16 + r;
    float v[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = acc[i][j / 4][j % 4] + bias[j];
    finish16<false, kNone, kAny>(e, row, col, v, row < nq ? n : 0);
  }
  __builtin_amdgcn_s_waitcnt(0x0f70);   // a wave leaves no load to LDS behind
}

template <int QT>
hipError_t go_tiles(const MatArg& x, const MatArg& w, const Epilogue& e, int64_t rows, int k, int n, hipStream_t s) {
  const auto kernel = &tile_mx4_kernel<QT>;
  static LdsLimit limit;
  if (const hipError_t no = limit.allow(kernel, sizeof(TileLds<QT>)); no != hipSuccess) return no;
  const int ptiles = int(div_up(n, 128));
  const int64_t most = (kMaxBlocks - 8) / ptiles * (32 * QT);   // rows of one launch
  for (int64_t first = 0; first < rows; first += most) {
    const int64_t count = rows - first < most ? rows - first : most;
    Epilogue part = e;
    part.r = rows_from(e.r, first);
    part.y = rows_from(e.y, first);
    const int tiles = int(ptiles * int64_t(div_up(count, 32 * QT)));
    kernel<<<(tiles + 7) / 8 * 8, kTileThreads, sizeof(TileLds<QT>), s>>>(w, mx4_rows_from(x, first), n, count, k, part, ptiles, tiles);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_mx4(const MatArg& x, const MatArg& w, const float* bias, int act, const MatArg& r,
                             const MatArg& y, int64_t rows, int k, int n, hipStream_t s) {
  const Epilogue e{bias, act, r, MatArg{nullptr, nullptr, 0, 0, GS_MAT_F32}, y};
  if (rows_fwd_takes(k, n) && rows > 16) return launch_rows_mx4(x, w, e, rows, k, n, s);
  GSK_PROF("linear_mx4", s);
  const int64_t tiles = int64_t(div_up(n, 128)) * div_up(rows, 128);
  if (tiles > 64) {
    if (x.type != GS_MAT_MX4) return launch_tile_nt(w, x, n, rows, k, e, s);
    return tiles <= 256 ? go_tiles<2>(x, w, e, rows, k, n, s) : go_tiles<4>(x, w, e, rows, k, n, s);
  }
  if (x.type == GS_MAT_MX4) return go<GS_MAT_MX4, false>(x, w, e, rows, k, n, s);
  if (x.type == GS_MAT_MX8) return k < 16 ? go<GS_MAT_MX8, true>(x, w, e, rows, k, n, s) : go<GS_MAT_MX8, false>(x, w, e, rows, k, n, s);
  return k < 16 ? go<GS_MAT_BF16, true>(x, w, e, rows, k, n, s) : go<GS_MAT_BF16, false>(x, w, e, rows, k, n, s);
}

}  // namespace gsk
