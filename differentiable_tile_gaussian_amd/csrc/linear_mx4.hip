// gs_linear_fwd with the weight in MX4: y = act(x W^T + b) + r.
//
// Operands are taken in steps of 128 k: lane l holds, of row l % 16, the block of 32 k that
// starts at 32 (l / 16), which is 16 bytes of MX4 and its scale byte.  With x in MX4 too a step is one
// 16x16x128 product of scaled 4-bit elements, whose sums are exact to float32's (4096 k of random
// codes: 5e-8 of the result, a float32 chain 8e-8).  x in bfloat16 or MX8 and the decoded weight
// are exact in bfloat16 and take four 16x16x32 products.  (The matrix cores' product of 8-bit
// with 4-bit elements is twice as fast, but it drops the low bits of what it adds: 4.5e-5 of the
// result, which an MX8 or float32 y would show.)
#include <type_traits>

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

// run(x, epilogue, rows) for parts of at most `most` rows, which a launch takes.
template <class Run>
hipError_t in_parts(const MatArg& x, const Epilogue& e, int64_t rows, int64_t most, Run run) {
  for (int64_t first = 0; first < rows; first += most) {
    const int64_t count = rows - first < most ? rows - first : most;
    Epilogue part = e;
    part.r = rows_from(e.r, first);
    part.y = rows_from(e.y, first);
    const hipError_t no = run(x.type == GS_MAT_MX4 ? mx4_rows_from(x, first) : rows_from(x, first), part, count);
    if (no != hipSuccess) return no;
  }
  return hipSuccess;
}

// ------------------------------------------------------------- few rows, and any size and type

// A block takes 64 columns by 16 QT rows and its waves share the contraction, each loading its
// operands into registers one step ahead; the waves' sums are joined through LDS in order.  Bounded by
// latency: with few rows there is little to read but the weight (1 row 1024 to 1024: 6.2 us; 4096 to
// 4096, 8.9 MB: a call every 12 us; operands loaded when they are needed 20).
constexpr int waves_of(int qt) { return qt == 4 ? 4 : 8; }   // 64 KiB of sums at most

template <int XT, int QT, bool NARROW>
__global__ void __launch_bounds__(waves_of(QT) * 64) linear_mx4_kernel(MatArg W, MatArg X, int np, int64_t nq, int nk, Epilogue e) {
  constexpr bool kX4 = XT == GS_MAT_MX4;
  constexpr int kWaves = waves_of(QT);
  __shared__ f32x4 sums[kWaves * QT * 4 * 64];   // [wave][QT][tile][lane]
  const int lane = threadIdx.x % 64, g = lane / 16, r = lane % 16;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int p0 = blockIdx.y * 64;
  const int64_t q0 = int64_t(blockIdx.x) * (16 * QT);
  const uint32_t wp = uint32_t(mx4_pitch(W)), xp = kX4 ? uint32_t(mx4_pitch(X)) : 0u;
  const Buffer wb = buffer_at(W.p + int64_t(p0) * wp), ws = buffer_at(W.s + int64_t(p0) * W.lds);
  const Buffer xb = buffer_at(kX4 ? X.p + q0 * xp : nullptr), xs = buffer_at(kX4 ? X.s + q0 * X.lds : nullptr);
  const int steps = (nk + 127) / 128;
  Block4 w[4];
  std::conditional_t<kX4, Block4, BlockX<XT, NARROW>> x[QT];
  auto fetch = [&](int s) {   // past the end: the weight is absent
    const int block = s * 4 + g, left = nk - block * 32;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int row = r / 4 * 16 + t * 4 + r % 4;   // a lane's tiles: 16 consecutive columns
      w[t].load(wb, ws, row, wp, uint32_t(W.lds), p0 + row < np, block, left);
    }
#pragma unroll
    for (int i = 0; i < QT; ++i) {
      const int64_t row = q0 + i * 16 + r;
      if constexpr (kX4)
        x[i].load(xb, xs, i * 16 + r, xp, uint32_t(X.lds), row < nq, block, left);
      else
        x[i].load(X, row < nq ? row : nq - 1, block * 32, nk, row < nq);
    }
  };
  fetch(wave);
  float bias[16];
  const int col = p0 + g * 16, n = np - col < 16 ? np - col : 16;
  load_bias16(e.bias, col, wave < QT ? n : 0, bias);
  f32x4 acc[QT][4];
#pragma unroll
  for (int i = 0; i < QT; ++i)
#pragma unroll
    for (int t = 0; t < 4; ++t) acc[i][t] = f32x4{0, 0, 0, 0};
  for (int s = wave; s < steps; s += kWaves) {
    const int left = nk - (s * 4 + g) * 32;
    if constexpr (kX4) {
      u32x4 wq[4], xq[QT];
      uint32_t wsc[4], xsc[QT];
#pragma unroll
      for (int t = 0; t < 4; ++t) wq[t] = mx4_keep(w[t].q, left), wsc[t] = w[t].scale;
#pragma unroll
      for (int i = 0; i < QT; ++i) xq[i] = mx4_keep(x[i].q, left), xsc[i] = x[i].scale;
      fetch(s + kWaves);
#pragma unroll
      for (int i = 0; i < QT; ++i)
#pragma unroll
        for (int t = 0; t < 4; ++t) acc[i][t] = product4(wq[t], wsc[t], xq[i], xsc[i], acc[i][t]);
    } else {
      bf16x8 wo[4][4], xo[QT][4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        w[t].keep(left);
        w[t].operands(wo[t]);
      }
#pragma unroll
      for (int i = 0; i < QT; ++i) {
        x[i].settle();
        x[i].operands(xo[i]);
      }
      fetch(s + kWaves);
#pragma unroll
      for (int i = 0; i < QT; ++i)
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int h = 0; h < 4; ++h) acc[i][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wo[t][h], xo[i][h], acc[i][t], 0, 0, 0);
    }
  }
#pragma unroll
  for (int i = 0; i < QT; ++i)
#pragma unroll
    for (int t = 0; t < 4; ++t) sums[((wave * QT + i) * 4 + t) * 64 + lane] = acc[i][t];
  __syncthreads();
  if (wave >= QT) return;
  const int64_t row = q0 + wave * 16 + r;
  float v[16];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    f32x4 total = sums[(wave * 4 + t) * 64 + lane];
#pragma unroll
    for (int o = 1; o < kWaves; ++o) total += sums[((o * QT + wave) * 4 + t) * 64 + lane];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[4 * t + i] = total[i] + bias[4 * t + i];
  }
  finish16<false, kNone, kAny>(e, row, col, v, row < nq ? n : 0);
}

template <int XT, int QT, bool NARROW>
hipError_t go(const MatArg& x, const MatArg& w, const Epilogue& e, int64_t rows, int k, int n, hipStream_t s) {
  return in_parts(x, e, rows, kMaxBlocks / 2 * (16 * QT), [&](const MatArg& part, const Epilogue& to, int64_t count) {
    linear_mx4_kernel<XT, QT, NARROW>
        <<<dim3(div_up(count, 16 * QT), div_up(n, 64)), waves_of(QT) * 64, 0, s>>>(w, part, n, count, k, to);
    return hipGetLastError();
  });
}

// Rows of a block: 16 where there are no more, else as many as leave 128 blocks, half the card: a block
// of 64 rows reads the weight a quarter as often as one of 16, but with fewer blocks the card's reads are not
// all under way.
template <int XT, bool NARROW>
hipError_t by_rows(const MatArg& x, const MatArg& w, const Epilogue& e, int64_t rows, int k, int n, hipStream_t s) {
  const int64_t across = div_up(n, 64);
  if (rows <= 16 || across * div_up(rows, 32) < 128) return go<XT, 1, NARROW>(x, w, e, rows, k, n, s);
  return across * div_up(rows, 64) < 128 ? go<XT, 2, NARROW>(x, w, e, rows, k, n, s) : go<XT, 4, NARROW>(x, w, e, rows, k, n, s);
}

// ------------------------------------------------------------- by tiles, x in MX4 or MX8

// Tiles of 128 columns by 32 QT rows, 64 x 16 QT for each of four waves, in steps of 256 k (x in MX4)
// or 128 k (MX8): 128 bytes of a row, a line.  LDS holds the operands as they are in memory: a wave's
// load takes a line of eight rows and writes 1 KiB of LDS without passing through registers, the 16-byte
// pieces of a row permuted by its number so that a fragment's 16 rows are read from different
// banks.  (A load of 64 bytes of sixteen rows takes twice the time, 40 cycles of the address unit.)  x
// in MX8 and its weight are decoded to bfloat16 behind LDS, which moves a quarter to a half of
// the bytes that way.
//
// A block takes one tile after another, and its loads run ahead of its products by kStages - 1 steps, into
// the next tile too: what a tile costs beside its products is latency.  One barrier a step.
//
// Scales are four bytes a row and 128 k, of which a lane reads its own; they come through registers (any
// alignment), kParts of them at a time, into one of two places.
//
// 8160 rows 4096 to 1024 from MX8: 63 us (1090 TFLOP/s, the rate of the library's plain bfloat16
// product of these sizes); by the counters (in a short run, at 77 us) the matrix cores are busy in 40 % of the cycles
// and vector instructions, the decodes and theirs, issue in 39.  The weight of that form is still loaded 64 bytes of
// a row at a time.  8160 rows 1024 to 4096 from MX4 with gelu: 46 us (1.5 PFLOP/s), of which gelu takes 9 and the
// stores 6; without both and the loads 26 would be left, the steps' latency with two blocks a compute unit.  (In
// a short run, at 54 us: matrix cores 13 % of the cycles, vector issue 41, 22 instructions a wave and result.)
constexpr int kTileThreads = 256;

template <int XT, int QT_>
struct Tile {
  static constexpr bool kX4 = XT == GS_MAT_MX4;
  static constexpr int QT = QT_, BP = 128, BQ = 32 * QT, kP = BP / 16, kQ = BQ / 16;
  static constexpr int kSub = kX4 ? 2 : 1, kHalves = kX4 ? 1 : 2;   // 128 k parts of a step; 16-byte parts of a lane's 32 k
  static constexpr int kStages = kX4 ? 2 : 3, kParts = kX4 ? 4 : 2;
  static constexpr int kW = kP * kSub, kX = kQ * 2;   // KiB, and loads, of a step
  static constexpr int kLoads = (kW + kX) / 4;
  struct Lds {
    uint8_t stage[kStages][(kW + kX) * 1024];
    uint8_t scales[2][256][4 * kParts];   // 16 (kP + kQ) rows are used
    float bias[kStages][BP];   // of as many tiles as loads run ahead, where a tile is one step
  };
};

// Loads to LDS of 16 or 4 bytes a lane, from off + more on, to `to` (the same in all lanes) and on.
__device__ __forceinline__ void load16_to_lds(Buffer from, uint32_t off, int more, void* to) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (__attribute__((address_space(3))) void*)to, 16, int(off), more, 0, 0);
}
__device__ __forceinline__ void load4_to_lds(Buffer from, uint32_t off, int more, void* to) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (__attribute__((address_space(3))) void*)to, 4, int(off), more, 0, 0);
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

// The row of W whose products are row r of fragment f: a lane's four result tiles are 16 consecutive
// columns.
__device__ inline int weight_row(int f, int r) { return f / 4 * 64 + r / 4 * 16 + f % 4 * 4 + r % 4; }

template <class T>
__global__ void __launch_bounds__(kTileThreads, 2) tile_mx4_kernel(MatArg W, MatArg X, int np, int64_t nq, int nk, Epilogue e,
                                                                    int ptiles, int tiles) {
  constexpr int QT = T::QT, kP = T::kP, kQ = T::kQ, kH = T::kHalves, kSub = T::kSub, kStages = T::kStages, kParts = T::kParts;
  constexpr bool kX4 = T::kX4;
  constexpr int kAhead = (kStages - 2) * T::kLoads;   // loads on their way behind those of a step
  extern __shared__ __align__(16) uint8_t lds_bytes[];
  typename T::Lds& lds = *reinterpret_cast<typename T::Lds*>(lds_bytes);
  const int lane = threadIdx.x % 64, g = lane / 16, r = lane % 16;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), wp = wave % 2, wq = wave / 2;
  const int blocks = (nk + 31) / 32, parts = (blocks + 3) / 4, steps = (parts + kSub - 1) / kSub;
  const uint32_t wpitch = uint32_t(mx4_pitch(W)), xpitch = kX4 ? uint32_t(mx4_pitch(X)) : uint32_t(X.ld);
  // the block's tiles, by turns: tile_of gives an XCD neighbouring ones
  const int turns = (tiles + 7) / 8 * 8;
  auto valid_from = [&](int turn) {
    while (turn < turns && tile_of(turn, tiles) >= tiles) turn += gridDim.x;
    return turn;
  };

  // ---- loads to LDS, for step `step` of the tile of turn `ahead`: of a wave's kW / 4 and kX / 4 KiB; with a
  // tile's first step its bias.  A line's lanes: row lane / 8 of eight, and of it piece lane % 8 ^ row.
  const int row8 = lane / 8, piece = (lane % 8) ^ row8;
  int ahead = valid_from(blockIdx.x), step = 0, to = 0, bias_to = 0;
  Buffer wb = buffer_at(nullptr), xb = buffer_at(nullptr);
  uint32_t woff[T::kW / 4], xoff[T::kX / 4], boff = kAbsent;
  const Buffer bb = buffer_at(e.bias);
  auto point = [&]() {
    const bool there = ahead < turns;
    const int tile = there ? tile_of(ahead, tiles) : 0, p0 = tile % ptiles * T::BP;
    const int64_t q0 = int64_t(tile / ptiles) * T::BQ;
    wb = buffer_at(W.p + int64_t(p0) * wpitch);
    xb = buffer_at(X.p + q0 * xpitch);
#pragma unroll
    for (int j = 0; j < T::kW / 4; ++j) {
      const int unit = wave * (T::kW / 4) + j;
      const int row = kSub == 2 ? weight_row(unit / 2, unit % 2 * 8 + row8) : weight_row(unit, r);
      woff[j] = there && p0 + row < np ? row * wpitch + (kSub == 2 ? piece : g) * 16 : kAbsent;
    }
#pragma unroll
    for (int j = 0; j < T::kX / 4; ++j) {
      const int row = (wave * (T::kX / 4) + j) * 8 + row8;
      xoff[j] = there && q0 + row < nq ? row * xpitch + piece * 16 : kAbsent;
    }
    const int c = p0 + int(threadIdx.x) % T::BP;
    boff = there && e.bias && c < np ? c * 4 : kAbsent;
  };
  // The same number of loads every time, so that the waits' count holds.
  auto issue = [&]() {
    if (step == 0) {   // (one more on its way only makes the waits longer; the upper waves write the same)
      load4_to_lds(bb, boff, 0, lds.bias[bias_to] + wave % 2 * 64);
      bias_to = bias_to + 1 < kStages ? bias_to + 1 : 0;
    }
    uint8_t *wto = lds.stage[to] + wave * (T::kW / 4) * 1024, *xto = lds.stage[to] + (T::kW + wave * (T::kX / 4)) * 1024;
    bool w_in = true, x_in = true;
    if ((step + 1) * (128 * kSub) > nk) {   // the last step: pieces that exist
      w_in = (step * kSub) * 4 + (kSub == 2 ? piece : g) < blocks;
      x_in = kX4 ? w_in : step * 128 + piece * 16 < nk;
    }
#pragma unroll
    for (int j = 0; j < T::kW / 4; ++j) load16_to_lds(wb, w_in ? woff[j] : kAbsent, step * 64 * kSub, wto + j * 1024);
#pragma unroll
    for (int j = 0; j < T::kX / 4; ++j) load16_to_lds(xb, x_in ? xoff[j] : kAbsent, step * 128, xto + j * 1024);
    to = to + 1 < kStages ? to + 1 : 0;
    if (++step == steps) {
      step = 0;
      ahead = valid_from(ahead + gridDim.x);
      point();
    }
  };

  // ---- scales: the thread's row, kParts words at a time.  Absent ones are zero.
  const int sf = threadIdx.x / 16, srow = sf < kP ? weight_row(sf, r) : (sf - kP) * 16 + r;
  uint32_t sr[kParts];
  auto load_scales = [&](int turn, int part) {
    if (turn >= turns) return;
    const int tile = tile_of(turn, tiles), p0 = tile % ptiles * T::BP;
    const int64_t q0 = int64_t(tile / ptiles) * T::BQ;
    const bool there = sf < kP ? p0 + srow < np : sf < kP + kQ && q0 + srow < nq;
    const uint8_t* row = sf < kP ? W.s + (there ? p0 + srow : 0) * W.lds : X.s + (there ? q0 + srow : 0) * X.lds;
    const int at = part * 4, n = blocks - at;
    if (n >= 4 * kParts) {
      __builtin_memcpy(sr, row + at, 4 * kParts);
    } else {
      uint8_t byte[4 * kParts];
#pragma unroll
      for (int i = 0; i < 4 * kParts; ++i) byte[i] = row[at + (i < n ? i : 0)];
#pragma unroll
      for (int j = 0; j < kParts; ++j) {
        sr[j] = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) sr[j] |= (4 * j + i < n ? uint32_t(byte[4 * j + i]) : 0u) << (8 * i);
      }
    }
#pragma unroll
    for (int j = 0; j < kParts; ++j) sr[j] = there ? sr[j] : 0;
  };
  auto put_scales = [&](int half) { __builtin_memcpy(__builtin_assume_aligned(lds.scales[half][threadIdx.x], 4 * kParts), sr, 4 * kParts); };

  int turn = ahead, now = 0, half = 0, bias_at = 0;
  bool stores = false;   // the epilogue in front of this step has made all its stores
  static_assert(stores16(GS_MAT_MX8) == stores16(GS_MAT_BF16), "one wait for both");
  const bool f32 = e.y.type == GS_MAT_F32;
  load_scales(turn, 0);
  point();
#pragma unroll
  for (int d = 0; d < kStages - 1; ++d) issue();
  put_scales(0);
  while (turn < turns) {
    const int tile = tile_of(turn, tiles), p0 = tile % ptiles * T::BP, next = valid_from(turn + gridDim.x);
    const int64_t q0 = int64_t(tile / ptiles) * T::BQ;
    f32x4 acc[QT][4];
#pragma unroll
    for (int i = 0; i < QT; ++i)
#pragma unroll
      for (int t = 0; t < 4; ++t) acc[i][t] = f32x4{0, 0, 0, 0};
    constexpr int kSegment = kParts / kSub;   // steps
    for (int s0 = 0; s0 < steps; s0 += kSegment) {
      if (s0 + kSegment < steps)
        load_scales(turn, (s0 + kSegment) * kSub);
      else
        load_scales(next, 0);
      const int last = s0 + kSegment < steps ? s0 + kSegment : steps;
      for (int s = s0; s < last; ++s) {
        // the stores are younger than the loads that this step needs; memory operations end in order
        if (!stores)
          wait_loads_and_waves<kAhead>();
        else if (f32)
          wait_loads_and_waves<kAhead + stores16(GS_MAT_F32) * QT>();
        else
          wait_loads_and_waves<kAhead + stores16(GS_MAT_BF16) * QT>();
        stores = false;
        issue();
        const uint8_t* wdata = lds.stage[now] + wp * (4 * kSub * 1024);
        const uint8_t* xdata = lds.stage[now] + (T::kW + wq * (QT * 2)) * 1024 + r * 128;
        const uint8_t* wscale = lds.scales[half][wp * 64 + r] + (s - s0) * kSub * 4 + g;
        const uint8_t* xscale = lds.scales[half][kP * 16 + wq * (QT * 16) + r] + (s - s0) * kSub * 4 + g;
        now = now + 1 < kStages ? now + 1 : 0;
        u32x4 wf[kSub][4], xf[kSub][QT][kH];
        uint32_t wsc[kSub][4], xsc[kSub][QT];
#pragma unroll
        for (int sub = 0; sub < kSub; ++sub) {
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const int at = kSub == 2 ? r * 128 + ((sub * 4 + g) ^ (r & 7)) * 16 : lane * 16;
            wf[sub][t] = *reinterpret_cast<const u32x4*>(wdata + t * (kSub * 1024) + at);
            wsc[sub][t] = wscale[sub * 4 + t * (64 * kParts)];
          }
#pragma unroll
          for (int i = 0; i < QT; ++i) {
#pragma unroll
            for (int h = 0; h < kH; ++h)
              xf[sub][i][h] = *reinterpret_cast<const u32x4*>(xdata + i * 2048 + ((kX4 ? sub * 4 + g : g * 2 + h) ^ (r & 7)) * 16);
            xsc[sub][i] = xscale[sub * 4 + i * (64 * kParts)];
          }
        }
        if (nk % 128 && s == steps - 1) {   // the rows end inside (with zeros alone in x, an infinity behind W's end would count)
#pragma unroll
          for (int sub = 0; sub < kSub; ++sub) {
            const int left = nk - ((s * kSub + sub) * 4 + g) * 32;
#pragma unroll
            for (int t = 0; t < 4; ++t) wf[sub][t] = mx4_keep(wf[sub][t], left);
#pragma unroll
            for (int i = 0; i < QT; ++i) {
              if constexpr (kX4) {
                xf[sub][i][0] = mx4_keep(xf[sub][i][0], left);
              } else {
#pragma unroll
                for (int h = 0; h < kH; ++h) xf[sub][i][h] = left > h * 16 ? xf[sub][i][h] : u32x4{0, 0, 0, 0};
              }
            }
          }
        }
#pragma unroll
        for (int sub = 0; sub < kSub; ++sub) {
          if (sub > 0 && s * kSub + sub >= parts) break;
          if constexpr (kX4) {
#pragma unroll
            for (int i = 0; i < QT; ++i)
#pragma unroll
              for (int t = 0; t < 4; ++t) acc[i][t] = product4(wf[sub][t], wsc[sub][t], xf[sub][i][0], xsc[sub][i], acc[i][t]);
          } else {
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              bf16x8 wo[4], xo[QT];
#pragma unroll
              for (int t = 0; t < 4; ++t) wo[t] = mx4_to_bf16x8(wf[sub][t][h], mx8_scale(wsc[sub][t]));
#pragma unroll
              for (int i = 0; i < QT; ++i) {
                const float sc = mx8_scale(xsc[sub][i]);
                const u32x4 raw = xf[sub][i][h / 2];
                const u32x2 a = mx8_to_bf16x4(raw[h % 2 * 2], sc), b = mx8_to_bf16x4(raw[h % 2 * 2 + 1], sc);
                xo[i] = __builtin_bit_cast(bf16x8, u32x4{a[0], a[1], b[0], b[1]});
              }
#pragma unroll
              for (int i = 0; i < QT; ++i)
#pragma unroll
                for (int t = 0; t < 4; ++t) acc[i][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wo[t], xo[i], acc[i][t], 0, 0, 0);
            }
          }
        }
      }
      half ^= 1;
      put_scales(half);   // last read a segment ago, and all waves have met since
    }
    const int col = p0 + wp * 64 + g * 16, n = np - col < 16 ? np - col : 16;
    float bias[16];
    const f32x4* from = reinterpret_cast<const f32x4*>(lds.bias[bias_at] + wp * 64 + g * 16);
    const int biases = e.bias ? n : 0;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const f32x4 b = from[t];
#pragma unroll
      for (int j = 0; j < 4; ++j) bias[4 * t + j] = 4 * t + j < biases ? b[j] : 0.0f;
    }
    bias_at = bias_at + 1 < kStages ? bias_at + 1 : 0;
#pragma unroll
    for (int i = 0; i < QT; ++i) {
      const int64_t row = q0 + (wq * QT + i) * 16 + r;
      float v[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = acc[i][j / 4][j % 4] + bias[j];
      if (n < 16) {   // absent columns are what LDS held, and a block in MX8 takes them for zero
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = j < n ? v[j] : 0.0f;
      }
      finish16<false, kNone, kAny>(e, row, col, v, row < nq ? n : 0);
    }
    stores = p0 + T::BP <= np && q0 + T::BQ <= nq;
    turn = next;
  }
  __builtin_amdgcn_s_waitcnt(0x0f70);   // a wave leaves no load to LDS behind
}

template <int XT, int QT>
hipError_t go_tiles(const MatArg& x, const MatArg& w, const Epilogue& e, int64_t rows, int k, int n, hipStream_t s) {
  using T = Tile<XT, QT>;
  const auto kernel = &tile_mx4_kernel<T>;
  static LdsLimit limit;
  if (const hipError_t no = limit.allow(kernel, sizeof(typename T::Lds)); no != hipSuccess) return no;
  const int ptiles = int(div_up(n, 128));
  return in_parts(x, e, rows, (kMaxBlocks - 8) / ptiles * T::BQ, [&](const MatArg& part, const Epilogue& to, int64_t count) {
    const int tiles = int(ptiles * int64_t(div_up(count, T::BQ))), turns = (tiles + 7) / 8 * 8;
    kernel<<<turns < 512 ? turns : 512, kTileThreads, sizeof(typename T::Lds), s>>>(w, part, n, count, k, to, ptiles, tiles);
    return hipGetLastError();
  });
}

// Tiles of 64 rows where those of 128 would be one a compute unit or fewer (1000 rows 4096 to 4096 from
// MX4, 256 tiles: 23 us), else of 128, which reads the weight half as often.
template <int XT>
hipError_t by_tiles(const MatArg& x, const MatArg& w, const Epilogue& e, int64_t rows, int k, int n, hipStream_t s) {
  return int64_t(div_up(n, 128)) * div_up(rows, 128) <= 256 ? go_tiles<XT, 2>(x, w, e, rows, k, n, s)
                                                           : go_tiles<XT, 4>(x, w, e, rows, k, n, s);
}

}  // namespace

hipError_t launch_linear_mx4(const MatArg& x, const MatArg& w, const float* bias, int act, const MatArg& r,
                             const MatArg& y, int64_t rows, int k, int n, hipStream_t s) {
  const Epilogue e{bias, act, r, MatArg{nullptr, nullptr, 0, 0, GS_MAT_F32}, y};
  if (rows_fwd_takes(k, n) && rows > 16) return launch_rows_mx4(x, w, e, rows, k, n, s);
  GSK_PROF("linear_mx4", s);
  const int64_t tiles = int64_t(div_up(n, 128)) * div_up(rows, 128);
  // up to 64 tiles leave most of the card idle (700 rows 4096 to 1024 from MX8, 48 tiles: 28 us, by
  // tiles 31; 700 rows 1024 to 4096, 192 tiles, 16 us)
  if (tiles > 64) {
    if (x.type == GS_MAT_MX4) return by_tiles<GS_MAT_MX4>(x, w, e, rows, k, n, s);
    if (x.type == GS_MAT_MX8 && k % 16 == 0 && buffer_ok(x)) return by_tiles<GS_MAT_MX8>(x, w, e, rows, k, n, s);
    return in_parts(x, e, rows, (kMaxBlocks - 8) / div_up(n, 128) * 64,
                    [&](const MatArg& part, const Epilogue& to, int64_t count) { return launch_tile_nt(w, part, n, count, k, to, s); });
  }
  if (x.type == GS_MAT_MX4) return by_rows<GS_MAT_MX4, false>(x, w, e, rows, k, n, s);
  if (x.type == GS_MAT_MX8)
    return k < 16 ? by_rows<GS_MAT_MX8, true>(x, w, e, rows, k, n, s) : by_rows<GS_MAT_MX8, false>(x, w, e, rows, k, n, s);
  return k < 16 ? by_rows<GS_MAT_BF16, true>(x, w, e, rows, k, n, s) : by_rows<GS_MAT_BF16, false>(x, w, e, rows, k, n, s);
}

}  // namespace gsk
