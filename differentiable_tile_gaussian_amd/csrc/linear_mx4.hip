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
  float bias[16];
  load_bias16(e.bias, col, n, bias);
#pragma unroll
  for (int j = 0; j < 16; ++j) v[j] += bias[j];
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

// ------------------------------------------------------------- by tiles, x in MX4 or MX8

// Tiles of 128 columns by 32 QT rows, 64 x 16 QT for each of four waves, in steps of 128 k.  LDS holds
// the operands as they are in memory, in the order in which lanes take them: a fragment (16 rows,
// 128 k) of MX4 is 1 KiB, 16 bytes a lane, one of MX8 two such halves, which is also how a wave's load
// writes LDS without passing through registers.  x in MX8 and its weight are decoded to bfloat16
// behind LDS, which moves a quarter to a half of the bytes that way.
//
// A block takes one tile after another, and its loads run ahead of its products by kStages - 1 steps, into
// the next tile too: what a tile costs beside its products is latency (with a block to a tile, 8
// steps of which the loads and products take 7 us take 25).  One barrier a step.
//
// Scales are four bytes a row and step, of which a lane reads its own.  ALIGNED: they are whole
// aligned words and come with their step; otherwise through registers, kSegment steps at a time.
constexpr int kTileThreads = 256;

template <int XT, int QT_, bool ALIGNED_>
struct Tile {
  static constexpr bool kX4 = XT == GS_MAT_MX4, ALIGNED = ALIGNED_;
  static constexpr int QT = QT_, BP = 128, BQ = 32 * QT, kP = BP / 16, kQ = BQ / 16, kHalves = kX4 ? 1 : 2;
  static constexpr int kUnits = kP + kQ * kHalves, kLoads = kUnits / 4, kRows = 256;
  static constexpr int kStages = kX4 ? 4 : 3, kSegment = 4;
  struct Lds {
    uint8_t stage[kStages][kUnits * 1024];
    uint32_t scales[ALIGNED ? kStages : 2 * kSegment][kRows];   // 16 (kP + kQ) rows are used
    float bias[kStages][BP];   // of as many tiles as loads run ahead, where a tile is one step
  };
};

// A load of 16 bytes a lane from memory to LDS, at `to` (the same in all lanes) and 16 lane on.
__device__ inline void load_to_lds(Buffer from, uint32_t off, uint8_t* to) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (__attribute__((address_space(3))) void*)to, 16, int(off), 0, 0, 0);
}
__device__ inline void load_words_to_lds(Buffer from, uint32_t off, void* to) {   // 4 bytes a lane
  __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (__attribute__((address_space(3))) void*)to, 4, int(off), 0, 0, 0);
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

template <class T, int XT>
__global__ void __launch_bounds__(kTileThreads, 2) tile_mx4_kernel(MatArg W, MatArg X, int np, int64_t nq, int nk, Epilogue e,
                                                                    int ptiles, int tiles) {
  constexpr int QT = T::QT, kP = T::kP, kQ = T::kQ, kH = T::kHalves, kLoads = T::kLoads, kStages = T::kStages, kSegment = T::kSegment;
  constexpr bool kX4 = T::kX4, ALIGNED = T::ALIGNED;
  constexpr int kAhead = (kStages - 2) * (kLoads + ALIGNED);   // loads on their way behind those of a step
  extern __shared__ __align__(16) uint8_t lds_bytes[];
  typename T::Lds& lds = *reinterpret_cast<typename T::Lds*>(lds_bytes);
  const int lane = threadIdx.x % 64, g = lane / 16, r = lane % 16;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), wp = wave % 2, wq = wave / 2;
  const int blocks = (nk + 31) / 32, steps = (blocks + 3) / 4;
  const uint32_t wpitch = uint32_t(mx4_pitch(W)), xpitch = kX4 ? uint32_t(mx4_pitch(X)) : uint32_t(X.ld);
  // the block's tiles, by turns: tile_of gives an XCD neighbouring ones
  const int turns = (tiles + 7) / 8 * 8;
  auto valid_from = [&](int turn) {
    while (turn < turns && tile_of(turn, tiles) >= tiles) turn += gridDim.x;
    return turn;
  };

  // ---- loads to LDS: unit wave + 4 u of step `step` of the tile of turn `ahead`, and the thread's word of
  // scales (a wave's are all of W or all of x); with a tile's first step its bias
  const int sf = threadIdx.x / 16, srow = sf < kP ? weight_row(sf, r) : (sf - kP) * 16 + r;
  const bool of_w = wave < kP / 4;
  int ahead = valid_from(blockIdx.x), step = 0, to = 0, bias_to = 0;
  Buffer wb = buffer_at(nullptr), xb = buffer_at(nullptr), sb = buffer_at(nullptr);
  uint32_t off[kLoads], soff = kAbsent, boff = kAbsent;
  const Buffer bb = buffer_at(e.bias);
  int most[kLoads];    // steps in which the lane's 16 bytes exist
#pragma unroll
  for (int u = 0; u < kLoads; ++u) {
    const bool is_w = u < kP / 4;
    const int f = wave + 4 * u, k0 = is_w ? g * 32 : g * 32 + (f - kP) % kH * 16, n = is_w || kX4 ? blocks * 32 : nk;
    most[u] = (n - k0 + 127) / 128;
  }
  auto point = [&]() {
    const bool there = ahead < turns;
    const int tile = there ? tile_of(ahead, tiles) : 0, p0 = tile % ptiles * T::BP;
    const int64_t q0 = int64_t(tile / ptiles) * T::BQ;
    wb = buffer_at(W.p + int64_t(p0) * wpitch);
    xb = buffer_at(X.p + q0 * xpitch);
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const int f = wave + 4 * u;
      if (u < kP / 4) {
        const int row = weight_row(f, r);
        off[u] = there && p0 + row < np ? row * wpitch + g * 16 : kAbsent;
      } else {
        const int row = (f - kP) / kH * 16 + r;
        off[u] = there && q0 + row < nq ? row * xpitch + g * 16 * kH + (f - kP) % kH * 16 : kAbsent;
      }
    }
    if constexpr (ALIGNED) {
      sb = buffer_at(of_w ? W.s + p0 * W.lds : X.s + q0 * X.lds);
      const bool row = of_w ? p0 + srow < np : sf < kP + kQ && q0 + srow < nq;
      soff = there && row ? srow * uint32_t(of_w ? W.lds : X.lds) : kAbsent;
    }
    const int c = p0 + int(threadIdx.x) % T::BP;
    boff = there && e.bias && c < np ? c * 4 : kAbsent;
  };
  auto issue = [&]() {   // always, so that the waits' count holds
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const uint32_t at = off[u] + step * (u < kP / 4 ? 64 : 64 * kH);
      load_to_lds(u < kP / 4 ? wb : xb, step < most[u] ? at : kAbsent, lds.stage[to] + (wave + 4 * u) * 1024);
    }
    if constexpr (ALIGNED) load_words_to_lds(sb, step * 4 < blocks ? soff + step * 4 : kAbsent, lds.scales[to] + wave * 64);
    if (step == 0) {   // (one more on its way only makes the waits longer; the upper waves write the same)
      load_words_to_lds(bb, boff, lds.bias[bias_to] + wave % 2 * 64);
      bias_to = bias_to + 1 < kStages ? bias_to + 1 : 0;
    }
    to = to + 1 < kStages ? to + 1 : 0;
    if (++step == steps) {
      step = 0;
      ahead = valid_from(ahead + gridDim.x);
      point();
    }
  };

  // ---- scales of any alignment: the thread's row, 16 bytes (four steps) at a time.  Absent ones are zero.
  u32x4 sr[kSegment / 4];
  auto load_scales = [&](int turn, int s0) {
    if (ALIGNED || turn >= turns) return;
    const int tile = tile_of(turn, tiles), p0 = tile % ptiles * T::BP;
    const int64_t q0 = int64_t(tile / ptiles) * T::BQ;
    const bool there = sf < kP ? p0 + srow < np : sf < kP + kQ && q0 + srow < nq;
    const uint8_t* row = sf < kP ? W.s + (there ? p0 + srow : 0) * W.lds : X.s + (there ? q0 + srow : 0) * X.lds;
#pragma unroll
    for (int j = 0; j < kSegment / 4; ++j) {
      const int at = (s0 + j * 4) * 4, n = blocks - at;
      sr[j] = u32x4{0, 0, 0, 0};
      if (n >= 16) {
        __builtin_memcpy(&sr[j], row + at, 16);
      } else if (n > 0) {
        uint8_t byte[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) byte[i] = row[at + (i < n ? i : 0)];
#pragma unroll
        for (int i = 0; i < 16; ++i) sr[j][i / 4] |= (i < n ? uint32_t(byte[i]) : 0u) << (8 * (i % 4));
      }
      if (!there) sr[j] = u32x4{0, 0, 0, 0};
    }
  };
  auto put_scales = [&](int half) {
    if constexpr (!ALIGNED) {
#pragma unroll
      for (int j = 0; j < kSegment; ++j) lds.scales[half * kSegment + j][threadIdx.x] = sr[j / 4][j % 4];
    }
  };

  int turn = ahead, now = 0, half = 0, bias_at = 0;
  bool stores = false;   // the epilogue in front of this step has made all its stores
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
    const int segment = ALIGNED ? steps : kSegment;
    for (int s0 = 0; s0 < steps; s0 += segment) {
      if (s0 + segment < steps)
        load_scales(turn, s0 + segment);
      else
        load_scales(next, 0);
      const int last = s0 + segment < steps ? s0 + segment : steps;
      for (int s = s0; s < last; ++s) {
        // the stores are younger than the loads that this step needs
        if (!stores)
          wait_loads_and_waves<kAhead>();
        else if (f32)
          wait_loads_and_waves<kAhead + 4 * QT>();
        else
          wait_loads_and_waves<kAhead + 2 * QT>();
        stores = false;
        const uint8_t* data = lds.stage[now] + lane * 16;
        const uint8_t* scales = reinterpret_cast<const uint8_t*>(lds.scales[ALIGNED ? now : half * kSegment + s - s0]) + r * 4 + g;
        u32x4 wf[4], xf[QT][kH];
        uint32_t wsc[4], xsc[QT];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          wf[t] = *reinterpret_cast<const u32x4*>(data + (wp * 4 + t) * 1024);
          wsc[t] = scales[(wp * 4 + t) * 64];
        }
#pragma unroll
        for (int i = 0; i < QT; ++i) {
#pragma unroll
          for (int h = 0; h < kH; ++h) xf[i][h] = *reinterpret_cast<const u32x4*>(data + (kP + (wq * QT + i) * kH + h) * 1024);
          xsc[i] = scales[(kP + wq * QT + i) * 64];
        }
        issue();
        now = now + 1 < kStages ? now + 1 : 0;
        if (nk % 128 && s == steps - 1) {   // x ends inside the step (what W holds behind it meets zeros)
          const int left = nk - (s * 4 + g) * 32;
#pragma unroll
          for (int i = 0; i < QT; ++i) {
            if constexpr (kX4) {
              xf[i][0] = mx4_keep(xf[i][0], left);
            } else {
#pragma unroll
              for (int h = 0; h < kH; ++h) xf[i][h] = left > h * 16 ? xf[i][h] : u32x4{0, 0, 0, 0};
            }
          }
        }
        if constexpr (kX4) {
#pragma unroll
          for (int i = 0; i < QT; ++i)
#pragma unroll
            for (int t = 0; t < 4; ++t) acc[i][t] = product4(wf[t], wsc[t], xf[i][0], xsc[i], acc[i][t]);
        } else {
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            bf16x8 wo[4], xo[QT];
#pragma unroll
            for (int t = 0; t < 4; ++t) wo[t] = mx4_to_bf16x8(wf[t][h], mx8_scale(wsc[t]));
#pragma unroll
            for (int i = 0; i < QT; ++i) {
              const float sc = mx8_scale(xsc[i]);
              const u32x4 raw = xf[i][h / 2];
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
      finish16<false, kNone, kAny>(e, row, col, v, row < nq ? n : 0);
    }
    stores = p0 + T::BP <= np && q0 + T::BQ <= nq;
    turn = next;
  }
  __builtin_amdgcn_s_waitcnt(0x0f70);   // a wave leaves no load to LDS behind
}

template <int XT, int QT, bool ALIGNED>
hipError_t go_tiles(const MatArg& x, const MatArg& w, const Epilogue& e, int64_t rows, int k, int n, hipStream_t s) {
  using T = Tile<XT, QT, ALIGNED>;
  const auto kernel = &tile_mx4_kernel<T, XT>;
  static LdsLimit limit;
  if (const hipError_t no = limit.allow(kernel, sizeof(typename T::Lds)); no != hipSuccess) return no;
  const int ptiles = int(div_up(n, 128));
  const int64_t most = (kMaxBlocks - 8) / ptiles * T::BQ;   // rows of one launch
  for (int64_t first = 0; first < rows; first += most) {
    const int64_t count = rows - first < most ? rows - first : most;
    Epilogue part = e;
    part.r = rows_from(e.r, first);
    part.y = rows_from(e.y, first);
    const int tiles = int(ptiles * int64_t(div_up(count, T::BQ))), turns = (tiles + 7) / 8 * 8;
    kernel<<<turns < 512 ? turns : 512, kTileThreads, sizeof(typename T::Lds), s>>>(
        w, XT == GS_MAT_MX4 ? mx4_rows_from(x, first) : rows_from(x, first), n, count, k, part, ptiles, tiles);
  }
  return hipGetLastError();
}

template <int XT>
hipError_t by_tiles(const MatArg& x, const MatArg& w, const Epilogue& e, int64_t rows, int k, int n, hipStream_t s) {
  auto words = [](const MatArg& m) { return reinterpret_cast<uintptr_t>(m.s) % 4 == 0 && m.lds % 4 == 0; };
  const bool aligned = (k + 31) / 32 % 4 == 0 && words(x) && words(w);
  const bool few = int64_t(div_up(n, 128)) * div_up(rows, 128) <= 256;
  if (few) return aligned ? go_tiles<XT, 2, true>(x, w, e, rows, k, n, s) : go_tiles<XT, 2, false>(x, w, e, rows, k, n, s);
  return aligned ? go_tiles<XT, 4, true>(x, w, e, rows, k, n, s) : go_tiles<XT, 4, false>(x, w, e, rows, k, n, s);
}

}  // namespace

hipError_t launch_linear_mx4(const MatArg& x, const MatArg& w, const float* bias, int act, const MatArg& r,
                             const MatArg& y, int64_t rows, int k, int n, hipStream_t s) {
  const Epilogue e{bias, act, r, MatArg{nullptr, nullptr, 0, 0, GS_MAT_F32}, y};
  if (rows_fwd_takes(k, n) && rows > 16) return launch_rows_mx4(x, w, e, rows, k, n, s);
  GSK_PROF("linear_mx4", s);
  const int64_t tiles = int64_t(div_up(n, 128)) * div_up(rows, 128);
  if (tiles > 64) {
    if (x.type == GS_MAT_MX4) return by_tiles<GS_MAT_MX4>(x, w, e, rows, k, n, s);
    if (x.type == GS_MAT_MX8 && k % 16 == 0 && buffer_ok(x)) return by_tiles<GS_MAT_MX8>(x, w, e, rows, k, n, s);
    return launch_tile_nt(w, x, n, rows, k, e, s);
  }
  if (x.type == GS_MAT_MX4) return go<GS_MAT_MX4, false>(x, w, e, rows, k, n, s);
  if (x.type == GS_MAT_MX8) return k < 16 ? go<GS_MAT_MX8, true>(x, w, e, rows, k, n, s) : go<GS_MAT_MX8, false>(x, w, e, rows, k, n, s);
  return k < 16 ? go<GS_MAT_BF16, true>(x, w, e, rows, k, n, s) : go<GS_MAT_BF16, false>(x, w, e, rows, k, n, s);
}

}  // namespace gsk
