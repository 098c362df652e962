// Products of wide layers, bounded by the matrix cores: tiles of 128 columns by 32 QT rows of
// the result (64 x 16 QT for each of four waves), with the contraction in steps of 64 staged
// through registers into two LDS buffers.  The operands of the next D steps are in flight from
// memory and the next step's are written to LDS while the present one is computed, so that
// one barrier a step suffices and nothing waits for memory.
//
// 8160 rows, 4096 to 1024 (68 GFLOP), by the clock over many calls: from bfloat16 81 us (845
// TFLOP/s), from MX8 with a residual 81-85; the first hundreds of calls after a pause are slower
// while the card's clock settles (from MX8 91-93 us, which a trace of 39 calls shows).  The contraction
// over the rows for dW (4096 x 1024), in such a trace: 107 us (640 TFLOP/s).  What is left is
// LDS: a step's operands are written once and read twice by the waves beside its matrix
// instructions.
#include "linear.h"
#include "profile.h"

namespace gsk {
namespace {

constexpr int kThreads = 256;

// Ends a step: LDS writes done, all waves there; loads from memory stay in flight.
__device__ inline void step_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// The order in which a step's instructions are issued: a few operand reads, then four matrix
// instructions at a time with what the next ones need in between: an operand read or two, an
// LDS write of the step to come, a load from memory.  (Left to itself the compiler puts the
// writes first, and every wave waits for them in front of its first operand.)
template <int READS, int WRITES, int LOADS, int GROUPS, int I = 0>
__device__ inline void interleave() {
  constexpr int kFirst = READS / 4, kRest = READS - kFirst, kOver = GROUPS - 2;
  if constexpr (I == 0) __builtin_amdgcn_sched_group_barrier(0x100, kFirst, 0);
  if constexpr (I < GROUPS) {
    __builtin_amdgcn_sched_group_barrier(0x008, 4, 0);
    if constexpr (I < kOver) {
      constexpr int reads = (I + 1) * kRest / kOver - I * kRest / kOver;
      if constexpr (reads > 0) __builtin_amdgcn_sched_group_barrier(0x100, reads, 0);
    }
    constexpr int writes = (I + 1) * WRITES / GROUPS - I * WRITES / GROUPS;
    if constexpr (writes > 0) __builtin_amdgcn_sched_group_barrier(0x200, writes, 0);
    constexpr int loads = (I + 1) * LOADS / GROUPS - I * LOADS / GROUPS;
    if constexpr (loads > 0) __builtin_amdgcn_sched_group_barrier(0x020, loads, 0);
    interleave<READS, WRITES, LOADS, GROUPS, I + 1>();
  }
}

// Which tile a block takes: consecutive blocks go to different XCDs, each with its own L2, so
// an XCD is given neighbouring tiles (the P tiles of one Q tile after another).
__device__ inline int tile_of(int block, int tiles) {
  const int per = (tiles + 7) / 8;
  return block % 8 * per + block / 8;
}

// 16 values of a row as loaded: bfloat16 (two 16-byte words) or MX8 (one, and the scale).
template <int TYPE>
struct Unit {
  u32x4 a, b;
  uint32_t scale;
  __device__ void load(Buffer data, Buffer scales, uint32_t off, uint32_t soff) {
    a = buffer_load16(data, off);
    if constexpr (TYPE == GS_MAT_MX8)
      scale = buffer_load1(scales, soff);
    else
      b = buffer_load16(data, off + 16);
  }
  // Any width and alignment (matrix.h): to be settled before its use.
  uint32_t skip;
  template <bool NARROW>
  __device__ void load_any(const MatArg& m, int64_t row, int col, int cols, bool live) {
    Raw16<TYPE, NARROW> r;
    r.load(m, row, col, cols, live);
    a = u32x4{r.w[0], r.w[1], r.w[2], r.w[3]};
    if constexpr (TYPE != GS_MAT_MX8) b = u32x4{r.w[4], r.w[5], r.w[6], r.w[7]};
    scale = TYPE == GS_MAT_MX8 ? r.scale : 0;
    skip = r.skip;
  }
  __device__ void settle() {
    Raw16<TYPE, false> r;
#pragma unroll
    for (int i = 0; i < r.kWords; ++i) r.w[i] = i < 4 ? a[i] : b[i % 4];
    r.skip = skip;
    r.settle();
    a = u32x4{r.w[0], r.w[1], r.w[2], r.w[3]};
    if constexpr (TYPE != GS_MAT_MX8) b = u32x4{r.w[4], r.w[5], r.w[6], r.w[7]};
  }
  __device__ void operands(u32x4& p, u32x4& q) const {
    if constexpr (TYPE == GS_MAT_MX8) {
      const float s = mx8_scale(scale);
      const u32x2 w0 = mx8_to_bf16x4(a[0], s), w1 = mx8_to_bf16x4(a[1], s);
      const u32x2 w2 = mx8_to_bf16x4(a[2], s), w3 = mx8_to_bf16x4(a[3], s);
      p = u32x4{w0[0], w0[1], w1[0], w1[1]};
      q = u32x4{w2[0], w2[1], w3[0], w3[1]};
    } else {
      p = a;
      q = b;
    }
  }
};

// ------------------------------------------------- contraction contiguous in both operands

// out(q, p) = sum_k Q(q, k) P(p, k) for the rows q of Q (bfloat16 or MX8) and p of P
// (bfloat16).  kWhole: nk is a multiple of 16 and both are in buffers' reach.  An LDS row is 64 k, 128 bytes, whose 16-byte pieces are
// permuted by the row's number so that a fragment read's 16 rows fall into different banks;
// P's rows are stored so that a lane's four result tiles are 16 consecutive columns.
template <int QTYPE, int QT, int D, Reach HOW>
__global__ void __launch_bounds__(kThreads) tile_nt_kernel(MatArg P, MatArg Q, int np, int64_t nq, int nk, Epilogue e,
                                                            int ptiles, int tiles) {
  constexpr bool WHOLE = HOW == kWhole, kFew = HOW == kNarrow;
  constexpr int BP = 128, BQ = 32 * QT, kStep = (BP + BQ) * 128;
  extern __shared__ __align__(16) uint8_t lds[];
  const int tile = tile_of(blockIdx.x, tiles);
  if (tile >= tiles) return;
  const int p0 = tile % ptiles * BP;
  const int64_t q0 = int64_t(tile / ptiles) * BQ;
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, wp = wave % 2, wq = wave / 2;
  // a thread stages piece `piece` (16 k) of the rows row + 64 u
  const int row = threadIdx.x / 4, piece = threadIdx.x % 4;
  constexpr uint32_t kQ = element_bytes(QTYPE);
  const Buffer pb = buffer_at(P.p + int64_t(p0) * P.ld * 2), qb = buffer_at(Q.p + q0 * Q.ld * kQ);
  const Buffer sb = buffer_at(QTYPE == GS_MAT_MX8 ? Q.s + q0 * Q.lds : nullptr);
  uint32_t poff[BP / 64], qoff[BQ / 64], soff[BQ / 64];
#pragma unroll
  for (int u = 0; u < BP / 64; ++u)
    poff[u] = p0 + u * 64 + row < np ? (u * 64 + row) * uint32_t(P.ld) * 2 + piece * 32 : kAbsent;
#pragma unroll
  for (int u = 0; u < BQ / 64; ++u) {
    const bool in = q0 + u * 64 + row < nq;
    qoff[u] = in ? (u * 64 + row) * uint32_t(Q.ld) * kQ + piece * 16 * kQ : kAbsent;
    soff[u] = in ? (u * 64 + row) * uint32_t(Q.lds) + piece / 2 : kAbsent;
  }
  Unit<GS_MAT_BF16> pr[D][BP / 64];
  Unit<QTYPE> qr[D][BQ / 64];
  auto fetch = [&](int d, int k0) {
    const bool in = k0 + piece * 16 < nk;
    if constexpr (!WHOLE) {
      const int k = k0 + piece * 16;
#pragma unroll
      for (int u = 0; u < BP / 64; ++u) {
        const int at = p0 + u * 64 + row;
        pr[d][u].template load_any<kFew>(P, at < np ? at : np - 1, k, nk, at < np);
      }
#pragma unroll
      for (int u = 0; u < BQ / 64; ++u) {
        const int64_t at = q0 + u * 64 + row;
        qr[d][u].template load_any<kFew>(Q, at < nq ? at : nq - 1, k, nk, at < nq);
      }
      return;
    }
#pragma unroll
    for (int u = 0; u < BP / 64; ++u) pr[d][u].load(pb, pb, in ? poff[u] + k0 * 2 : kAbsent, 0);
#pragma unroll
    for (int u = 0; u < BQ / 64; ++u)
      qr[d][u].load(qb, sb, in ? qoff[u] + k0 * kQ : kAbsent, in ? soff[u] + k0 / 32 : kAbsent);
  };
  auto put = [&](uint8_t* at, int r, u32x4 a, u32x4 b) {
    const int s = (r >> 1) & 7;
    *reinterpret_cast<u32x4*>(at + r * 128 + ((piece * 2) ^ s) * 16) = a;
    *reinterpret_cast<u32x4*>(at + r * 128 + ((piece * 2 + 1) ^ s) * 16) = b;
  };
  auto stage = [&](int d, uint8_t* at) {
    u32x4 a, b;
#pragma unroll
    for (int u = 0; u < BP / 64; ++u) {
      const int r = u * 64 + row;
      if constexpr (!WHOLE) pr[d][u].settle();
      pr[d][u].operands(a, b);
      put(at, (r & ~63) | ((r & 12) << 2) | ((r & 48) >> 2) | (r & 3), a, b);
    }
#pragma unroll
    for (int u = 0; u < BQ / 64; ++u) {
      if constexpr (!WHOLE) qr[d][u].settle();
      qr[d][u].operands(a, b);
      put(at + BP * 128, u * 64 + row, a, b);
    }
  };
  f32x4 acc[QT][4];
#pragma unroll
  for (int i = 0; i < QT; ++i)
#pragma unroll
    for (int t = 0; t < 4; ++t) acc[i][t] = f32x4{0, 0, 0, 0};
  // a fragment's place within its rows: the row's number enters through bits 1-3 only
  const int r16 = lane % 16, g = lane / 16, sw = (r16 >> 1) & 7;
  const int frag0 = r16 * 128 + (g ^ sw) * 16, frag1 = r16 * 128 + ((g + 4) ^ sw) * 16;
  // loads of D steps are in flight: step s + 1 + d in set (s + d) % D
  fetch(0, 0);
  stage(0, lds);
#pragma unroll
  for (int d = 0; d < D; ++d) fetch(d, (d + 1) * 64);
  const int steps = (nk + 63) / 64;
  for (int s0 = 0; s0 < steps; s0 += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const int s = s0 + d;
      if (s >= steps) break;
      step_barrier();
      const uint8_t* now = lds + (s & 1) * kStep;
      bf16x8 pf[2][4], qf[2][QT];
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        const uint8_t* at = now + (kk ? frag1 : frag0);
#pragma unroll
        for (int t = 0; t < 4; ++t) pf[kk][t] = *reinterpret_cast<const bf16x8*>(at + (wp * 64 + t * 16) * 128);
#pragma unroll
        for (int i = 0; i < QT; ++i) qf[kk][i] = *reinterpret_cast<const bf16x8*>(at + (BP + (wq * QT + i) * 16) * 128);
      }
      stage(d, lds + (~s & 1) * kStep);   // past the end: zeros, not read
      fetch(d, (s + 1 + D) * 64);
#pragma unroll
      for (int kk = 0; kk < 2; ++kk)
#pragma unroll
        for (int i = 0; i < QT; ++i)
#pragma unroll
          for (int t = 0; t < 4; ++t)
            acc[i][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(pf[kk][t], qf[kk][i], acc[i][t], 0, 0, 0);
      interleave<2 * (4 + QT), (BP + BQ) / 32, (BP + BQ) / 32, 2 * QT>();
    }
  }
  const int col = p0 + wp * 64 + g * 16, n = np - col < 16 ? np - col : 16;
  float bias[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) bias[i] = e.bias && i < n ? e.bias[col + i] : 0.0f;
#pragma unroll
  for (int i = 0; i < QT; ++i) {
    const int64_t r = q0 + (wq * QT + i) * 16 + r16;
    float v[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = acc[i][j / 4][j % 4] + bias[j];
    finish16<false, kAny, kAny>(e, r, col, v, r < nq ? n : 0);
  }
}

// ------------------------------------------------- contraction over the operands' rows

// out(q, p) = sum_m Q(m, q) P(m, p) for m in the block's slice: the weight's gradient (Q =
// dz, bfloat16; P = x, bfloat16 or MX8).  kWhole: np and nq are multiples of 16 and
// both matrices in buffers' reach.  LDS holds 64 rows m
// as they are in memory (plus 32 bytes a row, so that eight rows fall into different banks),
// read transposed.
template <int PTYPE, int QT, int D, Reach HOW>
__global__ void __launch_bounds__(kThreads) tile_tn_kernel(MatArg P, MatArg Q, int np, int nq, int64_t rows,
                                                            int64_t per_slice, float* part, MatArg out, int ptiles,
                                                            int tiles, int slices) {
  constexpr bool WHOLE = HOW == kWhole, kFew = HOW == kNarrow;
  constexpr int BP = 128, BQ = 32 * QT, kPitchP = BP * 2 + 32, kPitchQ = BQ * 2 + 32;
  constexpr int kStep = 64 * (kPitchP + kPitchQ), kUP = BP / 64, kUQ = BQ / 64;
  extern __shared__ __align__(16) uint8_t lds[];
  // an XCD is given all the tiles of a slice, which share its rows; a few slices: neighbouring tiles
  const int slice = slices < 8 ? blockIdx.x / ((tiles + 7) / 8 * 8) : blockIdx.x / 8 / tiles * 8 + blockIdx.x % 8;
  const int tile = slices < 8 ? tile_of(blockIdx.x % ((tiles + 7) / 8 * 8), tiles) : blockIdx.x / 8 % tiles;
  if (tile >= tiles || slice >= slices) return;
  const int p0 = tile % ptiles * BP, q0 = tile / ptiles * BQ;
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, wp = wave % 2, wq = wave / 2;
  const int64_t first = int64_t(slice) * per_slice;
  const int64_t last = first + per_slice < rows ? first + per_slice : rows;
  // a thread stages 16 columns of kUP + kUQ row pieces: P's rows hold BP / 16 of them, Q's BQ / 16
  constexpr uint32_t kP = element_bytes(PTYPE);
  const int pm = threadIdx.x / (BP / 16), pc = threadIdx.x % (BP / 16) * 16;
  const int qm = threadIdx.x / (BQ / 16), qc = threadIdx.x % (BQ / 16) * 16;
  Unit<PTYPE> pr[D][kUP];
  Unit<GS_MAT_BF16> qr[D][kUQ];
  auto fetch = [&](int d, int64_t m0) {
    const Buffer pb = buffer_at(P.p + (m0 * P.ld + p0) * kP), qb = buffer_at(Q.p + (m0 * Q.ld + q0) * 2);
    const Buffer sb = buffer_at(PTYPE == GS_MAT_MX8 ? P.s + m0 * P.lds + p0 / 32 : nullptr);
    const int left = last - m0 < 64 ? int(last - m0) : 64;
    if constexpr (!WHOLE) {
#pragma unroll
      for (int u = 0; u < kUP; ++u) {
        const int m = pm + u * (kThreads * 16 / BP);
        const int64_t at = m0 + m < rows ? m0 + m : rows - 1;
        pr[d][u].template load_any<kFew>(P, at, p0 + pc, np, m < left);
      }
#pragma unroll
      for (int u = 0; u < kUQ; ++u) {
        const int m = qm + u * (kThreads * 16 / BQ);
        const int64_t at = m0 + m < rows ? m0 + m : rows - 1;
        qr[d][u].template load_any<kFew>(Q, at, q0 + qc, nq, m < left);
      }
      return;
    }
#pragma unroll
    for (int u = 0; u < kUP; ++u) {
      const int m = pm + u * (kThreads * 16 / BP);
      const bool in = m < left && p0 + pc < np;
      pr[d][u].load(pb, sb, in ? (m * uint32_t(P.ld) + pc) * kP : kAbsent, in ? m * uint32_t(P.lds) + pc / 32 : kAbsent);
    }
#pragma unroll
    for (int u = 0; u < kUQ; ++u) {
      const int m = qm + u * (kThreads * 16 / BQ);
      qr[d][u].load(qb, qb, m < left && q0 + qc < nq ? (m * uint32_t(Q.ld) + qc) * 2 : kAbsent, 0);
    }
  };
  auto stage = [&](int d, uint8_t* at) {
    u32x4 a, b;
#pragma unroll
    for (int u = 0; u < kUP; ++u) {
      uint8_t* o = at + (pm + u * (kThreads * 16 / BP)) * kPitchP + pc * 2;
      if constexpr (!WHOLE) pr[d][u].settle();
      pr[d][u].operands(a, b);
      *reinterpret_cast<u32x4*>(o) = a;
      *reinterpret_cast<u32x4*>(o + 16) = b;
    }
#pragma unroll
    for (int u = 0; u < kUQ; ++u) {
      uint8_t* o = at + 64 * kPitchP + (qm + u * (kThreads * 16 / BQ)) * kPitchQ + qc * 2;
      if constexpr (!WHOLE) qr[d][u].settle();
      qr[d][u].operands(a, b);
      *reinterpret_cast<u32x4*>(o) = a;
      *reinterpret_cast<u32x4*>(o + 16) = b;
    }
  };
  f32x4 acc[QT][4];
#pragma unroll
  for (int i = 0; i < QT; ++i)
#pragma unroll
    for (int t = 0; t < 4; ++t) acc[i][t] = f32x4{0, 0, 0, 0};
  const int m = lane / 16 * 8 + lane % 16 / 4, c = lane % 4 * 4;
  const int pat = m * kPitchP + (wp * 64 + c) * 2, qat = 64 * kPitchP + m * kPitchQ + (wq * QT * 16 + c) * 2;
  const int steps = last > first ? int((last - first + 63) / 64) : 0;
  if (steps > 0) {
    fetch(0, first);
    stage(0, lds);
#pragma unroll
    for (int d = 0; d < D; ++d) fetch(d, first + (d + 1) * 64);
  }
  for (int s0 = 0; s0 < steps; s0 += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const int s = s0 + d;
      if (s >= steps) break;
      step_barrier();
      const uint8_t* now = lds + (s & 1) * kStep;
      bf16x8 pf[2][4], qf[2][QT];
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
        for (int t = 0; t < 4; ++t) pf[kk][t] = read_transposed(now + pat + kk * 32 * kPitchP + t * 32, kPitchP);
#pragma unroll
        for (int i = 0; i < QT; ++i) qf[kk][i] = read_transposed(now + qat + kk * 32 * kPitchQ + i * 32, kPitchQ);
      }
      stage(d, lds + (~s & 1) * kStep);
      fetch(d, first + int64_t(s + 1 + D) * 64);
#pragma unroll
      for (int kk = 0; kk < 2; ++kk)
#pragma unroll
        for (int i = 0; i < QT; ++i)
#pragma unroll
          for (int t = 0; t < 4; ++t)
            acc[i][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(pf[kk][t], qf[kk][i], acc[i][t], 0, 0, 0);
      interleave<4 * (4 + QT), 2 * (kUP + kUQ), 2 * (kUP + kUQ), 2 * QT>();
    }
  }
#pragma unroll
  for (int i = 0; i < QT; ++i) {
    const int q = q0 + (wq * QT + i) * 16 + lane % 16;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int p = p0 + wp * 64 + t * 16 + lane / 16 * 4;
      if (q >= nq || p >= np) continue;
      const f32x4 v = acc[i][t];
      if (!WHOLE && p + 4 > np) {   // the last columns of an odd width
        for (int j = 0; p + j < np; ++j) {
          if (part)
            part[(int64_t(slice) * nq + q) * np + p + j] = v[j];
          else if (out.type == GS_MAT_F32)
            reinterpret_cast<float*>(out.p)[int64_t(q) * out.ld + p + j] = v[j];
          else
            reinterpret_cast<uint16_t*>(out.p)[int64_t(q) * out.ld + p + j] = uint16_t(pack_bf16(v[j], 0.0f));
        }
        continue;
      }
      if (part) {
        __builtin_memcpy(__builtin_assume_aligned(part + (int64_t(slice) * nq + q) * np + p, 4), &v, 16);
      } else if (out.type == GS_MAT_F32) {
        __builtin_memcpy(__builtin_assume_aligned(reinterpret_cast<float*>(out.p) + int64_t(q) * out.ld + p, 4), &v, 16);
      } else {
        const u32x2 w{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
        __builtin_memcpy(__builtin_assume_aligned(out.p + (int64_t(q) * out.ld + p) * 2, 2), &w, 8);
      }
    }
  }
}

template <int QTYPE, int QT, int D, Reach HOW>
hipError_t go_nt(const MatArg& P, const MatArg& Q, int np, int64_t nq, int nk, const Epilogue& e, hipStream_t s) {
  constexpr int kLds = 2 * (128 + 32 * QT) * 128;
  const auto kernel = &tile_nt_kernel<QTYPE, QT, D, HOW>;
  static LdsLimit limit;
  if (const hipError_t no = limit.allow(kernel, kLds); no != hipSuccess) return no;
  const int ptiles = int(div_up(np, 128)), tiles = int(ptiles * int64_t(div_up(nq, 32 * QT)));
  kernel<<<(tiles + 7) / 8 * 8, kThreads, kLds, s>>>(P, Q, np, nq, nk, e, ptiles, tiles);
  return hipGetLastError();
}

template <int PTYPE, int QT, int D, Reach HOW>
hipError_t go_tn(const MatArg& P, const MatArg& Q, int np, int nq, int64_t rows, int slices, float* part,
                 const MatArg& out, hipStream_t s) {
  constexpr int kLds = 2 * 64 * (128 * 2 + 32 + 32 * QT * 2 + 32);
  const auto kernel = &tile_tn_kernel<PTYPE, QT, D, HOW>;
  static LdsLimit limit;
  if (const hipError_t no = limit.allow(kernel, kLds); no != hipSuccess) return no;
  const int ptiles = int(div_up(np, 128)), tiles = ptiles * int(div_up(nq, 32 * QT));
  const int64_t per = ((rows + slices - 1) / slices + 63) / 64 * 64;
  const unsigned blocks = unsigned(slices < 8 ? (tiles + 7) / 8 * 8 * slices : (slices + 7) / 8 * 8 * tiles);
  kernel<<<blocks, kThreads, kLds, s>>>(P, Q, np, nq, rows, per, slices > 1 ? part : nullptr, out, ptiles, tiles, slices);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_tile_nt(const MatArg& P, const MatArg& Q, int np, int64_t nq, int nk, const Epilogue& e,
                          hipStream_t s) {
  // One 128 x 256 block a compute unit or two of 128 x 128: a long contraction runs better on
  // the larger (8160 x 4096 to 1024: 82 us, smaller tiles 89; from MX8 the two are level, 91 and
  // 93 in calls after a pause, so it has the smaller alone), but two blocks hide each other's epilogue (8160 x 1024 to 4096: 110 us and 106; with
  // gelu and a kept z 138 and 118).
  const bool big = nk >= 2048 && int64_t(div_up(np, 128)) * div_up(nq, 256) >= 192;
  const Reach how = nk < 16 ? kNarrow : nk % 16 == 0 && buffer_ok(P) && buffer_ok(Q) ? kWhole : kHeldIn;
  // Up to 128 tiles of 128 x 128 leave half the card idle: twice as many of half the rows (1500 x
  // 4096 to 768: 51 us and 38, 2000 x 1024 to 1024: 18.7 and 15.6; with more, as 1364 x 1136 to
  // 1664, 21.4 and 23.3).
  const bool few = int64_t(div_up(np, 128)) * div_up(nq, 128) <= 128;
  if (few && how != kNarrow) {
    if (Q.type == GS_MAT_MX8)
      return how == kWhole ? go_nt<GS_MAT_MX8, 2, 3, kWhole>(P, Q, np, nq, nk, e, s)
                           : go_nt<GS_MAT_MX8, 2, 2, kHeldIn>(P, Q, np, nq, nk, e, s);
    return how == kWhole ? go_nt<GS_MAT_BF16, 2, 3, kWhole>(P, Q, np, nq, nk, e, s)
                         : go_nt<GS_MAT_BF16, 2, 2, kHeldIn>(P, Q, np, nq, nk, e, s);
  }
  if (Q.type == GS_MAT_MX8)
    return how == kWhole    ? go_nt<GS_MAT_MX8, 4, 2, kWhole>(P, Q, np, nq, nk, e, s)
           : how == kHeldIn ? go_nt<GS_MAT_MX8, 4, 2, kHeldIn>(P, Q, np, nq, nk, e, s)
                            : go_nt<GS_MAT_MX8, 4, 1, kNarrow>(P, Q, np, nq, nk, e, s);
  if (how == kHeldIn) return go_nt<GS_MAT_BF16, 4, 2, kHeldIn>(P, Q, np, nq, nk, e, s);
  if (how == kNarrow) return go_nt<GS_MAT_BF16, 4, 1, kNarrow>(P, Q, np, nq, nk, e, s);
  return big ? go_nt<GS_MAT_BF16, 8, 3, kWhole>(P, Q, np, nq, nk, e, s)
             : go_nt<GS_MAT_BF16, 4, 2, kWhole>(P, Q, np, nq, nk, e, s);
}

// Slices of the rows: about one block a compute unit, at least 256 rows each (two blocks a unit
// double the partial sums: 8160 rows 512 to 1024 26 us, by one 21; 1364 rows 1664 to 1136 32
// and 20).
int tile_tn_slices(int64_t rows, int np, int nq) {
  const int64_t tiles = int64_t(div_up(np, 128)) * div_up(nq, 128);
  const int64_t want = tiles >= 256 ? 1 : (256 + tiles / 2) / tiles, most = rows < 512 ? 1 : rows / 256;
  return int(want < most ? want : most);
}

hipError_t launch_tile_tn(const MatArg& P, const MatArg& Q, int np, int nq, int64_t rows, int slices, float* part,
                          const MatArg& out, hipStream_t s) {
  const bool whole = np % 16 == 0 && nq % 16 == 0 && buffer_ok(P) && buffer_ok(Q);
  const Reach how = np < 16 || nq < 16 ? kNarrow : whole ? kWhole : kHeldIn;
  if (P.type == GS_MAT_MX8)
    return how == kWhole    ? go_tn<GS_MAT_MX8, 4, 4, kWhole>(P, Q, np, nq, rows, slices, part, out, s)
           : how == kHeldIn ? go_tn<GS_MAT_MX8, 4, 2, kHeldIn>(P, Q, np, nq, rows, slices, part, out, s)
                            : go_tn<GS_MAT_MX8, 4, 1, kNarrow>(P, Q, np, nq, rows, slices, part, out, s);
  return how == kWhole    ? go_tn<GS_MAT_BF16, 4, 4, kWhole>(P, Q, np, nq, rows, slices, part, out, s)
         : how == kHeldIn ? go_tn<GS_MAT_BF16, 4, 2, kHeldIn>(P, Q, np, nq, rows, slices, part, out, s)
                          : go_tn<GS_MAT_BF16, 4, 1, kNarrow>(P, Q, np, nq, rows, slices, part, out, s);
}

}  // namespace gsk
