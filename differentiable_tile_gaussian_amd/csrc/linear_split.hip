// Products with few rows (a view's code, a small batch): the result has too few tiles to fill
// the card, and what there is to do is reading the weight.  A block takes 16 PT columns by 16
// QT rows and its waves share the contraction, each loading its operands from memory
// straight into registers one step ahead; the waves' sums are joined through LDS in order.
// Bounded by latency (a launch, the weight's and the bias's loads, the join): one row 1024 to
// 1024 in 5.4 us, 4096 to 4096 in 11 us (33.5 MB of weight, 3.0 TB/s).
#include "linear.h"
#include "profile.h"

namespace gsk {
namespace {

// 16 k of a row (a lane's share of a step of 64, two products), in bfloat16.
struct Operands {
  bf16x8 a, b;
};

// As loaded: bfloat16 (two words) or MX8 (one, and the scale).  kWhole: nk is a multiple of 16
// and the matrix in buffers' reach.
template <int TYPE, Reach HOW>
struct Share {
  u32x4 a, b;
  uint32_t scale, skip;
  __device__ void load(const MatArg& m, Buffer data, Buffer scales, int64_t row0, int row, bool in, int k, int nk) {
    if constexpr (HOW == kWhole) {
      const bool there = in && k < nk;
      const uint32_t off = there ? (row * uint32_t(m.ld) + k) * element_bytes(TYPE) : kAbsent;
      a = buffer_load16(data, off);
      if constexpr (TYPE == GS_MAT_MX8)
        scale = buffer_load1(scales, there ? row * uint32_t(m.lds) + k / 32 : kAbsent);
      else
        b = buffer_load16(data, off + 16);
    } else {
      Raw16<TYPE, HOW == kNarrow> r;
      r.load(m, in ? row0 + row : row0, k, nk, in);
      a = u32x4{r.w[0], r.w[1], r.w[2], r.w[3]};
      if constexpr (TYPE != GS_MAT_MX8) b = u32x4{r.w[4], r.w[5], r.w[6], r.w[7]};
      scale = TYPE == GS_MAT_MX8 ? r.scale : 0;
      skip = r.skip;
    }
  }
  __device__ void settle() {
    if constexpr (HOW != kWhole) {
      Raw16<TYPE, false> r;
#pragma unroll
      for (int i = 0; i < r.kWords; ++i) r.w[i] = i < 4 ? a[i] : b[i % 4];
      r.skip = skip;
      r.settle();
      a = u32x4{r.w[0], r.w[1], r.w[2], r.w[3]};
      if constexpr (TYPE != GS_MAT_MX8) b = u32x4{r.w[4], r.w[5], r.w[6], r.w[7]};
    }
  }
  __device__ Operands operands() const {
    if constexpr (TYPE == GS_MAT_MX8) {
      const float s = mx8_scale(scale);
      const u32x2 w0 = mx8_to_bf16x4(a[0], s), w1 = mx8_to_bf16x4(a[1], s);
      const u32x2 w2 = mx8_to_bf16x4(a[2], s), w3 = mx8_to_bf16x4(a[3], s);
      return {__builtin_bit_cast(bf16x8, u32x4{w0[0], w0[1], w1[0], w1[1]}),
              __builtin_bit_cast(bf16x8, u32x4{w2[0], w2[1], w3[0], w3[1]})};
    } else {
      return {__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b)};
    }
  }
};

// Waves of a block: enough loads in flight with few rows, 64 KiB of sums at most with many.
__host__ __device__ constexpr int waves_for(int qt) { return qt == 4 ? 4 : 8; }

// out(q, p) = sum_k Q(q, k) P(p, k), P bfloat16, Q bfloat16 or MX8.
template <int QTYPE, int QT, int PT, Reach HOW>
__global__ void __launch_bounds__(waves_for(QT) * 64) split_nt_kernel(MatArg P, MatArg Q, int np, int64_t nq, int nk, Epilogue e) {
  constexpr int kWaves = waves_for(QT);
  extern __shared__ __align__(16) uint8_t lds[];
  f32x4* sums = reinterpret_cast<f32x4*>(lds);   // [wave][QT][PT][lane]
  const int lane = threadIdx.x % 64, g = lane / 16, r = lane % 16;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int p0 = blockIdx.y * (16 * PT);
  const int64_t q0 = int64_t(blockIdx.x) * (16 * QT);
  const Buffer pb = buffer_at(P.p + int64_t(p0) * P.ld * 2), qb = buffer_at(Q.p + q0 * Q.ld * element_bytes(QTYPE));
  const Buffer sb = buffer_at(QTYPE == GS_MAT_MX8 ? Q.s + q0 * Q.lds : nullptr);
  Share<GS_MAT_BF16, HOW> ps[PT];
  Share<QTYPE, HOW> qs[QT];
  auto fetch = [&](int step) {
    const int k = step * 64 + g * 16;
#pragma unroll
    for (int t = 0; t < PT; ++t) {
      const int row = r / 4 * (4 * PT) + t * 4 + r % 4;   // a lane's tiles: 4 PT consecutive columns
      ps[t].load(P, pb, pb, p0, row, p0 + row < np, k, nk);
    }
#pragma unroll
    for (int i = 0; i < QT; ++i) qs[i].load(Q, qb, sb, q0, i * 16 + r, q0 + i * 16 + r < nq, k, nk);
  };
  f32x4 acc[QT][PT];
#pragma unroll
  for (int i = 0; i < QT; ++i)
#pragma unroll
    for (int t = 0; t < PT; ++t) acc[i][t] = f32x4{0, 0, 0, 0};
  const int steps = (nk + 63) / 64;
  fetch(wave);
  // the 16 columns that a lane finishes (PT 2: the lower half's lanes have all 32)
  const int col = p0 + (PT == 4 ? g : g % 2) * 16, n = PT == 2 && g >= 2 ? 0 : np - col < 16 ? np - col : 16;
  float bias[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) bias[j] = e.bias && wave < QT && j < n ? e.bias[col + j] : 0.0f;
  for (int s = wave; s < steps; s += kWaves) {
    Operands po[PT], qo[QT];
#pragma unroll
    for (int t = 0; t < PT; ++t) {
      ps[t].settle();
      po[t] = ps[t].operands();
    }
#pragma unroll
    for (int i = 0; i < QT; ++i) {
      qs[i].settle();
      qo[i] = qs[i].operands();
    }
    fetch(s + kWaves);   // past the end: all absent
#pragma unroll
    for (int i = 0; i < QT; ++i)
#pragma unroll
      for (int t = 0; t < PT; ++t) {
        acc[i][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(po[t].a, qo[i].a, acc[i][t], 0, 0, 0);
        acc[i][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(po[t].b, qo[i].b, acc[i][t], 0, 0, 0);
      }
  }
#pragma unroll
  for (int i = 0; i < QT; ++i)
#pragma unroll
    for (int t = 0; t < PT; ++t) sums[((wave * QT + i) * PT + t) * 64 + lane] = acc[i][t];
  __syncthreads();
  if (wave >= QT) return;
  f32x4 total[PT];
#pragma unroll
  for (int t = 0; t < PT; ++t) total[t] = sums[(wave * PT + t) * 64 + lane];
#pragma unroll 2
  for (int w = 1; w < kWaves; ++w)
#pragma unroll
    for (int t = 0; t < PT; ++t) total[t] += sums[((w * QT + wave) * PT + t) * 64 + lane];
  const int64_t row = q0 + wave * 16 + r;
  float v[16];
  if constexpr (PT == 4) {
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = total[j / 4][j % 4];
  } else {
    // eight columns a lane to sixteen, by way of the first wave's place in LDS
    static_assert(PT == 2 && QT == 1, "one wave finishes");
#pragma unroll
    for (int t = 0; t < 2; ++t) sums[r * 8 + g * 2 + t] = total[t];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const f32x4 q = sums[r * 8 + g % 2 * 4 + t];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[4 * t + i] = q[i];
    }
  }
#pragma unroll
  for (int j = 0; j < 16; ++j) v[j] += bias[j];
  finish16<false, kAny, kAny>(e, row, col, v, row < nq ? n : 0);
}

template <int QTYPE, int QT, int PT, Reach HOW>
hipError_t go(const MatArg& P, const MatArg& Q, int np, int64_t nq, int nk, const Epilogue& e, hipStream_t s) {
  constexpr int kWaves = waves_for(QT), kLds = kWaves * QT * PT * 1024;
  split_nt_kernel<QTYPE, QT, PT, HOW>
      <<<dim3(div_up(nq, 16 * QT), div_up(np, 16 * PT)), kWaves * 64, kLds, s>>>(P, Q, np, nq, nk, e);
  return hipGetLastError();
}

template <int QTYPE, Reach HOW>
hipError_t by_rows(const MatArg& P, const MatArg& Q, int np, int64_t nq, int nk, const Epilogue& e, hipStream_t s) {
  // one row 1024 to 1024 by 32 columns a block: 5.4 us, by 64 7.5
  if (nq <= 16) return go<QTYPE, 1, 2, HOW>(P, Q, np, nq, nk, e, s);
  return nq <= 32 ? go<QTYPE, 2, 4, HOW>(P, Q, np, nq, nk, e, s) : go<QTYPE, 4, 4, HOW>(P, Q, np, nq, nk, e, s);
}

}  // namespace

bool split_nt_takes(const MatArg& P, const MatArg& Q, int np, int64_t nq) {
  return P.type == GS_MAT_BF16 && Q.type != GS_MAT_F32 && int64_t(div_up(np, 128)) * div_up(nq, 128) <= 64;
}

hipError_t launch_split_nt(const MatArg& P, const MatArg& Q, int np, int64_t nq, int nk, const Epilogue& e,
                           hipStream_t s) {
  const Reach how = nk < 16 ? kNarrow : nk % 16 == 0 && buffer_ok(P) && buffer_ok(Q) ? kWhole : kHeldIn;
  if (Q.type == GS_MAT_MX8)
    return how == kWhole    ? by_rows<GS_MAT_MX8, kWhole>(P, Q, np, nq, nk, e, s)
           : how == kHeldIn ? by_rows<GS_MAT_MX8, kHeldIn>(P, Q, np, nq, nk, e, s)
                            : by_rows<GS_MAT_MX8, kNarrow>(P, Q, np, nq, nk, e, s);
  return how == kWhole    ? by_rows<GS_MAT_BF16, kWhole>(P, Q, np, nq, nk, e, s)
         : how == kHeldIn ? by_rows<GS_MAT_BF16, kHeldIn>(P, Q, np, nq, nk, e, s)
                          : by_rows<GS_MAT_BF16, kNarrow>(P, Q, np, nq, nk, e, s);
}

}  // namespace gsk
