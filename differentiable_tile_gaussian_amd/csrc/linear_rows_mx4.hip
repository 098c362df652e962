// Linear layers of narrow width over many rows with the weight in MX4: linear_rows.hip's kernels,
// the weight decoded once a block on its way to LDS.  x is decoded in registers; y may be MX8.
// 1,000,003 rows 128 to 128 with silu from and to MX8 take 70-72 us (3.7 TB/s over 264 MB, by the counters all that
// moves), without it 57 (4.6; a copy of the same matrices 47): HBM beside the vector units, which issue
// in 62 % of the cycles (10 instructions a wave and result) with the matrix cores busy in 19 %.  From MX8
// to bfloat16 86-88 us without and with it (4.5 TB/s: HBM), from MX4 85, from bfloat16 102 (5.0), 48 columns
// of float32 with a residual 119 (4.3).
#include "linear_rows.h"

namespace gsk {
namespace {

constexpr int WT = GS_MAT_MX4;

template <int KC, int NC, int XT>
hipError_t by_output(const RowsArgs& a, hipStream_t s) {
  const bool r = a.e.r.p != nullptr;
  switch (a.e.y.type) {
    case GS_MAT_MX8:
      return r ? go<WT, KC, NC, XT, kNone, GS_MAT_MX8, GS_MAT_BF16>(a, s) : go<WT, KC, NC, XT, kNone, GS_MAT_MX8, kNone>(a, s);
    case GS_MAT_F32:
      return r ? go<WT, KC, NC, XT, kNone, GS_MAT_F32, GS_MAT_F32>(a, s) : go<WT, KC, NC, XT, kNone, GS_MAT_F32, kNone>(a, s);
    default:
      return r ? go<WT, KC, NC, XT, kNone, GS_MAT_BF16, GS_MAT_BF16>(a, s) : go<WT, KC, NC, XT, kNone, GS_MAT_BF16, kNone>(a, s);
  }
}

template <int KC, int NC>
hipError_t by_input(const RowsArgs& a, hipStream_t s) {
  switch (a.x.type) {
    case GS_MAT_MX4: return by_output<KC, NC, GS_MAT_MX4>(a, s);
    case GS_MAT_MX8: return by_output<KC, NC, GS_MAT_MX8>(a, s);
    default: return by_output<KC, NC, GS_MAT_BF16>(a, s);
  }
}

template <int KC>
hipError_t by_columns(const RowsArgs& a, hipStream_t s) {
  const int groups = (a.n + 63) / 64;
  if (split_for(div_up(a.rows, 128), groups) == groups) return by_input<KC, 1>(a, s);
  return groups <= 2 ? by_input<KC, 2>(a, s) : by_input<KC, 4>(a, s);
}

template <int XT>
hipError_t any_width(const RowsArgs& a, hipStream_t s) {
  if (a.k < 16) return go_any<WT, 1, XT, true>(a, s);
  switch ((a.k + 63) / 64) {
    case 1: return go_any<WT, 1, XT, false>(a, s);
    case 2: return go_any<WT, 2, XT, false>(a, s);
    default: return go_any<WT, 4, XT, false>(a, s);
  }
}

// As linear_rows.hip's: whole 16-column pieces, buffers, and a residual of y's type (of bfloat16 with
// a y in MX8) or none.
bool fast(const RowsArgs& a) {
  const Epilogue& e = a.e;
  if (a.k % 16 || a.n % 16 || !buffer_ok(a.x) || !buffer_ok(e.y) || !buffer_ok(e.r)) return false;
  return !e.r.p || e.r.type == (e.y.type == GS_MAT_F32 ? GS_MAT_F32 : GS_MAT_BF16);
}

}  // namespace

hipError_t launch_rows_mx4(const MatArg& x, const MatArg& w, const Epilogue& e, int64_t rows, int k, int n,
                           hipStream_t s) {
  const RowsArgs a{x, w, e, rows, k, n};
  if (fast(a)) return k <= 64 ? by_columns<1>(a, s) : k <= 128 ? by_columns<2>(a, s) : by_columns<4>(a, s);
  switch (x.type) {
    case GS_MAT_MX4: return any_width<GS_MAT_MX4>(a, s);
    case GS_MAT_MX8: return any_width<GS_MAT_MX8>(a, s);
    default: return any_width<GS_MAT_BF16>(a, s);
  }
}

}  // namespace gsk
