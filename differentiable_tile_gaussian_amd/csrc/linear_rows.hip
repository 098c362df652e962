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
#include "linear_rows.h"

namespace gsk {
namespace {

template <int KC, int NC, int XT>
hipError_t by_output(const RowsArgs& a, hipStream_t s) {
  constexpr int WT = GS_MAT_BF16;
  const bool f32 = a.e.y.type == GS_MAT_F32;
  if (a.e.z.p) return go<WT, KC, NC, XT, GS_MAT_MX8, GS_MAT_BF16, kNone>(a, s);
  if (a.e.r.p)
    return f32 ? go<WT, KC, NC, XT, kNone, GS_MAT_F32, GS_MAT_F32>(a, s) : go<WT, KC, NC, XT, kNone, GS_MAT_BF16, GS_MAT_BF16>(a, s);
  return f32 ? go<WT, KC, NC, XT, kNone, GS_MAT_F32, kNone>(a, s) : go<WT, KC, NC, XT, kNone, GS_MAT_BF16, kNone>(a, s);
}

template <int KC, int NC>
hipError_t by_input(const RowsArgs& a, hipStream_t s) {
  return a.x.type == GS_MAT_MX8 ? by_output<KC, NC, GS_MAT_MX8>(a, s) : by_output<KC, NC, GS_MAT_BF16>(a, s);
}

template <int KC>
hipError_t by_columns(const RowsArgs& a, hipStream_t s) {
  const int groups = (a.n + 63) / 64;
  if (split_for(div_up(a.rows, 128), groups) == groups) return by_input<KC, 1>(a, s);
  return groups <= 2 ? by_input<KC, 2>(a, s) : by_input<KC, 4>(a, s);
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
  if (k < 16) return mx ? go_any<GS_MAT_BF16, 1, GS_MAT_MX8, true>(a, s) : go_any<GS_MAT_BF16, 1, GS_MAT_BF16, true>(a, s);
  switch ((k + 63) / 64) {
    case 1: return mx ? go_any<GS_MAT_BF16, 1, GS_MAT_MX8, false>(a, s) : go_any<GS_MAT_BF16, 1, GS_MAT_BF16, false>(a, s);
    case 2: return mx ? go_any<GS_MAT_BF16, 2, GS_MAT_MX8, false>(a, s) : go_any<GS_MAT_BF16, 2, GS_MAT_BF16, false>(a, s);
    default: return mx ? go_any<GS_MAT_BF16, 4, GS_MAT_MX8, false>(a, s) : go_any<GS_MAT_BF16, 4, GS_MAT_BF16, false>(a, s);
  }
}

}  // namespace gsk
