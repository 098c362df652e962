// gs_lookup_fwd and gs_lookup_bwd: y[i] = scale table[index[i]] and its gradient.
//
// The forward is a stream: 4 to 64 lanes take a row, 8 columns each, and keep kRows rows in
// flight.  The backward adds the rows of one entry in the order of their places, without
// atomics: the indices are sorted (sort.hip's stable radix passes over the bits that the
// entries have), and the sorted list is cut into slots of equal length, however the entries are
// used.  A slot adds up its runs of equal entries in float32; the runs inside it are whole and are
// written, its first and last may go on next door and become two rows of partial sums, which form
// a sorted list again, 2 / kSlot as long.  A list of one slot has no neighbours and ends it.
#include "lookup.h"
#include "profile.h"

namespace gsk {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 4;

template <class I>
__device__ inline int64_t entry_of(const void* index, int64_t i, uint32_t entries) {
  const int64_t e = static_cast<const I*>(index)[i];
  return uint64_t(e) < entries ? e : -1;
}

template <class I, bool NARROW>
__global__ void __launch_bounds__(kThreads) lookup_kernel(MatArg table, const void* index, float scale, MatArg y,
                                                           int64_t rows, uint32_t entries, int cols, int lanes) {
  const int lane = threadIdx.x & (lanes - 1);
  const int per = kThreads / lanes;
  const int64_t row0 = int64_t(blockIdx.x) * (per * kRows) + threadIdx.x / lanes;
  const int col = (int(blockIdx.y) * lanes + lane) * 8;
  const Held c = held_at(col, cols);
  int64_t at[kRows];
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    const int64_t row = row0 + int64_t(u) * per;
    at[u] = entry_of<I>(index, row < rows ? row : rows - 1, entries);
  }
  Raw8 raw[kRows];
#pragma unroll
  for (int u = 0; u < kRows; ++u)
    raw[u] = NARROW ? load_raw8(table, at[u] < 0 ? 0 : at[u], col, cols - col) : load_held(table, at[u] < 0 ? 0 : at[u], c);
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    const int64_t row = row0 + int64_t(u) * per;
    float v[8];
    raw8_to_float(raw[u], table.type, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = at[u] < 0 ? 0.0f : v[i] * scale;
    if (row < rows && c.skip < 8) store8(y, row, NARROW ? col : c.at, v, NARROW ? cols - col : 8);
  }
}

// ------------------------------------------------------------- the gradient

__global__ void __launch_bounds__(kThreads) zero_rows_kernel(MatArg m, int64_t rows, int cols, int lanes) {
  const int lane = threadIdx.x & (lanes - 1), col = (int(blockIdx.y) * lanes + lane) * 8;
  const int64_t row = int64_t(blockIdx.x) * (kThreads / lanes) + threadIdx.x / lanes;
  const float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (row < rows && col < cols) store8(m, row, col, v, cols - col);
}

constexpr int kSlot = 64;      // places of a slot
constexpr int kFlight = 8;     // rows loaded ahead

struct SegArgs {
  MatArg src;               // the list's rows
  const uint32_t* key;      // their entries, ascending
  const uint32_t* order;    // place -> row of src (nullptr: the place itself)
  MatArg dst;
  float scale;
  uint32_t entries;
  int cols;
  int64_t count, slots;
  float* part;              // [2 slots][cols]
  uint32_t* part_key;
  int lanes;
};

template <bool NARROW>
__global__ void __launch_bounds__(kThreads) segment_sums_kernel(SegArgs a) {
  const int lane = threadIdx.x & (a.lanes - 1);
  const int64_t slot = int64_t(blockIdx.x) * (kThreads / a.lanes) + threadIdx.x / a.lanes;
  const int col = (int(blockIdx.y) * a.lanes + lane) * 8;
  if (slot >= a.slots) return;
  const Held c = held_at(col, a.cols);
  const bool own = NARROW ? col < a.cols : c.skip < 8;
  const int at = NARROW ? col : c.at, n = NARROW ? a.cols - col : 8;
  const int64_t first = slot * kSlot, last = first + kSlot < a.count ? first + kSlot : a.count;
  const MatArg part{reinterpret_cast<char*>(a.part), nullptr, a.cols, 0, GS_MAT_F32};
  float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  uint32_t key = a.key[first];
  bool head = a.slots > 1;    // the present run began at the slot's edge
  auto flush = [&](bool edge) {
    if (edge) {
      if (own) store8(part, 2 * slot + (head ? 0 : 1), at, sum, n);
    } else if (own && key < a.entries) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = sum[i] * a.scale;
      store8(a.dst, key, at, v, n);
    }
  };
  const uint32_t first_key = key;
  for (int64_t p0 = first; p0 < last; p0 += kFlight) {
    uint32_t keys[kFlight];
    Raw8 raw[kFlight];
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      const int64_t p = p0 + u < last ? p0 + u : last - 1;
      keys[u] = a.key[p];
      const int64_t row = a.order ? int64_t(a.order[p]) : p;
      raw[u] = NARROW ? load_raw8(a.src, row, col, n) : load_held(a.src, row, c);
    }
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      if (p0 + u >= last) break;
      if (keys[u] != key) {
        flush(head);
        head = false;
        key = keys[u];
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] = 0.0f;
      }
      float v[8];
      raw8_to_float(raw[u], a.src.type, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] += v[i];
    }
  }
  if (a.slots == 1) {
    flush(false);
    return;
  }
  flush(true);
  if (head) {    // one run alone: nothing is left for the other row
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] = 0.0f;
    if (own) store8(part, 2 * slot + 1, at, sum, n);
  }
  if (lane == 0 && blockIdx.y == 0) {
    a.part_key[2 * slot] = first_key;
    a.part_key[2 * slot + 1] = key;
  }
}

int lanes_for(int cols) {
  int lanes = 1;
  while (lanes < 64 && lanes * 8 < cols) lanes *= 2;
  return lanes;
}

inline size_t align256(size_t b) { return (b + 255) & ~size_t(255); }
inline int64_t slots_of(int64_t count) { return (count + kSlot - 1) / kSlot; }

// The sorted indices, the sort's space, and the lists of partial sums (two take turns).
struct BwdWs {
  uint32_t *key, *order;
  void* sort;
  float* part[2];
  uint32_t* part_key[2];
  size_t bytes;
};

BwdWs carve(void* ws, int64_t rows, int cols) {
  BwdWs w;
  char* p = static_cast<char*>(ws);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* r = p + at;
    at += align256(bytes);
    return r;
  };
  w.key = reinterpret_cast<uint32_t*>(take(size_t(rows) * 4));
  w.order = reinterpret_cast<uint32_t*>(take(size_t(rows) * 4));
  w.sort = take(sort_index_ws_bytes(rows));
  int64_t count = rows;
  for (int i = 0; i < 2; ++i) {
    count = 2 * slots_of(count);
    w.part[i] = reinterpret_cast<float*>(take(size_t(count) * cols * 4));
    w.part_key[i] = reinterpret_cast<uint32_t*>(take(size_t(count) * 4));
  }
  w.bytes = at;
  return w;
}

}  // namespace

hipError_t launch_lookup_fwd(const MatArg& table, const void* index, bool wide, float scale, const MatArg& y, int64_t rows,
                             int64_t entries, int cols, hipStream_t s) {
  const int lanes = lanes_for(cols);
  GSK_PROF("lookup_fwd", s);
  for_row_parts(rows, kThreads / lanes * kRows, [&](int64_t first, int64_t count, unsigned blocks) {
    const void* from = static_cast<const char*>(index) + first * (wide ? 8 : 4);
    const dim3 grid(blocks, div_up(cols, lanes * 8));
    const auto kernel = cols < 8 ? (wide ? &lookup_kernel<int64_t, true> : &lookup_kernel<int32_t, true>)
                                 : (wide ? &lookup_kernel<int64_t, false> : &lookup_kernel<int32_t, false>);
    kernel<<<grid, kThreads, 0, s>>>(table, from, scale, rows_from(y, first), count, uint32_t(entries), cols, lanes);
  });
  return hipGetLastError();
}

size_t lookup_bwd_ws_bytes(int64_t rows, int cols) { return carve(nullptr, rows, cols).bytes; }

hipError_t launch_lookup_bwd(const MatArg& dy, const void* index, bool wide, float scale, const MatArg& dtable, int64_t rows,
                             int64_t entries, int cols, void* ws, hipStream_t s) {
  const int lanes = lanes_for(cols);
  const unsigned across = div_up(cols, lanes * 8);
  {
    GSK_PROF("lookup_zero", s);
    for_row_parts(entries, kThreads / lanes, [&](int64_t first, int64_t count, unsigned blocks) {
      zero_rows_kernel<<<dim3(blocks, across), kThreads, 0, s>>>(rows_from(dtable, first), count, cols, lanes);
    });
  }
  if (rows == 0) return hipGetLastError();
  const BwdWs w = carve(ws, rows, cols);
  hipError_t e = launch_sort_index(index, wide, uint32_t(rows), uint32_t(entries), w.key, w.order, w.sort, s);
  if (e != hipSuccess) return e;
  SegArgs a{dy, w.key, w.order, dtable, scale, uint32_t(entries), cols, rows, slots_of(rows), w.part[0], w.part_key[0], lanes};
  for (int i = 0;; ++i) {
    GSK_PROF("lookup_sums", s);
    const auto kernel = cols < 8 ? &segment_sums_kernel<true> : &segment_sums_kernel<false>;
    kernel<<<dim3(div_up(a.slots, kThreads / lanes), across), kThreads, 0, s>>>(a);
    if (a.slots == 1) break;
    a.src = MatArg{reinterpret_cast<char*>(a.part), nullptr, cols, 0, GS_MAT_F32};
    a.key = a.part_key;
    a.order = nullptr;
    a.count = 2 * a.slots;
    a.slots = slots_of(a.count);
    a.part = w.part[(i + 1) % 2];
    a.part_key = w.part_key[(i + 1) % 2];
  }
  return hipGetLastError();
}

}  // namespace gsk
