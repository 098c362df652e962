// gs_lookup_fwd and gs_lookup_bwd: y[i] = scale table[index[i]] and its gradient.
//
// The forward is a stream: 4 to 64 lanes take a row, 8 columns each, and keep kRows rows in
// flight.  The backward adds the rows of one entry in the order of their places, without
// atomics: the indices are sorted (sort.hip's stable radix passes over the bits that the
// entries have), and the sorted list is cut into slots of equal length, however the entries are
// used.  The lanes of a slot add up its runs of equal entries in float32, and runs that reach into
// the next slots of the block are joined through LDS.  What goes on in another block becomes a row of
// partial sums, at most one at each end of a block, and a second kernel joins those: the block in
// which a run begins adds the rows of the blocks that it reaches.  The first kernel also marks the entries
// that have rows, and the second writes zeros to the others.
//
// The forward is bounded by what passes the L2s: a table that an XCD's 4 MB do not hold is fetched again and
// again from the cache behind them.  1,000,003 rows of 128 to bfloat16 from 65536 entries of float32 (34 MB) take
// 86 us: by the counters 343 MB of the 512 that the indices name come past the L2s, with 256 MB of
// stores 7.0 TB/s (3.5 with the table counted once).  A bfloat16 table takes 59 us, a float32 y from it 148 and from
// the float32 one 167.  Its backward takes 130: the sums 69, in which rows are fetched in the order of entries
// (4.4 TB/s by the counters), the sort 52 and the joins 9, launches and latency; 6,000,000 rows of 48 float32 442 us.
// 100,003 rows of 48 float32 to 4096 entries: 39 us, the sort 21, the sums 12, the joins 8.  (One
// atomic addition an element would be one launch, but its results would depend on their order.)
// Rows without an entry are one run like the others, whose sum nobody keeps: where they are most of
// many wide rows, its blocks' sums are read by one block (1,000,003 rows of 512 to 4096 entries: 314 us
// with 2 % of them, 528 with half, 747 with 98 %; of 128 columns 125 to 130).
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
    if (row < rows && c.skip < 8) store8_once(y, row, NARROW ? col : c.at, v, NARROW ? cols - col : 8);
  }
}

// ------------------------------------------------------------- the gradient

constexpr int kFlight = 8;     // rows loaded ahead
constexpr int kLong = 32;      // blocks' sums that a run's own lanes add
constexpr uint32_t kNoKey = 0xffffffffu;
// Of a slot, and of a block: no run goes on behind it; the last run, which begins in it; the only run,
// which began in front of it.
enum { kEnds = 0, kBegins = 1, kThrough = 2 };

struct SegArgs {
  MatArg src;               // the rows, in their places
  const uint32_t* key;      // entries, ascending
  const uint32_t* order;    // their places
  MatArg dst;
  float scale;
  uint32_t entries;
  int cols;
  int64_t count, slots, blocks;
  int per_slot, per_block;  // places
  float* part;              // [2 blocks][cols]: of a block, the run that came from before, the run that goes on
  uint32_t* flags;          // [blocks]
  uint8_t* marks;           // [entries]: whether it has rows
  int lanes;
};

// This thread's share of the columns: what is loaded (at), and whether its results are its own.
struct Share {
  Held c;
  int col, at, n;
  bool own;
};

template <bool NARROW>
__device__ inline Share share_of(const SegArgs& a) {
  Share s;
  s.col = (int(blockIdx.y) * a.lanes + (threadIdx.x & (a.lanes - 1))) * 8;
  s.c = held_at(s.col, a.cols);
  s.at = NARROW ? s.col : s.c.at;
  s.n = NARROW ? a.cols - s.col : 8;
  s.own = NARROW ? s.n > 0 : s.c.skip < 8;
  return s;
}

template <bool NARROW>
__device__ inline Raw8 load_share(const MatArg& m, int64_t row, const Share& s) {
  return NARROW ? load_raw8(m, row, s.col, s.n) : load_held(m, row, s.c);
}

__device__ inline void write_entry(const SegArgs& a, const Share& s, uint32_t key, const float sum[8]) {
  if (!s.own || key >= a.entries) return;
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = sum[i] * a.scale;
  store8(a.dst, key, s.at, v, s.n);
}

template <bool NARROW>
__global__ void __launch_bounds__(kThreads) segment_sums_kernel(SegArgs a) {
  __shared__ float heads[kThreads * 8];   // a slot's run that came from before
  __shared__ int states[kThreads];
  const int groups = kThreads / a.lanes, group = threadIdx.x / a.lanes;
  const bool leads = (threadIdx.x & (a.lanes - 1)) == 0 && blockIdx.y == 0;
  const int64_t slot = int64_t(blockIdx.x) * groups + group;
  const Share s = share_of<NARROW>(a);
  const int64_t first = slot * a.per_slot, last = first + a.per_slot < a.count ? first + a.per_slot : a.count;
  const MatArg part{reinterpret_cast<char*>(a.part), nullptr, a.cols, 0, GS_MAT_F32};
  float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  float* head = heads + threadIdx.x * 8;
  uint32_t key = kNoKey;
  int state = kEnds;
  bool block_head = false;    // group 0: its first run came from the block before
  if (slot < a.slots) {
    const uint32_t before = first > 0 ? a.key[first - 1] : kNoKey, behind = last < a.count ? a.key[last] : kNoKey;
    uint32_t keys[kFlight], places[kFlight];
    auto fetch = [&](int64_t p0) {
#pragma unroll
      for (int u = 0; u < kFlight; ++u) {
        const int64_t p = p0 + u < last ? p0 + u : last - 1;
        keys[u] = a.key[p];
        places[u] = a.order[p];
      }
    };
    fetch(first);
    key = keys[0];
    bool from_before = key == before;    // the present run began in front of the slot
    block_head = group == 0 && from_before;
    auto mark = [&]() {
      if (leads && key < a.entries) a.marks[key] = 1;
    };
    if (!from_before) mark();
    for (int64_t p0 = first; p0 < last; p0 += kFlight) {
      Raw8 raw[kFlight];
      uint32_t now[kFlight];
#pragma unroll
      for (int u = 0; u < kFlight; ++u) {
        // the rows of no entry, all alike, are not fetched for nothing
        raw[u] = load_share<NARROW>(a.src, keys[u] < a.entries ? places[u] : 0, s);
        now[u] = keys[u];
      }
      fetch(p0 + kFlight < last ? p0 + kFlight : p0);
#pragma unroll
      for (int u = 0; u < kFlight; ++u) {
        if (p0 + u >= last) break;
        if (now[u] != key) {
          if (!from_before) write_entry(a, s, key, sum);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (from_before) head[i] = sum[i];
            sum[i] = 0.0f;
          }
          from_before = false;
          key = now[u];
          mark();
        }
        float v[8];
        raw8_to_float(raw[u], a.src.type, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] += v[i];
      }
    }
    state = key != behind ? kEnds : from_before ? kThrough : kBegins;
    if (from_before) {
#pragma unroll
      for (int i = 0; i < 8; ++i) head[i] = sum[i];
    } else if (state == kEnds) {
      write_entry(a, s, key, sum);
    }
  }
  states[threadIdx.x] = state;
  __syncthreads();
  auto state_of = [&](int g) { return states[g * a.lanes]; };
  auto add_head = [&](int g) {
    const float* h = heads + (g * a.lanes + (threadIdx.x & (a.lanes - 1))) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] += h[i];
  };
  if (state == kBegins) {    // the run ends in a later slot of the block, or leaves it
    int g = group + 1;
    for (; g < groups; ++g) {
      add_head(g);
      if (state_of(g) != kThrough) break;
    }
    if (g < groups) {
      write_entry(a, s, key, sum);
    } else {
      if (s.own) store8(part, 2 * int64_t(blockIdx.x) + 1, s.at, sum, s.n);
      if (leads) a.flags[blockIdx.x] = kBegins;
    }
  }
  if (block_head) {
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] = head[i];
    int g = 0;
    while (state_of(g) == kThrough && ++g < groups) add_head(g);
    if (s.own) store8(part, 2 * int64_t(blockIdx.x), s.at, sum, s.n);
    if (leads && g == groups) a.flags[blockIdx.x] = kThrough;
  }
  if (leads && state == kEnds && (group == groups - 1 || slot == a.slots - 1)) a.flags[blockIdx.x] = kEnds;
}

// The runs that reach over a block's end, from the blocks in which they begin; and, behind the
// first `joins` blocks, the entries without rows.
template <bool NARROW>
__global__ void __launch_bounds__(kThreads) segment_joins_kernel(SegArgs a, unsigned joins) {
  __shared__ float sums[kThreads * 8];
  __shared__ int marked[kThreads], beyond;
  const int groups = kThreads / a.lanes, group = threadIdx.x / a.lanes;
  const int64_t block = int64_t(blockIdx.x) * groups + group;
  const Share s = share_of<NARROW>(a);
  if (blockIdx.x >= joins) {
    const int64_t first = int64_t(blockIdx.x - joins) * kThreads, mine = first + threadIdx.x;
    marked[threadIdx.x] = a.count > 0 && mine < a.entries ? a.marks[mine] : a.count > 0;
    __syncthreads();
    const float zeros[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int e = group; e < kThreads && first + e < a.entries; e += groups)
      if (!marked[e]) write_entry(a, s, uint32_t(first + e), zeros);
    return;
  }
  const MatArg part{reinterpret_cast<char*>(a.part), nullptr, a.cols, 0, GS_MAT_F32};
  auto add = [&](float sum[8], int64_t row) {
    float v[8];
    raw8_to_float(load_share<NARROW>(part, row, s), GS_MAT_F32, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] += v[i];
  };
  auto key_of = [&](int64_t block) { return a.key[(block + 1) * a.per_block - 1]; };   // (the last block's run does not go on)
  bool is_long = false;
  if (block < a.blocks && a.flags[block] == kBegins) {
    const uint32_t key = key_of(block);
    float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    add(sum, 2 * block + 1);
    int reach = 0;    // the blocks that the run reaches
    for (int i = 1; i <= kLong && reach == 0; i += 8) {
      uint32_t flag[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) flag[u] = a.flags[block + i + u < a.blocks ? block + i + u : a.blocks - 1];
#pragma unroll
      for (int u = 7; u >= 0; --u) reach = flag[u] != kThrough ? i + u : reach;
    }
    is_long = reach == 0;
    if (!is_long) {
#pragma unroll 4
      for (int i = 1; i <= reach; ++i) add(sum, 2 * (block + i));
      write_entry(a, s, key, sum);
    }
  }
  // the long ones, in the order of their blocks
  marked[threadIdx.x] = 0;
  __syncthreads();
  if (is_long && (threadIdx.x & (a.lanes - 1)) == 0) marked[group] = 1;
  __syncthreads();
  for (int g = 0; g < groups; ++g) {
    if (!marked[g]) continue;
    const int64_t from = int64_t(blockIdx.x) * groups + g;
    // the block in which the run ends
    constexpr int kLook = 4;
    int64_t end = from + 1;
    for (;; end += kThreads * kLook) {
      if (threadIdx.x == 0) beyond = kThreads * kLook;
      __syncthreads();
      int at = kThreads * kLook;
#pragma unroll
      for (int u = kLook - 1; u >= 0; --u) {
        const int64_t look = end + u * kThreads + threadIdx.x;
        at = a.flags[look < a.blocks ? look : a.blocks - 1] != kThrough ? u * kThreads + threadIdx.x : at;
      }
      if (at < kThreads * kLook) atomicMin(&beyond, at);
      __syncthreads();
      const int b = beyond;
      __syncthreads();
      if (b < kThreads * kLook) {
        end += b;
        break;
      }
    }
    float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (group == 0) add(sum, 2 * from + 1);
#pragma unroll 8
    for (int64_t at = from + 1 + group; at <= end; at += groups) add(sum, 2 * at);
#pragma unroll
    for (int i = 0; i < 8; ++i) sums[threadIdx.x * 8 + i] = sum[i];
    for (int d = groups / 2; d > 0; d /= 2) {
      __syncthreads();
      if (group < d) {
#pragma unroll
        for (int i = 0; i < 8; ++i) sums[threadIdx.x * 8 + i] = sum[i] += sums[(threadIdx.x + d * a.lanes) * 8 + i];
      }
    }
    if (group == 0) write_entry(a, s, key_of(from), sum);
    __syncthreads();
  }
}

int lanes_for(int cols) {
  int lanes = 1;
  while (lanes < 64 && lanes * 8 < cols) lanes *= 2;
  return lanes;
}

inline size_t align256(size_t b) { return (b + 255) & ~size_t(255); }

// Places of a slot: few enough to give each compute unit four waves.
int per_slot(int64_t rows, int lanes) {
  for (int n = 32; n > 8; n /= 2)
    if (rows * lanes / 64 / n >= 1024) return n;
  return 8;
}

// The sorted indices, the sort's space, and the partial sums.
struct BwdWs {
  uint32_t *key, *order, *flags;
  uint8_t* marks;
  void* sort;
  float* part;
  size_t bytes;
};

BwdWs carve(void* ws, int64_t rows, int cols, int64_t entries) {
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
  w.marks = reinterpret_cast<uint8_t*>(take(size_t(entries)));
  w.sort = take(sort_index_ws_bytes(rows));
  // at least as many blocks as fewer rows take (512 where slots are longest for their number)
  const int lanes = lanes_for(cols), n = per_slot(rows, lanes);
  const int64_t here = div_up(rows, int64_t(n) * (kThreads / lanes)), fewer = n > 8 ? 512 : 0, blocks = here > fewer ? here : fewer;
  w.flags = reinterpret_cast<uint32_t*>(take(size_t(blocks) * 4));
  w.part = reinterpret_cast<float*>(take(size_t(blocks) * 2 * cols * 4));
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

size_t lookup_bwd_ws_bytes(int64_t rows, int cols, int64_t entries) { return carve(nullptr, rows, cols, entries).bytes; }

hipError_t launch_lookup_bwd(const MatArg& dy, const void* index, bool wide, float scale, const MatArg& dtable, int64_t rows,
                             int64_t entries, int cols, void* ws, hipStream_t s) {
  const int lanes = lanes_for(cols);
  const unsigned across = div_up(cols, lanes * 8);
  const BwdWs w = carve(ws, rows, cols, entries);
  const int n = per_slot(rows, lanes), per_block = n * (kThreads / lanes);
  const SegArgs a{dy,      w.key, w.order, dtable,  scale,  uint32_t(entries), cols, rows, (rows + n - 1) / n, div_up(rows, per_block), n, per_block,
                  w.part, w.flags, w.marks, lanes};
  if (rows > 0) {
    const hipError_t e = launch_sort_index(index, wide, uint32_t(rows), uint32_t(entries), w.key, w.order, w.marks, w.sort, s);
    if (e != hipSuccess) return e;
    GSK_PROF("lookup_sums", s);
    const auto kernel = cols < 8 ? &segment_sums_kernel<true> : &segment_sums_kernel<false>;
    kernel<<<dim3(unsigned(a.blocks), across), kThreads, 0, s>>>(a);
  }
  GSK_PROF("lookup_joins", s);
  const auto kernel = cols < 8 ? &segment_joins_kernel<true> : &segment_joins_kernel<false>;
  const unsigned joins = a.blocks > 1 ? div_up(a.blocks, kThreads / lanes) : 0;
  kernel<<<dim3(joins + div_up(entries, kThreads), across), kThreads, 0, s>>>(a, joins);
  return hipGetLastError();
}

}  // namespace gsk
