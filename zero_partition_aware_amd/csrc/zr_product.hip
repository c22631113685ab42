// Products of weights that lie in the ranks' partitions with groups of rows
// (gfx950).
//
// Y[t, n] = sum_k X[t, k] W_g[n, k] for the rows t of group g: a layer's output
// (n = out, k = in) or the gradient of its input (n = in, k = out).  Depending
// on how the weight is stored, k or n is its fast axis; X's is k.
//
// With many rows the products bound it, and behind them the chip's power: MFMAs
// 16 x 16 x 32 on random values reach 2,070 TFLOP/s from registers alone (32 x 32 x
// 16: 1,800; both 2,380 on constant values, at a higher clock), so what counts is
// energy and no less than cycles: operands cross the LDS once a tile and step, in
// tiles as large as the registers hold, and go there straight from memory.  2048
// rows of 128256 x 4096: 1,703 us, 1,264 TFLOP/s; 16384 rows to eight 8192 x 2048
// unevenly: 506 us, 1,086, of which a tenth are tiles that are not full.  With few
// rows the weights' bytes do: 32 rows to eight 8192 x 2048, 268 MB, 58 us, 4.6 TB/s;
// one row of 50257 x 768, 77 MB, 14 us, 5.5.

#include <type_traits>
#include <vector>

#include "zr_tiles.h"

using namespace zr;

namespace {

constexpr int kMaxGroups = 128;   // of one launch

struct Group {
  int64_t w;                   // the weight's first element in the flat space
  int32_t row0, rows;
  int32_t tile0;               // tiles of earlier groups
};
struct ProductArgs {
  const char* part[ZR_MAX_WORLD];
  Group group[kMaxGroups];
  const uint16_t* x;
  void* y;
  float* partial;              // a tile of sums for each piece
  int64_t part_numel;
  double part_inverse;
  int64_t x_stride, y_stride;
  int32_t n;                   // groups
  int32_t depth, cols;         // k's and n's extent
  int32_t col_tiles, tiles, pieces;
  int32_t y_bf16, y_past, world;   // y_past: y goes past the caches
};

// A workgroup's tile of rows and columns, by waves of 16 x 16 blocks, and the
// LDS of kStages steps of kDepth k.
template <int kRows_, int kCols_, int kWavesR_, int kWavesC_, int kDepth_, int kStages_>
struct Shape {
  static constexpr int kRows = kRows_, kCols = kCols_, kDepth = kDepth_;
  static constexpr int kUnits = kDepth / 8, kPhases = kDepth / 32;
  static constexpr int kWavesR = kWavesR_, kWavesC = kWavesC_, kStages = kStages_;
  static constexpr int kThreads = 64 * kWavesR * kWavesC;
  static constexpr int kRowBlocks = kRows / kWavesR / 16, kColBlocks = kCols / kWavesC / 16;
  static constexpr int kXBytes = kRows * kDepth * 2, kWBytes = kCols * kDepth * 2;
  static constexpr int kStage = kXBytes + kWBytes;
  static constexpr int kXLoads = kXBytes / 16 / kThreads, kWLoads = kWBytes / 16 / kThreads;
  static constexpr int kLds = kStages * kStage;
  static_assert(kXLoads * kThreads * 16 == kXBytes && kWLoads * kThreads * 16 == kWBytes, "staging shape");
};

// A matrix whose rows run along k: the 16-byte units of a row's kDepth k are
// exchanged (xor) by its pair (64 k) or four (32 k) of rows, so that sixteen
// lanes that read one unit of sixteen rows use all 64 banks.
template <int kDepth>
__device__ __forceinline__ int exchanged_row(int r, int u) {
  static_assert(kDepth == 32 || kDepth == 64, "a row of LDS");
  return u ^ (kDepth == 64 ? r >> 1 & 7 : r >> 2 & 3);
}
template <int kDepth>
__device__ __forceinline__ int staged_row(int r, int u) { return r * (kDepth * 2) + (exchanged_row<kDepth>(r, u) << 4); }

// Where a weight's part lies: in partition a up to the byte `cut` (counted from the
// part's first one), in b from there to `end`.
struct Source {
  uintptr_t a, b;              // as if the part's first element lay there
  int64_t cut, end;
};
__device__ __forceinline__ Source source_of(const ProductArgs& p, int64_t first, int64_t span) {
  Source s;
  // off by one at most: the estimate has 53 bits
  int k = uniform(static_cast<int>(static_cast<double>(first) * p.part_inverse));
  if (first < k * p.part_numel) --k;
  if (first >= (k + 1) * p.part_numel) ++k;
  const int64_t at = first - k * p.part_numel, left = p.part_numel - at;
  s.cut = left * 2;
  s.end = s.cut + (span > left ? p.part_numel * 2 : 0);
  s.a = reinterpret_cast<uintptr_t>(p.part[k]) + at * 2;
  s.b = span > left ? reinterpret_cast<uintptr_t>(p.part[k + 1]) - s.cut : s.a;
  return s;
}

// Where an element of the flat space lies: the at-th of partition k.
struct Element {
  int32_t k;
  int64_t at;
};
__device__ __forceinline__ Element element_of(const ProductArgs& p, int64_t e) {
  // off by one at most: the estimate has 53 bits
  Element r;
  r.k = static_cast<int32_t>(static_cast<double>(e) * p.part_inverse);
  r.at = e - r.k * p.part_numel;
  if (r.at < 0) --r.k, r.at += p.part_numel;
  if (r.at >= p.part_numel) ++r.k, r.at -= p.part_numel;
  return r;
}

// The last `count` (1 to 8) elements of a unit, zeros behind them.
__device__ __forceinline__ u32x4 last_of(const u32x4& v, int count) {
  uint64_t lo = v[0] | static_cast<uint64_t>(v[1]) << 32, hi = v[2] | static_cast<uint64_t>(v[3]) << 32;
  const int by = 16 * (8 - count);
  if (by >= 64) lo = hi, hi = 0;
  const int rest = by & 63;
  lo = lo >> rest | hi << 1 << (63 - rest);
  hi >>= rest;
  return u32x4{static_cast<uint32_t>(lo), static_cast<uint32_t>(lo >> 32), static_cast<uint32_t>(hi),
               static_cast<uint32_t>(hi >> 32)};
}
// `count` elements one by one, zeros behind them; where(i): the i-th one's address.
// kAtOnce: all eight loads on their way together.
template <bool kAtOnce, typename F>
__device__ __forceinline__ u32x4 gathered(int count, F where) {
  if constexpr (kAtOnce) {
    uint16_t v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = *as_global<uint16_t>(where(i < count ? i : count - 1));
    u32x4 to;
#pragma unroll
    for (int i = 0; i < 8; i += 2)
      to[i / 2] = (i < count ? v[i] : 0u) | (i + 1 < count ? static_cast<uint32_t>(v[i + 1]) << 16 : 0u);
    return to;
  }
  uint64_t lo = 0, hi = 0;
#pragma unroll 1
  for (int i = 0; i < count; ++i) {
    const uint64_t v = *as_global<uint16_t>(where(i));
    if (i < 4) lo |= v << (16 * i);
    else hi |= v << (16 * (i - 4));
  }
  return u32x4{static_cast<uint32_t>(lo), static_cast<uint32_t>(lo >> 32), static_cast<uint32_t>(hi),
               static_cast<uint32_t>(hi >> 32)};
}
// The `count` (8 or fewer) elements at `from`, which lie together, zeros behind
// them.  before: so do eight that end with them.
__device__ __forceinline__ u32x4 row_end(const char* from, int count, bool before) {
  if (count >= 8) return load_at<u32x4, 2>(from);
  if (count > 0 && before) return last_of(load_at<u32x4, 2>(from + 2 * (count - 8)), count);
  return gathered<false>(count, [&](int i) { return from + 2 * i; });
}

// A matrix whose rows run along n: its 16-byte units are exchanged by the row's
// number, so that the four rows that 16 lanes of a transposing read take, and the
// four eight rows on that the next 16 do, lie in different banks.
__device__ __forceinline__ int exchanged_column(int k, int u) { return u ^ (4 * (k & 3)) ^ (2 * (k >> 3 & 1)); }
template <int C>
__device__ __forceinline__ int staged_column(int k, int u) { return k * (C * 2) + (exchanged_column(k, u) << 4); }

// a / b for 0 <= a < 2^23 and b > 0, in a few instructions.
__device__ __forceinline__ int quotient(int a, int b) {
  int q = static_cast<int>(static_cast<float>(a) * __builtin_amdgcn_rcpf(static_cast<float>(b)));
  q = uniform(q);              // off by one at most: |error| < 2^23 * 2^-22 / b + 1
  const int left = a - q * b;
  return left < 0 ? q - 1 : left >= b ? q + 1 : q;
}

// A tile's place.
struct Place {
  const uint16_t* x;           // its first row
  int64_t w;                   // its weight's first element
  int64_t row;                 // its first row in y
  int32_t col;                 // its first column
  int32_t rows, cols;          // of the tile, that are there
};
template <typename S>
__device__ __forceinline__ Place place_of(const ProductArgs& a, int tile) {
  int lo = 0, hi = a.n - 1;    // the last group that starts at or before the tile
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (a.group[mid].tile0 <= tile) lo = mid;
    else hi = mid - 1;
  }
  const Group& g = a.group[lo];
  // bands of eight tiles of rows, walked along the columns
  const int t = tile - g.tile0, row_tiles = (g.rows + S::kRows - 1) / S::kRows;
  const int band = quotient(t, 8 * a.col_tiles), at = t - band * 8 * a.col_tiles;
  const int height = row_tiles - 8 * band < 8 ? row_tiles - 8 * band : 8;
  const int over = quotient(at, height);
  const int r = (8 * band + at - over * height) * S::kRows, c = over * S::kCols;
  Place p;
  p.row = static_cast<int64_t>(g.row0) + r;
  p.x = a.x + p.row * a.x_stride;
  p.w = g.w;
  p.col = c;
  p.rows = g.rows - r < S::kRows ? g.rows - r : S::kRows;
  p.cols = a.cols - c < S::kCols ? a.cols - c : S::kCols;
  return p;
}

// What a unit behind the last k is read from.
__device__ const u32x4 kZeros = {0, 0, 0, 0};

// A thread's unit of each of the kGroups groups of kHigh rows of a step, as bytes:
// the group's are a uniform number, the thread's one of two, in a group that is
// all there and in the one that the last row is in.  Where a row is behind the
// last, one before it is read instead; it is never stored.
template <int kHigh>
struct RowUnits {
  uint32_t all, some;          // the thread's
  uint32_t step;               // bytes a row
  int32_t rows;
  __device__ __forceinline__ RowUnits(int r, int u, int rows_, int64_t step_)
      : step(static_cast<uint32_t>(step_)), rows(rows_) {
    const int last = (rows - 1) % kHigh;
    all = r * step + u * 16;
    some = (r < last ? r : last) * step + u * 16;
  }
  __device__ __forceinline__ uint32_t group(int j) const { return (j * kHigh < rows ? j * kHigh : 0) * step; }
  __device__ __forceinline__ uint32_t unit(int j) const {
    return (j * kHigh < rows ? (j + 1) * kHigh : kHigh) > rows ? some : all;
  }
};

// One step's units of a thread, in registers.
template <typename S>
struct Staged {
  u32x4 x[S::kXLoads], w[S::kWLoads];
};
// A thread's places in the steps of a tile that lies anywhere (kColumns: n is the
// weight's fast axis).  A unit on any address is one load, at the rate of an aligned
// one.
template <typename S, bool kColumns>
struct Anywhere {
  static constexpr int kWWide = kColumns ? S::kCols / 8 : S::kUnits, kWHigh = S::kThreads / kWWide;
  // Beside a Large tile's sums there are no registers for partitions smaller than
  // its part of the weight (they would spill: 2000 rows of 4097 x 4095, 177 to 278 us).
  static constexpr bool kFew = S::kRows <= 128;
  RowUnits<S::kThreads / S::kUnits> xu;
  RowUnits<kWHigh> wu;
  int x_k, w_row, w_unit;      // the first k of the thread's units of x; its row and unit of the weight's
  __device__ __forceinline__ Anywhere(const ProductArgs& a, const Place& p, int tid)
      : xu(tid / S::kUnits, tid % S::kUnits, p.rows, a.x_stride * 2),
        wu(tid / kWWide, unit_of(p, tid) / 8, kColumns ? S::kDepth : p.cols, (kColumns ? a.cols : a.depth) * 2),
        x_k(8 * (tid % S::kUnits)), w_row(tid / kWWide), w_unit(unit_of(p, tid)) {}
  // What is behind the last column is never stored: any unit that is there will do,
  // and the next row's elements behind a row's last.
  static __device__ __forceinline__ int unit_of(const Place& p, int tid) {
    const int u = 8 * (tid % kWWide);
    return kColumns && u >= p.cols ? 0 : u;
  }
  __device__ __forceinline__ void load(Staged<S>& s, const ProductArgs& a, const Place& p, int k0) const {
    const int left = a.depth - k0 < S::kDepth ? a.depth - k0 : S::kDepth;
    const char* rows = reinterpret_cast<const char*>(p.x) + static_cast<int64_t>(k0) * 2;
    const int64_t first = p.w + (kColumns ? static_cast<int64_t>(k0) * a.cols + p.col
                                          : static_cast<int64_t>(p.col) * a.depth + k0);
    const int64_t span = kColumns ? static_cast<int64_t>(left - 1) * a.cols + p.cols
                                  : static_cast<int64_t>(p.cols - 1) * a.depth + left;
    const Source src = source_of(a, first, span);
    uint32_t x_at[S::kXLoads], w_at[S::kWLoads];
#pragma unroll
    for (int j = 0; j < S::kXLoads; ++j) {
      uint32_t off = xu.unit(j);
      ZR_OPAQUE_IN(off, k0);
      x_at[j] = xu.group(j) + off;
    }
    bool plain = left == S::kDepth;
#pragma unroll
    for (int j = 0; j < S::kWLoads; ++j) {
      uint32_t off = wu.unit(j);
      ZR_OPAQUE_IN(off, k0);
      w_at[j] = wu.group(j) + off;
      plain = plain && (w_at[j] + 16ll <= src.cut || (w_at[j] >= src.cut && w_at[j] + 16ll <= src.end));
    }
    // Partitions so small that a step has parts of more than two: each unit's own.
    if constexpr (kFew) {
      if (left == S::kDepth && src.end < span * 2) {
        const char* from[S::kWLoads];
        bool alone = true;
#pragma unroll
        for (int j = 0; j < S::kWLoads; ++j) {
          const Element e = element_of(a, first + w_at[j] / 2);
          alone = alone && e.at + 8 <= a.part_numel;
          from[j] = a.part[e.k] + e.at * 2;
        }
        if (__ballot(!alone) == 0) {
#pragma unroll
          for (int j = 0; j < S::kXLoads; ++j) s.x[j] = load_at<u32x4, 2>(rows + x_at[j]);
#pragma unroll
          for (int j = 0; j < S::kWLoads; ++j) s.w[j] = load_at<u32x4, 2>(from[j]);
          return;
        }
      }
    }
    // A wave whose units are all whole and each in one partition: no branches
    // between its loads, so that each is waited for by itself.
    if (__ballot(!plain) == 0) {
#pragma unroll
      for (int j = 0; j < S::kXLoads; ++j) s.x[j] = load_at<u32x4, 2>(rows + x_at[j]);
#pragma unroll
      for (int j = 0; j < S::kWLoads; ++j)
        s.w[j] = load_at<u32x4, 2>(reinterpret_cast<const char*>((w_at[j] < src.cut ? src.a : src.b) + w_at[j]));
      return;
    }
#pragma unroll
    for (int j = 0; j < S::kXLoads; ++j) {
      s.x[j] = row_end(rows + x_at[j], left - x_k, a.depth >= 8);
    }
#pragma unroll
    for (int j = 0; j < S::kWLoads; ++j) {
      const int64_t at = w_at[j];
      const int count = !kColumns ? left - w_unit : j * kWHigh + w_row < left ? p.cols - w_unit : 0;
      // the eight to load: a unit's, or, behind k's end, those that end with its elements
      const int64_t from = kColumns || count >= 8 ? at : at - 2 * (8 - count);
      const bool in_a = from >= 0 && from + 16 <= src.cut, in_b = from >= src.cut && from + 16 <= src.end;
      auto in_two = [&](int i) {
        const int64_t e = at + 2 * i;
        return reinterpret_cast<const char*>((e < src.cut ? src.a : src.b) + e);
      };
      auto each = [&](int i) {
        const int64_t e = first + at / 2 + i, k = e / a.part_numel;
        return a.part[k] + (e - k * a.part_numel) * 2;
      };
      const int few = count < 8 ? count : 8;
      if (count <= 0) {
        s.w[j] = u32x4{0, 0, 0, 0};
      } else if ((in_a || in_b) && (kColumns || a.depth >= 8)) {
        s.w[j] = row_end(in_two(0), kColumns ? 8 : few, true);
      } else if (at + 2 * few <= src.end) {
        s.w[j] = gathered<true>(few, in_two);
      } else if constexpr (kFew) {   // in a third partition, or one after that
        const Element e = element_of(a, first + at / 2);
        const char* there = a.part[e.k] + e.at * 2;
        if (count >= 8 && e.at + 8 <= a.part_numel)
          s.w[j] = load_at<u32x4, 2>(there);
        else if (a.part_numel >= 8)
          s.w[j] = gathered<true>(few, [&](int i) {
            const int64_t r = e.at + i - a.part_numel;
            return r < 0 ? there + 2 * i : a.part[e.k + 1] + r * 2;
          });
        else
          s.w[j] = gathered<false>(few, each);
      } else {
        s.w[j] = gathered<false>(few, each);
      }
    }
    __builtin_amdgcn_s_waitcnt(0x0070 | 0x0f00);   // vmcnt(0), so that the plain steps' waits are what they need
  }
};
template <typename S, bool kColumns>
__device__ __forceinline__ void store_step(const Staged<S>& s, char* lds, int tid) {
#pragma unroll
  for (int j = 0; j < S::kXLoads; ++j) {
    const int at = j * S::kThreads + tid;
    *reinterpret_cast<u32x4*>(lds + staged_row<S::kDepth>(at / S::kUnits, at % S::kUnits)) = s.x[j];
  }
#pragma unroll
  for (int j = 0; j < S::kWLoads; ++j) {
    constexpr int kPerRow = kColumns ? S::kCols / 8 : S::kUnits;
    const int at = j * S::kThreads + tid, r = at / kPerRow, u = at % kPerRow;
    const int to = kColumns ? staged_column<S::kCols>(r, u) : staged_row<S::kDepth>(r, u);
    *reinterpret_cast<u32x4*>(lds + S::kXBytes + to) = s.w[j];
  }
}

// Steps straight into LDS: rows and partitions on 16 bytes, a tile's part of the
// weight (where n is its fast axis, a step's) in two partitions at most.
template <typename S, bool kColumns>
struct Direct {
  static constexpr int kXHigh = S::kThreads / S::kUnits;
  static constexpr int kWWide = kColumns ? S::kCols / 8 : S::kUnits, kWHigh = S::kThreads / kWWide;
  RowUnits<kXHigh> xu;
  RowUnits<kWHigh> wu;         // where n is the weight's fast axis all its rows are there
  const char* x;               // step 0 of the rows
  uintptr_t w;                 // and of the weight, as if all of it lay in partition k
  uintptr_t w_next;            // in partition k + 1
  int64_t cut;                 // bytes from step 0 to that partition
  int32_t k;
  bool whole;                  // all of the tile's part lies in partition k
  __device__ __forceinline__ Direct(const ProductArgs& a, const Place& p, int k0, int tid)
      : xu(tid / S::kUnits, x_unit(tid), p.rows, a.x_stride * 2),
        wu(tid / kWWide, kColumns && 8 * w_unit(tid) >= p.cols ? 0 : w_unit(tid), kColumns ? S::kDepth : p.cols,
           (kColumns ? a.cols : a.depth) * 2) {
    x = reinterpret_cast<const char*>(uniform(reinterpret_cast<int64_t>(p.x)));
    const int64_t first = p.w + (kColumns ? p.col : static_cast<int64_t>(p.col) * a.depth);
    const int64_t here = first + (kColumns ? static_cast<int64_t>(k0) * a.cols : 0);
    // off by one at most: the estimate has 53 bits
    k = uniform(static_cast<int>(static_cast<double>(here) * a.part_inverse));
    if (here < k * a.part_numel) --k;
    if (here >= (k + 1) * a.part_numel) ++k;
    cut = ((k + 1) * a.part_numel - first) * 2;
    w = uniform(static_cast<int64_t>(reinterpret_cast<uintptr_t>(a.part[k]) + (first - k * a.part_numel) * 2));
    w_next = beyond(a);
    whole = (kColumns ? static_cast<int64_t>(a.depth - 1) * a.cols + p.cols : static_cast<int64_t>(p.cols) * a.depth) * 2 <= cut;
  }
  // The unit of its row that a thread has in every group.
  static __device__ __forceinline__ int x_unit(int tid) {
    static_assert(kXHigh % 16 == 0, "the exchange is the same in each group");
    return exchanged_row<S::kDepth>(tid / S::kUnits, tid % S::kUnits);
  }
  static __device__ __forceinline__ int w_unit(int tid) {
    static_assert(kWHigh % 16 == 0, "the exchange is the same in each group");
    if constexpr (kColumns) return exchanged_column(tid / kWWide, tid % kWWide);
    else return exchanged_row<S::kDepth>(tid / kWWide, tid % kWWide);
  }
  __device__ __forceinline__ uintptr_t beyond(const ProductArgs& a) const {
    return k + 1 < a.world ? reinterpret_cast<uintptr_t>(a.part[k + 1]) - cut : 0;
  }
  // Where the weight's step at k0 lies: steps go on.
  template <bool kAny>
  __device__ __forceinline__ int64_t go_to(const ProductArgs& a, int k0) {
    const int64_t at = kColumns ? static_cast<int64_t>(k0) * a.cols * 2 : k0 * 2;
    if constexpr (kColumns && kAny) {
      while (at >= cut && k + 1 < a.world) {
        ++k;
        w = w_next;
        cut += a.part_numel * 2;
        w_next = beyond(a);
      }
    }
    return at;
  }
  // The step at k0, `at` from go_to.  kAny: of a tile that a partition's end cuts
  // perhaps, perhaps the last, with fewer than kDepth k.
  template <bool kAny>
  __device__ __forceinline__ void load(const ProductArgs& a, int k0, int64_t at, char* lds_x, char* lds_w, int tid,
                                       int wave) const {
    const uintptr_t zeros = reinterpret_cast<uintptr_t>(&kZeros);
    const int left = a.depth - k0;
    const uintptr_t rows = reinterpret_cast<uintptr_t>(x) + k0 * 2;
#pragma unroll
    for (int j = 0; j < S::kXLoads; ++j) {
      // (a uniform address and 32 bits of a lane's, not their sum kept in 64)
      uint32_t off = xu.unit(j);
      ZR_OPAQUE_IN(off, k0);
      uintptr_t there = rows + xu.group(j) + off;
      if constexpr (kAny)
        if (8 * x_unit(tid) >= left) there = zeros;
      __builtin_amdgcn_global_load_lds((const ZR_GLOBAL_AS void*)reinterpret_cast<const char*>(there),
                                       (ZR_LDS_AS void*)(lds_x + (j * S::kThreads + 64 * wave) * 16), 16, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < S::kWLoads; ++j) {
      uint32_t off = wu.unit(j);
      ZR_OPAQUE_IN(off, k0);
      const int64_t of_group = at + wu.group(j);
      uintptr_t there = w + of_group;
      if constexpr (kAny) there = of_group + off < cut ? there : w_next + of_group;
      there += off;
      if constexpr (kAny)
        if ((kColumns ? j * kWHigh + tid / kWWide : 8 * w_unit(tid)) >= left) there = zeros;
      __builtin_amdgcn_global_load_lds((const ZR_GLOBAL_AS void*)reinterpret_cast<const char*>(there),
                                       (ZR_LDS_AS void*)(lds_w + (j * S::kThreads + 64 * wave) * 16), 16, 0, 0);
    }
  }
};

template <typename S>
using Acc = f32x4[S::kColBlocks][S::kRowBlocks];

// The fragments of 32 k that a wave multiplies.
template <typename S>
struct Fragments {
  bf16x8 x[S::kRowBlocks], w[S::kColBlocks];
};

// Reads a staged step.  The weight is the MFMA's first operand: its columns n are
// the accumulators' rows, four of them one after the other in a lane, and X's
// rows the lanes.
template <typename S, bool kColumns>
struct Reader {
  int x, w;                    // a lane's places in the first blocks of a staged step
  __device__ __forceinline__ Reader(int lane, int wave) {
    const int wr = wave / S::kWavesC, wc = wave % S::kWavesC;
    const int u = exchanged_row<S::kDepth>(lane & 15, lane >> 4) << 4;
    x = (wr * S::kRowBlocks * 16 + (lane & 15)) * (S::kDepth * 2) + u;
    if constexpr (kColumns) {
      const int k = 8 * (lane >> 4) + (lane >> 2 & 3), c = wc * S::kColBlocks * 16 + 4 * (lane & 3);
      w = staged_column<S::kCols>(k, c / 8) + (c % 8) * 2;
    } else {
      w = (wc * S::kColBlocks * 16 + (lane & 15)) * (S::kDepth * 2) + u;
    }
  }
  // Blocks lie 16 rows apart, the same exchange in each; four units on is the
  // units' bit 2.
  static __device__ __forceinline__ bf16x8 row(const char* lds, int at, int b, int phase) {
    return __builtin_bit_cast(
        bf16x8, *reinterpret_cast<const u32x4*>(lds + (at ^ (phase << 6)) + b * (16 * S::kDepth * 2)));
  }
  __device__ __forceinline__ bf16x8 read_x(const char* lds_x, int b, int phase) const { return row(lds_x, x, b, phase); }
  __device__ __forceinline__ bf16x8 read_w(const char* lds_w, int b, int phase) const {
    static_assert(S::kColBlocks <= 4 && (S::kColBlocks & (S::kColBlocks - 1)) == 0, "a block is two units: bits 1 and 2");
    if constexpr (kColumns) return read_columns<S::kCols>(lds_w, (w ^ (b << 5)) + 32 * phase * (S::kCols * 2));
    else return row(lds_w, w, b, phase);
  }
  // All of a phase's.
  __device__ __forceinline__ void read(Fragments<S>& f, const char* lds, int phase) const {
#pragma unroll
    for (int b = 0; b < S::kRowBlocks; ++b) f.x[b] = read_x(lds, b, phase);
#pragma unroll
    for (int b = 0; b < S::kColBlocks; ++b) f.w[b] = read_w(lds + S::kXBytes, b, phase);
  }
};

template <typename S>
__device__ __forceinline__ void multiply(Acc<S>& acc, const Fragments<S>& f) {
#pragma unroll
  for (int i = 0; i < S::kColBlocks; ++i)
#pragma unroll
    for (int j = 0; j < S::kRowBlocks; ++j)
      acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f.w[i], f.x[j], acc[i][j], 0, 0, 0);
}

// All waves' LDS reads before it are done after it, and all but the last n of a
// wave's loads have arrived.
template <int n>
__device__ __forceinline__ void meet() {
  ZR_ORDERED();
  __builtin_amdgcn_s_waitcnt((n & 15) | ((n >> 4) << 14) | 0x0070);   // vmcnt(n), lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  ZR_ORDERED();
}

// 32 k of a step.  While they multiply, the next 32's fragments are read: one of
// the rows' behind the products of the one before it, so that their registers are
// the next one's but one, and the last is there when it is wanted.  Once all waves
// have a step's fragments, the step that is kStages on goes into its place, its
// loads between the products: a CU takes a wave's load in 16 cycles, and all
// waves' at once would hold up the products behind them.  The pointers are
// restricted so that the compiler sees that reads of a stage need not wait for
// what goes into another.
template <int kPhase, bool kAny, typename S, bool kColumns>
__device__ __forceinline__ void phase(const ProductArgs& a, const Direct<S, kColumns>& in,
                                      const Reader<S, kColumns>& reader, Acc<S>& acc, const Fragments<S>& now,
                                      Fragments<S>& then, int ahead_k, int64_t ahead_at,
                                      const char* __restrict from_x, const char* __restrict from_w,
                                      char* __restrict ahead_x, char* __restrict ahead_w, int tid, int wave) {
  constexpr bool kLast = kPhase == S::kPhases - 1;
  constexpr int kThen = kLast ? 0 : kPhase + 1;
  constexpr int kLoads = kLast ? S::kXLoads + S::kWLoads : 0;
  static_assert(S::kColBlocks <= S::kRowBlocks, "the weight's fragments behind as many products");
  if constexpr (kLast) {
    meet<(S::kXLoads + S::kWLoads) * (S::kStages - 2)>();
    in.template load<kAny>(a, ahead_k, ahead_at, ahead_x, ahead_w, tid, wave);
  }
  then.x[0] = reader.read_x(from_x, 0, kThen);
#pragma unroll
  for (int j = 0; j < S::kRowBlocks; ++j) {
#pragma unroll
    for (int i = 0; i < S::kColBlocks; ++i)
      acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(now.w[i], now.x[j], acc[i][j], 0, 0, 0);
    if (j + 1 < S::kRowBlocks) then.x[j + 1] = reader.read_x(from_x, j + 1, kThen);
    if (j < S::kColBlocks) then.w[j] = reader.read_w(from_w, j, kThen);
  }
  __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);                                               // LDS read
#pragma unroll
  for (int j = 0; j < S::kRowBlocks; ++j) {
    __builtin_amdgcn_sched_group_barrier(0x008, S::kColBlocks, 0);                                 // MFMAs
    if (j < S::kColBlocks) __builtin_amdgcn_sched_group_barrier(0x100, kColumns ? 3 : 2, 0);       // LDS reads
    else if (j + 1 < S::kRowBlocks) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    constexpr int kEach = (kLoads + S::kRowBlocks - 1) / S::kRowBlocks;
    if (kEach > 0 && j * kEach < kLoads) __builtin_amdgcn_sched_group_barrier(0x010, kEach, 0);    // loads
  }
  __builtin_amdgcn_sched_barrier(0);
}

// A piece of a tile: steps [s0, s1) of its sums.
struct Work {
  Place p;
  int s0, s1, id;
};
template <typename S>
__device__ __forceinline__ Work work_of(const ProductArgs& a, int block) {
  // Consecutive workgroups go round the eight XCDs: of 256, each XCD takes 32
  // neighbours, which share rows in its L2.
  const int all = a.tiles * a.pieces, round = block & ~255, now = all - round < 256 ? all - round : 256;
  const int xcd = block % 8, more = now % 8;
  Work w;
  w.id = round + xcd * (now / 8) + (xcd < more ? xcd : more) + (block - round) / 8;
  const int piece = a.pieces > 1 ? w.id / a.tiles : 0;
  w.p = place_of<S>(a, w.id - piece * a.tiles);
  const int64_t steps = (a.depth + S::kDepth - 1) / S::kDepth;
  w.s0 = 0;
  w.s1 = static_cast<int>(steps);
  if (a.pieces > 1) {
    w.s0 = static_cast<int>(piece * steps / a.pieces);
    w.s1 = static_cast<int>((piece + 1) * steps / a.pieces);
  }
  return w;
}

// kN sums of a lane, at a row of y and columns from c on, `left` of which are there.
template <int kN>
__device__ __forceinline__ void put_sums(const ProductArgs& a, int64_t at, int left, const u32x4& v) {   // bf16 or fp32
  constexpr int kSize = 16 / kN;
  char* p = static_cast<char*>(a.y) + at * kSize;
  if (left >= kN) {
    if (a.y_past) store_once_at<kSize>(p, v);
    else store_at<kSize>(p, v);
  } else {
#pragma unroll
    for (int e = 0; e < kN - 1; ++e)
      if (e < left) {
        if constexpr (kN == 8) reinterpret_cast<uint16_t*>(p)[e] = static_cast<uint16_t>(v[e / 2] >> (16 * (e & 1)));
        else reinterpret_cast<uint32_t*>(p)[e] = v[e];
      }
  }
}

// A piece's sums: into y, or, where there are others of its tile, into the
// workspace.  A lane has four columns of a row: 16 bytes of fp32.  For bf16 it
// exchanges four of one block for four of the next with the lane that has that
// row's following columns, so that both have eight.
template <typename S>
__device__ __forceinline__ void put_tile(const ProductArgs& a, const Work& k, const Acc<S>& acc, int lane, int wave) {
  ZR_OPAQUE(lane);             // places are worked out here, not kept over the products
  const int r0 = wave / S::kWavesC * S::kRowBlocks * 16, c0 = wave % S::kWavesC * S::kColBlocks * 16;
  const int q = lane >> 4;
#pragma unroll
  for (int j = 0; j < S::kRowBlocks; ++j) {
    const int r = r0 + 16 * j + (lane & 15);
    const bool there = r < k.p.rows;
    const int64_t at = (k.p.row + r) * a.y_stride + k.p.col;
#pragma unroll
    for (int i = 0; i < S::kColBlocks; i += 2) {
      if (a.pieces > 1 || !a.y_bf16) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int c = c0 + 16 * (i + h) + 4 * q;
          if (!there) continue;
          if (a.pieces > 1)
            *as_global<f32x4>(a.partial + static_cast<int64_t>(k.id) * (S::kRows * S::kCols) + r * S::kCols + c) =
                acc[i + h][j];
          else
            put_sums<4>(a, at + c, k.p.cols - c, __builtin_bit_cast(u32x4, acc[i + h][j]));
        }
      } else {
        const f32x4 &s = acc[i][j], &t = acc[i + 1][j];
        const u32x2 lo = exchange_rows(pack_bf16(s[0], s[1]), pack_bf16(t[0], t[1]));
        const u32x2 hi = exchange_rows(pack_bf16(s[2], s[3]), pack_bf16(t[2], t[3]));
        const int c = c0 + 16 * (i + (q & 1)) + 8 * (q >> 1);
        if (there) put_sums<8>(a, at + c, k.p.cols - c, u32x4{lo[0], hi[0], lo[1], hi[1]});
      }
    }
  }
}

template <typename S>
__device__ __forceinline__ void clear(Acc<S>& acc) {
#pragma unroll
  for (int i = 0; i < S::kColBlocks; ++i)
#pragma unroll
    for (int j = 0; j < S::kRowBlocks; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
}

// Rows and partitions on 16 bytes.  A workgroup goes through its pieces in one
// stream of steps: while a piece's last steps multiply, and while its sums leave,
// the next one's first are on their way.  (Each piece has a step for every stage,
// behind its last k of zeros.)
template <typename S, bool kColumns>
__global__ __launch_bounds__(S::kThreads, 2) void product_kernel(const ProductArgs a) {
  static_assert(S::kPhases == 2, "phases in step");
  __shared__ __align__(16) char lds[S::kLds];
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int all = a.tiles * a.pieces;
  int block = blockIdx.x;
  Work now = work_of<S>(a, block);
  Direct<S, kColumns> in(a, now.p, now.s0 * S::kDepth, tid);
  constexpr int kEnd = S::kStages * S::kStage;
  auto steps_end = [](const Work& k) { return k.s1 - k.s0 < S::kStages ? k.s0 + S::kStages : k.s1; };
#pragma unroll 1
  for (int i = 0; i < S::kStages; ++i) {
    char* to = lds + i * S::kStage;
    const int k = (now.s0 + i) * S::kDepth;
    const int64_t at = in.template go_to<true>(a, k);
    in.template load<true>(a, k, at, to, to + S::kXBytes, tid, wave);
  }
  meet<(S::kXLoads + S::kWLoads) * (S::kStages - 1)>();
  const Reader<S, kColumns> reader(lane, wave);
  Fragments<S> f[2];
  reader.read(f[0], lds, 0);
  Acc<S> acc = {};
  int cur = 0;
  // A step, while that at k0 of the piece that `in` is in takes its place.
  auto one = [&](auto any, int k0) {
    constexpr bool kAny = decltype(any)::value;
    const int next = cur + S::kStage == kEnd ? 0 : cur + S::kStage;
    const int64_t at = in.template go_to<kAny>(a, k0);
    char* to = lds + cur;
    const char *same = lds + cur, *other = lds + next;
    phase<0, kAny>(a, in, reader, acc, f[0], f[1], k0, at, same, same + S::kXBytes, nullptr, nullptr, tid, wave);
    phase<1, kAny>(a, in, reader, acc, f[1], f[0], k0, at, other, other + S::kXBytes, to, to + S::kXBytes, tid, wave);
    cur = next;
  };
  for (;;) {
    const int end = steps_end(now);
    int s = now.s0;
    // steps whose place a whole one of the same piece takes
    const int plain = a.depth / S::kDepth < now.s1 ? a.depth / S::kDepth : now.s1;
    if (in.whole) {
#pragma unroll 1
      for (; s + S::kStages < plain; ++s) one(std::false_type{}, (s + S::kStages) * S::kDepth);
    }
#pragma unroll 1
    for (; s + S::kStages < end; ++s) one(std::true_type{}, (s + S::kStages) * S::kDepth);
    block += gridDim.x;
    Work then = now;
    const bool more = block < all;
    if (more) {
      then = work_of<S>(a, block);
      in = Direct<S, kColumns>(a, then.p, then.s0 * S::kDepth, tid);
    }
    // behind the last piece zeros, unused
#pragma unroll 1
    for (int i = 0; i < S::kStages; ++i) one(std::true_type{}, more ? (then.s0 + i) * S::kDepth : a.depth);
    put_tile<S>(a, now, acc, lane, wave);
    if (!more) break;
    clear<S>(acc);
    now = then;
  }
  meet<0>();
}

// Rows or partitions anywhere: steps go through registers, kStages - 1 of them on
// their way, into two stages of LDS in turn (the other one's readers are behind the
// last barrier).  2000 rows of 4096 x 4096: 100 us where product_kernel takes 66.
// The rows' own addresses cost nothing (100 us on 16 bytes too); the registers and
// the fragments that are read only when they are wanted do.
template <typename S, bool kColumns>
__global__ __launch_bounds__(S::kThreads, 2) void product_any_kernel(const ProductArgs a) {
  constexpr int kAhead = S::kStages - 1;
  __shared__ __align__(16) char lds[2 * S::kStage];
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const Work k = work_of<S>(a, blockIdx.x);
  const Reader<S, kColumns> reader(lane, wave);
  const Anywhere<S, kColumns> in(a, k.p, tid);
  Acc<S> acc = {};
  Staged<S> next[kAhead];
  // (behind the last step that one again)
  auto load = [&](Staged<S>& to, int s) { in.load(to, a, k.p, (s < k.s1 ? s : k.s1 - 1) * S::kDepth); };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) load(next[i], k.s0 + i);
  int at = 0;
#pragma unroll 1
  for (int s0 = k.s0; s0 < k.s1; s0 += kAhead) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (s0 + i >= k.s1) break;
      store_step<S, kColumns>(next[i], lds + at, tid);
      lds_barrier();
      load(next[i], s0 + i + kAhead);
#pragma unroll
      for (int phase = 0; phase < S::kPhases; ++phase) {
        Fragments<S> f;
        reader.read(f, lds + at, phase);
        multiply<S>(acc, f);
      }
      at = S::kStage - at;
    }
  }
  put_tile<S>(a, k, acc, lane, wave);
}

// Adds up the pieces of each tile, in their order: four sums a thread, the
// columns of 1024 / kCols rows a workgroup.
constexpr int kJoinThreads = 256;
template <typename S>
__global__ __launch_bounds__(kJoinThreads) void product_join_kernel(const ProductArgs a) {
  constexpr int kParts = S::kRows * S::kCols / (4 * kJoinThreads);
  const int tile = blockIdx.x / kParts, at = 4 * ((blockIdx.x % kParts) * kJoinThreads + threadIdx.x);
  const Place p = place_of<S>(a, tile);
  const int r = at / S::kCols, c = at % S::kCols;
  if (r >= p.rows || c >= p.cols) return;
  const float* from = a.partial + static_cast<int64_t>(tile) * (S::kRows * S::kCols) + at;
  const int64_t step = static_cast<int64_t>(a.tiles) * (S::kRows * S::kCols);
  f32x4 sum = *as_global<f32x4>(from);
#pragma unroll 8
  for (int k = 1; k < a.pieces; ++k) sum += *as_global<f32x4>(from + k * step);
  const int64_t to = (p.row + r) * a.y_stride + p.col + c;
  if (!a.y_bf16) {
    put_sums<4>(a, to, p.cols - c, __builtin_bit_cast(u32x4, sum));
  } else {
    uint16_t* y = static_cast<uint16_t*>(a.y) + to;
    const u32x2 v = {pack_bf16(sum[0], sum[1]), pack_bf16(sum[2], sum[3])};
    if (c + 4 <= p.cols) {
      store_at<2>(y, v);
    } else {
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (c + e < p.cols) y[e] = static_cast<uint16_t>(v[e / 2] >> (16 * (e & 1)));
    }
  }
}

// Steps of 64 k, 128 bytes of a row each (of 32 k, twice the stages: rows in pieces
// of 64 bytes come a good deal slower).  Large fills a CU's registers with its
// sums; of the others a CU holds two workgroups, whose loads are on their way while
// the other one multiplies.  us at 4096 x 4096, the best cut of each:
//     rows      64   128   256   512  1024  2048  4096
//     Small     15    20    27    42    70   122   236
//     Low       16    17    24    32    47    85   159
//     Middle    18    21    26    34    51    69   130
//     Large     24    28    34    41    53    80   112
// Small, against Low with 32 rows to eight 8192 x 2048: 59 and 63.
using Large = Shape<256, 256, 2, 4, 64, 2>;
using Middle = Shape<128, 128, 2, 2, 64, 2>;
using Low = Shape<64, 128, 1, 4, 64, 3>;
using Small = Shape<32, 128, 1, 4, 64, 4>;
constexpr int kShapes = 4;
template <typename F>
void with_shape(int shape, F f) {
  if (shape == 0) f(Small{});
  else if (shape == 1) f(Low{});
  else if (shape == 2) f(Middle{});
  else f(Large{});
}

// ---------------------------------------------------------------------- host

#ifndef ZR_CUS
#define ZR_CUS 256   // the chip's; the kernels run on a smaller one in tests on the CPU
#endif
constexpr int64_t kCus = ZR_CUS;

template <typename S>
constexpr int64_t kSlots = kCus * (2 * S::kLds > 160 * 1024 ? 1 : 2);   // workgroups that the chip holds

// What a step costs where a CU has one workgroup and where it has two, and what a
// piece costs beside its steps, in us, measured at 4096 x 4096 with 1 to 4096 rows:
// straight into LDS, and by way of registers.  Elsewhere the second is low: 2304 x
// 768 with 1531 rows 22 for 30, 4097 x 4095 with 2000 rows 146 for 172 to 177.
struct Cost {
  double one, two, piece;
};
template <typename S>
constexpr Cost kCost[2] = {};
template <>
constexpr Cost kCost<Small>[2] = {{0.25, 0.5, 1}, {0.7, 0.9, 1}};
template <>
constexpr Cost kCost<Low>[2] = {{0.37, 0.6, 1}, {0.95, 1.15, 1}};
template <>
constexpr Cost kCost<Middle>[2] = {{0.8, 0.95, 2}, {1.1, 1.45, 2}};
template <>
constexpr Cost kCost<Large>[2] = {{1.45, 1.45, 5}, {2.2, 2.2, 5}};

// What a call has to do.
struct Load {
  int64_t steps, sums;         // of k; rows times columns
  bool any;                    // sizes or places that are no multiples of 16 bytes
};

// What a launch takes, about, with its sums in so many pieces: the rounds of its
// workgroups, and the second launch that joins the pieces, written and read.
template <typename S>
double cost_of(const Load& l, int64_t tiles, int64_t pieces) {
  const Cost& c = kCost<S>[l.any];
  const int64_t items = tiles * pieces;
  const double round = (items > kCus ? c.two : c.one) * static_cast<double>(ceil_div(l.steps, pieces)) + c.piece;
  const double join = pieces == 1 ? 0 : 3 + static_cast<double>(pieces * l.sums) * 4 * 0.32e-6;
  return static_cast<double>(ceil_div(items, kSlots<S>)) * round + join;
}
constexpr int64_t kMaxPieces = 64;
struct Cut {
  int64_t pieces;
  double cost;
};
// In how many pieces, of four steps or more, that is least.
template <typename S>
Cut cut_of(const Load& l, int64_t tiles) {
  Cut best{1, cost_of<S>(l, tiles, 1)};
  const int64_t most = std::min(std::min<int64_t>(kMaxPieces, l.steps / 4), kSlots<S> / std::max<int64_t>(tiles, 1));
  for (int64_t k = 2; k <= most; ++k) {
    const double cost = cost_of<S>(l, tiles, k);
    if (cost < best.cost) best = {k, cost};
  }
  return best;
}

// A launch holds fewer than 2^32 threads (what is cut has few tiles).
constexpr int64_t kMaxTiles = int64_t(1) << 22;

struct Launch {
  ProductArgs a;
  int shape;
  int64_t bytes;
};

// The call's launches; `a` has what they share.
template <typename S>
void add_launches(const ProductArgs& shared, const std::vector<Group>& groups, bool any, int shape,
                  std::vector<Launch>* out) {
  for (size_t k = 0; k < groups.size();) {
    Launch l{};
    l.a = shared;
    l.shape = shape;
    int64_t tiles = 0, rows = 0;
    l.a.col_tiles = static_cast<int32_t>(ceil_div(shared.cols, S::kCols));
    for (; k < groups.size() && l.a.n < kMaxGroups; ++k) {
      const int64_t more = ceil_div(groups[k].rows, S::kRows) * l.a.col_tiles;
      if (l.a.n > 0 && tiles + more > kMaxTiles) break;
      Group g = groups[k];
      g.tile0 = static_cast<int32_t>(std::min(tiles, kMaxTiles));
      l.a.group[l.a.n++] = g;
      tiles += more;
      rows += g.rows;
    }
    l.a.tiles = static_cast<int32_t>(std::min(tiles, kMaxTiles + 1));
    l.a.pieces = static_cast<int32_t>(cut_of<S>(Load{ceil_div(shared.depth, S::kDepth), rows * shared.cols, any}, tiles).pieces);
    l.bytes = l.a.pieces > 1 ? tiles * l.a.pieces * (S::kRows * S::kCols * 4) : 0;
    out->push_back(l);
  }
}

// The shape of a call's tiles: Small where no group has more rows than one of its
// tiles; of the others the one that costs least.
int shape_of(const std::vector<Group>& groups, int64_t rows, int64_t depth, int64_t cols, bool any) {
  int64_t most = 0;
  for (const Group& g : groups) most = std::max<int64_t>(most, g.rows);
  if (most <= Small::kRows) return 0;
  int best = 0;
  double least = 0;
  for (int k = 1; k < kShapes; ++k) {
    with_shape(k, [&](auto s) {
      using S = decltype(s);
      int64_t tiles = 0;
      for (const Group& g : groups) tiles += ceil_div(g.rows, S::kRows) * ceil_div(cols, S::kCols);
      const double cost = cut_of<S>(Load{ceil_div(depth, S::kDepth), rows * cols, any}, tiles).cost;
      if (best == 0 || cost < least) best = k, least = cost;
    });
  }
  return best;
}

// Rows of whole 16-byte units, X's and the weight's (columns: n is its fast axis).
bool whole_units(int64_t depth, int64_t cols, bool columns) { return depth % 8 == 0 && (!columns || cols % 8 == 0); }

// Checks a call and plans its launches.  `input`: the gradient of the input.
zr_status plan_product(const zr_plan* plan, const int64_t* params, const int64_t* counts, int64_t n, int64_t n_out,
                       int64_t n_in, int32_t in_major, bool input, std::vector<Launch>* out, int32_t* group) {
  if (!plan) return fail(ZR_ERR_INVALID, "plan is null");
  if (n < 0) return fail(ZR_ERR_INVALID, "n must be >= 0");
  if (n > 0 && (!params || !counts)) return fail(ZR_ERR_INVALID, "null param or count list");
  if (n_out < 1 || n_in < 1) return fail(ZR_ERR_INVALID, "n_out and n_in must be >= 1");
  // 32-bit offsets in a tile
  if (n_out >= (int64_t(1) << 22) || n_in >= (int64_t(1) << 22))
    return fail(ZR_ERR_UNSUPPORTED, "n_out or n_in of 2^22 or more");
  ProductArgs a{};
  a.depth = static_cast<int32_t>(input ? n_out : n_in);
  a.cols = static_cast<int32_t>(input ? n_in : n_out);
  std::vector<Group> groups;
  bool misplaced = false;      // a weight or a partition that does not begin on 16 bytes
  int64_t row = 0;
  for (int64_t k = 0; k < n; ++k) {
    const int64_t p = params[k];
    if (p < 0 || p >= static_cast<int64_t>(plan->params.size())) return fail(ZR_ERR_INVALID, "param id out of range");
    const ParamInfo& pi = plan->params[p];
    if (k == 0) *group = pi.group;
    if (pi.group != *group) return fail(ZR_ERR_INVALID, "params of one call must share a group");
    if (pi.numel != n_out * n_in) return fail(ZR_ERR_INVALID, "n_out * n_in must be the param's elements");
    if (counts[k] < 0) return fail(ZR_ERR_INVALID, "a count is negative");
    if (counts[k] >= (int64_t(1) << 31) || row + counts[k] >= (int64_t(1) << 31))
      return fail(ZR_ERR_UNSUPPORTED, "2^31 rows or more");
    if (counts[k] > 0) {
      Group g{};
      g.w = pi.offset;
      misplaced = misplaced || pi.offset % 8 != 0 || plan->groups[pi.group].part % 8 != 0;
      g.row0 = static_cast<int32_t>(row);
      g.rows = static_cast<int32_t>(counts[k]);
      groups.push_back(g);
    }
    row += counts[k];
  }
  const bool any = !whole_units(a.depth, a.cols, input != (in_major != 0)) || misplaced;
  const int shape = shape_of(groups, row, a.depth, a.cols, any);
  with_shape(shape, [&](auto s) { add_launches<decltype(s)>(a, groups, any, shape, out); });
  for (const Launch& l : *out)
    if (l.a.tiles > kMaxTiles) return fail(ZR_ERR_UNSUPPORTED, "more tiles than a launch holds");
  return ZR_OK;
}

template <typename S>
zr_status launch_product(const ProductArgs& a, bool columns, bool direct, hipStream_t stream) {
  const int64_t items = int64_t(a.tiles) * a.pieces;
  if (direct) {
    // as many workgroups as the chip holds
    const int64_t grid = std::min(items, kSlots<S>);
    auto* kernel = columns ? product_kernel<S, true> : product_kernel<S, false>;
    ZR_LAUNCH(grid, S::kThreads, stream, a, kernel);
  } else {
    auto* kernel = columns ? product_any_kernel<S, true> : product_any_kernel<S, false>;
    ZR_LAUNCH(items, S::kThreads, stream, a, kernel);
  }
  zr_status st = launched("product launch");
  if (st != ZR_OK || a.pieces == 1) return st;
  ZR_LAUNCH(a.tiles * (S::kRows * S::kCols / (4 * kJoinThreads)), kJoinThreads, stream, a, product_join_kernel<S>);
  return launched("product join launch");
}

zr_status run_product(const zr_plan* plan, const int64_t* params, const int64_t* counts, int64_t n, int64_t n_out,
                      int64_t n_in, int32_t in_major, const void* const* parts, const uint16_t* x, int64_t rows,
                      int64_t x_stride, void* y, zr_dtype y_dtype, int64_t y_stride, void* workspace,
                      int64_t workspace_bytes, bool input, hipStream_t stream) {
  return guarded([&]() -> zr_status {
    std::vector<Launch> launches;
    int32_t group = 0;
    zr_status st = plan_product(plan, params, counts, n, n_out, n_in, in_major, input, &launches, &group);
    if (st != ZR_OK) return st;
    if (!valid_dtype(y_dtype)) return fail(ZR_ERR_INVALID, "unsupported output dtype");
    if (rows < 0) return fail(ZR_ERR_INVALID, "rows must be >= 0");
    int64_t used = 0;
    for (int64_t k = 0; k < n; ++k) used += counts[k];
    if (used > rows) return fail(ZR_ERR_INVALID, "the counts add up to more than the rows");
    const int64_t depth = input ? n_out : n_in, cols = input ? n_in : n_out;
    if (x_stride < depth || y_stride < cols)
      return fail(ZR_ERR_INVALID, "a stride is smaller than its rows");
    if (x_stride >= (int64_t(1) << 22)) return fail(ZR_ERR_UNSUPPORTED, "an input stride of 2^22 or more");
    if (used == 0) return ZR_OK;
    if (!x || !aligned_to(x, 2)) return fail(ZR_ERR_INVALID, "the input is null or not element-aligned");
    if (!y || !aligned_to(y, dtype_size(y_dtype))) return fail(ZR_ERR_INVALID, "the output is null or not element-aligned");
    if (!parts) return fail(ZR_ERR_INVALID, "null partition list");
    const GroupInfo& gi = plan->groups[group];
    bool aligned = gi.part % 8 == 0;
    for (int64_t k = 0; k < n; ++k) {
      if (counts[k] == 0) continue;
      const ParamInfo& pi = plan->params[params[k]];
      for (int32_t r : pi.partitions) {
        if (!parts[r] || !aligned_to(parts[r], 2))
          return fail(ZR_ERR_INVALID, "partition " + std::to_string(r) + " is null or not element-aligned");
        aligned = aligned && aligned_to(parts[r], 16);
      }
      aligned = aligned && pi.offset % 8 == 0;
    }
    // The weight's fast axis is k where it is stored as the product sums it.
    const bool columns = input != (in_major != 0);
    for (const Launch& l : launches)
      if (l.bytes > 0 && (!workspace || !aligned_to(workspace, 16) || workspace_bytes < l.bytes))
        return fail(ZR_ERR_INVALID, "workspace is null, not 16-byte aligned or smaller than " +
                                        std::to_string(l.bytes) + " bytes");
    // An output that the last-level cache (256 MB) does not hold beside the inputs
    // would only drive those out of it: 16384 x 8192 from 2048, 268 MB in all, 417 us
    // past the caches and 445 through them; 8192 x 4096 from 4096, 67 MB, 191 and 187.
    const bool past = used * cols * dtype_size(y_dtype) > (int64_t(128) << 20);
    for (Launch& l : launches) {
      ProductArgs& a = l.a;
      for (int r = 0; r < gi.world; ++r) a.part[r] = static_cast<const char*>(parts[r]);
      a.x = x;
      a.y = y;
      a.partial = static_cast<float*>(workspace);
      a.part_numel = gi.part;
      a.part_inverse = 1.0 / static_cast<double>(gi.part);
      a.world = gi.world;
      a.x_stride = x_stride;
      a.y_stride = y_stride;
      a.y_bf16 = y_dtype == ZR_BF16;
      a.y_past = past;
      // a step's part of the weight, in two partitions at most
      const bool whole = aligned_to(x, 16) && x_stride % 8 == 0 && whole_units(depth, cols, columns);
      with_shape(l.shape, [&](auto s) {
        using S = decltype(s);
        const int64_t span = columns ? std::min<int64_t>(S::kDepth, depth) * cols : std::min<int64_t>(S::kCols, cols) * depth;
        st = launch_product<S>(a, columns, aligned && whole && span <= gi.part, stream);
      });
      if (st != ZR_OK) return st;
    }
    return ZR_OK;
  });
}

zr_status workspace_of(const zr_plan* plan, const int64_t* params, const int64_t* counts, int64_t n, int64_t n_out,
                       int64_t n_in, int32_t in_major, bool input, int64_t* bytes) {
  return guarded([&]() -> zr_status {
    if (!bytes) return fail(ZR_ERR_INVALID, "null output pointer");
    *bytes = 0;
    std::vector<Launch> launches;
    int32_t group = 0;
    const zr_status st = plan_product(plan, params, counts, n, n_out, n_in, in_major, input, &launches, &group);
    if (st != ZR_OK) return st;
    for (const Launch& l : launches) *bytes = std::max(*bytes, l.bytes);
    return ZR_OK;
  });
}

}  // namespace

extern "C" zr_status zr_linear_forward_workspace(const zr_plan* plan, const int64_t* params, const int64_t* counts,
                                                 int64_t n, int64_t n_out, int64_t n_in, int32_t in_major,
                                                 int64_t* bytes) {
  return workspace_of(plan, params, counts, n, n_out, n_in, in_major, false, bytes);
}

extern "C" zr_status zr_linear_input_grad_workspace(const zr_plan* plan, const int64_t* params,
                                                    const int64_t* counts, int64_t n, int64_t n_out, int64_t n_in,
                                                    int32_t in_major, int64_t* bytes) {
  return workspace_of(plan, params, counts, n, n_out, n_in, in_major, true, bytes);
}

extern "C" zr_status zr_linear_forward(const zr_plan* plan, const int64_t* params, const int64_t* counts, int64_t n,
                                       int64_t n_out, int64_t n_in, int32_t in_major, const void* const* parts,
                                       const uint16_t* x, int64_t rows, int64_t x_stride, void* y, zr_dtype y_dtype,
                                       int64_t y_stride, void* workspace, int64_t workspace_bytes,
                                       hipStream_t stream) {
  return run_product(plan, params, counts, n, n_out, n_in, in_major, parts, x, rows, x_stride, y, y_dtype, y_stride,
                     workspace, workspace_bytes, false, stream);
}

extern "C" zr_status zr_linear_input_grad(const zr_plan* plan, const int64_t* params, const int64_t* counts,
                                          int64_t n, int64_t n_out, int64_t n_in, int32_t in_major,
                                          const void* const* parts, const uint16_t* dy, int64_t rows,
                                          int64_t dy_stride, void* dx, zr_dtype dx_dtype, int64_t dx_stride,
                                          void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  return run_product(plan, params, counts, n, n_out, n_in, in_major, parts, dy, rows, dy_stride, dx, dx_dtype,
                     dx_stride, workspace, workspace_bytes, true, stream);
}
