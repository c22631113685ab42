// Products of weights that lie in the ranks' partitions with groups of rows
// (gfx950).
//
// Y[t, n] = sum_k X[t, k] W_g[n, k] for the rows t of group g: a layer's output
// (n = out, k = in) or the gradient of its input (n = in, k = out).  Depending
// on how the weight is stored, k or n is its fast axis; X's is k.

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
  int64_t x_stride, y_stride;
  int32_t n;                   // groups
  int32_t depth, cols;         // k's and n's extent
  int32_t col_tiles, tiles, pieces;
  int32_t y_bf16, world;
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

// Where a weight's tile lies: in partition a up to the element `cut` (counted
// from the tile's first one), in b from there on.  more: in others too.
struct Source {
  uintptr_t a, b;              // as if the tile's first element lay there
  int64_t cut;
  bool more;
};
__device__ __forceinline__ Source source_of(const ProductArgs& p, int64_t first, int64_t span) {
  Source s;
  const int64_t k = first / p.part_numel, at = first - k * p.part_numel;
  s.cut = p.part_numel - at;
  s.more = span > s.cut + p.part_numel;
  s.a = reinterpret_cast<uintptr_t>(p.part[k]) + at * 2;
  s.b = span > s.cut ? reinterpret_cast<uintptr_t>(p.part[k + 1]) - s.cut * 2 : s.a;
  return s;
}

// `count` (1 to 8) elements from the e-th of a tile on.
__device__ __forceinline__ u32x4 source_unit(const ProductArgs& p, const Source& s, int64_t first, int64_t e,
                                             int count) {
  const char* from = nullptr;
  if (s.more) {
    const int64_t k = (first + e) / p.part_numel, at = first + e - k * p.part_numel;
    if (at + count <= p.part_numel) from = p.part[k] + at * 2;
  } else if (e + count <= s.cut) {
    from = reinterpret_cast<const char*>(s.a + e * 2);
  } else if (e >= s.cut) {
    from = reinterpret_cast<const char*>(s.b + e * 2);
  }
  if (from && count == 8) return load_at<u32x4, 2>(from);
  u32x4 v = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (i >= count) continue;
    const char* q;
    if (from) {
      q = from + 2 * i;
    } else {
      const int64_t k = (first + e + i) / p.part_numel;
      q = p.part[k] + (first + e + i - k * p.part_numel) * 2;
    }
    v[i / 2] |= static_cast<uint32_t>(*as_global<uint16_t>(q)) << (16 * (i & 1));
  }
  return v;
}
__device__ __forceinline__ u32x4 row_unit(const uint16_t* x, int count) {
  if (count == 8) return load_at<u32x4, 2>(x);
  u32x4 v = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < count) v[i / 2] |= static_cast<uint32_t>(*as_global<uint16_t>(x + i)) << (16 * (i & 1));
  return v;
}

// A matrix whose rows run along n: its 16-byte units are exchanged by the row's
// number, so that the four rows that 16 lanes of a transposing read take, and the
// four eight rows on that the next 16 do, lie in different banks.
__device__ __forceinline__ int exchanged_column(int k, int u) { return u ^ (4 * (k & 3)) ^ (2 * (k >> 3 & 1)); }
template <int C>
__device__ __forceinline__ int staged_column(int k, int u) { return k * (C * 2) + (exchanged_column(k, u) << 4); }

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
  const int band = t / (8 * a.col_tiles), at = t - band * 8 * a.col_tiles;
  const int height = row_tiles - 8 * band < 8 ? row_tiles - 8 * band : 8;
  const int r = (8 * band + at % height) * S::kRows, c = at / height * S::kCols;
  Place p;
  p.row = static_cast<int64_t>(g.row0) + r;
  p.x = a.x + p.row * a.x_stride;
  p.w = g.w;
  p.col = c;
  p.rows = g.rows - r < S::kRows ? g.rows - r : S::kRows;
  p.cols = a.cols - c < S::kCols ? a.cols - c : S::kCols;
  return p;
}

// One step's units of a thread, in registers.
template <typename S>
struct Staged {
  u32x4 x[S::kXLoads], w[S::kWLoads];
};
// kColumns: n is the weight's fast axis.
template <typename S, bool kColumns>
__device__ __forceinline__ void load_step(Staged<S>& s, const ProductArgs& a, const Place& p, int k0, int tid) {
  const int left = a.depth - k0 < S::kDepth ? a.depth - k0 : S::kDepth;
#pragma unroll
  for (int j = 0; j < S::kXLoads; ++j) {
    const int at = j * S::kThreads + tid, r = at / S::kUnits, u = 8 * (at % S::kUnits);
    s.x[j] = u32x4{0, 0, 0, 0};
    if (r < p.rows && u < left)
      s.x[j] = row_unit(p.x + r * a.x_stride + k0 + u, left - u < 8 ? left - u : 8);
  }
  const int64_t first = p.w + (kColumns ? static_cast<int64_t>(k0) * a.cols + p.col
                                        : static_cast<int64_t>(p.col) * a.depth + k0);
  const int64_t span = kColumns ? static_cast<int64_t>(left - 1) * a.cols + p.cols
                                : static_cast<int64_t>(p.cols - 1) * a.depth + left;
  const Source src = source_of(a, first, span);
#pragma unroll
  for (int j = 0; j < S::kWLoads; ++j) {
    constexpr int kPerRow = kColumns ? S::kCols / 8 : S::kUnits;
    const int at = j * S::kThreads + tid, r = at / kPerRow, u = 8 * (at % kPerRow);
    const int high = kColumns ? left : p.cols, wide = kColumns ? p.cols : left;
    s.w[j] = u32x4{0, 0, 0, 0};
    if (r < high && u < wide)
      s.w[j] = source_unit(a, src, first, static_cast<int64_t>(r) * (kColumns ? a.cols : a.depth) + u,
                           wide - u < 8 ? wide - u : 8);
  }
}
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

// Whole steps straight into LDS: rows and partitions on 16 bytes, a tile's part
// of the weight (where n is its fast axis, a step's) in two partitions at most,
// or all in one (kCut false).
// Where a row or column is behind the last, the tile's first is read instead; it
// is never stored.
template <typename S, bool kColumns, bool kCut>
struct Direct {
  uint32_t x_off[S::kXLoads], w_off[S::kWLoads];   // a thread's bytes from a step's start
  const char* x;               // step 0 of the rows
  uintptr_t w;                 // and of the weight, as if all of it lay in partition k
  uintptr_t w_next;            // in partition k + 1
  int64_t cut;                 // bytes from step 0 to that partition
  int32_t k;
  __device__ __forceinline__ Direct(const ProductArgs& a, const Place& p, int k0, int tid) {
#pragma unroll
    for (int j = 0; j < S::kXLoads; ++j) {
      const int at = j * S::kThreads + tid, r = at / S::kUnits, u = exchanged_row<S::kDepth>(r, at % S::kUnits);
      x_off[j] = (r < p.rows ? r : 0) * static_cast<uint32_t>(a.x_stride * 2) + u * 16;
    }
#pragma unroll
    for (int j = 0; j < S::kWLoads; ++j) {
      if constexpr (kColumns) {
        constexpr int kPerRow = S::kCols / 8;
        const int at = j * S::kThreads + tid, r = at / kPerRow, u = exchanged_column(r, at % kPerRow);
        w_off[j] = r * static_cast<uint32_t>(a.cols * 2) + (8 * u < p.cols ? u : 0) * 16;
      } else {
        const int at = j * S::kThreads + tid, r = at / S::kUnits, u = exchanged_row<S::kDepth>(r, at % S::kUnits);
        w_off[j] = (r < p.cols ? r : 0) * static_cast<uint32_t>(a.depth * 2) + u * 16;
      }
    }
    x = reinterpret_cast<const char*>(p.x);
    const int64_t first = p.w + (kColumns ? p.col : static_cast<int64_t>(p.col) * a.depth);
    const int64_t here = first + (kColumns ? static_cast<int64_t>(k0) * a.cols : 0);
    k = static_cast<int>(here / a.part_numel);
    cut = ((k + 1) * a.part_numel - first) * 2;
    w = reinterpret_cast<uintptr_t>(a.part[k]) + (first - k * a.part_numel) * 2;
    w_next = beyond(a);
  }
  __device__ __forceinline__ uintptr_t beyond(const ProductArgs& a) const {
    return k + 1 < a.world ? reinterpret_cast<uintptr_t>(a.part[k + 1]) - cut : 0;
  }
  // Where the weight's step at k0 lies: steps go on.
  __device__ __forceinline__ int64_t go_to(const ProductArgs& a, int k0) {
    const int64_t at = kColumns ? static_cast<int64_t>(k0) * a.cols * 2 : k0 * 2;
    if constexpr (kColumns && kCut) {
      while (at >= cut) {
        ++k;
        w = w_next;
        cut += a.part_numel * 2;
        w_next = beyond(a);
      }
    }
    return at;
  }
  // The step at k0, `at` from go_to.
  __device__ __forceinline__ void load(int k0, int64_t at, char* lds_x, char* lds_w, int wave) const {
    const char* from = x + k0 * 2;
#pragma unroll
    for (int j = 0; j < S::kXLoads; ++j)
      __builtin_amdgcn_global_load_lds((const ZR_GLOBAL_AS void*)(from + x_off[j]),
                                       (ZR_LDS_AS void*)(lds_x + (j * S::kThreads + 64 * wave) * 16), 16, 0, 0);
#pragma unroll
    for (int j = 0; j < S::kWLoads; ++j) {
      uintptr_t there = w + at;
      if constexpr (kCut) there = at + w_off[j] < cut ? there : w_next + at;
      there += w_off[j];
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
  int x[S::kRowBlocks], w[S::kColBlocks];   // a lane's places in a staged step
  int lane;
  __device__ __forceinline__ Reader(int lane_, int wave) : lane(lane_) {
    const int wr = wave / S::kWavesC, wc = wave % S::kWavesC;
#pragma unroll
    for (int b = 0; b < S::kRowBlocks; ++b) x[b] = ((wr * S::kRowBlocks + b) * 16 + (lane & 15)) * (S::kDepth * 2);
    const int k = 8 * (lane >> 4) + (lane >> 2 & 3), c = 4 * (lane & 3);
#pragma unroll
    for (int b = 0; b < S::kColBlocks; ++b) {
      if constexpr (kColumns) {
        const int at = (wc * S::kColBlocks + b) * 16 + c;
        w[b] = staged_column<S::kCols>(k, at / 8) + (at % 8) * 2;
      } else {
        w[b] = ((wc * S::kColBlocks + b) * 16 + (lane & 15)) * (S::kDepth * 2);
      }
    }
  }
  __device__ __forceinline__ bf16x8 row(const char* lds, int at, int phase) const {
    const int u = exchanged_row<S::kDepth>(lane & 15, 4 * phase + (lane >> 4));
    return __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(lds + at + (u << 4)));
  }
  __device__ __forceinline__ void read(Fragments<S>& f, const char* lds_x, const char* lds_w, int phase) const {
#pragma unroll
    for (int b = 0; b < S::kRowBlocks; ++b) f.x[b] = row(lds_x, x[b], phase);
#pragma unroll
    for (int b = 0; b < S::kColBlocks; ++b) {
      if constexpr (kColumns) f.w[b] = read_columns<S::kCols>(lds_w, w[b] + 32 * phase * (S::kCols * 2));
      else f.w[b] = row(lds_w, w[b], phase);
    }
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
template <typename S, bool kColumns>
__device__ __forceinline__ void multiply_step(Acc<S>& acc, const Reader<S, kColumns>& reader, const char* lds) {
#pragma unroll
  for (int phase = 0; phase < S::kPhases; ++phase) {
    Fragments<S> f;
    reader.read(f, lds, lds + S::kXBytes, phase);
    multiply<S>(acc, f);
  }
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

// 32 k of a step.  While they multiply, the next 32's fragments are read.  Once
// all waves have a step's fragments, the step that is kStages on goes into its
// place, its loads between the products: a CU takes a wave's load in 16 cycles,
// and all waves' at once would hold up the products behind them.  The pointers
// are restricted so that the compiler sees that reads of a stage need not wait
// for what goes into another.
template <int kPhase, typename S, bool kColumns, bool kCut>
__device__ __forceinline__ void phase(const Direct<S, kColumns, kCut>& in, const Reader<S, kColumns>& reader,
                                      Acc<S>& acc, const Fragments<S>& now, Fragments<S>& then, int ahead_k,
                                      int64_t ahead_at, const char* __restrict cur, const char* __restrict next,
                                      char* __restrict ahead_x, char* __restrict ahead_w, int wave) {
  constexpr bool kLast = kPhase == S::kPhases - 1;
  if constexpr (kLast) {
    meet<(S::kXLoads + S::kWLoads) * (S::kStages - 2)>();
    reader.read(then, next, next + S::kXBytes, 0);
    in.load(ahead_k, ahead_at, ahead_x, ahead_w, wave);
  } else {
    reader.read(then, cur, cur + S::kXBytes, kPhase + 1);
  }
  multiply<S>(acc, now);
  // Reads behind the first products, loads between them, and nothing over the
  // phase's end.
  constexpr int kReads = S::kRowBlocks + S::kColBlocks * (kColumns ? 2 : 1), kProducts = S::kRowBlocks * S::kColBlocks;
  constexpr int kLoads = kLast ? S::kXLoads + S::kWLoads : 0;
  constexpr int kBehind = (kReads + kProducts - 1) / kProducts, kApart = kProducts / (kLoads > 0 ? kLoads : 1);
#pragma unroll
  for (int i = 0; i < kProducts; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                                     // MFMA
    if (i * kBehind < kReads) __builtin_amdgcn_sched_group_barrier(0x100, kBehind, 0);     // LDS read
    if (kApart > 0 && i % kApart == kApart / 2 && i / kApart < kLoads)
      __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);                                   // load
  }
  __builtin_amdgcn_sched_barrier(0);
}
// The whole steps [s, whole) through a ring of stages.
template <typename S, bool kColumns, bool kCut>
__device__ __forceinline__ void whole_steps(const ProductArgs& a, const Place& p, const Reader<S, kColumns>& reader,
                                            Acc<S>& acc, int s, int whole, char* lds, int tid, int wave) {
  static_assert(S::kPhases == 1 || S::kPhases == 2, "phases in step");
  Direct<S, kColumns, kCut> in(a, p, s * S::kDepth, tid);
  // behind the last step, the last is loaded again, unused
  auto step = [&](int n) { return (n < whole ? n : whole - 1) * S::kDepth; };
  constexpr int kEnd = S::kStages * S::kStage;
#pragma unroll
  for (int i = 0; i < S::kStages; ++i) {
    char* to = lds + i * S::kStage;
    const int k = step(s + i);
    const int64_t at = in.go_to(a, k);
    in.load(k, at, to, to + S::kXBytes, wave);
  }
  meet<(S::kXLoads + S::kWLoads) * (S::kStages - 1)>();
  Fragments<S> f[2];
  reader.read(f[0], lds, lds + S::kXBytes, 0);
  int cur = 0;
  auto one = [&](Fragments<S>& now, Fragments<S>& then) {
    const int next = cur + S::kStage == kEnd ? 0 : cur + S::kStage;
    const int k = step(s + S::kStages);
    const int64_t at = in.go_to(a, k);
    char* to = lds + cur;
    if constexpr (S::kPhases == 1) {
      phase<0>(in, reader, acc, now, then, k, at, lds + cur, lds + next, to, to + S::kXBytes, wave);
    } else {
      phase<0>(in, reader, acc, now, then, k, at, lds + cur, lds + next, to, to + S::kXBytes, wave);
      phase<1>(in, reader, acc, then, now, k, at, lds + cur, lds + next, to, to + S::kXBytes, wave);
    }
    cur = next;
    return ++s < whole;
  };
  if constexpr (S::kPhases == 1) {
#pragma unroll 1
    while (one(f[0], f[1]) && one(f[1], f[0])) {
    }
  } else {
#pragma unroll 1
    while (one(f[0], f[1])) {
    }
  }
  meet<0>();
}

// Four sums of a lane, at a row of y and columns from n on.
__device__ __forceinline__ void put_sums(const ProductArgs& a, int64_t row, int64_t n, const f32x4& s) {
  const int64_t at = row * a.y_stride + n;
  const int64_t left = a.cols - n;
  if (a.y_bf16) {
    uint16_t* y = static_cast<uint16_t*>(a.y) + at;
    const u32x2 v = {pack_bf16(s[0], s[1]), pack_bf16(s[2], s[3])};
    if (left >= 4) {
      store_at<2>(y, v);
    } else {
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (i < left) y[i] = static_cast<uint16_t>(v[i / 2] >> (16 * (i & 1)));
    }
  } else {
    float* y = static_cast<float*>(a.y) + at;
    if (left >= 4) {
      store_at<4>(y, s);
    } else {
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (i < left) y[i] = s[i];
    }
  }
}

// A wave's sums into y, 32 rows at a time by way of its own LDS, so that a row's
// columns leave together: a lane has four of them, of one row.  Rows of LDS are
// exchanged like staged ones.
template <typename S, bool kBf16>
__device__ __forceinline__ void store_tile(const ProductArgs& a, const Place& p, const Acc<S>& acc, char* lds, int lane,
                                           int wave) {
  constexpr int kSize = kBf16 ? 2 : 4, kRow = S::kColBlocks * 16 * kSize, kU = kRow / 16, kPer = 16 / kSize;
  static_assert(2 * 32 * kRow <= S::kStages * S::kStage / (S::kThreads / 64), "a wave's share of the LDS");
  static_assert((16 % kU == 0 || kU % 16 == 0) && S::kRowBlocks % 2 == 0, "units of a row, rows of a pass");
  constexpr int kRowsABank = kU < 16 ? 16 / kU : 1;   // rows that the 64 banks hold
  auto place = [&](int r, int u) { return r * kRow + ((u ^ (r / kRowsABank & ((kU < 16 ? kU : 16) - 1))) << 4); };
  const int r0 = wave / S::kWavesC * S::kRowBlocks * 16, c0 = wave % S::kWavesC * S::kColBlocks * 16;
#pragma unroll
  for (int j = 0; j < S::kRowBlocks / 2; ++j) {
    if (r0 + 32 * j >= p.rows) break;
    char* at = lds + (j & 1) * (32 * kRow);
#pragma unroll
    for (int i = 0; i < S::kColBlocks; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const f32x4& s = acc[i][2 * j + h];
        const int r = 16 * h + (lane & 15), q = lane >> 4;
        if constexpr (kBf16)
          *reinterpret_cast<u32x2*>(at + place(r, 2 * i + (q >> 1)) + 8 * (q & 1)) =
              u32x2{pack_bf16(s[0], s[1]), pack_bf16(s[2], s[3])};
        else
          *reinterpret_cast<f32x4*>(at + place(r, 4 * i + q)) = s;
      }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int q = 0; q < 32 * kU / 64; ++q) {
      const int r = q * (64 / kU) + lane / kU, u = lane % kU, c = c0 + u * kPer;
      const u32x4 v = *reinterpret_cast<const u32x4*>(at + place(r, u));
      if (r0 + 32 * j + r >= p.rows || c >= p.cols) continue;
      char* y = static_cast<char*>(a.y) + ((p.row + r0 + 32 * j + r) * a.y_stride + p.col + c) * kSize;
      if (c + kPer <= p.cols) {
        store_at<kSize>(y, v);
      } else {
#pragma unroll
        for (int e = 0; e < kPer - 1; ++e)
          if (c + e < p.cols) {
            if constexpr (kBf16) reinterpret_cast<uint16_t*>(y)[e] = static_cast<uint16_t>(v[e / 2] >> (16 * (e & 1)));
            else reinterpret_cast<uint32_t*>(y)[e] = v[e];
          }
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
}

template <typename S, bool kColumns, bool kDirect>
__global__ __launch_bounds__(S::kThreads) void product_kernel(const ProductArgs a) {
  __shared__ __align__(16) char lds[S::kStages * S::kStage];
  const int tid = threadIdx.x, lane = tid & 63, w = uniform(tid >> 6);
  // Consecutive workgroups go round the eight XCDs: of the 256 that run at
  // once, each XCD takes 32 neighbours, which share rows in its L2.
  const int round = blockIdx.x & ~255;
  const int now = static_cast<int>(gridDim.x) - round < 256 ? gridDim.x - round : 256;
  const int xcd = blockIdx.x % 8, more = now % 8;
  const int id = round + xcd * (now / 8) + (xcd < more ? xcd : more) + (blockIdx.x - round) / 8;
  const int piece = id / a.tiles, tile = id - piece * a.tiles;
  const Place p = place_of<S>(a, tile);
  const int64_t all = (a.depth + S::kDepth - 1) / S::kDepth;
  const int s0 = static_cast<int>(piece * all / a.pieces), s1 = static_cast<int>((piece + 1) * all / a.pieces);
  const Reader<S, kColumns> reader(lane, w);
  Acc<S> acc = {};
  int s = s0;
  if constexpr (kDirect) {
    const int whole = s1 < a.depth / S::kDepth ? s1 : a.depth / S::kDepth;
    if (s < whole) {
      // the tile's part of the weight, all of one partition or not
      const int64_t first = p.w + (kColumns ? 0 : static_cast<int64_t>(p.col) * a.depth);
      const int64_t end = p.w + (kColumns ? static_cast<int64_t>(a.cols) : p.col + p.cols) * a.depth;
      if (first / a.part_numel == (end - 1) / a.part_numel)
        whole_steps<S, kColumns, false>(a, p, reader, acc, s, whole, lds, tid, w);
      else
        whole_steps<S, kColumns, true>(a, p, reader, acc, s, whole, lds, tid, w);
      s = whole;
    }
  }
  if (s < s1) {
    Staged<S> next;
    load_step<S, kColumns>(next, a, p, s * S::kDepth, tid);
    for (; s < s1; ++s) {
      lds_barrier();
      store_step<S, kColumns>(next, lds, tid);
      lds_barrier();
      if (s + 1 < s1) load_step<S, kColumns>(next, a, p, (s + 1) * S::kDepth, tid);
      multiply_step<S, kColumns>(acc, reader, lds);
    }
  }
  if (a.pieces == 1) {
    lds_barrier();             // the stages are read
    char* own = lds + w * (S::kStages * S::kStage / (S::kThreads / 64));
    if (a.y_bf16) store_tile<S, true>(a, p, acc, own, lane, w);
    else store_tile<S, false>(a, p, acc, own, lane, w);
    return;
  }
  const int wr = w / S::kWavesC, wc = w % S::kWavesC;
#pragma unroll
  for (int j = 0; j < S::kRowBlocks; ++j) {
    const int r = (wr * S::kRowBlocks + j) * 16 + (lane & 15);
    if (r >= p.rows) continue;
#pragma unroll
    for (int i = 0; i < S::kColBlocks; ++i) {
      const int c = (wc * S::kColBlocks + i) * 16 + 4 * (lane >> 4);
      *as_global<f32x4>(a.partial + static_cast<int64_t>(id) * (S::kRows * S::kCols) + r * S::kCols + c) = acc[i][j];
    }
  }
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
  for (int k = 1; k < a.pieces; ++k) sum += *as_global<f32x4>(from + k * step);
  put_sums(a, p.row + r, p.col + c, sum);
}

using Large = Shape<256, 256, 2, 4, 64, 2>;
using Small = Shape<32, 128, 1, 4, 64, 4>;

// ---------------------------------------------------------------------- host

constexpr int64_t kCus = 256;

// How many pieces the sums of a launch are cut into.
int32_t pieces_of(int64_t tiles, int64_t steps, int64_t slots) {
  if (tiles * 2 > slots) return 1;
  return static_cast<int32_t>(std::max<int64_t>(1, std::min(slots / tiles, steps / 4)));
}

// A launch holds fewer than 2^32 threads (what is cut has few tiles).
constexpr int64_t kMaxTiles = int64_t(1) << 22;

struct Launch {
  ProductArgs a;
  bool small;
  int64_t bytes;
};

// The call's launches; `a` has what they share.
template <typename S>
void add_launches(const ProductArgs& shared, const std::vector<Group>& groups, bool small,
                  std::vector<Launch>* out) {
  for (size_t k = 0; k < groups.size();) {
    Launch l{};
    l.a = shared;
    l.small = small;
    int64_t tiles = 0;
    l.a.col_tiles = static_cast<int32_t>(ceil_div(shared.cols, S::kCols));
    for (; k < groups.size() && l.a.n < kMaxGroups; ++k) {
      const int64_t more = ceil_div(groups[k].rows, S::kRows) * l.a.col_tiles;
      if (l.a.n > 0 && tiles + more > kMaxTiles) break;
      Group g = groups[k];
      g.tile0 = static_cast<int32_t>(std::min(tiles, kMaxTiles));
      l.a.group[l.a.n++] = g;
      tiles += more;
    }
    l.a.tiles = static_cast<int32_t>(std::min(tiles, kMaxTiles + 1));
    l.a.pieces = pieces_of(tiles, ceil_div(shared.depth, S::kDepth), small ? 2 * kCus : kCus);
    l.bytes = l.a.pieces > 1 ? tiles * l.a.pieces * (S::kRows * S::kCols * 4) : 0;
    out->push_back(l);
  }
}

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
      g.row0 = static_cast<int32_t>(row);
      g.rows = static_cast<int32_t>(counts[k]);
      groups.push_back(g);
    }
    row += counts[k];
  }
  (void)in_major;
  int64_t large = 0;
  for (const Group& g : groups) large = std::max<int64_t>(large, g.rows);
  if (large > 64) add_launches<Large>(a, groups, false, out);
  else add_launches<Small>(a, groups, true, out);
  for (const Launch& l : *out)
    if (l.a.tiles > kMaxTiles) return fail(ZR_ERR_UNSUPPORTED, "more tiles than a launch holds");
  return ZR_OK;
}

template <typename S>
zr_status launch_product(const ProductArgs& a, bool columns, bool direct, hipStream_t stream) {
  auto* kernel = columns ? (direct ? product_kernel<S, true, true> : product_kernel<S, true, false>)
                         : (direct ? product_kernel<S, false, true> : product_kernel<S, false, false>);
  ZR_LAUNCH(a.tiles * a.pieces, S::kThreads, stream, a, kernel);
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
    for (Launch& l : launches) {
      ProductArgs& a = l.a;
      for (int r = 0; r < gi.world; ++r) a.part[r] = static_cast<const char*>(parts[r]);
      a.x = x;
      a.y = y;
      a.partial = static_cast<float*>(workspace);
      a.part_numel = gi.part;
      a.world = gi.world;
      a.x_stride = x_stride;
      a.y_stride = y_stride;
      a.y_bf16 = y_dtype == ZR_BF16;
      // a step's part of the weight, in two partitions at most
      const int64_t wide = columns ? cols : depth;
      const int64_t span = columns ? (l.small ? Small::kDepth : Large::kDepth) * cols
                                   : (l.small ? Small::kCols : Large::kCols) * depth;
      const bool direct = aligned && aligned_to(x, 16) && x_stride % 8 == 0 && wide % 8 == 0 && span <= gi.part;
      st = l.small ? launch_product<Small>(a, columns, direct, stream)
                   : launch_product<Large>(a, columns, direct, stream);
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
