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
  int32_t y_bf16;
};

constexpr int kDepth = 64;     // k of a staged tile
constexpr int kUnits = kDepth / 8;

// A workgroup's tile of rows and columns, by waves of 32 x 32 blocks, with
// kStages tiles of LDS.
template <int kRows_, int kCols_, int kWavesR_, int kWavesC_, int kStages_>
struct Shape {
  static constexpr int kRows = kRows_, kCols = kCols_;
  static constexpr int kWavesR = kWavesR_, kWavesC = kWavesC_, kStages = kStages_;
  static constexpr int kThreads = 64 * kWavesR * kWavesC;
  static constexpr int kRowBlocks = kRows / kWavesR / 32, kColBlocks = kCols / kWavesC / 32;
  static constexpr int kXBytes = kRows * kDepth * 2, kWBytes = kCols * kDepth * 2;
  static constexpr int kStage = kXBytes + kWBytes;
  static constexpr int kXLoads = kXBytes / 16 / kThreads, kWLoads = kWBytes / 16 / kThreads;
  static_assert(kXLoads * kThreads * 16 == kXBytes && kWLoads * kThreads * 16 == kWBytes, "staging shape");
};

// A matrix whose rows run along k: 128 bytes of a row, its 16-byte units
// exchanged (xor) by the row's number, so that eight lanes that read one unit of
// eight rows use all banks.
__device__ __forceinline__ int staged_row(int r, int u) { return r * (kDepth * 2) + ((u ^ (r & 7)) << 4); }

// Where a weight's tile lies: in partition a up to the element `cut` (counted
// from the tile's first one), in b from there on.  more: in others too.
struct Source {
  const char* a;
  const char* b;               // both as if the tile's first element lay there
  int64_t cut;
  bool more;
};
__device__ __forceinline__ Source source_of(const ProductArgs& p, int64_t first, int64_t span) {
  Source s;
  const int64_t k = first / p.part_numel, at = first - k * p.part_numel;
  s.cut = p.part_numel - at;
  s.more = span > s.cut + p.part_numel;
  s.a = p.part[k] + at * 2;
  s.b = span > s.cut ? p.part[k + 1] - s.cut * 2 : s.a;
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
    from = s.a + e * 2;
  } else if (e >= s.cut) {
    from = s.b + e * 2;
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
  const int left = a.depth - k0 < kDepth ? a.depth - k0 : kDepth;
#pragma unroll
  for (int j = 0; j < S::kXLoads; ++j) {
    const int at = j * S::kThreads + tid, r = at / kUnits, u = 8 * (at % kUnits);
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
    constexpr int kPerRow = kColumns ? S::kCols / 8 : kUnits;
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
    *reinterpret_cast<u32x4*>(lds + staged_row(at / kUnits, at % kUnits)) = s.x[j];
  }
#pragma unroll
  for (int j = 0; j < S::kWLoads; ++j) {
    constexpr int kPerRow = kColumns ? S::kCols / 8 : kUnits;
    const int at = j * S::kThreads + tid, r = at / kPerRow, u = at % kPerRow;
    const int to = kColumns ? staged<S::kCols>(r, u) : staged_row(r, u);
    *reinterpret_cast<u32x4*>(lds + S::kXBytes + to) = s.w[j];
  }
}

// Whole steps straight into LDS: rows and partitions on 16 bytes, a step's part
// of the weight in two partitions at most.  Where a row or column is behind the
// last, the tile's first is read instead; it is never stored.
template <typename S, bool kColumns>
struct Direct {
  uint32_t x_off[S::kXLoads], w_off[S::kWLoads];   // bytes from the step's start
  __device__ __forceinline__ Direct(const ProductArgs& a, const Place& p, int tid) {
#pragma unroll
    for (int j = 0; j < S::kXLoads; ++j) {
      const int at = j * S::kThreads + tid, r = at / kUnits, u = (at % kUnits) ^ (r & 7);
      x_off[j] = (r < p.rows ? r : 0) * static_cast<uint32_t>(a.x_stride * 2) + u * 16;
    }
#pragma unroll
    for (int j = 0; j < S::kWLoads; ++j) {
      if constexpr (kColumns) {
        constexpr int kPerRow = S::kCols / 8;
        const int at = j * S::kThreads + tid, r = at / kPerRow, u = exchanged(r, at % kPerRow);
        w_off[j] = r * static_cast<uint32_t>(a.cols * 2) + (8 * u < p.cols ? u : 0) * 16;
      } else {
        const int at = j * S::kThreads + tid, r = at / kUnits, u = (at % kUnits) ^ (r & 7);
        w_off[j] = (r < p.cols ? r : 0) * static_cast<uint32_t>(a.depth * 2) + u * 16;
      }
    }
  }
  __device__ __forceinline__ void load(const ProductArgs& a, const Place& p, int k0, char* lds, int w) const {
    const char* x = reinterpret_cast<const char*>(p.x + k0);
#pragma unroll
    for (int j = 0; j < S::kXLoads; ++j)
      __builtin_amdgcn_global_load_lds((const ZR_GLOBAL_AS void*)(x + x_off[j]),
                                       (ZR_LDS_AS void*)(lds + (j * S::kThreads + 64 * w) * 16), 16, 0, 0);
    const int64_t first = p.w + (kColumns ? static_cast<int64_t>(k0) * a.cols + p.col
                                          : static_cast<int64_t>(p.col) * a.depth + k0);
    const int64_t span = kColumns ? static_cast<int64_t>(kDepth - 1) * a.cols + p.cols
                                  : static_cast<int64_t>(p.cols - 1) * a.depth + kDepth;
    const Source s = source_of(a, first, span);
#pragma unroll
    for (int j = 0; j < S::kWLoads; ++j) {
      const char* from = (static_cast<int64_t>(w_off[j]) < 2 * s.cut ? s.a : s.b) + w_off[j];
      __builtin_amdgcn_global_load_lds((const ZR_GLOBAL_AS void*)from,
                                       (ZR_LDS_AS void*)(lds + S::kXBytes + (j * S::kThreads + 64 * w) * 16), 16,
                                       0, 0);
    }
  }
};

template <typename S>
using Acc = f32x16[S::kColBlocks][S::kRowBlocks];

// A staged step's products.  The weight is the MFMA's first operand: its
// columns n are the accumulators' rows, four of them one after the other in a
// lane, and X's rows the lanes.
template <typename S, bool kColumns>
struct Reader {
  int x[S::kRowBlocks], w[S::kColBlocks];   // a lane's places in a staged step
  int lane;
  __device__ __forceinline__ Reader(int lane_, int wave) : lane(lane_) {
    const int wr = wave / S::kWavesC, wc = wave % S::kWavesC;
#pragma unroll
    for (int b = 0; b < S::kRowBlocks; ++b) x[b] = ((wr * S::kRowBlocks + b) * 32 + (lane & 31)) * (kDepth * 2);
    const int g = lane >> 4, q = lane & 15;
    const int k = 8 * (g >> 1) + (q >> 2), c = 16 * (g & 1) + 4 * (q & 3);
#pragma unroll
    for (int b = 0; b < S::kColBlocks; ++b) {
      if constexpr (kColumns) {
        const int at = (wc * S::kColBlocks + b) * 32 + c;
        w[b] = staged<S::kCols>(k, at / 8) + (at % 8) * 2;
      } else {
        w[b] = ((wc * S::kColBlocks + b) * 32 + (lane & 31)) * (kDepth * 2);
      }
    }
  }
  __device__ __forceinline__ bf16x8 row(const char* lds, int at, int phase) const {
    const int u = (2 * phase + (lane >> 5)) ^ (lane & 7);
    return __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(lds + at + (u << 4)));
  }
  __device__ __forceinline__ void multiply(Acc<S>& acc, const char* lds) const {
#pragma unroll
    for (int phase = 0; phase < kDepth / 16; ++phase) {
      bf16x8 xf[S::kRowBlocks], wf[S::kColBlocks];
#pragma unroll
      for (int b = 0; b < S::kRowBlocks; ++b) xf[b] = row(lds, x[b], phase);
#pragma unroll
      for (int b = 0; b < S::kColBlocks; ++b) {
        if constexpr (kColumns)
          wf[b] = read_columns<S::kCols>(lds + S::kXBytes, w[b] + 16 * phase * (S::kCols * 2));
        else
          wf[b] = row(lds + S::kXBytes, w[b], phase);
      }
#pragma unroll
      for (int i = 0; i < S::kColBlocks; ++i)
#pragma unroll
        for (int j = 0; j < S::kRowBlocks; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wf[i], xf[j], acc[i][j], 0, 0, 0);
    }
  }
};

template <int n>
__device__ __forceinline__ void wait_loads() {   // all but the last n have arrived
  __builtin_amdgcn_s_waitcnt((n & 15) | ((n >> 4) << 14) | 0x0f70);
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
  const int64_t all = (a.depth + kDepth - 1) / kDepth;
  const int s0 = static_cast<int>(piece * all / a.pieces), s1 = static_cast<int>((piece + 1) * all / a.pieces);
  const Reader<S, kColumns> reader(lane, w);
  Acc<S> acc = {};
  int s = s0;
  if constexpr (kDirect) {
    const int whole = s1 < a.depth / kDepth ? s1 : a.depth / kDepth;
    if (s < whole) {
      const Direct<S, kColumns> in(a, p, tid);
      // behind the last step, the last is loaded again, unused
      auto step = [&](int n) { return (n < whole ? n : whole - 1) * kDepth; };
      constexpr int kAhead = S::kStages - 1, kLoads = S::kXLoads + S::kWLoads;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) in.load(a, p, step(s + i), lds + i * S::kStage, w);
      int now_at = 0, next_at = kAhead * S::kStage;
      for (; s < whole; ++s) {
        wait_loads<kLoads * (kAhead - 1)>();
        lds_barrier();
        in.load(a, p, step(s + kAhead), lds + next_at, w);
        reader.multiply(acc, lds + now_at);
        now_at = now_at + S::kStage == S::kStages * S::kStage ? 0 : now_at + S::kStage;
        next_at = next_at + S::kStage == S::kStages * S::kStage ? 0 : next_at + S::kStage;
      }
      wait_loads<0>();
    }
  }
  if (s < s1) {
    Staged<S> next;
    load_step<S, kColumns>(next, a, p, s * kDepth, tid);
    for (; s < s1; ++s) {
      lds_barrier();
      store_step<S, kColumns>(next, lds, tid);
      lds_barrier();
      if (s + 1 < s1) load_step<S, kColumns>(next, a, p, (s + 1) * kDepth, tid);
      reader.multiply(acc, lds);
    }
  }
  const int wr = w / S::kWavesC, wc = w % S::kWavesC;
#pragma unroll
  for (int j = 0; j < S::kRowBlocks; ++j) {
    const int r = (wr * S::kRowBlocks + j) * 32 + (lane & 31);
    if (r >= p.rows) continue;
#pragma unroll
    for (int i = 0; i < S::kColBlocks; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const f32x4 sums = {acc[i][j][4 * v], acc[i][j][4 * v + 1], acc[i][j][4 * v + 2], acc[i][j][4 * v + 3]};
        const int c = (wc * S::kColBlocks + i) * 32 + 8 * v + 4 * (lane >> 5);
        if (a.pieces > 1)
          *as_global<f32x4>(a.partial + static_cast<int64_t>(id) * (S::kRows * S::kCols) + r * S::kCols + c) = sums;
        else if (c < p.cols)
          put_sums(a, p.row + r, p.col + c, sums);
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

using Large = Shape<256, 256, 2, 4, 2>;
using Small = Shape<32, 128, 1, 4, 4>;

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
    l.a.pieces = pieces_of(tiles, ceil_div(shared.depth, kDepth), small ? 2 * kCus : kCus);
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
      a.x_stride = x_stride;
      a.y_stride = y_stride;
      a.y_bf16 = y_dtype == ZR_BF16;
      // a step's part of the weight, in two partitions at most
      const int64_t wide = columns ? cols : depth;
      const int64_t span = columns ? kDepth * cols : (l.small ? Small::kCols : Large::kCols) * depth;
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
