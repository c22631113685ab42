// The embedding table's operators (gfx950): rows looked up in the ranks'
// partitions, and the table's gradient by sorted tokens into main_grad.
// Both are HBM-bound streams over rows: no product is large enough for MFMA.

#include "zr_layers.h"

using namespace zr;

namespace {

// Token ids of either width.
struct Tokens {
  const void* ids;
  int32_t wide;  // 1: int64, 0: int32
};
__device__ __forceinline__ int64_t token_at(const Tokens& t, int64_t i) {
  return t.wide ? as_global<int64_t>(t.ids)[i] : as_global<int32_t>(t.ids)[i];
}

// ---------------------------------------------------------------- lookup ---

struct LookupArgs {
  const void* parts[ZR_MAX_WORLD];
  Tokens tokens;
  void* out;
  int64_t n, vocab, dim, out_stride;
  int64_t base, part;     // the table's flat offset; partition elements
  double part_inverse;
  float scale;
  int32_t chunks;         // pieces of kLookupCols columns per row
};

constexpr int kLookupWaves = 4;
template <typename T> constexpr int kVec = 16 / static_cast<int>(sizeof(T));
template <typename T> constexpr int kLookupCols = 64 * kVec<T> * 4;

template <typename T>
__device__ __forceinline__ T scaled(T x, float s);
template <>
__device__ __forceinline__ float scaled(float x, float s) { return x * s; }
template <>
__device__ __forceinline__ uint16_t scaled(uint16_t x, float s) {
  return static_cast<uint16_t>(pack_bf16(bf16_lo(x) * s, 0.0f));
}
template <typename T>
__device__ __forceinline__ u32x4 scaled_vec(u32x4 w, float s) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = sizeof(T) == 2 ? pack_bf16(bf16_lo(w[i]) * s, bf16_hi(w[i]) * s)
                          : float_bits(bits_float(w[i]) * s);
  return w;
}

// out[i, c] = rnd(scale * table[token_i, c]).  One wave copies one piece of
// up to kLookupCols columns of one row, 16 bytes a lane and four loads in
// flight; the partition that holds the piece is found once a wave, and only
// a piece that a partition border cuts goes element by element.  An id
// outside [0, vocab) gives a row of +0 and reads nothing.
template <typename T>
__global__ __launch_bounds__(64 * kLookupWaves) void lookup_kernel(const LookupArgs a) {
  constexpr int V = kVec<T>, C = kLookupCols<T>;
  const int lane = threadIdx.x & 63;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kLookupWaves + uniform(static_cast<int>(threadIdx.x >> 6));
  const int64_t row = unit / a.chunks;
  if (row >= a.n) return;
  const int64_t c0 = (unit - row * a.chunks) * C;
  const int64_t len = a.dim - c0 < C ? a.dim - c0 : C;
  const int64_t t = uniform(token_at(a.tokens, row));
  T* out = static_cast<T*>(a.out) + row * a.out_stride + c0;
  const bool valid = t >= 0 && t < a.vocab;
  const int64_t f = a.base + (valid ? t * a.dim + c0 : 0);
  // f < 2^53, so the quotient is off by one at most.
  int64_t k = static_cast<int64_t>(static_cast<double>(f) * a.part_inverse);
  if (k * a.part > f) --k;
  if ((k + 1) * a.part <= f) ++k;
  if (!valid || f + len <= (k + 1) * a.part) {
    const T* src = valid ? static_cast<const T*>(a.parts[k]) + (f - k * a.part) : nullptr;
    if (len >= V) {
      // The last lane of a row that is no multiple of V takes its last V
      // columns, some of them twice.
      u32x4 x[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int64_t c = (u * 64 + lane) * V, d = c + V <= len ? c : len - V;
        x[u] = u32x4{0, 0, 0, 0};
        if (valid && c < len) x[u] = load_at<u32x4, sizeof(T)>(src + d);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int64_t c = (u * 64 + lane) * V, d = c + V <= len ? c : len - V;
        // zeros are not scaled: -0 or NaN would come of a negative or infinite scale
        if (c < len) store_at<sizeof(T)>(out + d, valid ? scaled_vec<T>(x[u], a.scale) : u32x4{0, 0, 0, 0});
      }
    } else if (lane < len) {
      out[lane] = valid ? scaled<T>(src[lane], a.scale) : T(0);
    }
    return;
  }
  for (int64_t e = lane; e < len; e += 64) {
    while (f + e >= (k + 1) * a.part) ++k;
    out[e] = scaled<T>(static_cast<const T*>(a.parts[k])[f + e - k * a.part], a.scale);
  }
}

// -------------------------------------------------------------- gradient ---
//
// main_grad[row] (+)= scale * sum of dY over the tokens with that row's id.
// 1. sort: the positions of the tokens whose row meets the window, row after
//    row (in no particular order of the rows) and in their own order within a
//    row;
// 2. sum: pieces of 8 to 64 sorted positions, each summed by waves of its own
//    in that order.  A row whose tokens lie in one piece is added to
//    main_grad at once; one that spans pieces leaves a partial sum per piece;
// 3. join: the partial sums of such a row, added in the order of the pieces.
// The pieces are cut by position and never by row, so that a token that fills
// half the batch is spread over the GPU like any other; and nothing depends
// on which wave comes first, so the sums have the same bits on every run.

constexpr int kSortWaves = 16;
constexpr int kSortRows = 1024;   // rows one workgroup sorts, at most

struct EmbedWork {       // the caller's workspace
  int32_t* count;        // sorted positions
  int32_t* pos;          // their places in the batch
  int32_t* row;          // their rows, relative to the window's first row
  float* partial;        // [pieces][2][cols]: a piece's first and last run
};

struct SortArgs {
  Tokens tokens;
  EmbedWork w;
  int64_t n, row0;
  int32_t rows;           // the window's rows: [row0, row0 + rows)
  int32_t shift;          // 2^shift workgroups
  // first micro-batch only: rows without tokens are zeroed
  float* main_grad;       // null otherwise; where the table's element 0 lies
  int64_t dim, first, last;
  int32_t zero_all;       // every row first, those with tokens too
};

// kGroup times 64 ids of a wave's share at once.  A row r of the window is kept
// as r mod 2^shift (its workgroup) above r / 2^shift (its place there), less
// the first such number of the workgroup that reads it: below the count of that
// workgroup's rows for its own.  Every workgroup handles every id, so the
// instructions for each are what the sort takes: whole groups need no check of
// their ends, and what the wave has in common is counted by its scalar unit.
constexpr int kGroup = 8;
constexpr int kAhead = 4;   // groups that a wave loads at once
constexpr int kHits = 512;  // tokens of its workgroup's rows that a wave keeps
using Rows = uint32_t[kGroup];
template <typename Id>
__device__ __forceinline__ void load_rows(const SortArgs& a, int64_t i, int64_t end, int lane,
                                          uint32_t base, Rows& r) {
  const auto* ids = as_global<Id>(a.tokens.ids) + i;
  // Positions fit in 32 bits.  A 64-bit comparison here, taken by a branch and
  // by a select, is compiled (ROCm 7.2) to a select on another condition.
  const int count = min(static_cast<int>(end - i), 64 * kGroup);
  Id t[kGroup];
  if (count == 64 * kGroup) {
#pragma unroll
    for (int g = 0; g < kGroup; ++g) t[g] = ids[lane + 64 * g];
  } else {   // behind the end the last id, unused
#pragma unroll
    for (int g = 0; g < kGroup; ++g) t[g] = ids[min(lane + 64 * g, count - 1)];
  }
#pragma unroll
  for (int g = 0; g < kGroup; ++g) {
    const uint64_t row = static_cast<uint64_t>(static_cast<int64_t>(t[g])) - static_cast<uint64_t>(a.row0);
    const bool in = row < static_cast<uint32_t>(a.rows) && lane + 64 * g < count;
    r[g] = (in ? __builtin_rotateright32(static_cast<uint32_t>(row), a.shift) : ~0u) - base;   // ~0 is no row's
  }
}
__device__ __forceinline__ int lanes_before(uint64_t lanes, int lane) {
  return __popcll(lanes & ((1ull << lane) - 1));
}

// What a wave keeps of its share: the tokens of its workgroup's rows, in order.
struct Hits {
  int32_t pos[kHits];
  uint16_t row[kHits];     // in the workgroup's order
};

// Counts each row of this workgroup, with the row of the first such lane at
// once (one token may fill half the batch), and the tokens of earlier ones.
__device__ __forceinline__ void count_rows(const Rows& r, int64_t i, uint32_t base, uint32_t span, int lane,
                                           int32_t* place, Hits& hits, int* found, int* before) {
#pragma unroll
  for (int g = 0; g < kGroup; ++g) {
    *before += __popcll(__ballot(r[g] > ~base));
    const bool mine = r[g] < span;
    const uint64_t all = __ballot(mine);
    if (!all) continue;
    const int leader = __builtin_ctzll(all);
    const uint32_t one = __builtin_amdgcn_readlane(static_cast<int>(r[g]), leader);
    const int same = __popcll(__ballot(r[g] == one));
    if (mine) {
      if (lane == leader) atomicAdd(&place[one], same);
      else if (r[g] != one) atomicAdd(&place[r[g]], 1);
      const int at = *found + lanes_before(all, lane);
      if (at < kHits) {
        hits.pos[at] = static_cast<int32_t>(i) + 64 * g + lane;
        hits.row[at] = static_cast<uint16_t>(r[g]);
      }
    }
    *found += __popcll(all);
  }
}
// Puts the positions of 64 lanes where their rows' next ones belong; a lane
// with row >= span has none.  Lanes of one row find each other by a ballot for
// the first lane's row, and the next one's; where more than kTries rows meet,
// by a ballot for each bit of the row.
constexpr int kTries = 3;
__device__ __forceinline__ void place_rows(const EmbedWork& w, uint32_t row, int32_t pos, int shift,
                                           uint32_t span, int bits, int lane, int32_t* place) {
  bool left = row < span;
  uint64_t todo = __ballot(left);
  for (int t = 0; todo; ++t) {
    uint64_t same = todo;
    bool mine = left;
    if (t < kTries) {
      const uint32_t one = __builtin_amdgcn_readlane(static_cast<int>(row), __builtin_ctzll(todo));
      mine = left && row == one;
      same = __ballot(mine);
    } else {
      for (int b = 0; b < bits; ++b) {
        const int64_t bit = -static_cast<int64_t>((row >> b) & 1);
        same &= ~(__ballot(bit) ^ bit);
      }
    }
    if (mine) {
      const int p = place[row], rank = lanes_before(same, lane);
      w.pos[p + rank] = pos;
      w.row[p + rank] = static_cast<int32_t>(row << shift) + static_cast<int>(blockIdx.x);
      if ((same >> lane) == 1) place[row] = p + rank + 1;   // the row's last lane
      left = false;
    }
    // the next lanes read what these wrote: in order in a wave, no wait needed
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    todo = t < kTries ? todo & ~same : 0;
  }
}

// Zeros to the table's elements in the window, a run of them to each wave of
// the launch; stores that drain while the ids are sorted.
__device__ __forceinline__ void zero_window(const SortArgs& a, int w, int lane) {
  float* p = a.main_grad + a.first;
  const int64_t n = a.last - a.first;
  const int lead = static_cast<int>(-(reinterpret_cast<uintptr_t>(p) / 4) & 3);   // to 16 bytes
  const int64_t vecs = n > lead ? (n - lead) / 4 : 0, done = lead + 4 * vecs;
  if (blockIdx.x == 0 && w == 0) {
    if (lane < lead && lane < n) p[lane] = 0.0f;
    if (done + lane < n) p[done + lane] = 0.0f;   // three at most
  }
  const int64_t waves = static_cast<int64_t>(gridDim.x) * kSortWaves, k = blockIdx.x * int64_t(kSortWaves) + w;
  const int64_t each = ((vecs + waves - 1) / waves + 63) & ~int64_t(63);
  const int64_t end = (k + 1) * each < vecs ? (k + 1) * each : vecs;
  for (int64_t v = k * each + lane; v < end; v += 64)
    *as_global<f32x4>(p + lead + 4 * v) = f32x4{0, 0, 0, 0};
}

// Workgroup g sorts the tokens of the rows r with r mod 2^shift = g (the
// commonest ids are often neighbours: taken apart, no workgroup has many of
// them).  It counts, over the whole batch, the tokens of earlier workgroups
// (its first place in the order) and those of each row of its own, by wave,
// and keeps these; then every wave places what it kept, in order, behind what
// earlier rows and earlier waves have.  Every workgroup reads all ids (from
// L2), so that one launch sorts and nothing waits for another workgroup.  What
// bounds it: three chains of LDS accesses, one after the other.  Measured,
// launch included, 32768 ids over 16032 rows, a 17th of them the same: 15 us
// (7 for the loads, 4 to count, 5 to place), 20 where every 64 ids are looked
// through again to be placed; all the same 26 (42); neighbouring rows together
// cost 3 us more.
template <typename Id>
__global__ __launch_bounds__(64 * kSortWaves) void embed_sort_kernel(const SortArgs a) {
  __shared__ int32_t place[kSortWaves][kSortRows];
  __shared__ int32_t wave_sum[kSortWaves];
  __shared__ int32_t before_s;
  __shared__ uint8_t empty[kSortRows];
  __shared__ Hits hits[kSortWaves];
  const int tid = threadIdx.x, lane = tid & 63, w = uniform(tid >> 6);
  const int own = blockIdx.x;
  const uint32_t span = (a.rows - own + (1 << a.shift) - 1) >> a.shift;   // its rows
  for (int i = lane; i < span; i += 64) place[w][i] = 0;
  if (tid == 0) before_s = 0;
  __syncthreads();
  const int64_t share = (a.n + 64 * kSortWaves - 1) / (64 * kSortWaves) * 64;
  const int64_t i0 = w * share, i1 = i0 + share < a.n ? i0 + share : a.n;
  constexpr int kStep = 64 * kGroup;
  const uint32_t base = a.shift ? static_cast<uint32_t>(own) << (32 - a.shift) : 0;
  int before = 0, found = 0;
  {
    Rows r[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (i0 + k * kStep < i1) load_rows<Id>(a, i0 + k * kStep, i1, lane, base, r[k]);
    if (a.main_grad && a.zero_all) zero_window(a, w, lane);
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (i0 + k * kStep < i1)
        count_rows(r[k], i0 + k * kStep, base, span, lane, place[w], hits[w], &found, &before);
  }
  for (int64_t i = i0 + kAhead * kStep; i < i1; i += kStep) {
    Rows r;
    load_rows<Id>(a, i, i1, lane, base, r);
    count_rows(r, i, base, span, lane, place[w], hits[w], &found, &before);
  }
  if (lane == 0) atomicAdd(&before_s, before);
  __syncthreads();
  // One thread a row: its count, then an exclusive scan over the rows.
  int count = 0;
  if (tid < span)
    for (int v = 0; v < kSortWaves; ++v) count += place[v][tid];
  int scan = count;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int up = __shfl_up(scan, d);
    if (lane >= d) scan += up;
  }
  if (lane == 63) wave_sum[w] = scan;
  __syncthreads();
  int at = before_s + scan - count;
  for (int v = 0; v < w; ++v) at += wave_sum[v];
  empty[tid] = count == 0;
  if (blockIdx.x == gridDim.x - 1 && tid == 64 * kSortWaves - 1) *a.w.count = at + count;
  if (tid < span)
    for (int v = 0; v < kSortWaves; ++v) {
      const int c = place[v][tid];
      place[v][tid] = at;
      at += c;
    }
  __syncthreads();
  const int bits = 32 - __builtin_clz(span);
  if (found <= kHits) {
    for (int h = 0; h < found; h += 64) {
      const int k = min(h + lane, found - 1);
      const uint32_t row = h + lane < found ? hits[w].row[k] : ~0u;
      place_rows(a.w, row, hits[w].pos[k], a.shift, span, bits, lane, place[w]);
    }
  } else {   // more than it keeps: its share again
    for (int64_t i = i0; i < i1; i += kStep) {
      Rows r;
      load_rows<Id>(a, i, i1, lane, base, r);
#pragma unroll
      for (int g = 0; g < kGroup; ++g)
        place_rows(a.w, r[g], static_cast<int32_t>(i) + 64 * g + lane, a.shift, span, bits, lane, place[w]);
    }
  }
  if (!a.main_grad || a.zero_all) return;
  // Zeros to the rows without tokens, a wave to a row.
  for (int r = w; r < span; r += kSortWaves) {
    if (!empty[r]) continue;
    const int64_t e = (a.row0 + own + (static_cast<int64_t>(r) << a.shift)) * a.dim;
    const int64_t f = e > a.first ? e : a.first, l = e + a.dim < a.last ? e + a.dim : a.last;
    float* p = a.main_grad + f;
    const int n = static_cast<int>(l - f);
    const int lead = static_cast<int>(-(reinterpret_cast<uintptr_t>(p) / 4) & 3);   // to 16 bytes
    if (lane < lead && lane < n) p[lane] = 0.0f;
    int c = lead + 4 * lane;
    for (; c + 4 <= n; c += 256) *as_global<f32x4>(p + c) = f32x4{0, 0, 0, 0};
    for (; c < n; ++c) p[c] = 0.0f;
  }
}

struct SumArgs {
  const void* dy;
  EmbedWork w;
  float* main_grad;            // where the table's element 0 lies
  int64_t dy_stride, row0, first, last;
  int32_t dim, piece, cols;    // positions per piece; columns of a partial sum
  float scale;
};

// Four columns of a row's gradient into main_grad, clipped to the window.
template <bool kFirst>
__device__ __forceinline__ void put_row(const SumArgs& a, int64_t row, int col, f32x4 s) {
  const int64_t e = (a.row0 + row) * a.dim + col;
  s *= a.scale;
  if (col + 4 <= a.dim && e >= a.first && e + 4 <= a.last) {
    float* p = a.main_grad + e;
    store_at<4>(p, (kFirst ? f32x4{0, 0, 0, 0} : load_at<f32x4, 4>(p)) + s);
  } else {
    f32x4 old{0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (!kFirst && col + j < a.dim && e + j >= a.first && e + j < a.last) old[j] = a.main_grad[e + j];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (col + j < a.dim && e + j >= a.first && e + j < a.last) a.main_grad[e + j] = old[j] + s[j];
  }
}

// Four columns of a row of dY, used once.
__device__ __forceinline__ u32x2 load4(const uint16_t* p) {
  return load_once_at<u32x2, 2>(p);
}
__device__ __forceinline__ f32x4 load4(const float* p) {
  return load_once_at<f32x4, 4>(p);
}
__device__ __forceinline__ u32x2 load_some(const uint16_t* p, int n) {
  u32x2 x{0, 0};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j < n) x[j / 2] |= static_cast<uint32_t>(p[j]) << (16 * (j & 1));
  return x;
}
__device__ __forceinline__ f32x4 load_some(const float* p, int n) {
  f32x4 x{0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j < n) x[j] = p[j];
  return x;
}
__device__ __forceinline__ f32x4 widen4(u32x2 w) {
  return f32x4{bf16_lo(w[0]), bf16_hi(w[0]), bf16_lo(w[1]), bf16_hi(w[1])};
}
__device__ __forceinline__ f32x4 widen4(f32x4 x) { return x; }
// The values from the n-th on, n < 4, moved to the front.
__device__ __forceinline__ f32x4 from(f32x4 x, int n) {
  if (n & 1) x = f32x4{x[1], x[2], x[3], x[3]};
  if (n & 2) x = f32x4{x[2], x[3], x[3], x[3]};
  return x;
}

constexpr int kSumVecs = 2;                     // groups of four columns of a lane
constexpr int kSumCols = 64 * 4 * kSumVecs;     // columns of a wave
// Positions of a batch; with main_grad's rows in flight too, as many as leave
// room for a second workgroup on a CU (128 registers).
template <bool kFirst> constexpr int kSumRows = kFirst ? 4 : 3;

// The rows of dY of a batch of positions, and the rows of main_grad that runs
// end in among them.
template <typename T, bool kFirst>
struct Batch {
  using Vec = decltype(load4(static_cast<const T*>(nullptr)));
  Vec x[kSumRows<kFirst>][kSumVecs];
  f32x4 old[kFirst ? 1 : kSumRows<kFirst>][kSumVecs];
};

// One wave sums one piece (at most 64) of the sorted positions over kSumCols
// columns.  Its lanes hold the piece's positions and rows; two batches of
// rows are on their way at any time, main_grad's among them.  A lane that the
// rows' end cuts reads the last four columns and moves its own to the front.
//
// What bounds it: HBM, with rows of dY in no order.  Rows of dY are read past
// the caches (they are used once, and main_grad's lines would give way to
// them), and the waves of a workgroup take neighbouring columns of the same
// rows.  Measured, 32768 tokens of 4096 bf16 columns of which 27000 lie in a
// window of 16032 rows, sort and join included: 107 us in the _first form, 135
// with ordinary loads, 111 with workgroups of one wave; 117 us added, 119 with
// ordinary loads or four positions a batch.  Every row twice, in no order: 113
// us in the _first form (141 with ordinary loads), 146 added (189, and 154 with
// four positions).
constexpr int kSumWaves = 8;
template <typename T, bool kFirst, bool kTiny>   // kTiny: rows of fewer than four columns
__global__ __launch_bounds__(64 * kSumWaves) void embed_sum_kernel(const SumArgs a) {
  constexpr int kRows = kSumRows<kFirst>;
  const int lane = threadIdx.x & 63, w = uniform(static_cast<int>(threadIdx.x >> 6));
  const int wave = blockIdx.y * (blockDim.x >> 6) + w;   // of those that share the columns
  if (wave * kSumCols >= a.dim) return;
  const int p0 = blockIdx.x * a.piece;
  const int at = p0 + lane;
  const int count = *a.w.count;
  if (p0 >= count) return;
  const int n = count - p0 < a.piece ? count - p0 : a.piece;
  const int my_pos = a.w.pos[at < count ? at : count - 1];
  const int my_row = a.w.row[at < count ? at : count - 1];
  const int my_next = at + 1 < count ? a.w.row[at + 1] : -1;
  const uint64_t ends = __ballot(my_row != my_next);       // positions that end a run
  // and whose rows lie in the window whole
  const int64_t my_first = (a.row0 + my_row) * a.dim;
  const uint64_t quick = __ballot(my_first >= a.first && my_first + a.dim <= a.last);
  bool head = p0 > 0 && a.w.row[p0 - 1] == __builtin_amdgcn_readfirstlane(my_row);   // began earlier
  const int c0 = wave * kSumCols + 4 * lane;
  int c_in[kSumVecs];
#pragma unroll
  for (int u = 0; u < kSumVecs; ++u) {
    const int c = c0 + 256 * u;
    c_in[u] = c + 4 <= a.dim ? c : c < a.dim && !kTiny ? a.dim - 4 : 0;
  }
  const bool cut = a.dim & 3;
  f32x4 s[kSumVecs] = {};

  auto load = [&](Batch<T, kFirst>& b, int p) {
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      // behind the piece the last row is asked for again, unused
      const int i = p + k < n ? p + k : n - 1;
      const T* src = static_cast<const T*>(a.dy) +
                     static_cast<int64_t>(__builtin_amdgcn_readlane(my_pos, i)) * a.dy_stride;
#pragma unroll
      for (int u = 0; u < kSumVecs; ++u)
        b.x[k][u] = kTiny ? load_some(src, a.dim) : load4(src + c_in[u]);
      if constexpr (!kFirst && !kTiny) {
        if (p + k < n && ((ends & quick) >> i & 1)) {
          const float* row = a.main_grad + (a.row0 + __builtin_amdgcn_readlane(my_row, i)) * a.dim;
#pragma unroll
          for (int u = 0; u < kSumVecs; ++u) b.old[k][u] = load_at<f32x4, 4>(row + c_in[u]);
        }
      }
    }
  };
  auto add = [&](const Batch<T, kFirst>& b, int p) {
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const int i = p + k;
      if (i < n) {
#pragma unroll
        for (int u = 0; u < kSumVecs; ++u) {
          const f32x4 x = widen4(b.x[k][u]);
          s[u] += cut ? from(x, (c0 + 256 * u - c_in[u]) & 3) : x;
        }
        if (ends >> i & 1) {
          const int row = __builtin_amdgcn_readlane(my_row, i);
          const bool whole = !kTiny && (quick >> i & 1);
#pragma unroll
          for (int u = 0; u < kSumVecs; ++u) {
            const int c = c0 + 256 * u;
            if (c < a.dim) {
              if (head) {
                *as_global<f32x4>(a.w.partial + int64_t(blockIdx.x) * 2 * a.cols + c) = s[u];
              } else if (whole) {
                float* p = a.main_grad + (a.row0 + row) * a.dim + c;
                const f32x4 o = kFirst ? f32x4{0, 0, 0, 0} : b.old[kFirst ? 0 : k][u];
                const f32x4 v = (cut ? from(o, (c - c_in[u]) & 3) : o) + s[u] * a.scale;
                if (c + 4 <= a.dim) {
                  store_at<4>(p, v);
                } else {
#pragma unroll
                  for (int j = 0; j < 3; ++j)
                    if (c + j < a.dim) p[j] = v[j];
                }
              } else {
                put_row<kFirst>(a, row, c, s[u]);
              }
            }
            s[u] = f32x4{0, 0, 0, 0};
          }
          head = false;
        }
      }
    }
  };
  Batch<T, kFirst> b0, b1;
  load(b0, 0);
  for (int p = 0; p < n; p += 2 * kRows) {
    load(b1, p + kRows);
    add(b0, p);
    load(b0, p + 2 * kRows);
    add(b1, p + kRows);
  }
  if (ends >> (n - 1) & 1) return;
  // The last run goes on behind the piece.
#pragma unroll
  for (int u = 0; u < kSumVecs; ++u) {
    const int c = c0 + 256 * u;
    if (c < a.dim)
      *as_global<f32x4>(a.w.partial + (int64_t(blockIdx.x) * 2 + (head ? 0 : 1)) * a.cols + c) = s[u];
  }
}

// The rows that span pieces: workgroup (piece, kJoinCols columns) adds up the
// run that starts in its piece and goes on behind it, if there is one: its
// waves add an eighth of the pieces each, in their order.  With rows of three
// tokens on average most pieces end inside a run, so what counts is how few
// loads wait for each other: the run's pieces are counted 64 at a time.
constexpr int kJoinVecs = 4, kJoinCols = 256 * kJoinVecs, kJoinWaves = 8;
template <bool kFirst>
__global__ __launch_bounds__(64 * kJoinWaves) void embed_join_kernel(const SumArgs a) {
  __shared__ f32x4 part[kJoinWaves][kJoinVecs][64];
  const int lane = threadIdx.x & 63, w = uniform(static_cast<int>(threadIdx.x >> 6));
  const int64_t p0 = static_cast<int64_t>(blockIdx.x) * a.piece, p1 = p0 + a.piece;
  // asked for together, though what lies behind the count is not set
  const int64_t end = static_cast<int64_t>(gridDim.x) * a.piece;   // the last piece's first position
  const int64_t there = p1 + lane * a.piece;
  int first_row = a.w.row[there < end ? there : end];
  const int count = *a.w.count, row = a.w.row[p1], last = a.w.row[p1 - 1];
  const int before = a.w.row[p0 > 0 ? p0 - 1 : 0];
  if (p1 >= count || last != row || (p0 > 0 && before == row)) return;
  int64_t links = 0;   // pieces that follow
  for (;;) {
    const int64_t p = p1 + (links + lane) * a.piece;
    const uint64_t on = __ballot(p < count && first_row == row);
    const int more = on == ~0ull ? 64 : __builtin_ctzll(~on);
    links += more;
    if (more < 64) break;
    const int64_t q = p1 + (links + lane) * a.piece;
    first_row = a.w.row[q < end ? q : end];
  }
  const int64_t each = (links + kJoinWaves - 1) / kJoinWaves;
  const int64_t j1 = (w + 1) * each < links ? (w + 1) * each : links;
  const int c0 = blockIdx.y * kJoinCols + 4 * lane;
  const float* first = a.w.partial + (blockIdx.x * int64_t(2) + 1) * a.cols;
  const float* next = first + a.cols;
  f32x4 s[kJoinVecs] = {};
  int64_t c_in[kJoinVecs];   // columns behind the last are read as the first, unused
#pragma unroll
  for (int u = 0; u < kJoinVecs; ++u) c_in[u] = c0 + 256 * u < a.dim ? c0 + 256 * u : 0;
  if (w == 0) {
#pragma unroll
    for (int u = 0; u < kJoinVecs; ++u) s[u] = *as_global<f32x4>(first + c_in[u]);
  }
  constexpr int kDeep = 4;
  for (int64_t j = w * each; j < j1; j += kDeep) {
    f32x4 x[kDeep][kJoinVecs];
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      const int64_t link = j + d < j1 ? j + d : j1 - 1;
#pragma unroll
      for (int u = 0; u < kJoinVecs; ++u) x[d][u] = *as_global<f32x4>(next + link * 2 * a.cols + c_in[u]);
    }
#pragma unroll
    for (int d = 0; d < kDeep; ++d)
      if (j + d < j1) {
#pragma unroll
        for (int u = 0; u < kJoinVecs; ++u) s[u] += x[d][u];
      }
  }
#pragma unroll
  for (int u = 0; u < kJoinVecs; ++u) part[w][u][lane] = s[u];
  __syncthreads();
  const int c = c0 + 256 * w;   // a group of columns for each of the first waves
  if (w < kJoinVecs && c < a.dim) {
    f32x4 sum = part[0][w][lane];
#pragma unroll
    for (int v = 1; v < kJoinWaves; ++v) sum += part[v][w][lane];
    put_row<kFirst>(a, row, c, sum);
  }
}
static_assert(kJoinVecs <= kJoinWaves, "a wave for each group of columns");

// Positions per piece: enough pieces to fill the chip, and no more partial
// sums than that takes.  Measured, sum and join: 32768 tokens of 4096 columns
// 77 us with 64 positions, 82 with 32, 85 with 16 (_first form; 103, 104 and
// 110 added); 8192 of 768 columns 14 us with 8, 16 with 16, 31 with 64 and 17
// with 4.
int64_t piece_of(int64_t n, int64_t dim) {
  const int64_t waves = ceil_div(dim, kSumCols);
  int64_t piece = 64;   // positions that a wave's lanes hold
  while (piece > 8 && ceil_div(n, piece) * waves < 2048) piece /= 2;
  return piece;
}

struct Shape {
  int64_t piece, pieces, cols, pos, row, partial, bytes;   // offsets in the workspace
};
Shape shape_of(int64_t n, int64_t dim) {
  Shape s;
  s.piece = piece_of(n, dim);
  s.pieces = ceil_div(n, s.piece);
  s.cols = ceil_div(dim, 4) * 4;
  s.pos = 256;
  s.row = s.pos + ceil_div(4 * n, 256) * 256;
  s.partial = s.row + ceil_div(4 * n, 256) * 256;
  s.bytes = s.partial + (s.pieces > 1 ? s.pieces * 2 * s.cols * 4 : 0);
  return s;
}

zr_status check_table(const zr_plan* plan, int64_t param, int64_t dim, int64_t n) {
  if (!plan) return fail(ZR_ERR_INVALID, "plan is null");
  if (param < 0 || param >= static_cast<int64_t>(plan->params.size()))
    return fail(ZR_ERR_INVALID, "param id out of range");
  if (dim < 1 || plan->params[param].numel % dim)
    return fail(ZR_ERR_INVALID, "dim must be >= 1 and divide the param's elements");
  if (dim >= (int64_t(1) << 24)) return fail(ZR_ERR_UNSUPPORTED, "dim of 2^24 or more");
  if (n < 0) return fail(ZR_ERR_INVALID, "n must be >= 0");
  // positions in 32 bits, and the sum's and the join's threads within a launch
  if (n >= (int64_t(1) << 28)) return fail(ZR_ERR_UNSUPPORTED, "2^28 tokens or more");
  return ZR_OK;
}

zr_status check_tokens(const void* tokens, zr_index type, int64_t n) {
  if (type != ZR_I32 && type != ZR_I64) return fail(ZR_ERR_INVALID, "unsupported token type");
  if (n > 0 && (!tokens || !aligned_to(tokens, type == ZR_I64 ? 8 : 4)))
    return fail(ZR_ERR_INVALID, "tokens is null or not element-aligned");
  return ZR_OK;
}

template <typename T, bool kFirst>
void launch_sum(const SumArgs& a, int64_t pieces, hipStream_t stream) {
  const int64_t waves = ceil_div(a.dim, kSumCols), here = std::min<int64_t>(waves, kSumWaves);
  const dim3 grid(pieces, ceil_div(waves, here));
  if (a.dim < 4) ZR_LAUNCH(grid, 64 * here, stream, a, embed_sum_kernel<T, kFirst, true>);
  else ZR_LAUNCH(grid, 64 * here, stream, a, embed_sum_kernel<T, kFirst, false>);
}

zr_status run_embedding(const zr_plan* plan, int64_t param, int64_t dim, const void* tokens,
                        zr_index token_type, int64_t n, float scale, const void* dy,
                        zr_dtype dy_dtype, int64_t dy_stride, float* main_grad,
                        int64_t window_base, int64_t window_len, void* workspace,
                        int64_t workspace_bytes, bool first, hipStream_t stream) {
  return guarded([&]() -> zr_status {
    zr_status st = check_table(plan, param, dim, n);
    if (st != ZR_OK) return st;
    st = check_tokens(tokens, token_type, n);
    if (st != ZR_OK) return st;
    if (!valid_dtype(dy_dtype)) return fail(ZR_ERR_INVALID, "unsupported gradient dtype");
    if (n > 0 && (!dy || !aligned_to(dy, dtype_size(dy_dtype))))
      return fail(ZR_ERR_INVALID, "dy is null or not element-aligned");
    if (dy_stride < dim) return fail(ZR_ERR_INVALID, "dy_stride must be >= dim");
    Clip clip;
    st = clip_param(plan, param, main_grad, window_base, window_len, &clip);
    if (st != ZR_OK) return st;
    const Shape s = shape_of(n, dim);
    if (!workspace || !aligned_to(workspace, 16) || workspace_bytes < s.bytes)
      return fail(ZR_ERR_INVALID, "workspace is null, not 16-byte aligned or smaller than " +
                                      std::to_string(s.bytes) + " bytes");
    if (clip.first == clip.last || (n == 0 && !first)) return ZR_OK;
    char* ws = static_cast<char*>(workspace);
    const EmbedWork w{reinterpret_cast<int32_t*>(ws), reinterpret_cast<int32_t*>(ws + s.pos),
                      reinterpret_cast<int32_t*>(ws + s.row),
                      reinterpret_cast<float*>(ws + s.partial)};
    float* table = main_grad + clip.place;
    SortArgs sa{};
    sa.tokens = Tokens{tokens, token_type == ZR_I64};
    sa.w = w;
    sa.n = n;
    sa.row0 = clip.first / dim;
    const int64_t rows = ceil_div(clip.last, dim) - sa.row0;
    if (rows >= (int64_t(1) << 30)) return fail(ZR_ERR_UNSUPPORTED, "2^30 rows or more in the window");
    sa.rows = static_cast<int32_t>(rows);
    // as many workgroups as the chip has CUs, where each has a row and none too many
    sa.shift = 0;
    while ((int64_t(1) << sa.shift) < 256 && (int64_t(2) << sa.shift) <= rows) ++sa.shift;
    while ((rows >> sa.shift) >= kSortRows) ++sa.shift;
    sa.main_grad = first ? table : nullptr;
    // Zeroing rows that the tokens will write again costs less than waiting
    // for the ids' count, where there are few tokens (of the batch: how many lie
    // in the window is not known here).  The whole call: 333
    // tokens of 16753 rows of 1001 columns 19.2 us against 20.8, 8192 of 50257
    // rows of 768 46 both ways, 16384 of them 45.7 against 44.5 (back to back).
    sa.zero_all = n <= rows / 4;
    sa.dim = dim;
    sa.first = clip.first;
    sa.last = clip.last;
    auto* sort = token_type == ZR_I64 ? embed_sort_kernel<int64_t> : embed_sort_kernel<int32_t>;
    ZR_LAUNCH(1 << sa.shift, 64 * kSortWaves, stream, sa, sort);
    st = launched("embedding sort launch");
    if (st != ZR_OK || n == 0) return st;
    SumArgs a{};
    a.dy = dy;
    a.w = w;
    a.main_grad = table;
    a.dy_stride = dy_stride;
    a.dim = static_cast<int32_t>(dim);
    a.row0 = sa.row0;
    a.first = clip.first;
    a.last = clip.last;
    a.piece = static_cast<int32_t>(s.piece);
    a.cols = static_cast<int32_t>(s.cols);
    a.scale = scale;
    if (dy_dtype == ZR_BF16) {
      if (first) launch_sum<uint16_t, true>(a, s.pieces, stream);
      else launch_sum<uint16_t, false>(a, s.pieces, stream);
    } else {
      if (first) launch_sum<float, true>(a, s.pieces, stream);
      else launch_sum<float, false>(a, s.pieces, stream);
    }
    st = launched("embedding sum launch");
    if (st != ZR_OK || s.pieces == 1) return st;
    const dim3 grid(s.pieces - 1, ceil_div(dim, kJoinCols));
    if (first) ZR_LAUNCH(grid, 64 * kJoinWaves, stream, a, embed_join_kernel<true>);
    else ZR_LAUNCH(grid, 64 * kJoinWaves, stream, a, embed_join_kernel<false>);
    return launched("embedding join launch");
  });
}

}  // namespace

extern "C" zr_status zr_embedding_lookup(const zr_plan* plan, int64_t param, int64_t dim,
                                         const void* const* parts, zr_dtype dtype,
                                         const void* tokens, zr_index token_type, int64_t n,
                                         float scale, void* out, int64_t out_stride,
                                         hipStream_t stream) {
  return guarded([&]() -> zr_status {
    zr_status st = check_table(plan, param, dim, n);
    if (st != ZR_OK) return st;
    st = check_tokens(tokens, token_type, n);
    if (st != ZR_OK) return st;
    if (!valid_dtype(dtype)) return fail(ZR_ERR_INVALID, "unsupported element dtype");
    const int64_t es = dtype_size(dtype);
    if (out_stride < dim) return fail(ZR_ERR_INVALID, "out_stride must be >= dim");
    if (n > 0 && (!out || !aligned_to(out, es)))
      return fail(ZR_ERR_INVALID, "out is null or not element-aligned");
    if (!parts) return fail(ZR_ERR_INVALID, "parts is null");
    const ParamInfo& pi = plan->params[param];
    const GroupInfo& gi = plan->groups[pi.group];
    LookupArgs a{};
    for (int32_t k = 0; k < gi.world; ++k) {
      // only the partitions that hold some of the table are read
      if ((k + 1) * gi.part <= pi.offset || k * gi.part >= pi.offset + pi.numel) continue;
      if (!parts[k] || !aligned_to(parts[k], es))
        return fail(ZR_ERR_INVALID, "partition " + std::to_string(k) + " is null or misaligned");
      a.parts[k] = parts[k];
    }
    if (n == 0) return ZR_OK;
    a.tokens = Tokens{tokens, token_type == ZR_I64};
    a.out = out;
    a.n = n;
    a.vocab = pi.numel / dim;
    a.dim = dim;
    a.out_stride = out_stride;
    a.base = pi.offset;
    a.part = gi.part;
    a.part_inverse = 1.0 / static_cast<double>(gi.part);
    a.scale = scale;
    const int64_t cols = dtype == ZR_BF16 ? kLookupCols<uint16_t> : kLookupCols<float>;
    a.chunks = static_cast<int32_t>(ceil_div(dim, cols));
    const int64_t grid = ceil_div(n * a.chunks, kLookupWaves);
    if (!fits_launch(grid, 64 * kLookupWaves))
      return fail(ZR_ERR_UNSUPPORTED, "too many rows for one call");
    if (dtype == ZR_BF16) ZR_LAUNCH(grid, 64 * kLookupWaves, stream, a, lookup_kernel<uint16_t>);
    else ZR_LAUNCH(grid, 64 * kLookupWaves, stream, a, lookup_kernel<float>);
    return launched("embedding lookup launch");
  });
}

extern "C" zr_status zr_ipg_embedding_workspace(const zr_plan* plan, int64_t param, int64_t dim,
                                                int64_t n, int64_t window_base,
                                                int64_t window_len, int64_t* bytes) {
  return guarded([&]() -> zr_status {
    if (!bytes) return fail(ZR_ERR_INVALID, "null output pointer");
    zr_status st = check_table(plan, param, dim, n);
    if (st != ZR_OK) return st;
    Clip clip;
    st = clip_param(plan, param, reinterpret_cast<const float*>(4), window_base, window_len, &clip);
    if (st != ZR_OK) return st;
    *bytes = shape_of(n, dim).bytes;
    return ZR_OK;
  });
}

extern "C" zr_status zr_ipg_accumulate_embedding(
    const zr_plan* plan, int64_t param, int64_t dim, const void* tokens, zr_index token_type,
    int64_t n, float scale, const void* dy, zr_dtype dy_dtype, int64_t dy_stride,
    float* main_grad, int64_t window_base, int64_t window_len, void* workspace,
    int64_t workspace_bytes, hipStream_t stream) {
  return run_embedding(plan, param, dim, tokens, token_type, n, scale, dy, dy_dtype, dy_stride,
                       main_grad, window_base, window_len, workspace, workspace_bytes, false,
                       stream);
}

extern "C" zr_status zr_ipg_accumulate_embedding_first(
    const zr_plan* plan, int64_t param, int64_t dim, const void* tokens, zr_index token_type,
    int64_t n, float scale, const void* dy, zr_dtype dy_dtype, int64_t dy_stride,
    float* main_grad, int64_t window_base, int64_t window_len, void* workspace,
    int64_t workspace_bytes, hipStream_t stream) {
  return run_embedding(plan, param, dim, tokens, token_type, n, scale, dy, dy_dtype, dy_stride,
                       main_grad, window_base, window_len, workspace, workspace_bytes, true,
                       stream);
}
