// Activation checkpoints in 8 bits and the weight gradients taken from them
// (gfx950).
//
// A checkpoint of X [rows, cols] is one e4m3 code per element and one scale
// byte per row and 32 columns, E + 127 for the scale 2^E: the least E >= -110
// with max |x| <= 448 * 2^E over the block's finite values.  No value is
// clipped, the scale adds no rounding of its own, and code * 2^E is exact in
// bf16 and fp32, so restoring rounds nothing and the gradient's products are
// those of bf16 values.  Rows of codes are padded to whole blocks with zeros,
// so every row of codes starts on 32 bytes whatever cols is.

#include <tuple>
#include <vector>

#include "zr_tiles.h"

using namespace zr;

namespace {

constexpr int kBlock = 32;      // columns that share a scale
constexpr int kMinExp = -110;   // 2^-119, the least code's value, is a normal bf16

// ------------------------------------------------------ store and restore ---

struct ActArgs {
  const void* x;          // rows of x, or (restore) of codes
  void* out;              // rows of codes, or (restore) of out
  uint8_t* scales;
  int64_t total;          // groups of eight columns in all rows
  int64_t cols, stride;   // stride of the rows of x / out
  int32_t row_groups;     // groups of eight columns per row of codes
};

constexpr int kActThreads = 256;

// A thread's group of eight columns: its row and first column.
__device__ __forceinline__ bool act_group(const ActArgs& a, int64_t* row, int* col) {
  const int64_t base = static_cast<int64_t>(blockIdx.x) * kActThreads;
  const int64_t r = base / a.row_groups;
  const uint32_t off = static_cast<uint32_t>(base - r * a.row_groups) + threadIdx.x;
  const uint32_t more = off / static_cast<uint32_t>(a.row_groups);
  *row = r + more;
  *col = 8 * static_cast<int>(off - more * a.row_groups);
  return base + threadIdx.x < a.total;
}

__device__ __forceinline__ void load8(const uint16_t* p, int left, float* x) {
  if (left >= 8) {
    const u32x4 w = load_at<u32x4, 2>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = bf16_lo(w[i]), x[2 * i + 1] = bf16_hi(w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = i < left ? bf16_lo(p[i]) : 0.0f;
  }
}
__device__ __forceinline__ void load8(const float* p, int left, float* x) {
  if (left >= 8) {
    const f32x4 u = load_at<f32x4, 4>(p), v = load_at<f32x4, 4>(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = u[i], x[4 + i] = v[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = i < left ? p[i] : 0.0f;
  }
}

// The largest of a lane's value and those of the three lanes it shares a block
// with: lanes exchanged in pairs, then pairs in fours.
__device__ __forceinline__ uint32_t block_max(uint32_t top) {
  constexpr int kPairs = 0xb1, kFours = 0x4e;   // quad_perm [1,0,3,2] and [2,3,0,1]
  top = max(top, static_cast<uint32_t>(
                     __builtin_amdgcn_mov_dpp(static_cast<int>(top), kPairs, 0xf, 0xf, true)));
  return max(top, static_cast<uint32_t>(
                      __builtin_amdgcn_mov_dpp(static_cast<int>(top), kFours, 0xf, 0xf, true)));
}

// A thread codes eight columns; four neighbours share a block's scale.  Bound
// by HBM: 8192 x 14336 bf16 in 65 us (5.5 TB/s), 67 with exchanges through
// LDS, 64 and 70 with two and four groups a thread; 8192 x 4096 in 21 us, 23
// and 27 with two and four.
template <typename T>
__global__ __launch_bounds__(kActThreads) void act_quantize_kernel(const ActArgs a) {
  int64_t row;
  int col;
  if (!act_group(a, &row, &col)) return;   // whole blocks leave together
  float x[8];
  load8(static_cast<const T*>(a.x) + row * a.stride + col, static_cast<int>(a.cols) - col, x);
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = float_bits(x[i]) & 0x7fffffffu;
    top = b < 0x7f800000u && b > top ? b : top;
  }
  top = block_max(top);
  // top = 1.m * 2^(e-127) <= 1.75 * 2^(8+E); subnormals end at kMinExp.
  int e = static_cast<int>(top >> 23) - 127 - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = max(e, kMinExp);
  const float inverse = bits_float(static_cast<uint32_t>(127 - e) << 23);
  u32x2 w;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    x[i] = (float_bits(x[i]) & 0x7fffffffu) < 0x7f800000u ? x[i] * inverse
                                                          : bits_float(0x7fc00000u);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * i], x[4 * i + 1], 0, false);
    w[i] = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * i + 2], x[4 * i + 3], v, true);
  }
  const int64_t pitch = 8 * static_cast<int64_t>(a.row_groups);
  *as_global<u32x2>(static_cast<char*>(a.out) + row * pitch + col) = w;
  if (col % kBlock == 0) a.scales[row * (pitch / kBlock) + col / kBlock] = e + 127;
}

// Eight codes times their block's scale.  Bound by HBM: 8192 x 14336 to bf16 in
// 63 us (5.6 TB/s).  Stores past the caches take 61, but what reads the values
// next then waits for HBM: 140 us with a reader, 135 so.
template <typename T>
__global__ __launch_bounds__(kActThreads) void act_dequantize_kernel(const ActArgs a) {
  int64_t row;
  int col;
  if (!act_group(a, &row, &col) || col >= a.cols) return;
  const int64_t pitch = 8 * static_cast<int64_t>(a.row_groups);
  const u32x2 w = *as_global<u32x2>(static_cast<const char*>(a.x) + row * pitch + col);
  const float s = bits_float(static_cast<uint32_t>(a.scales[row * (pitch / kBlock) + col / kBlock]) << 23);
  float x[8];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(w[i], false);
    const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(w[i], true);
    x[4 * i] = lo[0] * s, x[4 * i + 1] = lo[1] * s;
    x[4 * i + 2] = hi[0] * s, x[4 * i + 3] = hi[1] * s;
  }
  T* out = static_cast<T*>(a.out) + row * a.stride + col;
  const int left = static_cast<int>(a.cols) - col;
  if constexpr (sizeof(T) == 2) {
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
    if (left >= 8) {
      store_at<2>(out, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) out[i] = static_cast<T>(v[i / 2] >> (16 * (i & 1)));
    }
  } else {
    if (left >= 8) {
      store_at<4>(out, f32x4{x[0], x[1], x[2], x[3]});
      store_at<4>(out + 4, f32x4{x[4], x[5], x[6], x[7]});
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) out[i] = x[i];
    }
  }
}

// ------------------------------------------------------- weight gradients ---
//
// dW[o, i] = sum over tokens t of dY[t, o] * X^[t, i], added to main_grad.
// Both operands lie token by token, so the sum runs over their slow axis.  A
// workgroup of 2 x 4 waves owns 256 x 256 weights, 128 x 64 a wave in the
// accumulators.  Tiles of 64 tokens go into one of two LDS buffers: dY's
// straight from memory where its rows lie on 16 bytes (through registers
// otherwise), X's through registers, where it is decoded once for the
// workgroup.  The transposing LDS read hands each lane of a 32x32x16 MFMA the
// eight tokens of its column.  The 16-byte units of a staged row are exchanged
// (xor) by four times the token's number mod 4, so that the four rows that 16
// lanes read, and the two blocks that 32 do, lie in different banks: 3.0 cycles
// a read, 4.0 with half the distance and 8.0 without.  One barrier a tile:
// while a tile multiplies, the next fragments, the next tile's stores and the
// loads of the one after it are under way (phase below).
//
// What bounds it: the instructions between the MFMAs.  The MFMAs of a tile
// take 2050 cycles of a SIMD, the loop about 2900; without the staging of
// either operand it takes 2400, with dY through registers 3100.  Smaller tiles
// read and store more for each product.  Measured at 4096 x 4096 weights and
// 8192 tokens: 1332 TFLOP/s, 1240 with rows that do not lie on 16 bytes; with
// dY through registers 1207, and of that kind 256 x 128 tiles of four waves,
// two workgroups a CU, 1042, four waves of 128 x 128 1156.  (One full round of
// tiles: weights of few tiles or few tokens were not compared.)

constexpr int kMaxItems = 16;

constexpr int kTileOut = 256;   // columns of dY per workgroup
constexpr int kTileIn = 256;    // columns of X per workgroup
constexpr int kDepth = 64;      // tokens per staged tile
constexpr int kWavesOut = 2, kWavesIn = 4;
constexpr int kThreads = 64 * kWavesOut * kWavesIn;

struct Item {
  const uint16_t* dy;
  const uint8_t* codes;
  const uint8_t* scales;
  float* grad;                 // where the weight's element 0 lies
  int64_t dy_stride, tokens;
  int64_t first, last;         // the weight's elements in the window
  int64_t out, in;             // dY's and X's columns
  int64_t pitch;               // bytes per row of codes
  int32_t out_tile0, in_tile0; // first tiles that meet the window
  int32_t out_tiles, in_tiles;
  int16_t in_major;            // weight stored [in][out] rather than [out][in]
  int16_t direct;              // dY's rows lie on 16 bytes
  // The first `whole` tiles are one workgroup's each; the others' tokens are
  // cut into `pieces`, a workgroup each.
  int32_t whole, pieces;
  int32_t whole0, piece0, cut0;   // whole tiles, pieces and cut tiles of earlier items
};
struct LinearArgs {
  Item item[kMaxItems];
  float* partial;              // a tile of sums for each piece
  int32_t n;
  int32_t first;               // main_grad is written, not added to
  int32_t whole;               // whole tiles in all
};

// One step's share of a thread: rows of dY and of X's codes, in registers
// between their loads and their places in LDS.
constexpr int kOutUnits = kTileOut / 8, kOutRows = kThreads / kOutUnits;
constexpr int kOutLoads = kDepth / kOutRows;
constexpr int kInUnits = kTileIn / 16, kInRows = kThreads / kInUnits;
constexpr int kInLoads = kDepth / kInRows;
static_assert(kOutLoads * kOutRows == kDepth && kInLoads * kInRows == kDepth, "staging shape");

struct StagedOut {
  u32x4 v[kOutLoads];
};
struct StagedIn {
  u32x4 v[kInLoads];
  uint32_t scale[kInLoads];
};

// Where a thread's units of a tile come from.  A unit behind the matrix's last
// column is read from the tile's first instead: its columns are never stored.
struct Loader {
  const char* dy;              // row 0 of the tile's columns
  const char* codes;
  const char* scales;
  int64_t dy_step, x_step, s_step;   // bytes per token
  uint32_t dy_off, x_off, s_off;     // this thread's first unit
  uint32_t direct_off;               // and that of dY straight into LDS
  int32_t dy_row, x_row, dy_left;    // its rows; dY's columns from its unit on

  __device__ __forceinline__ Loader(const Item& it, int64_t o0, int64_t i0, int tid) {
    int u = 8 * (tid % kOutUnits), v = 16 * (tid % kInUnits);
    if (o0 + u >= it.out) u = 0;
    if (i0 + v >= it.pitch) v = 0;
    dy_row = tid / kOutUnits;
    x_row = tid / kInUnits;
    dy_step = it.dy_stride * 2;
    x_step = it.pitch;
    s_step = it.pitch / kBlock;
    dy = reinterpret_cast<const char*>(it.dy) + o0 * 2;
    codes = reinterpret_cast<const char*>(it.codes) + i0;
    scales = reinterpret_cast<const char*>(it.scales) + i0 / kBlock;
    dy_off = dy_row * static_cast<uint32_t>(dy_step) + 2 * u;
    int d = 8 * exchanged(dy_row, tid % kOutUnits);
    if (o0 + d >= it.out) d = 0;
    direct_off = dy_row * static_cast<uint32_t>(dy_step) + 2 * d;
    x_off = x_row * static_cast<uint32_t>(x_step) + v;
    s_off = x_row * static_cast<uint32_t>(s_step) + v / kBlock;
    dy_left = static_cast<int>(it.out - o0 < kTileOut ? it.out - o0 : kTileOut) - u;
  }
  // The whole tile's tokens from t on, all there.  A unit that the row's end
  // cuts is read whole: it ends in the next row.
  template <int kJ0, int kJ1>
  __device__ __forceinline__ void load_dy(StagedOut& s, int64_t t) const {
    const char* d = dy + t * dy_step;
#pragma unroll
    for (int j = kJ0; j < kJ1; ++j)
      s.v[j] = load_at<u32x4, 2>(d + (dy_off + j * (kOutRows * static_cast<uint32_t>(dy_step))));
  }
  // dY straight into LDS, where a wave's 64 units lie one after the other: the
  // exchange is made by what each lane reads.  Units on 16 bytes.
  __device__ __forceinline__ void direct_dy(char* lds, int64_t t, int w) const {
    const char* d = dy + t * dy_step;
#pragma unroll
    for (int j = 0; j < kOutLoads; ++j)
      __builtin_amdgcn_global_load_lds(
          (const ZR_GLOBAL_AS void*)(d + (direct_off + j * (kOutRows * static_cast<uint32_t>(dy_step)))),
          (ZR_LDS_AS void*)(lds + (w * (64 / kOutUnits) + j * kOutRows) * (kTileOut * 2)),
          16, 0, 0);
  }
  __device__ __forceinline__ void load_x(StagedIn& s, int64_t t) const {
    const char* x = codes + t * x_step;
    const char* c = scales + t * s_step;
#pragma unroll
    for (int j = 0; j < kInLoads; ++j) {
      s.v[j] = *as_global<u32x4>(x + (x_off + j * (kInRows * static_cast<uint32_t>(x_step))));
      s.scale[j] = *as_global<uint8_t>(c + (s_off + j * (kInRows * static_cast<uint32_t>(s_step))));
    }
  }
  // The same for `tokens` tokens, fewer than kDepth perhaps, up to the last.
  __device__ __forceinline__ void load_some(StagedOut& o, StagedIn& i, int64_t t, int64_t tokens) const {
    const char* d = dy + t * dy_step;
    const char* x = codes + t * x_step;
    const char* c = scales + t * s_step;
#pragma unroll
    for (int j = 0; j < kOutLoads; ++j) {
      o.v[j] = u32x4{0, 0, 0, 0};
      if (dy_row + j * kOutRows < tokens) {
        const char* p = d + (dy_off + j * (kOutRows * static_cast<uint32_t>(dy_step)));
        if (dy_left >= 8) {
          o.v[j] = load_at<u32x4, 2>(p);
        } else {
#pragma unroll
          for (int e = 0; e < 7; ++e)
            if (e < dy_left)
              o.v[j][e / 2] |= static_cast<uint32_t>(as_global<uint16_t>(p)[e]) << (16 * (e & 1));
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kInLoads; ++j) {
      i.v[j] = u32x4{0, 0, 0, 0};
      i.scale[j] = 127;
      if (x_row + j * kInRows < tokens) {
        i.v[j] = *as_global<u32x4>(x + (x_off + j * (kInRows * static_cast<uint32_t>(x_step))));
        i.scale[j] = *as_global<uint8_t>(c + (s_off + j * (kInRows * static_cast<uint32_t>(s_step))));
      }
    }
  }
};

// A staged tile in LDS: dY's columns, then X's, decoded.
constexpr int kOutBytes = kDepth * kTileOut * 2, kInBytes = kDepth * kTileIn * 2;
constexpr int kStage = kOutBytes + kInBytes;

template <int kJ0, int kJ1>
__device__ __forceinline__ void store_dy(const StagedOut& s, char* lds, int tid) {
#pragma unroll
  for (int j = kJ0; j < kJ1; ++j)
    *reinterpret_cast<u32x4*>(lds + staged<kTileOut>(tid / kOutUnits + j * kOutRows, tid % kOutUnits)) =
        s.v[j];
}
__device__ __forceinline__ void store_x(const StagedIn& s, char* lds, int tid) {
#pragma unroll
  for (int j = 0; j < kInLoads; ++j) {
    const float scale = bits_float(s.scale[j] << 23);
    u32x4 w[2];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      w[e / 2][2 * (e & 1)] = __builtin_bit_cast(
          uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(s.v[j][e], scale, false));
      w[e / 2][2 * (e & 1) + 1] = __builtin_bit_cast(
          uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(s.v[j][e], scale, true));
    }
    // Every other unit at a time costs the store two of sixteen cycles; a
    // choice between the two halves by the lane would cost more.
    const int k = tid / kInUnits + j * kInRows, u = 2 * (tid % kInUnits);
    *reinterpret_cast<u32x4*>(lds + staged<kTileIn>(k, u)) = w[0];
    *reinterpret_cast<u32x4*>(lds + staged<kTileIn>(k, u + 1)) = w[1];
  }
}

constexpr int kOutBlocks = kTileOut / kWavesOut / 32;   // 32-column blocks of a wave
constexpr int kInBlocks = kTileIn / kWavesIn / 32;

using Acc = f32x16[kOutBlocks][kInBlocks];

// The fragments of sixteen tokens that a wave multiplies.
struct Fragments {
  bf16x8 d[kOutBlocks], x[kInBlocks];
};
struct Reader {
  int d[kOutBlocks], x[kInBlocks];   // a lane's places in a staged tile's halves
  __device__ __forceinline__ Reader(int lane, int w) {
    const int g = lane >> 4, q = lane & 15;
    const int k = 8 * (g >> 1) + (q >> 2), c = 16 * (g & 1) + 4 * (q & 3);
#pragma unroll
    for (int b = 0; b < kOutBlocks; ++b) {
      const int at = (w / kWavesIn) * (32 * kOutBlocks) + 32 * b + c;
      d[b] = staged<kTileOut>(k, at / 8) + (at % 8) * 2;
    }
#pragma unroll
    for (int b = 0; b < kInBlocks; ++b) {
      const int at = (w % kWavesIn) * (32 * kInBlocks) + 32 * b + c;
      x[b] = staged<kTileIn>(k, at / 8) + (at % 8) * 2;
    }
  }
  __device__ __forceinline__ void read(Fragments& f, const char* dy, const char* in, int k) const {
#pragma unroll
    for (int b = 0; b < kOutBlocks; ++b) f.d[b] = read_columns<kTileOut>(dy, d[b] + k * (kTileOut * 2));
#pragma unroll
    for (int b = 0; b < kInBlocks; ++b) f.x[b] = read_columns<kTileIn>(in, x[b] + k * (kTileIn * 2));
  }
};

template <bool kInMajor>
__device__ __forceinline__ void multiply(Acc& acc, const Fragments& f) {
#pragma unroll
  for (int i = 0; i < kOutBlocks; ++i)
#pragma unroll
    for (int j = 0; j < kInBlocks; ++j)
      acc[i][j] = kInMajor
                      ? __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.x[j], f.d[i], acc[i][j], 0, 0, 0)
                      : __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.d[i], f.x[j], acc[i][j], 0, 0, 0);
}

// What the pipelined loop keeps in registers.
struct Pipe {
  StagedOut dy;    // the next tile's, unless dY goes straight into LDS
  StagedIn x;      // the next tile's
  Fragments f[2];
};

// Sixteen tokens of tile n: while they multiply, the next sixteen's fragments
// are read and a third of tile n + 1 is put into LDS.
template <bool kInMajor, bool kDirect, int kPhase>
__device__ __forceinline__ void phase(Acc& acc, Pipe& r, const Loader& in, const Reader& reader,
                                      const char* cur, char* next_dy, char* next_x, int64_t t1,
                                      int64_t t2, int tid) {
  constexpr int kPhases = kDepth / 16, kParts = kPhases - 1;
  static_assert(kPhases == 4, "four phases in step");
  Fragments& next = r.f[(kPhase + 1) & 1];
  if constexpr (kPhase == kParts) {
    if constexpr (kDirect) __builtin_amdgcn_s_waitcnt(0x0f70);   // vmcnt(0): dY is there
    lds_barrier();
    reader.read(next, next_dy, next_x, 0);
    in.load_x(r.x, t2);
  } else {
    reader.read(next, cur, cur + kOutBytes, 16 * (kPhase + 1));
    if constexpr (kDirect) {
      if constexpr (kPhase == 0) in.direct_dy(next_dy, t1, uniform(tid >> 6));
    } else {
      constexpr int d0 = kOutLoads * kPhase / kParts, d1 = kOutLoads * (kPhase + 1) / kParts;
      store_dy<d0, d1>(r.dy, next_dy, tid);
      in.load_dy<d0, d1>(r.dy, t2);
    }
    // X last: it was asked for after the last barrier
    if constexpr (kPhase == kParts - 1) store_x(r.x, next_x, tid);
  }
  multiply<kInMajor>(acc, r.f[kPhase & 1]);
  // Three reads behind each of the first MFMAs, and nothing over the phase's
  // end (measured, 4096 x 4096 weights over 8192 tokens: 208 us; two reads
  // each 212, one and two in turn 217, the compiler's own order 231).
  constexpr int kReads = 2 * (kOutBlocks + kInBlocks);
#pragma unroll
  for (int i = 0; i < kReads / 3; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // MFMA
    __builtin_amdgcn_sched_group_barrier(0x100, 3, 0);   // LDS read
  }
  __builtin_amdgcn_sched_group_barrier(0x008, kOutBlocks * kInBlocks - kReads / 3, 0);
  __builtin_amdgcn_sched_barrier(0);
}

// Tile n, with the tokens of tiles n + 1 and n + 2 from t1 and t2 on.  The
// pointers are restricted so that the compiler sees that reads of the current
// buffer need not wait for what goes into the other.
template <bool kInMajor, bool kDirect>
__device__ __forceinline__ void step(Acc& acc, Pipe& r, const Loader& in, const Reader& reader,
                                     const char* __restrict cur, char* __restrict next_dy,
                                     char* __restrict next_x, int64_t t1, int64_t t2, int tid) {
  phase<kInMajor, kDirect, 0>(acc, r, in, reader, cur, next_dy, next_x, t1, t2, tid);
  phase<kInMajor, kDirect, 1>(acc, r, in, reader, cur, next_dy, next_x, t1, t2, tid);
  phase<kInMajor, kDirect, 2>(acc, r, in, reader, cur, next_dy, next_x, t1, t2, tid);
  phase<kInMajor, kDirect, 3>(acc, r, in, reader, cur, next_dy, next_x, t1, t2, tid);
}

// `steps` whole tiles of tokens from t0 on.
template <bool kInMajor, bool kDirect>
__device__ __forceinline__ void whole_tiles(const Loader& in, const Reader& reader, int64_t t0,
                                            int steps, char* lds, Acc& acc, int tid) {
  Pipe r;
  // behind the last tile, the last is loaded and staged again, unused
  auto tile = [&](int n) { return t0 + static_cast<int64_t>(n < steps ? n : steps - 1) * kDepth; };
  if constexpr (kDirect) {
    in.direct_dy(lds, t0, uniform(tid >> 6));
  } else {
    in.load_dy<0, kOutLoads>(r.dy, t0);
    store_dy<0, kOutLoads>(r.dy, lds, tid);
    in.load_dy<0, kOutLoads>(r.dy, tile(1));
  }
  in.load_x(r.x, t0);
  store_x(r.x, lds + kOutBytes, tid);
  in.load_x(r.x, tile(1));
  if constexpr (kDirect) __builtin_amdgcn_s_waitcnt(0x0f70);   // vmcnt(0)
  lds_barrier();
  reader.read(r.f[0], lds, lds + kOutBytes, 0);
  int stage = 0;
#pragma unroll 1
  for (int n = 0; n < steps; ++n) {
    const char* cur = lds + stage;
    stage = kStage - stage;
    char* next = lds + stage;
    step<kInMajor, kDirect>(acc, r, in, reader, cur, next, next + kOutBytes, tile(n + 1), tile(n + 2),
                            tid);
  }
}

// The tile's sums over the tokens [t0, t1), added to the MFMAs' accumulators:
// a block's rows are the weight's stored rows, its columns a row's elements.
template <bool kInMajor, bool kDirect>
__device__ __forceinline__ void tile_sums(const Item& it, int64_t o0, int64_t i0, int64_t t0,
                                          int64_t t1, char* lds, Acc& acc) {
  const int tid = threadIdx.x;
  const Loader in(it, o0, i0, tid);
  const Reader reader(tid & 63, uniform(tid >> 6));
  // Whole tiles of tokens.  The matrix's last row cannot be read past its end,
  // and a row of fewer than eight columns ends behind the next row.
  const int64_t end = it.out % 8 && t1 == it.tokens ? t1 - 1 : t1;
  const int steps = it.out < 8 || end < t0 ? 0 : static_cast<int>((end - t0) / kDepth);
  if (steps > 0) {
    if (kDirect || it.direct) whole_tiles<kInMajor, true>(in, reader, t0, steps, lds, acc, tid);
    else whole_tiles<kInMajor, false>(in, reader, t0, steps, lds, acc, tid);
    t0 += static_cast<int64_t>(steps) * kDepth;
  }
  for (; t0 < t1; t0 += kDepth) {
    StagedOut dy;
    StagedIn x;
    in.load_some(dy, x, t0, t1 - t0);
    __builtin_amdgcn_s_waitcnt(0x0f70);   // vmcnt(0): nothing goes into LDS any more
    lds_barrier();
    store_dy<0, kOutLoads>(dy, lds, tid);
    store_x(x, lds + kOutBytes, tid);
    lds_barrier();
#pragma unroll 1
    for (int k = 0; k < kDepth; k += 16) {
      Fragments f;
      reader.read(f, lds, lds + kOutBytes, k);
      multiply<kInMajor>(acc, f);
    }
  }
}

// A tile's place: its first columns of dY and X.  Bands of eight tiles of dY's
// columns are walked along X's columns.
template <bool kInMajor>
struct Place {
  int64_t o0, i0;
  bool whole;                  // all its weights are there and in the window
  __device__ __forceinline__ Place(const Item& it, int tile) {
    const int band = tile / (8 * it.in_tiles), at = tile - band * 8 * it.in_tiles;
    const int height = it.out_tiles - 8 * band < 8 ? it.out_tiles - 8 * band : 8;
    o0 = static_cast<int64_t>(it.out_tile0 + 8 * band + at % height) * kTileOut;
    i0 = static_cast<int64_t>(it.in_tile0 + at / height) * kTileIn;
    const int64_t r = kInMajor ? i0 : o0, c = kInMajor ? o0 : i0;
    const int64_t rows = kInMajor ? it.in : it.out, cols = kInMajor ? it.out : it.in;
    const int high = kInMajor ? kTileIn : kTileOut, wide = kInMajor ? kTileOut : kTileIn;
    whole = r + high <= rows && c + wide <= cols && r * cols + c >= it.first &&
            (r + high - 1) * cols + c + wide <= it.last;
  }
};

// kCount of the sixteen sums that a lane has of block (i, j), from the v0-th
// on, into main_grad: stored rows 8 * (v / 4) + v % 4, one column a lane.
template <int kCount, bool kInMajor, typename V>
__device__ __forceinline__ void put_sums(const Item& it, const Place<kInMajor>& at, bool first, int w,
                                         int lane, int i, int j, int v0, const V& sums) {
  const int64_t o = at.o0 + (w / kWavesIn) * (32 * kOutBlocks) + 32 * i;
  const int64_t c = at.i0 + (w % kWavesIn) * (32 * kInBlocks) + 32 * j;
  const int64_t cols = kInMajor ? it.out : it.in, rows = kInMajor ? it.in : it.out;
  const int64_t row = (kInMajor ? c : o) + 4 * (lane >> 5);
  const int64_t col = (kInMajor ? o : c) + (lane & 31);
  if (at.whole) {
    float* p = it.grad + row * cols + col;
    float old[kCount] = {};
    if (!first) {
#pragma unroll
      for (int v = 0; v < kCount; ++v)
        old[v] = *as_global<float>(p + (8 * ((v0 + v) / 4) + ((v0 + v) & 3)) * cols);
    }
#pragma unroll
    for (int v = 0; v < kCount; ++v)
      *as_global<float>(p + (8 * ((v0 + v) / 4) + ((v0 + v) & 3)) * cols) = old[v] + sums[v];
  } else {
    auto place = [&](int v) { return (row + 8 * ((v0 + v) / 4) + ((v0 + v) & 3)) * cols + col; };
    auto there = [&](int v) {
      return row + 8 * ((v0 + v) / 4) + ((v0 + v) & 3) < rows && col < cols &&
             place(v) >= it.first && place(v) < it.last;
    };
    if (first) {
#pragma unroll
      for (int v = 0; v < kCount; ++v)
        if (there(v)) it.grad[place(v)] = 0.0f + sums[v];
    } else {   // all asked for before the first is used
      float old[kCount] = {};
      bool in[kCount];
#pragma unroll
      for (int v = 0; v < kCount; ++v)
        if ((in[v] = there(v))) old[v] = it.grad[place(v)];
#pragma unroll
      for (int v = 0; v < kCount; ++v)
        if (in[v]) it.grad[place(v)] = old[v] + sums[v];
    }
  }
}

// kDirect: every item's dY lies on 16 bytes.
template <bool kInMajor, bool kDirect>
__global__ __launch_bounds__(kThreads, 2) void linear_kernel(const LinearArgs a) {
  __shared__ __align__(16) char lds[2 * kStage];
  const int tid = threadIdx.x, lane = tid & 63, w = uniform(tid >> 6);
  // Consecutive workgroups go round the eight XCDs: of the 256 that run at
  // once, each XCD takes 32 neighbours, which share columns in its L2.
  const int round = blockIdx.x & ~255;
  const int now = static_cast<int>(gridDim.x) - round < 256 ? gridDim.x - round : 256;
  const int xcd = blockIdx.x % 8, more = now % 8;
  const int id = round + xcd * (now / 8) + (xcd < more ? xcd : more) + (blockIdx.x - round) / 8;
  int k = 0, tile;
  int64_t t0 = 0, t1;
  float* partial = nullptr;
  if (id < a.whole) {
    while (k + 1 < a.n && a.item[k + 1].whole0 <= id) ++k;
    tile = id - a.item[k].whole0;
    t1 = a.item[k].tokens;
  } else {
    const int piece = id - a.whole;
    while (k + 1 < a.n && a.item[k + 1].piece0 <= piece) ++k;
    const Item& it = a.item[k];
    const int cut = it.out_tiles * it.in_tiles - it.whole;
    const int p = (piece - it.piece0) / cut;
    tile = it.whole + (piece - it.piece0) % cut;
    const int64_t steps = (it.tokens + kDepth - 1) / kDepth;
    t0 = p * steps / it.pieces * kDepth;
    t1 = p + 1 < it.pieces ? (p + 1) * steps / it.pieces * kDepth : it.tokens;
    partial = a.partial + static_cast<int64_t>(piece) * (kTileOut * kTileIn);
  }
  const Item& it = a.item[k];
  const Place<kInMajor> at(it, tile);
  Acc acc = {};
  tile_sums<kInMajor, kDirect>(it, at.o0, at.i0, t0, t1, lds, acc);
#pragma unroll
  for (int i = 0; i < kOutBlocks; ++i)
#pragma unroll
    for (int j = 0; j < kInBlocks; ++j) {
      if (partial) {
#pragma unroll
        for (int v = 0; v < 4; ++v)
          *as_global<f32x4>(partial + (((i * kInBlocks + j) * 4 + v) * kThreads + tid) * 4) =
              f32x4{acc[i][j][4 * v], acc[i][j][4 * v + 1], acc[i][j][4 * v + 2], acc[i][j][4 * v + 3]};
      } else {
        put_sums<16>(it, at, a.first, w, lane, i, j, 0, acc[i][j]);
      }
    }
}

// Adds up the pieces of the cut tiles, in their order: a workgroup for each
// four rows of each block.
constexpr int kJoins = kOutBlocks * kInBlocks * 4;
template <bool kInMajor>
__global__ __launch_bounds__(kThreads) void linear_join_kernel(const LinearArgs a) {
  const int tid = threadIdx.x, cut = blockIdx.x / kJoins, part = blockIdx.x % kJoins;
  int k = 0;
  while (k + 1 < a.n && a.item[k + 1].cut0 <= cut) ++k;
  const Item& it = a.item[k];
  const int tile = cut - it.cut0;
  const int64_t step = static_cast<int64_t>(it.out_tiles * it.in_tiles - it.whole) * (kTileOut * kTileIn);
  const float* p = a.partial + (static_cast<int64_t>(it.piece0) + tile) * (kTileOut * kTileIn) +
                   (part * kThreads + tid) * 4;
  f32x4 sum = *as_global<f32x4>(p);
  // Four pieces at a time are asked for before the first is added (seven of 36
  // tiles: 1.4 us less than one after the other; eight at a time no better).
  for (int n = 1; n < it.pieces; n += 4) {
    f32x4 x[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (n + u < it.pieces) x[u] = *as_global<f32x4>(p + (n + u) * step);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (n + u < it.pieces) sum += x[u];
  }
  const int block = part / 4;
  put_sums<4>(it, Place<kInMajor>(it, it.whole + tile), a.first, uniform(tid >> 6), tid & 63,
              block / kInBlocks, block % kInBlocks, 4 * (part % 4), sum);
}

zr_status check_rows(const void* codes, const uint8_t* scales, int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 1) return fail(ZR_ERR_INVALID, "rows must be >= 0 and cols >= 1");
  if (cols >= (int64_t(1) << 30)) return fail(ZR_ERR_UNSUPPORTED, "2^30 columns or more");
  if (rows > 0 && (!codes || !aligned_to(codes, 16) || !scales))
    return fail(ZR_ERR_INVALID, "codes or scales is null, or codes is not 16-byte aligned");
  return ZR_OK;
}

zr_status act_args(const void* x, zr_dtype dtype, int64_t rows, int64_t cols, int64_t stride,
                   const void* codes, const uint8_t* scales, const char* name, ActArgs* a,
                   int64_t* grid) {
  zr_status st = check_rows(codes, scales, rows, cols);
  if (st != ZR_OK) return st;
  if (!valid_dtype(dtype)) return fail(ZR_ERR_INVALID, "unsupported element dtype");
  if (stride < cols) return fail(ZR_ERR_INVALID, std::string(name) + "_stride must be >= cols");
  if (rows > 0 && (!x || !aligned_to(x, dtype_size(dtype))))
    return fail(ZR_ERR_INVALID, std::string(name) + " is null or not element-aligned");
  a->scales = const_cast<uint8_t*>(scales);
  a->cols = cols;
  a->stride = stride;
  a->row_groups = static_cast<int32_t>(ceil_div(cols, kBlock) * (kBlock / 8));
  if (rows > (int64_t(1) << 32) / a->row_groups ||
      !fits_launch(ceil_div(rows * a->row_groups, kActThreads), kActThreads))
    return fail(ZR_ERR_UNSUPPORTED, "too many elements for one call");
  a->total = rows * a->row_groups;
  *grid = ceil_div(a->total, kActThreads);
  return ZR_OK;
}

// Checks the items of a call and builds their launch arguments (those that
// meet the window, in calls of kMaxItems).
zr_status linear_items(const zr_plan* plan, const zr_linear_grad* items, int64_t n,
                       const float* main_grad, int64_t window_base, int64_t window_len,
                       bool first, std::vector<Item>* out) {
  if (!plan) return fail(ZR_ERR_INVALID, "plan is null");
  if (n < 0) return fail(ZR_ERR_INVALID, "n must be >= 0");
  if (n > 0 && !items) return fail(ZR_ERR_INVALID, "null item list");
  std::vector<int64_t> seen;
  int32_t group = -1;
  for (int64_t k = 0; k < n; ++k) {
    const zr_linear_grad& z = items[k];
    if (z.param < 0 || z.param >= static_cast<int64_t>(plan->params.size()))
      return fail(ZR_ERR_INVALID, "param id out of range");
    const ParamInfo& pi = plan->params[z.param];
    if (group < 0) group = pi.group;
    if (pi.group != group) return fail(ZR_ERR_INVALID, "params of one call must share a group");
    Clip clip;
    zr_status st = clip_param(plan, z.param, main_grad, window_base, window_len, &clip);
    if (st != ZR_OK) return st;
    seen.push_back(z.param);
    if (z.n_out < 1 || z.n_in < 1 || z.n_out > pi.numel || pi.numel % z.n_out ||
        pi.numel / z.n_out != z.n_in)
      return fail(ZR_ERR_INVALID, "n_out * n_in must be the param's elements");
    st = check_rows(z.codes, z.scales, z.tokens, z.n_in);
    if (st != ZR_OK) return st;
    // 32-bit offsets in a tile, and tiles counted in 32 bits
    if (z.n_in >= (int64_t(1) << 24) || z.dy_stride >= (int64_t(1) << 24) ||
        z.tokens >= (int64_t(1) << 31))
      return fail(ZR_ERR_UNSUPPORTED, "n_in or dy_stride of 2^24, or tokens of 2^31, or more");
    if (z.dy_stride < z.n_out) return fail(ZR_ERR_INVALID, "dy_stride must be >= n_out");
    if (z.tokens > 0 && (!z.dy || !aligned_to(z.dy, 2)))
      return fail(ZR_ERR_INVALID, "dy is null or not element-aligned");
    if (clip.first == clip.last || (z.tokens == 0 && !first)) continue;
    Item it{};
    it.dy = z.dy;
    it.codes = z.codes;
    it.scales = z.scales;
    it.grad = const_cast<float*>(main_grad) + clip.place;
    it.dy_stride = z.dy_stride;
    it.tokens = z.tokens;
    it.first = clip.first;
    it.last = clip.last;
    it.out = z.n_out;
    it.in = z.n_in;
    it.pitch = ceil_div(z.n_in, kBlock) * kBlock;
    it.in_major = z.in_major != 0;
    it.direct = aligned_to(z.dy, 16) && z.dy_stride % 8 == 0;
    // Tiles of the stored rows that meet the window; within a row, all.
    const int64_t row = it.in_major ? it.out : it.in;
    const int64_t high = it.in_major ? kTileIn : kTileOut, wide = it.in_major ? kTileOut : kTileIn;
    const int64_t r0 = clip.first / row / high, r1 = ceil_div(ceil_div(clip.last, row), high);
    const int64_t all = ceil_div(row, wide);
    if ((r1 - r0) * all > 0x3fffffff) return fail(ZR_ERR_UNSUPPORTED, "weight too large for one call");
    (it.in_major ? it.in_tile0 : it.out_tile0) = static_cast<int32_t>(r0);
    it.in_tiles = static_cast<int32_t>(it.in_major ? r1 - r0 : all);
    it.out_tiles = static_cast<int32_t>(it.in_major ? all : r1 - r0);
    out->push_back(it);
  }
  // One storage order's items together, and tiles with most tokens first: the
  // last to start are the shortest.
  std::stable_sort(out->begin(), out->end(), [](const Item& a, const Item& b) {
    return std::make_tuple(a.in_major, b.tokens) < std::make_tuple(b.in_major, a.tokens);
  });
  std::sort(seen.begin(), seen.end());
  if (std::adjacent_find(seen.begin(), seen.end()) != seen.end())
    return fail(ZR_ERR_INVALID, "param listed twice in one call");
  return ZR_OK;
}

// The items that one launch takes from the k-th on: of one storage order, and at
// most kMaxItems.  Where rows of dY lie does not matter, or it would show in how
// the sums are cut; and two kinds in one launch fill the chip together (768 x 768
// and 2304 x 768 weights over 8192 tokens, one of each kind: 57 us, 76 in a
// launch each).
size_t launch_end(const std::vector<Item>& items, size_t k) {
  size_t e = k + 1;
  while (e < items.size() && e < k + kMaxItems && items[e].in_major == items[k].in_major) ++e;
  return e;
}

// How many pieces the tokens of a tile in the last round are cut into, where
// `rest` tiles are left for the chip's 256 CUs (one workgroup each): the number
// with the least time in the model below, in 256ths of the time that a tile of
// tokens takes (1.6 us).  Cutting costs the join's launch and the pieces'
// writes and reads, 256 kB each: 3 tiles, and 13 more when every CU has a
// piece.  Measured, cut and not, back to back: 2304 x 768 and 768 x 768 weights
// over 8192 tokens (36 tiles, 7 pieces each; with 5 and 4 pieces 1 us less and 3
// more) 59 and 162 us; 2560 x 2560 over 4096 (100 tiles, 2 pieces) 71 and 88;
// 1024 x 1024 over 2048 (16 tiles, 6 pieces) 30 and 45; 160 x 2451 over 1164 (10
// tiles, 4 pieces) 22 and 36; 14336 x 4096 over 8192 (896 tiles, the last 128
// in 2 pieces) 793 and 825 us.
constexpr int kCus = 256;
int32_t pieces_of(int64_t steps, int64_t rest) {
  int64_t best = 1, least = 256 * steps;
  for (int64_t p = 2; p * rest <= kCus && 2 * p <= steps; ++p) {
    const int64_t cost = 256 * ceil_div(steps, p) + 3 * 256 + 13 * rest * p;
    if (cost < least) best = p, least = cost;
  }
  return static_cast<int32_t>(best);
}

// The launch of up to kMaxItems items: which tiles are one workgroup's, and
// which are cut along their tokens so that the last round fills the chip.
struct Launch {
  LinearArgs a;
  int64_t grid = 0, cut = 0, bytes = 0;   // workgroups, cut tiles, workspace
};
zr_status plan_launch(const Item* items, size_t n, bool first, Launch* out) {
  LinearArgs& a = out->a;
  a = LinearArgs{};
  a.first = first;
  a.n = static_cast<int32_t>(n);
  int64_t all = 0, tiles = 0;   // tiles, and those with tokens
  for (size_t k = 0; k < n; ++k) {
    const int64_t count = int64_t(items[k].out_tiles) * items[k].in_tiles;
    all += count;
    if (items[k].tokens > 0) tiles += count;
  }
  // a workgroup each, and no more pieces than CUs
  if (!fits_launch(all + kCus, kThreads))
    return fail(ZR_ERR_UNSUPPORTED, "weights too large for one call");
  // Tiles of the last round.  Those without tokens, which come last and which
  // only the first micro-batch's form writes, do not count: the other tiles'
  // sums are cut into the same pieces in both forms.
  const int64_t rest = tiles % kCus;
  int64_t before = 0, whole = 0, pieces = 0;
  for (size_t k = 0; k < n; ++k) {
    Item& it = a.item[k] = items[k];
    const int64_t count = int64_t(it.out_tiles) * it.in_tiles;
    const int64_t steps = ceil_div(it.tokens, kDepth);
    it.pieces = rest > 0 ? pieces_of(steps, rest) : 1;   // one without tokens
    it.whole = static_cast<int32_t>(
        it.pieces > 1 ? std::min(count, std::max<int64_t>(0, tiles - rest - before)) : count);
    it.whole0 = static_cast<int32_t>(whole);
    it.piece0 = static_cast<int32_t>(pieces);
    it.cut0 = static_cast<int32_t>(out->cut);
    before += count;
    whole += it.whole;
    out->cut += count - it.whole;
    pieces += (count - it.whole) * it.pieces;
  }
  a.whole = static_cast<int32_t>(whole);
  out->grid = whole + pieces;
  out->bytes = pieces * (kTileOut * kTileIn * 4);
  return ZR_OK;
}

zr_status run_linear(const zr_plan* plan, const zr_linear_grad* items, int64_t n,
                     float* main_grad, int64_t window_base, int64_t window_len, void* workspace,
                     int64_t workspace_bytes, bool first, hipStream_t stream) {
  return guarded([&]() -> zr_status {
    std::vector<Item> todo;
    zr_status st = linear_items(plan, items, n, main_grad, window_base, window_len, first, &todo);
    if (st != ZR_OK) return st;
    std::vector<Launch> launches;
    for (size_t k = 0, e; k < todo.size(); k = e) {
      e = launch_end(todo, k);
      launches.emplace_back();
      Launch& l = launches.back();
      st = plan_launch(&todo[k], e - k, first, &l);
      if (st != ZR_OK) return st;
      if (l.bytes > 0 && (!workspace || !aligned_to(workspace, 16) || workspace_bytes < l.bytes))
        return fail(ZR_ERR_INVALID, "workspace is null, not 16-byte aligned or smaller than " +
                                        std::to_string(l.bytes) + " bytes");
      l.a.partial = static_cast<float*>(workspace);
    }
    for (const Launch& l : launches) {
      const bool in_major = l.a.item[0].in_major;
      // Where all of dY lies on 16 bytes, a kernel without the other kind's loop
      // spills no registers: 33.3 us for two weights of 1024 x 1024 over 2048
      // tokens (33.7), 11.3 for 2048 x 2048 over 64 (11.8).
      const bool direct = std::all_of(l.a.item, l.a.item + l.a.n, [](const Item& it) { return it.direct; });
      auto* kernel = in_major ? (direct ? linear_kernel<true, true> : linear_kernel<true, false>)
                              : (direct ? linear_kernel<false, true> : linear_kernel<false, false>);
      ZR_LAUNCH(l.grid, kThreads, stream, l.a, kernel);
      st = launched("linear gradient launch");
      if (st != ZR_OK) return st;
      if (l.cut == 0) continue;
      auto* join = in_major ? linear_join_kernel<true> : linear_join_kernel<false>;
      ZR_LAUNCH(l.cut * kJoins, kThreads, stream, l.a, join);
      st = launched("linear gradient join launch");
      if (st != ZR_OK) return st;
    }
    return ZR_OK;
  });
}

}  // namespace

extern "C" zr_status zr_act_layout(int64_t cols, int64_t* code_pitch, int64_t* scale_pitch) {
  return guarded([&]() -> zr_status {
    if (!code_pitch && !scale_pitch) return fail(ZR_ERR_INVALID, "null output pointer");
    if (cols < 1) return fail(ZR_ERR_INVALID, "cols must be >= 1");
    if (cols >= (int64_t(1) << 30)) return fail(ZR_ERR_UNSUPPORTED, "2^30 columns or more");
    if (code_pitch) *code_pitch = ceil_div(cols, kBlock) * kBlock;
    if (scale_pitch) *scale_pitch = ceil_div(cols, kBlock);
    return ZR_OK;
  });
}

extern "C" zr_status zr_act_quantize(const void* x, zr_dtype dtype, int64_t rows, int64_t cols,
                                     int64_t x_stride, uint8_t* codes, uint8_t* scales,
                                     hipStream_t stream) {
  return guarded([&]() -> zr_status {
    ActArgs a{};
    int64_t grid = 0;
    const zr_status st = act_args(x, dtype, rows, cols, x_stride, codes, scales, "x", &a, &grid);
    if (st != ZR_OK || rows == 0) return st;
    a.x = x;
    a.out = codes;
    if (dtype == ZR_BF16) ZR_LAUNCH(grid, kActThreads, stream, a, act_quantize_kernel<uint16_t>);
    else ZR_LAUNCH(grid, kActThreads, stream, a, act_quantize_kernel<float>);
    return launched("activation quantize launch");
  });
}

extern "C" zr_status zr_act_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows,
                                       int64_t cols, void* out, zr_dtype dtype,
                                       int64_t out_stride, hipStream_t stream) {
  return guarded([&]() -> zr_status {
    ActArgs a{};
    int64_t grid = 0;
    const zr_status st = act_args(out, dtype, rows, cols, out_stride, codes, scales, "out", &a, &grid);
    if (st != ZR_OK || rows == 0) return st;
    a.x = codes;
    a.out = out;
    if (dtype == ZR_BF16) ZR_LAUNCH(grid, kActThreads, stream, a, act_dequantize_kernel<uint16_t>);
    else ZR_LAUNCH(grid, kActThreads, stream, a, act_dequantize_kernel<float>);
    return launched("activation dequantize launch");
  });
}

extern "C" zr_status zr_ipg_linear_workspace(const zr_plan* plan, const zr_linear_grad* items,
                                             int64_t n, int64_t window_base, int64_t window_len,
                                             int64_t* bytes) {
  return guarded([&]() -> zr_status {
    if (!bytes) return fail(ZR_ERR_INVALID, "null output pointer");
    *bytes = 0;
    std::vector<Item> todo;
    zr_status st = linear_items(plan, items, n, reinterpret_cast<const float*>(4), window_base,
                                window_len, true, &todo);
    if (st != ZR_OK) return st;
    for (size_t k = 0, e; k < todo.size(); k = e) {
      e = launch_end(todo, k);
      Launch l;
      st = plan_launch(&todo[k], e - k, true, &l);
      if (st != ZR_OK) return st;
      *bytes = std::max(*bytes, l.bytes);
    }
    return ZR_OK;
  });
}

extern "C" zr_status zr_ipg_accumulate_linear(const zr_plan* plan, const zr_linear_grad* items,
                                              int64_t n, float* main_grad, int64_t window_base,
                                              int64_t window_len, void* workspace,
                                              int64_t workspace_bytes, hipStream_t stream) {
  return run_linear(plan, items, n, main_grad, window_base, window_len, workspace,
                    workspace_bytes, false, stream);
}

extern "C" zr_status zr_ipg_accumulate_linear_first(const zr_plan* plan,
                                                    const zr_linear_grad* items, int64_t n,
                                                    float* main_grad, int64_t window_base,
                                                    int64_t window_len, void* workspace,
                                                    int64_t workspace_bytes, hipStream_t stream) {
  return run_linear(plan, items, n, main_grad, window_base, window_len, workspace,
                    workspace_bytes, true, stream);
}
