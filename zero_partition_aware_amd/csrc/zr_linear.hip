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

#include <vector>

#include "zr_layers.h"

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
    const u32x4 w = *as_global<u32x4_a2>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = bf16_lo(w[i]), x[2 * i + 1] = bf16_hi(w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = i < left ? bf16_lo(p[i]) : 0.0f;
  }
}
__device__ __forceinline__ void load8(const float* p, int left, float* x) {
  if (left >= 8) {
    const f32x4 u = *as_global<f32x4_a4>(p), v = *as_global<f32x4_a4>(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = u[i], x[4 + i] = v[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = i < left ? p[i] : 0.0f;
  }
}

// A thread codes eight columns; four neighbours share a block's scale.
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
  top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 1)));
  top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 2)));
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

// Eight codes times their block's scale.
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
      *as_global<u32x4_a2>(out) = v;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) out[i] = static_cast<T>(v[i / 2] >> (16 * (i & 1)));
    }
  } else {
    if (left >= 8) {
      *as_global<f32x4_a4>(out) = f32x4{x[0], x[1], x[2], x[3]};
      *as_global<f32x4_a4>(out + 4) = f32x4{x[4], x[5], x[6], x[7]};
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
// Both operands lie token by token, so the sum runs over their slow axis:
// tiles of kDepth tokens are staged in LDS as bf16 (X decoded once, on the
// way in), and the transposing LDS read hands each lane of an MFMA its eight
// tokens of one column.  16-byte units of a staged row are exchanged by the
// token's number (xor), which spreads the four rows that 16 lanes read over
// all banks.

using bf16x8 = __bf16 __attribute__((ext_vector_type(8)));
using s16x4 = short __attribute__((ext_vector_type(4)));
using f32x16 = float __attribute__((ext_vector_type(16)));

constexpr int kMaxItems = 16;
constexpr int kDepth = 64;      // tokens per staged tile
constexpr int kTile = 128;      // columns of dY and of X per workgroup
constexpr int kThreads = 256;   // 2 x 2 waves of 64 x 64

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
  int32_t tile0;               // tiles of earlier items
  int32_t in_major;            // weight stored [in][out] rather than [out][in]
};
struct LinearArgs {
  Item item[kMaxItems];
  int32_t n;
  int32_t first;               // main_grad is written, not added to
};

// Byte offset of the 16-byte unit u of staged row k.
__device__ __forceinline__ int staged(int k, int u) {
  return k * (kTile * 2) + ((u ^ (2 * (k & 3))) << 4);
}

__device__ __forceinline__ bf16x8 read_columns(const char* lds, int at) {
  using lds_s16x4 = __attribute__((address_space(3))) s16x4;
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(lds + at));
  const s16x4 hi =
      __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(lds + at + 4 * (kTile * 2)));
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

__global__ __launch_bounds__(kThreads) void linear_kernel(const LinearArgs a) {
  __shared__ __align__(16) char lds[2][kDepth * kTile * 2];
  const int tid = threadIdx.x, lane = tid & 63, w = uniform(tid >> 6);
  int k = 0;
  while (k + 1 < a.n && a.item[k + 1].tile0 <= static_cast<int>(blockIdx.x)) ++k;
  const Item& it = a.item[k];
  const int tile = blockIdx.x - it.tile0;
  const int64_t o0 = static_cast<int64_t>(it.out_tile0 + tile / it.in_tiles) * kTile;
  const int64_t i0 = static_cast<int64_t>(it.in_tile0 + tile % it.in_tiles) * kTile;
  f32x16 acc[2][2] = {};
  // A lane's place in the transposing read of a 16-token, 32-column block.
  const int g = lane >> 4, q = lane & 15;
  const int k_lane = 8 * (g >> 1) + (q >> 2);
  const int c_lane = 16 * (g & 1) + 4 * (q & 3);
  for (int64_t t0 = 0; t0 < it.tokens; t0 += kDepth) {
    __syncthreads();
    // dY: 64 rows of 16 units of eight bf16.
    for (int j = tid; j < kDepth * (kTile / 8); j += kThreads) {
      const int r = j / (kTile / 8), u = j % (kTile / 8);
      const int64_t t = t0 + r, c = o0 + 8 * u;
      u32x4 v{0, 0, 0, 0};
      if (t < it.tokens && c < it.out) {
        const uint16_t* p = it.dy + t * it.dy_stride + c;
        if (c + 8 <= it.out) {
          v = *as_global<u32x4_a2>(p);
        } else {
          for (int e = 0; e < it.out - c; ++e)
            v[e / 2] |= static_cast<uint32_t>(p[e]) << (16 * (e & 1));
        }
      }
      *reinterpret_cast<u32x4*>(lds[0] + staged(r, u)) = v;
    }
    // X: 64 rows of 16 units of eight codes, decoded.
    for (int j = tid; j < kDepth * (kTile / 8); j += kThreads) {
      const int r = j / (kTile / 8), u = j % (kTile / 8);
      const int64_t t = t0 + r, c = i0 + 8 * u;
      u32x4 v{0, 0, 0, 0};
      if (t < it.tokens && c < it.pitch) {
        const u32x2 x = *as_global<u32x2>(it.codes + t * it.pitch + c);
        const float s = bits_float(
            static_cast<uint32_t>(it.scales[t * (it.pitch / kBlock) + c / kBlock]) << 23);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          v[2 * e] = __builtin_bit_cast(
              uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[e], s, false));
          v[2 * e + 1] = __builtin_bit_cast(
              uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[e], s, true));
        }
      }
      *reinterpret_cast<u32x4*>(lds[1] + staged(r, u)) = v;
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < kDepth; kk += 16) {
      bf16x8 d[2], x[2];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int cd = (w >> 1) * 64 + 32 * b + c_lane, cx = (w & 1) * 64 + 32 * b + c_lane;
        d[b] = read_columns(lds[0], staged(kk + k_lane, cd / 8) + (cd % 8) * 2);
        x[b] = read_columns(lds[1], staged(kk + k_lane, cx / 8) + (cx % 8) * 2);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(d[i], x[j], acc[i][j], 0, 0, 0);
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int64_t o = o0 + (w >> 1) * 64 + 32 * i + 8 * (v / 4) + 4 * (lane >> 5) + (v & 3);
        const int64_t c = i0 + (w & 1) * 64 + 32 * j + (lane & 31);
        const int64_t e = it.in_major ? c * it.out + o : o * it.in + c;
        if (o < it.out && c < it.in && e >= it.first && e < it.last)
          it.grad[e] = (a.first ? 0.0f : it.grad[e]) + acc[i][j][v];
      }
}

zr_status check_rows(const void* codes, const uint8_t* scales, int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 1) return fail(ZR_ERR_INVALID, "rows must be >= 0 and cols >= 1");
  if (cols >= (int64_t(1) << 30) || rows >= (int64_t(1) << 40))
    return fail(ZR_ERR_UNSUPPORTED, "2^30 columns or 2^40 rows or more");
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
  a->total = rows * a->row_groups;
  *grid = ceil_div(a->total, kActThreads);
  if (*grid > 0x7fffffff) return fail(ZR_ERR_UNSUPPORTED, "too many elements for one call");
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
    if (z.n_out >= (int64_t(1) << 30)) return fail(ZR_ERR_UNSUPPORTED, "2^30 outputs or more");
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
    // Tiles of the stored rows that meet the window; within a row, all.
    const int64_t row = it.in_major ? it.out : it.in;
    const int64_t r0 = clip.first / row / kTile, r1 = ceil_div(ceil_div(clip.last, row), kTile);
    const int64_t all = ceil_div(row, kTile);
    if ((r1 - r0) * all > 0x3fffffff) return fail(ZR_ERR_UNSUPPORTED, "weight too large for one call");
    (it.in_major ? it.in_tile0 : it.out_tile0) = static_cast<int32_t>(r0);
    it.in_tiles = static_cast<int32_t>(it.in_major ? r1 - r0 : all);
    it.out_tiles = static_cast<int32_t>(it.in_major ? all : r1 - r0);
    out->push_back(it);
  }
  std::sort(seen.begin(), seen.end());
  if (std::adjacent_find(seen.begin(), seen.end()) != seen.end())
    return fail(ZR_ERR_INVALID, "param listed twice in one call");
  return ZR_OK;
}

zr_status run_linear(const zr_plan* plan, const zr_linear_grad* items, int64_t n,
                     float* main_grad, int64_t window_base, int64_t window_len, void* workspace,
                     int64_t workspace_bytes, bool first, hipStream_t stream) {
  return guarded([&]() -> zr_status {
    std::vector<Item> todo;
    zr_status st = linear_items(plan, items, n, main_grad, window_base, window_len, first, &todo);
    if (st != ZR_OK) return st;
    (void)workspace;
    (void)workspace_bytes;
    for (size_t b = 0; b < todo.size(); b += kMaxItems) {
      LinearArgs a{};
      a.first = first;
      int64_t tiles = 0;
      for (size_t k = b; k < todo.size() && k < b + kMaxItems; ++k) {
        todo[k].tile0 = static_cast<int32_t>(tiles);
        tiles += int64_t(todo[k].out_tiles) * todo[k].in_tiles;
        a.item[a.n++] = todo[k];
      }
      if (tiles > 0x7fffffff) return fail(ZR_ERR_UNSUPPORTED, "weights too large for one call");
      linear_kernel<<<tiles, kThreads, 0, stream>>>(a);
      st = launched("linear gradient launch");
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
    if (dtype == ZR_BF16) act_quantize_kernel<uint16_t><<<grid, kActThreads, 0, stream>>>(a);
    else act_quantize_kernel<float><<<grid, kActThreads, 0, stream>>>(a);
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
    if (dtype == ZR_BF16) act_dequantize_kernel<uint16_t><<<grid, kActThreads, 0, stream>>>(a);
    else act_dequantize_kernel<float><<<grid, kActThreads, 0, stream>>>(a);
    return launched("activation dequantize launch");
  });
}

extern "C" zr_status zr_ipg_linear_workspace(const zr_plan* plan, const zr_linear_grad* items,
                                             int64_t n, int64_t window_base, int64_t window_len,
                                             int64_t* bytes) {
  return guarded([&]() -> zr_status {
    if (!bytes) return fail(ZR_ERR_INVALID, "null output pointer");
    std::vector<Item> todo;
    const zr_status st = linear_items(plan, items, n, reinterpret_cast<const float*>(4),
                                      window_base, window_len, true, &todo);
    if (st != ZR_OK) return st;
    *bytes = 0;
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
