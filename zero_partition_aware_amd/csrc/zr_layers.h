// Host and device helpers shared by the layer operators' translation units
// (zr_embed.hip, zr_linear.hip).  Not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <string>

#include "zr_internal.h"

namespace zr {

using u32x2 = uint32_t __attribute__((ext_vector_type(2)));
using u32x4 = uint32_t __attribute__((ext_vector_type(4)));
using f32x4 = float __attribute__((ext_vector_type(4)));
using bf16x2 = __bf16 __attribute__((ext_vector_type(2)));

// Address spaces, and the launch of kernel __VA_ARGS__ over `grid` workgroups of
// `block` lanes.  A CPU build of these files, for bounds checking, has its own.
#ifndef ZR_GLOBAL_AS
#define ZR_GLOBAL_AS __attribute__((address_space(1)))
#define ZR_LDS_AS __attribute__((address_space(3)))
#define ZR_LAUNCH(grid, block, stream, args, ...) __VA_ARGS__<<<(grid), (block), 0, (stream)>>>(args)
#endif

// Global-memory pointers (rather than generic ones): no flat instructions.
template <typename T>
__device__ __forceinline__ const ZR_GLOBAL_AS T* as_global(const void* p) {
  return (const ZR_GLOBAL_AS T*)p;
}
template <typename T>
__device__ __forceinline__ ZR_GLOBAL_AS T* as_global(void* p) {
  return (ZR_GLOBAL_AS T*)p;
}

// Vector accesses that assume no more than kAlign bytes' alignment, the
// elements' own: the GPU's global loads and stores take any address, so rows of
// an odd number of elements need no path of their own.  (An aligned type would
// lose its alignment as a template argument.)
template <typename V, int kAlign>
__device__ __forceinline__ V load_at(const void* p) {
  typedef V __attribute__((aligned(kAlign))) U;
  return *(const ZR_GLOBAL_AS U*)p;
}
template <typename V, int kAlign>
__device__ __forceinline__ V load_once_at(const void* p) {   // past the caches
  typedef V __attribute__((aligned(kAlign))) U;
  return __builtin_nontemporal_load((const ZR_GLOBAL_AS U*)p);
}
template <int kAlign, typename V>
__device__ __forceinline__ void store_at(void* p, V v) {
  typedef V __attribute__((aligned(kAlign))) U;
  *(ZR_GLOBAL_AS U*)p = v;
}

__device__ __forceinline__ float bits_float(uint32_t u) { return __builtin_bit_cast(float, u); }
__device__ __forceinline__ uint32_t float_bits(float f) { return __builtin_bit_cast(uint32_t, f); }
__device__ __forceinline__ float bf16_lo(uint32_t w) { return bits_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return bits_float(w & 0xffff0000u); }
// Two fp32 values to bf16, each rounded to nearest even (one instruction).
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, bf16x2{static_cast<__bf16>(lo), static_cast<__bf16>(hi)});
}
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ int64_t uniform(int64_t x) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(x));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(x >> 32));
  return static_cast<int64_t>((static_cast<uint64_t>(hi) << 32) | lo);
}

// Runs a C entry's body; no C++ exception leaves it.
template <typename F>
zr_status guarded(F body) {
  clear_error();
  try {
    return body();
  } catch (...) {
    return fail(ZR_ERR_OOM, "unexpected host error");
  }
}

inline bool valid_dtype(zr_dtype d) { return d == ZR_BF16 || d == ZR_FP32; }
inline int64_t dtype_size(zr_dtype d) { return d == ZR_BF16 ? 2 : 4; }
inline bool aligned_to(const void* p, int64_t s) { return reinterpret_cast<uintptr_t>(p) % s == 0; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// A launch holds fewer than 2^32 threads along an axis.
inline bool fits_launch(int64_t blocks, int64_t threads) { return blocks <= 0xffffffffll / threads; }

inline zr_status launched(const char* what) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(ZR_ERR_HIP, std::string(what) + ": " + hipGetErrorString(e));
  return ZR_OK;
}

// A parameter's elements inside a main_grad window: [first, last) relative to
// the parameter, and where the parameter's element 0 would lie in the window
// (negative when the window starts inside the parameter).
struct Clip {
  int64_t first = 0, last = 0, place = 0;
};

// Checks a (param, window) pair as zr_ipg_accumulate does.
inline zr_status clip_param(const zr_plan* plan, int64_t p, const float* main_grad,
                            int64_t window_base, int64_t window_len, Clip* out) {
  if (p < 0 || p >= static_cast<int64_t>(plan->params.size()))
    return fail(ZR_ERR_INVALID, "param id out of range");
  if (window_base < 0 || window_len < 0)
    return fail(ZR_ERR_INVALID, "window base and length must be >= 0");
  const ParamInfo& pi = plan->params[p];
  const int64_t padded = plan->groups[pi.group].padded;
  if (window_len > padded || window_base > padded - window_len)
    return fail(ZR_ERR_INVALID, "window runs past the group's padded flat space");
  if (window_len > 0 && (!main_grad || !aligned_to(main_grad, 4)))
    return fail(ZR_ERR_INVALID, "main_grad is null or not element-aligned");
  out->first = std::max(pi.offset, window_base) - pi.offset;
  out->last = std::min(pi.offset + pi.numel, window_base + window_len) - pi.offset;
  if (out->last < out->first) out->last = out->first;
  out->place = pi.offset - window_base;
  return ZR_OK;
}

}  // namespace zr
