// Matrix-core tiles in LDS, shared by the layer operators' products
// (zr_linear.hip, zr_product.hip).  Not part of the ABI.
#pragma once

#include "zr_layers.h"

namespace zr {

using bf16x8 = __bf16 __attribute__((ext_vector_type(8)));
using s16x4 = short __attribute__((ext_vector_type(4)));
using f32x16 = float __attribute__((ext_vector_type(16)));

// A tile in LDS of tokens (or whatever else a sum runs over) and C columns:
// 16-byte units (8 bf16) of a token's row, exchanged by the token's number.
__device__ __forceinline__ int exchanged(int k, int u) { return u ^ (4 * (k & 3)); }
template <int C>
__device__ __forceinline__ int staged(int k, int u) {
  return k * (C * 2) + (exchanged(k, u) << 4);
}

// The eight tokens of one column that a lane of an MFMA takes, from the
// 16-token, 32-column block whose place `at` the lane has.
template <int C>
__device__ __forceinline__ bf16x8 read_columns(const char* lds, int at) {
  using lds_s16x4 = ZR_LDS_AS s16x4;
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(lds + at));
  const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(lds + at + 4 * (C * 2)));
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// All waves' LDS accesses before it are done after it; loads from global
// memory stay in flight.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// The lanes of a wave in four rows of sixteen: those of rows 1 and 3 give their x
// for the y of the lanes in the row before.
__device__ __forceinline__ u32x2 exchange_rows(uint32_t x, uint32_t y) {
  const auto r = __builtin_amdgcn_permlane16_swap(x, y, false, false);
  return u32x2{r[0], r[1]};
}

}  // namespace zr
