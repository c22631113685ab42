// CPU build of the layer operators' HIP sources (zr_embed.hip, zr_linear.hip),
// for bounds checking under AddressSanitizer and UndefinedBehaviorSanitizer.
//
// These kernels exchange values between the lanes of a wave, share LDS and meet
// at barriers, so every lane of a workgroup runs as a coroutine of its own
// (waves.cpp): it runs until it reaches an operation of its whole wave or a
// barrier, and goes on when all the lanes that are left have reached the same
// one.  Lanes that reach different ones end the program.  LDS is a static array,
// whose bounds AddressSanitizer checks like any other's, and a load into LDS
// arrives only when it is waited for.  This header stands in for
// <hip/hip_runtime.h> when the sources are compiled for the host.
#pragma once

#include <hip/hip_runtime_api.h>   // the runtime's types and declarations

#include <cstddef>
#include <cstdint>
#include <cstring>

#define __global__
#define __device__
#define __forceinline__ inline
#define __shared__ static
#define __launch_bounds__(...)
#define __align__(n) __attribute__((aligned(n)))
#define ZR_GLOBAL_AS
#define ZR_LDS_AS

struct zr_emu_dim {
  unsigned x = 0, y = 0, z = 0;
};
extern zr_emu_dim zr_emu_block, zr_emu_thread, zr_emu_grid, zr_emu_size;
#define blockIdx zr_emu_block
#define threadIdx zr_emu_thread
#define gridDim zr_emu_grid
#define blockDim zr_emu_size

// ------------------------------------------------------------------ launches

void zr_emu_run(dim3 grid, unsigned block, void* kernel, void (*body)(const void*), const void* args);
template <typename Args>
struct zr_emu_call {
  void (*kernel)(Args);
  const Args* args;
};
template <typename Args>
void zr_emu_launch(void (*kernel)(Args), dim3 grid, unsigned block, const Args& args) {
  const zr_emu_call<Args> call{kernel, &args};
  zr_emu_run(grid, block, reinterpret_cast<void*>(kernel),
             [](const void* c) {
               const auto* p = static_cast<const zr_emu_call<Args>*>(c);
               p->kernel(*p->args);
             },
             &call);
}
#define ZR_LAUNCH(grid, block, stream, args, ...) zr_emu_launch(__VA_ARGS__, dim3(grid), (block), args)

// --------------------------------------------------------- wave operations

enum zr_emu_op { kFirstLane, kReadLane, kBallot, kShiftUp, kQuadPerm, kTranspose, kMfma, kWaveSync };
// Gives the lane's input to the operation and returns its result.
void zr_emu_wave(zr_emu_op op, const void* in, size_t in_bytes, void* out, size_t out_bytes);
void zr_emu_barrier();

inline int zr_emu_first(int x) {
  int r;
  zr_emu_wave(kFirstLane, &x, sizeof(x), &r, sizeof(r));
  return r;
}
inline int zr_emu_two(zr_emu_op op, int x, int y) {
  const int in[2] = {x, y};
  int r;
  zr_emu_wave(op, in, sizeof(in), &r, sizeof(r));
  return r;
}
inline uint64_t __ballot(int x) {
  uint64_t r;
  zr_emu_wave(kBallot, &x, sizeof(x), &r, sizeof(r));
  return r;
}
inline int __shfl_up(int x, unsigned d) { return zr_emu_two(kShiftUp, x, static_cast<int>(d)); }
template <typename T>
T min(T a, T b) { return b < a ? b : a; }
template <typename T>
T max(T a, T b) { return a < b ? b : a; }
inline int __popcll(uint64_t x) { return __builtin_popcountll(x); }
inline void __syncthreads() { zr_emu_barrier(); }
inline void zr_emu_fence(int, const char* scope, const char* = nullptr) {
  if (!std::strcmp(scope, "wavefront")) zr_emu_wave(kWaveSync, nullptr, 0, nullptr, 0);
}
inline int atomicAdd(int* p, int x) {
  const int old = *p;
  *p += x;
  return old;
}
#define __builtin_amdgcn_readfirstlane(x) zr_emu_first(static_cast<int>(x))
#define __builtin_amdgcn_readlane(x, lane) zr_emu_two(kReadLane, (x), static_cast<int>(lane))
#define __builtin_amdgcn_mov_dpp(x, control, rows, banks, bound) zr_emu_two(kQuadPerm, (x), (control))
#define __builtin_amdgcn_fence(...) zr_emu_fence(__VA_ARGS__)
#define __builtin_amdgcn_s_barrier() zr_emu_barrier()
#define __builtin_amdgcn_sched_group_barrier(...) ((void)0)
#define __builtin_amdgcn_sched_barrier(x) ((void)0)

// ------------------------------------------------------- numbers and matrices

using zr_emu_s16x4 = short __attribute__((ext_vector_type(4)));
using zr_emu_f32x2 = float __attribute__((ext_vector_type(2)));

uint8_t zr_emu_e4m3(float x);
float zr_emu_e4m3_value(uint8_t code);

inline int zr_emu_cvt_pk_fp8(float lo, float hi, int old, bool high) {
  const uint32_t v = zr_emu_e4m3(lo) | (static_cast<uint32_t>(zr_emu_e4m3(hi)) << 8);
  const uint32_t o = static_cast<uint32_t>(old);
  return static_cast<int>(high ? (o & 0xffffu) | (v << 16) : (o & 0xffff0000u) | v);
}
inline zr_emu_f32x2 zr_emu_cvt_pk_f32(uint32_t codes, bool high) {
  const uint32_t v = high ? codes >> 16 : codes;
  return zr_emu_f32x2{zr_emu_e4m3_value(v & 0xff), zr_emu_e4m3_value((v >> 8) & 0xff)};
}
// Two codes times a power of two, as bf16 patterns: exact.
inline uint32_t zr_emu_cvt_scale(uint32_t codes, float scale, bool high) {
  const zr_emu_f32x2 v = zr_emu_cvt_pk_f32(codes, high) * scale;
  return (__builtin_bit_cast(uint32_t, float(v[0])) >> 16) |
         (__builtin_bit_cast(uint32_t, float(v[1])) & 0xffff0000u);
}
template <typename F>
inline F zr_emu_mfma(const void* a, const void* b, const F& c) {
  unsigned char bytes[96];
  std::memcpy(bytes, a, 16);
  std::memcpy(bytes + 16, b, 16);
  std::memcpy(bytes + 32, &c, 64);
  F r;
  zr_emu_wave(kMfma, bytes, sizeof(bytes), &r, sizeof(r));
  return r;
}
inline zr_emu_s16x4 zr_emu_transpose(const void* p) {
  zr_emu_s16x4 own, r;
  std::memcpy(&own, p, sizeof(own));   // checked here
  zr_emu_wave(kTranspose, &own, sizeof(own), &r, sizeof(r));
  return r;
}
// Sixteen bytes a lane into LDS, lane after lane from `lds` on; there after the
// next wait.
void zr_emu_lds_later(void* lds, const void* data);
void zr_emu_wait();
inline void zr_emu_load_lds(const void* p, void* lds, int bytes, int, int) {
  unsigned char v[16];
  if (bytes != 16) __builtin_trap();
  std::memcpy(v, p, 16);
  zr_emu_lds_later(lds, v);
}
#define __builtin_amdgcn_cvt_pk_fp8_f32(lo, hi, old, high) zr_emu_cvt_pk_fp8((lo), (hi), (old), (high))
#define __builtin_amdgcn_cvt_pk_f32_fp8(codes, high) zr_emu_cvt_pk_f32((codes), (high))
#define __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, scale, high) zr_emu_cvt_scale((codes), (scale), (high))
#define __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, x, y, z) zr_emu_mfma(&(a), &(b), (c))
#define __builtin_amdgcn_ds_read_tr16_b64_v4i16(p) zr_emu_transpose(p)
#define __builtin_amdgcn_global_load_lds(...) zr_emu_load_lds(__VA_ARGS__)
#define __builtin_amdgcn_s_waitcnt(x) zr_emu_wait()
