// Buffers, plans and random numbers of the drivers that run kernels on the CPU
// under AddressSanitizer + UndefinedBehaviorSanitizer.  Every buffer has exactly
// the size that the call asks for, with the end of its allocation behind it and
// poisoned bytes before it.
#pragma once

#include <sanitizer/asan_interface.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <memory>
#include <string>
#include <vector>

#include "zr.h"

extern bool zr_emu_waves_backwards;
extern long long zr_emu_workgroups;
std::map<std::string, long long>& zr_emu_coverage();
float zr_emu_e4m3_value(uint8_t code);

namespace {

#define CHECK(cond, ...)                                        \
  do {                                                          \
    if (!(cond)) {                                              \
      std::fprintf(stderr, "FAIL %s:%d: ", __FILE__, __LINE__); \
      std::fprintf(stderr, __VA_ARGS__);                        \
      std::fprintf(stderr, " (%s)\n", zr_last_error());         \
      std::abort();                                             \
    }                                                           \
  } while (0)

struct Rng {
  uint64_t s;
  explicit Rng(uint64_t seed) : s(seed * 0x9E3779B97F4A7C15ull + 1) {}
  uint64_t next() {
    uint64_t z = (s += 0x9E3779B97F4A7C15ull);
    z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
    z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
    return z ^ (z >> 31);
  }
  int64_t uni(int64_t lo, int64_t hi) { return lo + static_cast<int64_t>(next() % uint64_t(hi - lo + 1)); }
  bool one_in(int n) { return uni(1, n) == 1; }
  template <typename T>
  T pick(std::initializer_list<T> v) { return v.begin()[next() % v.size()]; }
};

const float kNaN = std::nanf("");
uint16_t bf16_of(float x) {   // values that bf16 holds
  uint32_t b;
  std::memcpy(&b, &x, 4);
  return static_cast<uint16_t>(b >> 16);
}
float bf16_value(uint16_t h) {
  const uint32_t b = static_cast<uint32_t>(h) << 16;
  float x;
  std::memcpy(&x, &b, 4);
  return x;
}

// `bytes` bytes, `off` behind a 16-byte boundary, that end where their
// allocation ends.
struct Buf {
  static constexpr size_t kGuard = 64;
  unsigned char* block;
  unsigned char* p;
  size_t pre, bytes;
  Buf(size_t bytes_, size_t off, int fill = 0xA5) : pre(kGuard + off), bytes(bytes_) {
    block = static_cast<unsigned char*>(std::malloc(pre + bytes));
    p = block + pre;
    std::memset(block, fill, pre + bytes);
    __asan_poison_memory_region(block, pre & ~size_t(7));
  }
  ~Buf() {
    __asan_unpoison_memory_region(block, pre);
    for (size_t i = pre & ~size_t(7); i < pre; ++i) CHECK(block[i] == 0xA5, "store before a buffer");
    std::free(block);
  }
  Buf(const Buf&) = delete;
  template <typename T>
  T* as() { return reinterpret_cast<T*>(p); }
};

// A matrix of bf16 or fp32 rows of `cols` elements, `stride` apart, that ends
// behind the last row's last element.
struct Rows {
  int64_t n, cols, stride;
  bool bf16;
  Buf b;
  Rows(int64_t n_, int64_t cols_, int64_t stride_, bool bf16_, int64_t off)
      : n(n_), cols(cols_), stride(stride_), bf16(bf16_),
        b(size_t(n ? (n - 1) * stride + cols : 0) * (bf16 ? 2 : 4), size_t(off) * (bf16 ? 2 : 4)) {
    for (int64_t i = 0; n && i < (n - 1) * stride + cols; ++i) put(i, kNaN);
  }
  void put(int64_t i, float x) {
    if (bf16) b.as<uint16_t>()[i] = bf16_of(x);
    else b.as<float>()[i] = x;
  }
  float at(int64_t i) { return bf16 ? bf16_value(b.as<uint16_t>()[i]) : b.as<float>()[i]; }
  zr_dtype type() const { return bf16 ? ZR_BF16 : ZR_FP32; }
};

struct Plan {
  zr_plan* h = nullptr;
  int64_t total = 0, padded = 0, part = 0;
  Plan(std::vector<int64_t> numels, int world) {
    std::vector<zr_param> ps;
    for (int64_t n : numels) ps.push_back(zr_param{n, 0});
    const zr_group g{world, 1};
    CHECK(zr_plan_buckets(ps.data(), int64_t(ps.size()), &g, 1, int64_t(1) << 40, 0, 1, &h) == ZR_OK, "plan");
    zr_plan_group_info(h, 0, &total, &padded, &part, nullptr);
  }
  ~Plan() { zr_plan_free(h); }
  int64_t offset(int64_t p) {
    int64_t o = 0;
    zr_plan_param_offset(h, p, &o);
    return o;
  }
};

// A window: a rank's partition, the whole space, or any piece of it.
void window(Rng& r, const Plan& plan, int world, int64_t* base, int64_t* length) {
  switch (r.uni(0, 2)) {
    case 0: *base = r.uni(0, world - 1) * plan.part, *length = plan.part; break;
    case 1: *base = 0, *length = plan.padded; break;
    default: *base = r.uni(0, plan.padded - 1), *length = r.uni(0, plan.padded - *base);
  }
}

}  // namespace
