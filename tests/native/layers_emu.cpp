// Bounds and value check of the layer operators' kernels, run on the CPU.
//
// Built together with the library's own sources (zr_embed.hip, zr_linear.hip
// compiled as C++ with tests/native/emu_waves on the include path, zr_plan.cpp)
// under AddressSanitizer + UndefinedBehaviorSanitizer.  Every buffer, workspaces
// among them, has exactly the size that the call asks for, with the end of its
// allocation behind it and poisoned bytes before it.  Values are small whole
// numbers (in the gaps between rows, in rows that must not be read and in what a
// call must write NaN), so that sums are exact in any order and outputs are
// compared for equality with plain loops in 64 bits.
//
// usage: layers_emu <cases> [first seed]; seeds below 0 are the large lists of
// weights

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

struct Ids {
  Buf b;
  bool wide;
  std::vector<int64_t> t;
  Ids(Rng& r, int64_t n, int64_t vocab, bool wide_) : b(size_t(n) * (wide_ ? 8 : 4), wide_ ? 8 : 4), wide(wide_), t(n) {
    const int kind = int(r.uni(0, 3));
    const int64_t common = r.uni(0, vocab - 1);
    for (int64_t i = 0; i < n; ++i) {
      t[i] = kind == 0 ? r.uni(0, vocab - 1) : kind == 1 ? r.uni(0, std::min<int64_t>(vocab - 1, 5))
             : kind == 2 && !r.one_in(3) ? common : r.uni(0, vocab - 1);
      if (r.one_in(8)) t[i] = r.pick<int64_t>({-1, -100, vocab, vocab + 7, INT32_MAX, INT32_MIN});
      if (wide && r.one_in(40)) t[i] = r.pick<int64_t>({INT64_MAX, INT64_MIN, int64_t(1) << 32, (int64_t(1) << 32) + 1});
      if (wide) b.as<int64_t>()[i] = t[i];
      else b.as<int32_t>()[i] = int32_t(t[i]);
    }
  }
  zr_index type() const { return wide ? ZR_I64 : ZR_I32; }
};

int64_t columns(Rng& r, int64_t most) {
  const int64_t near = r.pick<int64_t>({4, 8, 64, 256, 512, 1024, 2048, 4096, 8192}) + r.uni(-3, 3);
  return std::max<int64_t>(1, std::min(most, r.one_in(3) ? r.uni(1, 40) : near));
}

// ------------------------------------------------------------------- lookup

void lookup_case(Rng& r, int seed) {
  const int world = int(r.pick<int64_t>({1, 2, 3, 8, 64}));
  const int64_t dim = columns(r, 9000), vocab = r.uni(1, std::max<int64_t>(1, 60000 / dim)), lead = r.uni(0, 9);
  const int64_t n = r.uni(0, std::max<int64_t>(1, std::min<int64_t>(60, 60000 / dim)));
  const bool bf16 = r.one_in(2);
  Plan plan(lead ? std::vector<int64_t>{lead, vocab * dim, r.uni(1, 20)} : std::vector<int64_t>{vocab * dim, 7}, world);
  const int64_t param = lead ? 1 : 0, o = plan.offset(param);
  std::vector<std::unique_ptr<Rows>> parts;
  std::vector<const void*> ptrs;
  for (int k = 0; k < world; ++k) {
    parts.emplace_back(new Rows(1, plan.part, plan.part, bf16, r.uni(0, 3)));
    for (int64_t i = 0; i < plan.part; ++i) parts.back()->put(i, float(r.uni(-100, 100)));
    const bool holds = (k + 1) * plan.part > o && k * plan.part < o + vocab * dim;
    ptrs.push_back(holds ? parts.back()->b.p : nullptr);
  }
  Ids ids(r, n, vocab, r.one_in(2));
  const float scale = r.pick({1.0f, 0.5f, -2.0f, float(INFINITY)});
  Rows out(n, dim, dim + r.pick<int64_t>({0, 0, 1, 8}), bf16, r.uni(0, 7));
  const int64_t row = out.stride;
  CHECK(zr_embedding_lookup(plan.h, param, dim, ptrs.data(), out.type(), n ? ids.b.p : nullptr, ids.type(), n,
                            scale, out.b.p, row, nullptr) == ZR_OK, "seed %d", seed);
  for (int64_t i = 0; i < n; ++i)
    for (int64_t c = 0; c < row && i * row + c < (n - 1) * row + dim; ++c) {
      const float got = out.at(i * row + c);
      if (c >= dim) {
        CHECK(std::isnan(got), "seed %d: wrote between rows", seed);
      } else if (ids.t[i] < 0 || ids.t[i] >= vocab) {
        CHECK(got == 0 && !std::signbit(got), "seed %d: row %ld column %ld %g", seed, long(i), long(c), got);
      } else {
        const int64_t f = o + ids.t[i] * dim + c;
        const float want = parts[f / plan.part]->at(f % plan.part) * scale;
        CHECK(got == want || (std::isnan(got) && std::isnan(want)), "seed %d: row %ld column %ld %g for %g", seed,
              long(i), long(c), got, want);
      }
    }
}

// -------------------------------------------------------- embedding gradient

void embedding_case(Rng& r, int seed) {
  const int world = int(r.pick<int64_t>({1, 1, 2, 3, 8}));
  const bool many_rows = r.one_in(4);
  const int64_t dim = many_rows ? r.uni(1, 9) : columns(r, 9000);
  const int64_t vocab = many_rows ? r.pick<int64_t>({255, 256, 257, 511, 513, 1500, 5000}) + r.uni(0, 3)
                                  : r.uni(1, std::max<int64_t>(1, 40000 / dim));
  const int64_t n = std::min<int64_t>(
      200000 / dim + 1, (dim < 10 && r.one_in(4) ? 20000 : r.pick<int64_t>({0, 1, 7, 64, 65, 200, 700, 2100, 9000})) + r.uni(0, 3));
  const bool bf16 = r.one_in(2), first = r.one_in(2);
  const int64_t lead = r.uni(0, 9);
  Plan plan(lead ? std::vector<int64_t>{lead, vocab * dim, r.uni(1, 20)} : std::vector<int64_t>{vocab * dim, 7}, world);
  const int64_t param = lead ? 1 : 0, o = plan.offset(param);
  int64_t base, length;
  window(r, plan, world, &base, &length);
  Ids ids(r, n, vocab, r.one_in(2));
  Rows dy(n, dim, dim + r.pick<int64_t>({0, 0, 1, 8}), bf16, r.uni(0, 7));
  const float scale = r.pick({1.0f, 0.5f, -2.0f});
  Rows grad(1, length, length, false, r.uni(0, 3));
  std::vector<double> want(length);
  for (int64_t i = 0; i < length; ++i) {
    want[i] = double(r.uni(-100, 100));
    const bool in_table = base + i >= o && base + i < o + vocab * dim;
    grad.put(i, first && in_table ? kNaN : float(want[i]));
    if (first && in_table) want[i] = 0;
  }
  for (int64_t i = 0; i < n; ++i) {
    const int64_t t = ids.t[i];
    if (t < 0 || t >= vocab || o + (t + 1) * dim <= base || o + t * dim >= base + length) continue;   // NaN, not read
    for (int64_t c = 0; c < dim; ++c) {
      const float x = float(r.uni(-8, 8));
      dy.put(i * dy.stride + c, x);
      const int64_t f = o + t * dim + c - base;
      if (f >= 0 && f < length) want[f] += double(scale) * x;
    }
  }
  int64_t bytes = -1;
  CHECK(zr_ipg_embedding_workspace(plan.h, param, dim, n, base, length, &bytes) == ZR_OK, "seed %d", seed);
  Buf ws(size_t(bytes), 0);
  CHECK((first ? zr_ipg_accumulate_embedding_first : zr_ipg_accumulate_embedding)(
            plan.h, param, dim, n ? ids.b.p : nullptr, ids.type(), n, scale, n ? dy.b.p : nullptr, dy.type(),
            dy.stride, grad.b.as<float>(), base, length, ws.p, bytes, nullptr) == ZR_OK, "seed %d", seed);
  for (int64_t i = 0; i < length; ++i)
    CHECK(double(grad.at(i)) == want[i], "seed %d: element %ld of %ld+%ld: %g for %g", seed, long(i), long(base),
          long(length), grad.at(i), want[i]);
}

// -------------------------------------------------------------- checkpoints

// The code of a whole number of at most 8 bits' worth that e4m3 holds.
uint8_t code_of(float x) {
  for (int c = 0; c < 256; ++c)
    if (zr_emu_e4m3_value(uint8_t(c)) == x && std::signbit(x) == (c >= 128)) return uint8_t(c);
  CHECK(false, "%g is no code", x);
}

void checkpoint_case(Rng& r, int seed) {
  const int64_t cols = columns(r, 5000), rows = r.uni(0, std::max<int64_t>(1, std::min<int64_t>(700, 30000 / cols)));
  const int64_t blocks = (cols + 31) / 32;
  const bool bf16 = r.one_in(2);
  Rows x(rows, cols, cols + r.pick<int64_t>({0, 0, 1, 8}), bf16, r.uni(0, 7));
  Buf codes(size_t(rows * blocks * 32), 0, 0x55), scales(size_t(rows * blocks), size_t(r.uni(0, 15)));
  // eighths of a scale in each block, whose largest is 256 of them or 448
  std::vector<int> e(rows * blocks);
  std::vector<float> v(rows * blocks * 32, 0.0f);
  for (int64_t i = 0; i < rows; ++i)
    for (int64_t b = 0; b < blocks; ++b) {
      const int s = int(e[i * blocks + b] = int(r.uni(-20, 20)));
      for (int64_t c = 32 * b; c < std::min(cols, 32 * b + 32); ++c) {
        const float m = c == 32 * b ? r.pick({256.0f, -448.0f}) : float(r.uni(-15, 15));
        v[i * blocks * 32 + c] = c > 32 * b && r.one_in(50) ? r.pick({kNaN, float(INFINITY)}) : m;
        x.put(i * x.stride + c, std::ldexp(v[i * blocks * 32 + c], s));
      }
    }
  CHECK(zr_act_quantize(x.b.p, x.type(), rows, cols, x.stride, codes.p, scales.p, nullptr) == ZR_OK, "seed %d", seed);
  for (int64_t i = 0; i < rows * blocks; ++i)
    CHECK(scales.p[i] == e[i] + 127, "seed %d: scale %d for %d", seed, scales.p[i], e[i] + 127);
  for (size_t i = 0; i < v.size(); ++i) {
    const float got = zr_emu_e4m3_value(codes.p[i]);
    CHECK(std::isfinite(v[i]) ? got == v[i] : std::isnan(got), "seed %d: code %g for %g", seed, got, v[i]);
  }
  Rows back(rows, cols, cols + r.pick<int64_t>({0, 0, 1, 8}), r.one_in(2), r.uni(0, 7));
  CHECK(zr_act_dequantize(codes.p, scales.p, rows, cols, back.b.p, back.type(), back.stride, nullptr) == ZR_OK,
        "seed %d", seed);
  for (int64_t i = 0; i < rows; ++i)
    for (int64_t c = 0; c < back.stride && i * back.stride + c < (rows - 1) * back.stride + cols; ++c) {
      const float got = back.at(i * back.stride + c);
      if (c >= cols || !std::isfinite(v[i * blocks * 32 + c]))
        CHECK(std::isnan(got), "seed %d: %g for NaN", seed, got);
      else
        CHECK(got == std::ldexp(v[i * blocks * 32 + c], e[i * blocks + c / 32]), "seed %d: value", seed);
    }
}

// --------------------------------------------------------- weight gradients

struct Layer {
  int64_t out, in, tokens;
  bool in_major;
  std::unique_ptr<Rows> dy;
  std::unique_ptr<Buf> codes, scales;
  std::vector<double> grad;
};

void linear_call(Rng& r, int seed, std::vector<Layer>& layers, int world, bool whole = false) {
  std::vector<int64_t> numels{r.uni(1, 9)};
  std::vector<zr_linear_grad> items;
  uint8_t code[17];
  for (int i = -8; i <= 8; ++i) code[i + 8] = code_of(float(i));
  for (Layer& l : layers) {
    const int64_t blocks = (l.in + 31) / 32;
    // rows of dY on 16 bytes, off them, or apart by a multiple of them
    const int64_t stride = r.one_in(2) ? (l.out + 7) / 8 * 8 : l.out + r.pick<int64_t>({0, 1, 3});
    l.dy.reset(new Rows(l.tokens, l.out, stride, true, r.one_in(2) ? 0 : r.uni(1, 7)));
    l.codes.reset(new Buf(size_t(l.tokens * blocks * 32), 0, 0x7f));   // NaN behind the last column
    l.scales.reset(new Buf(size_t(l.tokens * blocks), size_t(r.uni(0, 15)), 0xA5));
    l.grad.assign(size_t(l.out * l.in), 0.0);
    std::vector<double> x(l.in);
    for (int64_t t = 0; t < l.tokens; ++t) {
      for (int64_t b = 0; b < blocks; ++b) l.scales->p[t * blocks + b] = uint8_t(126 + r.uni(0, 2));
      for (int64_t i = 0; i < l.in; ++i) {
        const int v = int(r.uni(-8, 8));
        l.codes->p[t * blocks * 32 + i] = code[v + 8];
        x[i] = std::ldexp(double(v), l.scales->p[t * blocks + i / 32] - 127);
      }
      for (int64_t o = 0; o < l.out; ++o) {
        const float d = float(r.uni(-4, 4));
        l.dy->put(t * stride + o, d);
        double* g = &l.grad[l.in_major ? o : o * l.in];
        const int64_t step = l.in_major ? l.out : 1;
        for (int64_t i = 0; i < l.in; ++i) g[i * step] += double(d) * x[i];
      }
    }
    items.push_back(zr_linear_grad{int64_t(numels.size()), l.out, l.in, l.tokens,
                                   l.tokens ? l.dy->b.as<uint16_t>() : nullptr, stride,
                                   l.tokens ? l.codes->p : nullptr, l.tokens ? l.scales->p : nullptr, l.in_major});
    numels.push_back(l.out * l.in);
  }
  Plan plan(numels, world);
  int64_t base, length;
  window(r, plan, world, &base, &length);
  if (whole) base = 0, length = plan.padded;
  const bool first = r.one_in(2);
  Rows grad(1, length, length, false, r.uni(0, 3));
  std::vector<double> want(length);
  for (int64_t i = 0; i < length; ++i) {
    want[i] = double(r.uni(-100, 100));
    grad.put(i, float(want[i]));
  }
  for (size_t k = 0; k < layers.size(); ++k) {
    const int64_t o = plan.offset(int64_t(k) + 1) - base;
    for (int64_t e = 0; e < layers[k].out * layers[k].in; ++e)
      if (o + e >= 0 && o + e < length) {
        if (first) grad.put(o + e, kNaN), want[o + e] = 0;
        want[o + e] += layers[k].grad[e];
      }
  }
  int64_t bytes = -1;
  CHECK(zr_ipg_linear_workspace(plan.h, items.data(), int64_t(items.size()), base, length, &bytes) == ZR_OK,
        "seed %d", seed);
  Buf ws(size_t(bytes), 0);
  CHECK((first ? zr_ipg_accumulate_linear_first : zr_ipg_accumulate_linear)(
            plan.h, items.data(), int64_t(items.size()), grad.b.as<float>(), base, length, bytes ? ws.p : nullptr,
            bytes, nullptr) == ZR_OK, "seed %d", seed);
  for (int64_t i = 0; i < length; ++i)
    CHECK(double(grad.at(i)) == want[i], "seed %d: element %ld of %ld+%ld: %g for %g", seed, long(i), long(base),
          long(length), grad.at(i), want[i]);
}

void linear_case(Rng& r, int seed) {
  std::vector<Layer> layers(size_t(r.pick<int64_t>({1, 1, 2, 3, 20})));
  const bool small = layers.size() > 3;
  for (Layer& l : layers) {
    auto side = [&] { return small || r.one_in(2) ? r.uni(1, 40) : r.pick<int64_t>({32, 64, 256, 512}) + r.uni(-3, 9); };
    l.out = side();
    l.in = side();
    l.tokens = r.one_in(6) ? 0 : small ? r.uni(1, 70) : r.pick<int64_t>({1, 16, 64, 128, 300, 700}) + r.uni(0, 3);
    if (l.out * l.in > 300 * 300) l.tokens = std::min<int64_t>(l.tokens, 200);
    l.in_major = r.one_in(2);
  }
  linear_call(r, seed, layers, int(r.pick<int64_t>({1, 1, 2, 3})));
}

// 260 tiles, four more than CUs: the last four, of the layer with the fewest
// tokens, are cut along them, and its other 23 are not; more than eight tiles of
// dY's columns lie beside several of X's.  (The other layers have many tiles of
// few weights.)
void rounds_case(Rng& r, int seed, bool in_major) {
  std::vector<Layer> layers(4);
  auto layer = [&](int64_t out, int64_t in, int64_t tokens) {
    return Layer{out, in, tokens, in_major, {}, {}, {}, {}};
  };
  layers[0] = layer(256 * 64 + r.uni(1, 256), 5, 390);
  layers[1] = layer(256 * 8 + r.uni(1, 256), 512 + r.uni(1, 256), 321 + r.uni(0, 60));
  layers[2] = layer(3, 256 * 64 + r.uni(1, 256), 385);
  layers[3] = layer(9, 256 * 102 + r.uni(1, 256), 385);
  linear_call(r, seed, layers, 1, true);
}

}  // namespace

int main(int argc, char** argv) {
  const int cases = argc > 1 ? std::atoi(argv[1]) : 40;
  const int first = argc > 2 ? std::atoi(argv[2]) : 0;
  for (int c = first; c < first + cases; ++c) {
    Rng r(static_cast<uint64_t>(c));
    zr_emu_waves_backwards = r.one_in(2);
    if (c < 0) {
      rounds_case(r, c, c % 2);
      continue;
    }
    switch (c % 4) {
      case 0: lookup_case(r, c); break;
      case 1: embedding_case(r, c); break;
      case 2: checkpoint_case(r, c); break;
      case 3: linear_case(r, c); break;
    }
  }
  std::printf("layer emulation ok: %d cases, %lld workgroups\n", cases, zr_emu_workgroups);
  for (const auto& kv : zr_emu_coverage()) std::printf("launches %lld %s\n", kv.second, kv.first.c_str());
  return 0;
}
