// Bounds and value check of the grouped products' kernels, run on the CPU.
//
// Built together with zr_product.hip (as C++, with tests/native/emu_waves on the
// include path) under AddressSanitizer + UndefinedBehaviorSanitizer.  Values are
// small whole numbers (NaN in the gaps between rows, in partitions' other
// elements and in what a call must write), so that sums are exact in any order
// and outputs are compared for equality with plain loops.
//
// usage: products_emu <cases> [first seed]

#include "emu_cases.h"

namespace {

void product_case(Rng& r, int seed) {
  const bool input = r.one_in(2), in_major = r.one_in(2), small = r.one_in(2), even = r.one_in(2);
  const int world = int(r.pick<int64_t>({1, 1, 2, 3, 8, 64}));
  auto side = [&] {
    const int64_t s = r.one_in(3) ? r.uni(1, 40) : r.pick<int64_t>({64, 128, 192, 256, 320, 400}) + r.uni(-3, 9);
    return even ? (s + 7) / 8 * 8 : s;
  };
  int64_t n_out = side(), n_in = side();
  if (r.one_in(3)) {   // sums in pieces
    (input ? n_out : n_in) = r.uni(520, 900) / 8 * 8 + (even ? 0 : r.uni(0, 7));
    (input ? n_in : n_out) = r.uni(1, 20) * (even ? 8 : 1);
  }
  // sizes whose tiles are large, and whose sums are in pieces too
  const bool wide = !small && r.one_in(3);
  if (wide) {
    const bool pieces = r.one_in(2);
    (input ? n_out : n_in) = r.uni(pieces ? 225 : 17, pieces ? 240 : 22) * 8 + (even ? 0 : r.uni(1, 7));
    (input ? n_in : n_out) = r.uni(17, 20) * 8 + (even ? 0 : r.uni(1, 7));
  }
  const bool deep = !wide && r.one_in(6);   // pieces of few tiles
  if (deep) {
    (input ? n_out : n_in) = r.uni(300, 310) * 8 + (even ? 0 : r.uni(1, 7));
    (input ? n_in : n_out) = r.uni(1, 5) * 8 + (even ? 0 : r.uni(1, 7));
  }
  if (even && r.one_in(4)) (input ? n_out : n_in) -= r.uni(1, 7);   // a last unit of k that is not whole
  const int64_t experts = wide || deep ? 1 : r.pick<int64_t>({1, 1, 2, 3, 5, 140});
  const int64_t depth = input ? n_out : n_in, cols = input ? n_in : n_out;
  const int64_t lead = even ? 8 * r.uni(0, 2) : r.uni(0, 9);
  std::vector<int64_t> numels, params, counts;
  if (lead) numels.push_back(lead);
  const int64_t weights = experts > 5 ? 2 : experts;
  for (int64_t k = 0; k < weights; ++k) numels.push_back(n_out * n_in);
  int64_t total = 0;
  for (int64_t n : numels) total += n;
  // partitions of whole eights
  numels.push_back(even ? 8 * world - total % (8 * world) : r.uni(1, 20));
  Plan plan(numels, world);
  int64_t rows = 0;
  for (int64_t k = 0; k < experts; ++k) {
    params.push_back((lead ? 1 : 0) + (experts > 5 ? r.uni(0, 1) : k));
    int64_t c = r.one_in(4) ? 0 : small || experts > 5 ? r.uni(1, experts > 5 ? 3 : 64) : r.pick<int64_t>({1, 65, 128, 200, 257, 300});
    if (wide) c = depth > 1000 ? r.uni(130, 160) : r.uni(400, 500);
    else if (deep) c = r.pick<int64_t>({1, 30, 40, 64, 66, 80});
    else if (depth * cols > 200 * 200) c = std::min<int64_t>(c, 130);
    counts.push_back(c);
    rows += c;
  }
  if (!small && rows && experts <= 5 && r.one_in(2)) {
    rows += 65 - std::min<int64_t>(counts[0], 65);
    counts[0] = std::max<int64_t>(counts[0], 65);
  }
  const int64_t used = rows;
  rows += r.pick<int64_t>({0, 0, 3});
  std::vector<std::unique_ptr<Rows>> parts;
  std::vector<const void*> ptrs;
  for (int k = 0; k < world; ++k) {
    parts.emplace_back(new Rows(1, plan.part, plan.part, true, even ? 0 : r.uni(0, 3)));
    bool holds = false;
    for (int64_t e = 0; e < experts; ++e) {
      const int64_t o = plan.offset(params[size_t(e)]);
      if (!counts[size_t(e)] || o >= (k + 1) * plan.part || o + n_out * n_in <= k * plan.part) continue;
      holds = true;
      for (int64_t f = std::max(o, k * plan.part); f < std::min(o + n_out * n_in, (k + 1) * plan.part); ++f)
        parts.back()->put(f - k * plan.part, float(int(uint64_t(f) * 2654435761u >> 7) % 5 - 2));
    }
    ptrs.push_back(holds ? parts.back()->b.p : nullptr);
  }
  auto weight = [&](int64_t e, int64_t o, int64_t i) {
    const int64_t f = plan.offset(params[size_t(e)]) + (in_major ? i * n_out + o : o * n_in + i);
    return parts[size_t(f / plan.part)]->at(f % plan.part);
  };
  Rows x(rows, depth, even ? (depth + 7) / 8 * 8 + r.pick<int64_t>({0, 8}) : depth + r.pick<int64_t>({0, 1, 5}), true,
         even ? 0 : r.uni(0, 7));
  for (int64_t t = 0; t < used; ++t)
    for (int64_t k = 0; k < depth; ++k) x.put(t * x.stride + k, float(r.uni(-2, 2)));
  Rows y(rows, cols, cols + r.pick<int64_t>({0, 0, 1, 8}), r.one_in(2), r.uni(0, 7));
  int64_t bytes = 0;
  CHECK((input ? zr_linear_input_grad_workspace : zr_linear_forward_workspace)(
            plan.h, params.data(), counts.data(), experts, n_out, n_in, in_major, &bytes) == ZR_OK, "seed %d", seed);
  Buf ws(size_t(bytes), 0);
  CHECK((input ? zr_linear_input_grad : zr_linear_forward)(
            plan.h, params.data(), counts.data(), experts, n_out, n_in, in_major, ptrs.data(), x.b.as<uint16_t>(),
            rows, x.stride, y.b.p, y.type(), y.stride, bytes ? ws.p : nullptr, bytes, nullptr) == ZR_OK, "seed %d",
        seed);
  std::vector<float> w(size_t(depth * cols));
  int64_t t = 0;
  for (int64_t e = 0; e <= experts; ++e) {
    const int64_t end = e < experts ? t + counts[size_t(e)] : rows;
    if (e < experts && end > t)
      for (int64_t n = 0; n < cols; ++n)
        for (int64_t k = 0; k < depth; ++k) w[size_t(n * depth + k)] = input ? weight(e, k, n) : weight(e, n, k);
    for (; t < end; ++t) {
      for (int64_t n = 0; n < y.stride && t * y.stride + n < (rows - 1) * y.stride + cols; ++n) {
        const float got = y.at(t * y.stride + n);
        if (n >= cols || e == experts) {
          CHECK(std::isnan(got), "seed %d: wrote where it must not", seed);
          continue;
        }
        float want = 0;
        for (int64_t k = 0; k < depth; ++k) want += x.at(t * x.stride + k) * w[size_t(n * depth + k)];
        if (y.bf16) {   // to nearest even: whole numbers past 256 round
          uint32_t b;
          std::memcpy(&b, &want, 4);
          b = (b + 0x7fff + (b >> 16 & 1)) & 0xffff0000u;
          std::memcpy(&want, &b, 4);
        }
        CHECK(got == want, "seed %d: row %ld column %ld (%ld x %ld, input %d, in_major %d): %g for %g", seed, long(t),
              long(n), long(n_out), long(n_in), input, in_major, got, want);
      }
    }
  }
}

}  // namespace

int main(int argc, char** argv) {
  const int cases = argc > 1 ? std::atoi(argv[1]) : 40;
  const int first = argc > 2 ? std::atoi(argv[2]) : 0;
  for (int c = first; c < first + cases; ++c) {
    Rng r(static_cast<uint64_t>(c));
    zr_emu_waves_backwards = r.one_in(2);
    product_case(r, c);
  }
  std::printf("product emulation ok: %d cases, %lld workgroups\n", cases, zr_emu_workgroups);
  for (const auto& kv : zr_emu_coverage()) std::printf("launches %lld %s\n", kv.second, kv.first.c_str());
  return 0;
}
