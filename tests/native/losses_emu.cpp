// Bounds and value check of the losses' kernels, run on the CPU.
//
// Built together with zr_loss.hip (as C++, with tests/native/emu_waves on the
// include path) under AddressSanitizer + UndefinedBehaviorSanitizer, and compared
// with the formulas in 64 bits.
//
// usage: losses_emu <cases> [first seed]; seeds below 0 are rows that are longer
// than a workgroup's registers

#include "emu_cases.h"

namespace {

const double kInf = INFINITY;

// z - its row's gaps, with masked places.
void fill_logits(Rng& r, Rows& z, int64_t row, int64_t vocab) {
  const int kind = int(r.uni(0, 9));
  for (int64_t v = 0; v < vocab; ++v) {
    float x = float(r.uni(-64, 64)) / 8;
    if (kind == 0 && !r.one_in(10)) x = -INFINITY;
    if (kind == 1 && !r.one_in(10)) x = -3.3895314e38f;
    if (kind == 2) x = -INFINITY;
    if (kind == 3) x = -3.3895314e38f;
    if (kind == 4) x += 1024;
    z.put(row * z.stride + v, x);
  }
}

void loss_case(Rng& r, int seed, int64_t rows, int64_t vocab, bool bf16, double masked) {
  const bool distill = r.one_in(2), wide = r.one_in(2), in_place = r.one_in(4), grad = in_place || !r.one_in(5);
  const int64_t top = distill ? r.pick<int64_t>({1, 2, 7, 33, 64, 65, 200, 1024}) : 1;
  const double tau = r.pick({1.0, 0.5, 2.0});
  Rows z(rows, vocab, vocab + r.pick<int64_t>({0, 0, 1, 8}), bf16, r.uni(0, 7));
  std::vector<double> was(size_t(rows * vocab));
  for (int64_t i = 0; i < rows; ++i) {
    fill_logits(r, z, i, vocab);
    for (int64_t v = 0; v < vocab; ++v) was[size_t(i * vocab + v)] = z.at(i * z.stride + v);
  }
  Rows g(in_place ? 0 : rows, vocab, vocab + r.pick<int64_t>({0, 0, 1, 8}), bf16, r.uni(0, 7));
  Rows& out = in_place ? z : g;
  const int64_t is = distill ? top + r.uni(0, 2) : 1, ts = top + r.uni(0, 2);
  Buf ids(size_t(rows ? (rows - 1) * is + top : 0) * (wide ? 8 : 4), wide ? 8 : 4);
  std::vector<int64_t> id(size_t(rows * top));
  const bool teacher_bf16 = r.one_in(2);
  Rows t(rows, top, ts, teacher_bf16, r.uni(0, 3));
  Rows per(6, std::max<int64_t>(rows, 1), std::max<int64_t>(rows, 1), false, 1);   // weight, old, ref, advantage, loss, logp
  const int64_t ps = per.stride;
  for (int64_t i = 0; i < rows; ++i) {
    const bool none = r.uni(0, 99) < masked * 100;
    const int64_t common = r.uni(0, vocab - 1);
    for (int64_t j = 0; j < top; ++j) {
      int64_t k = r.one_in(4) ? common : r.uni(0, vocab - 1);
      if (none || (distill && r.one_in(6))) k = r.pick<int64_t>({-1, -100, vocab, INT32_MAX, INT32_MIN});
      if (none && wide && r.one_in(3)) k = r.pick<int64_t>({INT64_MAX, INT64_MIN, int64_t(1) << 32});
      id[size_t(i * top + j)] = k;
      if (wide) ids.as<int64_t>()[i * is + j] = k;
      else ids.as<int32_t>()[i * is + j] = int32_t(k);
      t.put(i * ts + j, r.one_in(12) ? -INFINITY : float(r.uni(-40, 40)) / 8);
    }
    per.put(i, r.one_in(8) ? 0.0f : float(r.uni(1, 16)) / 16);
    per.put(ps + i, -float(r.uni(0, 40)) / 8);
    per.put(2 * ps + i, -float(r.uni(0, 40)) / 8);
    per.put(3 * ps + i, r.one_in(10) ? 0.0f : float(r.uni(-16, 16)) / 8);
  }
  const bool weighted = !r.one_in(4), kl = r.one_in(2);
  const double beta = kl ? 0.25 : 0.0, lo = 0.2, hi = 0.28;
  int64_t bytes = 0;
  CHECK(zr_loss_workspace(rows, vocab, top, z.type(), &bytes) == ZR_OK, "seed %d", seed);
  Buf ws(size_t(bytes), 0);
  float* p = per.b.as<float>();
  void* gp = grad ? (rows ? static_cast<void*>(out.b.p) : static_cast<void*>(z.b.p)) : nullptr;
  const zr_status st =
      distill ? zr_distill_loss(z.b.p, z.type(), rows, vocab, z.stride, ids.p, wide ? ZR_I64 : ZR_I32, is, t.b.p,
                                t.type(), ts, top, weighted ? p : nullptr, tau, p + 4 * ps, gp, out.stride,
                                bytes ? ws.p : nullptr, bytes, nullptr)
              : zr_policy_loss(z.b.p, z.type(), rows, vocab, z.stride, ids.p, wide ? ZR_I64 : ZR_I32, p + ps,
                               kl ? p + 2 * ps : nullptr, p + 3 * ps, weighted ? p : nullptr, lo, hi, beta, tau,
                               p + 4 * ps, p + 5 * ps, gp, out.stride, bytes ? ws.p : nullptr, bytes, nullptr);
  CHECK(st == ZR_OK, "seed %d", seed);
  for (int64_t i = 0; i < rows; ++i) {
    const double* x = &was[size_t(i * vocab)];
    double m = -kInf, s = 0;
    for (int64_t v = 0; v < vocab; ++v) m = std::max(m, x[v]);
    for (int64_t v = 0; v < vocab && m > -kInf; ++v) s += std::exp((x[v] - m) / tau);
    auto logq = [&](int64_t v) { return (x[v] - m) / tau - std::log(s); };
    const double w = weighted ? per.at(i) : 1.0;
    std::vector<double> target(size_t(vocab), 0.0);
    double want = 0, lp = 0, coef = 0, size = 0;
    if (distill) {
      double tm = -kInf, tsum = 0;
      auto there = [&](int64_t j) {
        const int64_t k = id[size_t(i * top + j)];
        return k >= 0 && k < vocab && t.at(i * ts + j) > -INFINITY;
      };
      for (int64_t j = 0; j < top; ++j)
        if (there(j)) tm = std::max(tm, double(t.at(i * ts + j)));
      if (tm > -kInf && m > -kInf && w != 0) {
        for (int64_t j = 0; j < top; ++j)
          if (there(j)) tsum += std::exp((t.at(i * ts + j) - tm) / tau);
        for (int64_t j = 0; j < top; ++j) {
          if (!there(j)) continue;
          const int64_t k = id[size_t(i * top + j)];
          const double l = (t.at(i * ts + j) - tm) / tau - std::log(tsum), q = std::exp(l);
          target[size_t(k)] += q;
          if (q > 0) want += q * (l - logq(k));
          if (q > 0 && logq(k) > -kInf) size += q * (std::fabs(l) + std::fabs(logq(k)));
        }
        want *= w * tau * tau;
        size *= w * tau * tau;
        coef = w * tau;
      }
    } else {
      const int64_t k = id[size_t(i)];
      if (k >= 0 && k < vocab && m > -kInf) {
        lp = logq(k);
        const double ratio = std::exp(lp - per.at(ps + i)), adv = per.at(3 * ps + i);
        const double held = std::min(std::max(ratio, 1 - lo), 1 + hi);
        want = -std::min(ratio * adv, held * adv);
        double slope = ratio * adv <= held * adv ? -ratio * adv : 0;
        size = std::fabs(want) * (1 + std::fabs(lp));
        if (kl) {
          const double d = per.at(2 * ps + i) - lp;
          want += beta * (d == kInf ? kInf : std::exp(d) - d - 1);
          slope += beta * (1 - std::exp(d));
          size += beta * std::exp(d) * (2 + std::fabs(d));
        }
        want = w == 0 ? 0 : want * w;
        coef = w == 0 ? 0 : -slope * w / tau;
        target[size_t(k)] = 1;
      }
      const double got = per.at(5 * ps + i);
      if (std::fabs(lp) > 3e38) lp = -kInf;   // past fp32
      CHECK(got == lp || std::fabs(got - lp) <= 2e-6 * (1 + std::fabs(lp)), "seed %d row %ld: logp %.9g for %.9g", seed,
            long(i), got, lp);
    }
    const double got = per.at(4 * ps + i);
    if (std::fabs(want) > 3e38) want = std::copysign(kInf, want);   // past fp32
    if (std::fabs(coef) > 3e38) continue;
    CHECK(got == want || std::fabs(got - want) <= 4e-6 * (size + std::fabs(want)), "seed %d row %ld: loss %g for %g",
          seed, long(i), got, want);
    for (int64_t v = 0; grad && v < out.stride && i * out.stride + v < (rows - 1) * out.stride + vocab; ++v) {
      const double gv = out.at(i * out.stride + v);
      if (v >= vocab) {
        CHECK(std::isnan(gv), "seed %d: wrote between rows", seed);
        continue;
      }
      const double q = coef == 0 ? 0 : std::exp(logq(v));
      const double wv = coef == 0 ? 0 : coef * (q - target[size_t(v)]);
      const double tol = std::fabs(coef) * 1e-5 * (q + target[size_t(v)]) + (bf16 ? std::fabs(wv) / 256 : 0) + 1e-30;
      CHECK(gv == wv || std::fabs(gv - wv) <= tol, "seed %d row %ld column %ld of %ld: %g for %g", seed, long(i),
            long(v), long(vocab), gv, wv);
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
    const bool bf16 = r.one_in(2);
    if (c < 0) {
      // rows of one workgroup of each size, the largest longer than its registers,
      // and on a small chip several of them to one
      const int64_t lanes[] = {256, 512, 1024};
      const int64_t vocab = lanes[-c % 3] * 16 * (bf16 ? 8 : 4) * (-c % 3 == 2 ? 5 : 3) / 4 + r.uni(0, 9);
      loss_case(r, c, r.one_in(2) ? 70 : 129, vocab, bf16, 0.97);
      continue;
    }
    const int64_t rows = r.pick<int64_t>({0, 1, 2, 5, 130});
    const int64_t vocab =
        r.one_in(3) ? r.uni(1, 40)
                    : std::min<int64_t>(rows > 5 ? 1100 : 40000,
                                        r.pick<int64_t>({256, 1000, 1024, 4096, 8192, 16384, 33000}) + r.uni(-9, 9));
    loss_case(r, c, rows, vocab, bf16, 0.25);
  }
  std::printf("loss emulation ok: %d cases, %lld workgroups\n", cases, zr_emu_workgroups);
  for (const auto& kv : zr_emu_coverage()) std::printf("launches %lld %s\n", kv.second, kv.first.c_str());
  return 0;
}
