// The losses' kernels at the ends of what their arguments may hold, run on the
// CPU: rows that a case gives value by value, in the form that takes a row to a
// workgroup and in the one that cuts it into pieces, with the gradient in a
// buffer of its own and over the logits, against the formulas in 64 bits.
//
// Built as losses_emu.cpp is.
//
// usage: loss_edges_emu <section>

#include <functional>

#include "emu_cases.h"

namespace {

const double kInf = INFINITY;
const double kU = 1.0 / (1 << 24);   // half a step of fp32, relative

// One row of the policy loss.
struct PolicyRow {
  std::function<float(int64_t)> z;   // its logits
  int64_t token = 0;
  float old = 0, ref = 0, advantage = 1, weight = 1;
};
struct Want {
  double loss = 0, logp = 0, coef = 0, size = 0;   // size: how much loss and coef change with logp
  std::vector<double> q;
};

struct Policy {
  int64_t vocab;
  bool bf16 = false;
  double kl = 0, tau = 1, clip_low = 0.2, clip_high = 0.28;
};

Want want_of(const Policy& c, const PolicyRow& row, const std::vector<double>& z) {
  Want w;
  double m = -kInf, s = 0;
  for (double x : z) m = x != x ? x : std::max(m, x);
  for (double x : z) s += std::exp((x - m) / c.tau);
  auto log_q = [&](int64_t v) { return (z[size_t(v)] - m) / c.tau - std::log(s); };
  for (int64_t v = 0; v < c.vocab; ++v) w.q.push_back(std::exp(log_q(v)));
  w.logp = log_q(row.token);
  const double a = row.advantage, r = std::exp(w.logp - row.old);
  auto times = [&](double x) { return a == 0 && x == kInf ? 0 : x * a; };
  const double held = std::min(std::max(r, 1 - c.clip_low), 1 + c.clip_high);
  w.loss = -std::min(times(r), held * a);
  double slope = times(r) <= held * a ? -times(r) : 0;
  w.size = std::fabs(slope);
  if (c.kl != 0) {
    const double d = row.ref - w.logp, e = std::expm1(d);
    w.loss += c.kl * (e == kInf ? e : e - d);
    slope -= c.kl * e;
    w.size += std::fabs(c.kl) * (1 + std::exp(d));
  }
  w.loss *= row.weight;
  w.size *= row.weight;
  w.coef = -row.weight * slope / c.tau;
  if (row.weight == 0) w.loss = w.coef = w.size = 0;
  return w;
}

// An error that fp32 may make, or the same that is no finite number of fp32.
bool same(double got, double want, double tolerance) {
  if (std::fabs(want) >= 0x1.ffffffp127) want = std::copysign(kInf, want);
  return got == want || (got != got && want != want) || std::fabs(got - want) <= tolerance;
}

int g_cases = 0;

// zeros: rows of weight 0, whose loss and gradient are +0 in every bit.
void check_policy(const char* what, const Policy& c, const std::vector<PolicyRow>& list, bool in_place) {
  const int64_t n = int64_t(list.size()), V = c.vocab;
  Rows z(n, V, V + 1, c.bf16, 1), g(in_place ? 0 : n, V, V, c.bf16, 3);
  Rows& out = in_place ? z : g;
  std::vector<std::vector<double>> was(list.size(), std::vector<double>(static_cast<size_t>(V)));
  Buf tokens(size_t(n) * 8, 0);
  Rows per(6, n, n, false, 0);   // old, ref, advantage, weight, loss, logp
  for (int64_t i = 0; i < n; ++i) {
    const PolicyRow& row = list[size_t(i)];
    for (int64_t v = 0; v < V; ++v) {
      z.put(i * z.stride + v, row.z(v));
      was[size_t(i)][size_t(v)] = z.at(i * z.stride + v);
    }
    tokens.as<int64_t>()[i] = row.token;
    per.put(i, row.old);
    per.put(n + i, row.ref);
    per.put(2 * n + i, row.advantage);
    per.put(3 * n + i, row.weight);
  }
  int64_t bytes = 0;
  CHECK(zr_loss_workspace(n, V, 1, z.type(), &bytes) == ZR_OK, "%s", what);
  Buf ws(size_t(bytes), 0);
  float* p = per.b.as<float>();
  CHECK(zr_policy_loss(z.b.p, z.type(), n, V, z.stride, tokens.p, ZR_I64, p, c.kl != 0 ? p + n : nullptr, p + 2 * n,
                       p + 3 * n, c.clip_low, c.clip_high, c.kl, c.tau, p + 4 * n, p + 5 * n, out.b.p, out.stride,
                       bytes ? ws.p : nullptr, bytes, nullptr) == ZR_OK, "%s", what);
  // q is off by U (3 |ln q| + 3 ln V + V / 256 + 210) of it (exponents' roundings,
  // the exponential's, the adds), log q by the row's part of that, exp by its
  // argument's error and 8 U
  const double part = kU * (3 * std::log(double(V)) + double(V) / 256 + 210), half = c.bf16 ? 1.0 / 256 : kU;
  for (int64_t i = 0; i < n; ++i) {
    const PolicyRow& row = list[size_t(i)];
    const Want w = want_of(c, row, was[size_t(i)]);
    const double off = part + 4 * kU * std::fabs(w.logp), loss = per.at(4 * n + i), lp = per.at(5 * n + i);
    CHECK(same(lp, w.logp, off), "%s row %ld: logp %.9g for %.9g", what, long(i), lp, w.logp);
    CHECK(same(loss, w.loss, 1.01 * (off + 8 * kU) * w.size + 2 * kU * std::fabs(w.loss) + 1e-37),
          "%s row %ld: loss %.9g for %.9g", what, long(i), loss, w.loss);
    for (int64_t v = 0; v < V; ++v) {
      const double got = out.at(i * out.stride + v);
      if (row.weight == 0) {
        const bool zero = got == 0 && !std::signbit(got);
        CHECK(zero, "%s row %ld column %ld: a gradient of %g where the weight is 0", what, long(i), long(v), got);
        continue;
      }
      const double q = w.q[size_t(v)], t = v == row.token, to = w.coef * (q - t);
      const double rel = q * (part + 3 * kU * (q > 0 ? std::min(-std::log(q), 100.0) : 0)) + 8 * kU * t;
      const double tolerance = 1.01 * (std::fabs(w.coef) * rel + (off + 8 * kU) * w.size / c.tau * std::fabs(q - t) +
                                       half * std::fabs(to)) + 1e-37 * (1 + std::min(std::fabs(w.coef), 1e30));
      CHECK(to != 0 || got == 0, "%s row %ld column %ld: %g for 0", what, long(i), long(v), got);
      CHECK(same(got, to, tolerance), "%s row %ld column %ld: %.9g for %.9g (multiple %.9g)", what, long(i), long(v), got,
            to, w.coef);
    }
  }
  ++g_cases;
}

// In every form: a row to a workgroup, in pieces; both dtypes; in place and not.
void in_all_forms(const char* what, Policy c, const std::vector<PolicyRow>& list) {
  for (int64_t vocab : {301, 20003})
    for (bool bf16 : {false, true})
      for (bool in_place : {false, true}) {
        c.vocab = vocab;
        c.bf16 = bf16;
        check_policy(what, c, list, in_place);
      }
}

float plain(int64_t v) { return float(int(v * 37 % 65) - 32) / 8; }
// plain, but x at column `at`
std::function<float(int64_t)> with(int64_t at, float x) {
  return [=](int64_t v) { return v == at ? x : plain(v); };
}

// Rows of weight 0 hold anything.
void weights() {
  std::vector<PolicyRow> rows;
  for (float x : {0.0f, kNaN, INFINITY, -INFINITY, 3e38f, -3e38f}) {
    PolicyRow r;
    r.z = with(5, x);
    r.token = 7;
    r.old = -5;
    r.ref = -6;
    r.weight = 0;
    rows.push_back(r);
    r.token = 5;
    rows.push_back(r);
    r.advantage = r.old = r.ref = kNaN;
    rows.push_back(r);
    r.weight = -0.0f;
    rows.push_back(r);
  }
  // a clipped row, whose multiple is 0 too, and rows that count, among them
  PolicyRow r;
  r.z = plain;
  r.token = 3;
  r.old = -100;
  rows.insert(rows.begin() + 2, r);
  r.old = -7;
  rows.push_back(r);
  r.z = with(9, kNaN);
  rows.push_back(r);
  r.old = -100;
  rows.push_back(r);
  in_all_forms("weight 0", Policy{0}, rows);
  in_all_forms("weight 0, kl", Policy{0, false, 0.25}, rows);
}

// The KL term alone, with a reference anywhere.
void references() {
  std::vector<PolicyRow> rows;
  PolicyRow r;
  r.z = plain;
  r.token = 11;
  r.advantage = 0;
  r.old = -5;
  r.weight = 0.75f;
  for (float x : {-100.0f, -1e6f, -1.7e7f, -3e7f, -1e8f, -1e9f, -3e38f, -INFINITY, 20.0f, 60.0f, INFINITY, kNaN}) {
    r.ref = x;
    rows.push_back(r);
  }
  for (int k = 0; k < 40; ++k) {   // next to the row's own, and around it
    r.ref = -13.0f + 0.31f * float(k);
    rows.push_back(r);
  }
  // a token that the policy masks
  r.z = with(11, -INFINITY);
  r.ref = -3;
  rows.push_back(r);
  in_all_forms("reference", Policy{0, false, 1.0}, rows);
  in_all_forms("reference, kl < 0", Policy{0, false, -0.01, 1.5}, rows);
}

// Ratios that fp32 does not hold, with advantages of any size, and references as
// far above the policy.
void ratios() {
  std::vector<PolicyRow> rows;
  PolicyRow r;
  r.z = plain;
  r.token = 2;
  for (float old : {-100.0f, -200.0f, -500.0f, -900.0f, -1e9f, -INFINITY, 100.0f, 1e9f, INFINITY})
    for (float a : {-0.5f, -3.0f, -1e-10f, -1e-30f, 0.0f, 0.5f, 1e-30f}) {
      r.old = old;
      r.advantage = a;
      rows.push_back(r);
    }
  // small weights hold them again
  r.weight = 1e-20f;
  r.advantage = -1;
  for (float old : {-90.0f, -100.0f, -120.0f}) {
    r.old = old;
    rows.push_back(r);
  }
  in_all_forms("ratio", Policy{0}, rows);
  rows.clear();
  r.advantage = 0;
  for (float ref : {70.0f, 85.0f, 100.0f, 500.0f, 1e9f}) {
    r.ref = ref;
    rows.push_back(r);
  }
  in_all_forms("reference above", Policy{0, false, 1e-12}, rows);
}

// Rows around 10^8 binary orders from 0, where a row's maximum is no longer the
// base of its exponentials.
void far_rows() {
  for (double tau : {1.0, 1e-8, 1e8}) {
    const double at = 1e8 * std::log(2.0) * tau;
    std::vector<PolicyRow> rows;
    PolicyRow r;
    r.token = 3;
    r.old = -4;
    for (double sign : {-1.0, 1.0})
      for (int k = -8; k <= 20; ++k) {
        // a step of fp32 there is 2^-24 to 2^-23 of it, several units of the exponent
        const double first = sign * at * (1 + k * 0x1p-23), step = at * 0x1p-23;
        r.z = [=](int64_t v) { return float(v % 5 ? first - step * double(v % 5) : first); };
        rows.push_back(r);
        r.z = [=](int64_t v) { return v % 7 ? float(first) : plain(v); };
        rows.push_back(r);
        r.weight = 1e-6f;
        rows.push_back(r);
        r.weight = 1;
      }
    Policy c{0, false, 0, tau};
    for (int64_t vocab : {301, 5003}) {
      c.vocab = vocab;
      check_policy("far", c, rows, false);
    }
  }
}

// Multiples of q that fp32 does not hold, over columns that are masked, far below and
// not: each column's own gradient may be one that it does.
void multiples() {
  std::vector<PolicyRow> rows;
  PolicyRow r;
  r.token = 7;
  r.advantage = -0.5f;
  for (int kind = 0; kind < 3; ++kind) {
    r.z = [=](int64_t v) {
      if (v % 11 == 3) return kind == 0 ? -INFINITY : kind == 1 ? -150.0f : -3e38f;
      return v == 7 && kind == 2 ? -40.0f : plain(v);
    };
    for (float old : {-80.0f, -92.0f, -95.0f, -98.0f, -110.0f, -150.0f, -200.0f, -600.0f}) {
      r.old = old;
      rows.push_back(r);
    }
  }
  in_all_forms("multiple", Policy{0}, rows);
  r.advantage = 0;
  r.old = -5;
  rows.clear();
  for (float ref : {80.0f, 85.0f, 90.0f, 120.0f, 300.0f}) {
    r.ref = ref;
    rows.push_back(r);
  }
  in_all_forms("multiple of the KL term", Policy{0, false, 1.0, 0.5}, rows);
}

}  // namespace

int main(int argc, char** argv) {
  const std::map<std::string, void (*)()> sections = {{"weights", weights}, {"references", references}, {"ratios", ratios}, {"far", far_rows},
                                                          {"multiples", multiples}};
  const auto it = sections.find(argc > 1 ? argv[1] : "");
  CHECK(it != sections.end(), "no such section");
  it->second();
  std::printf("loss edges ok: %d calls, %lld workgroups\n", g_cases, zr_emu_workgroups);
  return 0;
}
