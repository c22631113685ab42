// Losses over a vocabulary's logits and their gradients (gfx950).
//
// For a row z of logits and the temperature tau, with q = softmax(z / tau):
//   distillation  L = w tau^2 sum_j p_j (log p_j - log q[id_j]),
//                 dL/dz = w tau (q - sum_{j: id_j = v} p_j),
//                 p = softmax(t / tau) over the teacher's entries;
//   policy        L = w (-min(r A, clip(r) A) + kl k),  r = exp(lp - old),
//                 k = exp(ref - lp) - (ref - lp) - 1,   lp = log q[a],
//                 dL/dz = dL/dlp / tau ([v = a] - q).
// Both gradients are one multiple of q with corrections at few columns, so one
// kernel serves both: statistics of the row, a handful of numbers, the row
// written.  Maxima are exact, exponentials and sums over a row fp32.  log q, how
// far it is from old and ref, and what the loss is put together from are 64-bit: a
// ratio may be past fp32, and next to the clip's border it decides between a
// gradient and none (by log q, which is as good as the row's fp32 sum: the header
// gives the bound).  The exponentials and logarithms themselves are fp32 with the
// exponent apart: functions of 64 bits held wave 0, and all waves behind it, for
// 6,000 cycles a row.

#include <cmath>
#include <cstddef>
#include <type_traits>

#include "zr_layers.h"

using namespace zr;

namespace {

constexpr int kMaxTop = 1024;      // a row's entries, kept in LDS
constexpr int kMaxChunks = 64;     // pieces of a row, one a lane

// (12 bytes more, the scalars in 64 bits, cost 0.1 us a launch: 8 rows of 50257 fp32
// 11.67 and 11.45 us.)
struct LossArgs {
  const void* logits;
  void* grad;                      // null: losses only
  int64_t stride, grad_stride;
  const void* ids;                 // a row's entries: tokens, or the teacher's
  const void* teacher;             // null: the policy loss
  int64_t ids_stride, teacher_stride;
  const float* weight;             // null: 1
  const float *old_logp, *ref_logp, *advantage;
  float *loss, *logp;
  double tau, inverse_tau;
  float c;                         // log2(e) / tau
  float clip_low, clip_high;       // the ratio's borders, and their logarithms
  double log_low, log_high;
  float kl;
  int32_t wide, teacher_bf16;
  int64_t rows;
  int32_t vocab, top;
  // a row in pieces
  int32_t chunks, chunk;           // how many, of how many vectors each
  float* stats;                    // [row][chunk] maximum and sum
  float* picked;                   // [row][entry] its logit
  int32_t* counter;                // rows taken beyond the first of each workgroup; null: every gridDim.x-th
};

// -------------------------------------------------------------- a row's data

// Elements of 16 bytes.
template <typename T>
constexpr int kPer = 16 / static_cast<int>(sizeof(T));

template <typename T>
__device__ __forceinline__ float element(const u32x4& v, int k) {
  if constexpr (sizeof(T) == 2) return k & 1 ? bf16_hi(v[k / 2]) : bf16_lo(v[k / 2]);
  else return bits_float(v[k]);
}
template <typename T>
__device__ __forceinline__ float one(const T* p) {
  if constexpr (sizeof(T) == 2) return bf16_lo(*as_global<uint16_t>(p));
  else return *as_global<float>(p);
}
template <typename T>
__device__ __forceinline__ void put_one(T* p, float x) {
  if constexpr (sizeof(T) == 2) *as_global<uint16_t>(p) = static_cast<uint16_t>(pack_bf16(x, 0.0f));
  else *as_global<float>(p) = x;
}
template <typename T>
__device__ __forceinline__ u32x4 filled(float x) {   // x: exact in bf16
  const uint32_t w = sizeof(T) == 2 ? (float_bits(x) >> 16) | (float_bits(x) & 0xffff0000u) : float_bits(x);
  return u32x4{w, w, w, w};
}
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
// e^x of any size: the power's fraction in fp32, its whole part in the exponent of 64
// bits.  What is past that is past fp32 with any fp32 factor too: 0 and infinity.
__device__ __forceinline__ double exp_of(double x) {
  const double p = __builtin_fmax(__builtin_fmin(x * 1.4426950408889634, 1100.0), -1100.0);   // no NaN
  const double n = __builtin_rint(p);
  const double r = __builtin_ldexp(static_cast<double>(exp2_fast(static_cast<float>(p - n))), static_cast<int>(n));
  return x != x ? x : r;
}
// The natural logarithm of s > 0, off by some 2^-24: of its mantissa in fp32, and
// the exponent apart.
__device__ __forceinline__ double log_of(float s) {
  if (!(s < INFINITY)) return s;
  const uint32_t b = float_bits(s);
  int n = static_cast<int>(b >> 23) - 127;
  float f = bits_float((b & 0x7fffffu) | 0x3f800000u);
  if (f > 1.41421356f) f *= 0.5f, ++n;
  return n * 0.69314718055994531 + static_cast<double>(__builtin_amdgcn_logf(f) * 0.69314718f);
}
// exp(d) - 1 and exp(d) - d - 1, of an fp32 exponential or series, neither from the
// other where that would cancel.
struct AboveOne {
  double exp, line;
};
__device__ __forceinline__ AboveOne above_one(double d) {
  const float x = static_cast<float>(d);
  if (x > -0.5f && x < 0.5f) {   // d^2 (1/2 + d/6 + ... + d^7/9!)
    float r = 1.0f / 362880;
    r = __builtin_fmaf(r, x, 1.0f / 40320);
    r = __builtin_fmaf(r, x, 1.0f / 5040);
    r = __builtin_fmaf(r, x, 1.0f / 720);
    r = __builtin_fmaf(r, x, 1.0f / 120);
    r = __builtin_fmaf(r, x, 1.0f / 24);
    r = __builtin_fmaf(r, x, 1.0f / 6);
    r = __builtin_fmaf(r, x, 0.5f);
    const double line = r * d * d;
    return {d + line, line};
  }
  const double e = exp_of(d) - 1.0;
  return {e, e == INFINITY ? e : e - d};
}

// The maximum of some logits and the sum of 2^(c (z - maximum)) over them.  A NaN
// is in the sum, not the maximum.
struct Stats {
  float m, s;
};
constexpr Stats kNoStats{-INFINITY, 0.0f};
__device__ __forceinline__ float base(float m) { return m == -INFINITY ? 0.0f : m; }
__device__ __forceinline__ Stats joined(const Stats& a, const Stats& b, float c) {
  Stats r;
  r.m = a.m > b.m ? a.m : b.m;
  const float at = base(r.m);
  r.s = a.s * exp2_fast((a.m - at) * c) + b.s * exp2_fast((b.m - at) * c);
  return r;
}

// 2^(c (z - m)) for many z, m the same in all lanes.  Fast: an FMA and the
// exponential, and then `fix` once for all that is off by the rounding of c m.
// There m is held where c m is under 10^8, so that the rounding is a few units: the
// sum of a row whose maximum lies further out is not between 1 and its length (it
// may be 0 or infinite), which tells those rows (logits of the type's lowest value,
// all of a row's perhaps).  Otherwise the difference is taken first and stays finite.
struct Powers {
  float m, c, mc, fix;
  __device__ __forceinline__ Powers(float m_, float c_) : m(m_), c(c_), mc(m_ * c_), fix(1.0f) {}
  static __device__ __forceinline__ Powers fast(float m, float c) {
    const float most = 1e8f / c;
    m = m > most ? most : m < -most ? -most : m;
    Powers p(m, c);
    p.fix = exp2_fast(-__builtin_fmaf(m, c, -p.mc));
    return p;
  }
  template <bool kFast>
  __device__ __forceinline__ float of(float z) const {
    return exp2_fast(kFast ? __builtin_fmaf(z, c, -mc) : (z - m) * c);
  }
};
template <typename T>
__device__ __forceinline__ float top_of(float m, const u32x4& v) {
#pragma unroll
  for (int k = 0; k < kPer<T>; k += 2) m = __builtin_fmaxf(__builtin_fmaxf(m, element<T>(v, k)), element<T>(v, k + 1));
  return m;
}
template <bool kFast, typename T>
__device__ __forceinline__ float sum_of(const u32x4& v, const Powers& p) {
  float s = 0.0f;
#pragma unroll
  for (int k = 0; k < kPer<T>; ++k) s += p.of<kFast>(element<T>(v, k));
  return s;
}
template <bool kFast, typename T>
__device__ __forceinline__ u32x4 gradient(const u32x4& v, const Powers& p, float scale) {
  u32x4 g;
  float x[kPer<T>];
#pragma unroll
  for (int k = 0; k < kPer<T>; ++k) x[k] = p.of<kFast>(element<T>(v, k)) * scale;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (sizeof(T) == 2) g[k] = pack_bf16(x[2 * k], x[2 * k + 1]);
    else g[k] = float_bits(x[k]);
  }
  return g;
}
// The statistics of a workgroup's waves, put together in every wave: a power of
// two of them, one a lane.
template <int kWaves>
__device__ __forceinline__ Stats over_waves(const Stats* wave, float c) {
  const Stats own = wave[threadIdx.x % kWaves];
  Stats st = own;
#pragma unroll
  for (int d = 1; d < kWaves; d *= 2) {
    const float o = __shfl_xor(st.m, d);
    st.m = o > st.m ? o : st.m;
  }
  st.s *= exp2_fast((own.m - base(st.m)) * c);
#pragma unroll
  for (int d = 1; d < kWaves; d *= 2) st.s += __shfl_xor(st.s, d);
  return st;
}

// Values unpacked in one pass are not kept for the next: the registers hold the
// packed ones.
template <int kVecs>
__device__ __forceinline__ void keep_packed(u32x4 (&x)[kVecs]) {
#pragma unroll
  for (int i = 0; i < kVecs; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t w = x[i][k];
      ZR_OPAQUE(w);
      x[i][k] = w;
    }
}

__device__ __forceinline__ Stats over_wave(Stats r, float c) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    Stats o;
    o.m = __shfl_xor(r.m, d);
    o.s = __shfl_xor(r.s, d);
    // the same order in both lanes
    r = (threadIdx.x & d) ? joined(o, r, c) : joined(r, o, c);
  }
  return r;
}
__device__ __forceinline__ float most_of_wave(float x) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const float o = __shfl_xor(x, d);
    x = o > x ? o : x;
  }
  return x;
}
template <typename V>
__device__ __forceinline__ V sum_of_wave(V x) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) x += __shfl_xor(x, d);
  return x;
}

// ------------------------------------------------------------- a row's entries

// A row's entries in LDS: their columns (-1: none), what is subtracted from q
// there, and their logits.  Four columns are read at a time: each row's lie on 16
// bytes.
template <bool kTeacher>
struct alignas(16) Entries {
  static constexpr int kTop = kTeacher ? kMaxTop : 4;
  int32_t id[kTop];
  float p[kTop];
  float z[kTop];
  int32_t used;                // one of the below
};
static_assert(sizeof(Entries<true>) % 16 == 0 && offsetof(Entries<true>, id) == 0, "the second row's too");
// What is asked of a row: nothing; all; of the policy's rows of weight 0 the
// log-probability, with a loss and a gradient of 0 whatever their logits are.
enum { kNothing, kAll, kLogpOnly };
// And what else a workgroup shares.
template <bool kTeacher, int kWaves>
struct Shared {
  Entries<kTeacher> row[2];
  Stats wave[kWaves];
  double coef;
  int32_t next;
};

__device__ __forceinline__ int32_t entry_id(const LossArgs& a, int64_t row, int j) {
  const int64_t at = row * a.ids_stride + j;
  if (a.wide) {
    const int64_t id = as_global<int64_t>(a.ids)[at];
    return id >= 0 && id < a.vocab ? static_cast<int32_t>(id) : -1;
  }
  const int32_t id = as_global<int32_t>(a.ids)[at];
  return id >= 0 && id < a.vocab ? id : -1;
}
__device__ __forceinline__ float teacher_logit(const LossArgs& a, int64_t row, int j) {
  const int64_t at = row * a.teacher_stride + j;
  return a.teacher_bf16 ? bf16_lo(as_global<uint16_t>(a.teacher)[at]) : as_global<float>(a.teacher)[at];
}
__device__ __forceinline__ float weight_of(const LossArgs& a, int64_t row) {
  return a.weight ? as_global<float>(a.weight)[row] : 1.0f;
}

// What wave 0 keeps of a row's teacher: the logarithm of the sum of exp(t /
// tau), and sum p t / tau over the entries.
struct Teacher {
  double lse = 0.0, mean = 0.0;
};

// A wave's first 64 entries of a row and the row's numbers, asked for.
struct Asked {
  int32_t id;
  float t, weight, advantage, old_logp, ref_logp;
};
template <bool kTeacher>
__device__ __forceinline__ Asked ask(const LossArgs& a, int64_t row, int lane) {
  Asked q{-1, 0.0f, 1.0f, 0.0f, 0.0f, 0.0f};
  if (lane < a.top) {
    q.id = entry_id(a, row, lane);
    if constexpr (kTeacher) q.t = teacher_logit(a, row, lane);
  }
  q.weight = weight_of(a, row);
  if constexpr (!kTeacher) {
    q.advantage = as_global<float>(a.advantage)[row];
    q.old_logp = as_global<float>(a.old_logp)[row];
    if (a.ref_logp) q.ref_logp = as_global<float>(a.ref_logp)[row];
  }
  return q;
}

// One wave: puts the row's entries into LDS and finds out what is asked of the
// row: nothing where it has no entry in the vocabulary (for the teacher's, none
// above -inf, or no weight).
template <bool kTeacher>
__device__ __forceinline__ void put_asked(const LossArgs& a, int64_t row, const Asked& q, Entries<kTeacher>& e,
                                          int lane) {
  bool some = false;
  for (int j = lane; j < a.top; j += 64) {
    int32_t id = j < 64 ? q.id : entry_id(a, row, j);
    if constexpr (kTeacher) {
      const float t = j < 64 ? q.t : teacher_logit(a, row, j);
      if (t == -INFINITY) id = -1;   // no probability, no matter what q is
      e.p[j] = t;
    } else {
      e.p[j] = 1.0f;
    }
    e.id[j] = id;
    some = some || id >= 0;
  }
  // four at a time are compared below
  if (kTeacher && lane < (-a.top & 3)) e.id[a.top + lane] = -1;
  const bool weighted = q.weight != 0.0f;
  int used = __ballot(some) != 0 && (!kTeacher || weighted);
  if (!kTeacher && used && !weighted) used = kLogpOnly;
  if (lane == 0) e.used = used;
}

// The same wave, of a row that counts: the entries' logits (kLogits; otherwise
// they are there already) and the teacher's probabilities, those of one column
// added up.
template <typename T, bool kTeacher, bool kLogits>
__device__ __forceinline__ Teacher finish_entries(const LossArgs& a, int64_t row, Entries<kTeacher>& e, int lane) {
  Teacher t;
  const T* z = static_cast<const T*>(a.logits) + row * a.stride;
  if constexpr (kLogits)
    for (int j = lane; j < a.top; j += 64)
      if (e.id[j] >= 0) e.z[j] = one(z + e.id[j]);
  if constexpr (kTeacher) {
    float m = -INFINITY;
    for (int j = lane; j < a.top; j += 64)
      if (e.id[j] >= 0) m = e.p[j] > m ? e.p[j] : m;
    m = most_of_wave(m);
    double s = 0.0, mean = 0.0;
    for (int j = lane; j < a.top; j += 64) {
      if (e.id[j] < 0) continue;
      const float d = e.p[j] - m, x = exp2_fast(d * a.c);
      s += x;
      if (x != 0.0f) mean += static_cast<double>(x) * d;
      e.p[j] = x;
    }
    s = sum_of_wave(s);
    mean = sum_of_wave(mean);
    const float part = 1.0f / static_cast<float>(s);
    for (int j = lane; j < a.top; j += 64) e.p[j] = e.id[j] < 0 ? 0.0f : e.p[j] * part;
    // both less m / tau
    t.lse = log_of(static_cast<float>(s));
    t.mean = mean * static_cast<double>(part) * a.inverse_tau;
  }
  return t;
}

// Wave 0, with the row's statistics and the entries' logits: the loss, and the
// multiple of q in the gradient.
template <bool kTeacher>
__device__ __forceinline__ double finish_row(const LossArgs& a, int64_t row, const Entries<kTeacher>& sh,
                                             const Asked& of_row, const Teacher& t, const Stats& st, int lane,
                                             bool store) {
  const double log_s = log_of(st.s);
  if constexpr (kTeacher) {
    // log q[id] = (z - m) / tau - log s
    double cross = 0.0;
    for (int j = lane; j < a.top; j += 64)
      if (sh.id[j] >= 0 && sh.p[j] != 0.0f)
        cross += sh.p[j] * ((static_cast<double>(sh.z[j]) - st.m) * a.inverse_tau - log_s);
    cross = sum_of_wave(cross);
    if (lane == 0 && store)
      a.loss[row] = static_cast<float>(of_row.weight * a.tau * a.tau * ((t.mean - t.lse) - cross));
    return of_row.weight * a.tau;
  } else {
    const double lp = (static_cast<double>(sh.z[0]) - st.m) * a.inverse_tau - log_s;
    // (The KL term first, and 64 bits only where a value is used: with all of them
    // at once the row's registers spill, 777 rows of 50257 fp32 39.7 us for 37.8.)
    const float w = of_row.weight, adv = of_row.advantage;
    double loss = 0.0, slope = 0.0;
    if (a.ref_logp) {
      const AboveOne e = above_one(of_row.ref_logp - lp);
      loss = a.kl * e.line;
      slope = a.kl * e.exp;
    }
    const double over = lp - of_row.old_logp;
    const bool cut = (adv > 0.0f && over > a.log_high) || (adv < 0.0f && over < a.log_low);
    if (cut) {
      loss -= static_cast<double>(adv) * (adv > 0.0f ? a.clip_high : a.clip_low);
    } else {
      double gain = exp_of(over);
      gain = adv == 0.0f && gain == INFINITY ? 0.0 : gain * adv;   // an infinite ratio times 0 is 0
      loss -= gain;
      slope += gain;
    }
    if (lane == 0 && store) {
      a.loss[row] = w == 0.0f ? 0.0f : static_cast<float>(w * loss);
      a.logp[row] = static_cast<float>(lp);
    }
    return w * slope * a.inverse_tau;
  }
}
// A row that does not count.
template <bool kTeacher>
__device__ __forceinline__ void put_nothing(const LossArgs& a, int64_t row) {
  a.loss[row] = 0.0f;
  if constexpr (!kTeacher) a.logp[row] = 0.0f;
}

// The gradient at the entries' columns inside [v0, v1), over what the row's
// pass wrote there.  The p of one column are added up, in their order; entries of
// one column write one value.
template <typename T, int kThreads, bool kTeacher>
__device__ __forceinline__ void put_entries(const LossArgs& a, T* out, const Entries<kTeacher>& e, float coef,
                                            const Stats& st, int v0, int v1) {
  const float part = 1.0f / st.s;
  for (int j = threadIdx.x; j < a.top; j += kThreads) {
    const int32_t id = e.id[j];
    if (id < v0 || id >= v1) continue;
    float p = kTeacher ? 0.0f : e.p[0];
    if constexpr (kTeacher) {
#pragma unroll 4
      for (int i = 0; i < a.top; i += 4) {
        const u32x4 other = *reinterpret_cast<const u32x4*>(&e.id[i]);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (static_cast<int32_t>(other[k]) == id) p += e.p[i + k];
      }
    }
    put_one(out + id, coef * (exp2_fast((e.z[j] - st.m) * a.c) * part - p));
  }
}

// A policy row whose multiple of q may not be an fp32 number, though its columns'
// gradients are: in 64 bits, element by element.
__device__ __forceinline__ bool is_wide(float coef) { return __builtin_fabsf(coef) > 1e30f; }
template <typename T, int kThreads>
__device__ __forceinline__ void put_wide(const LossArgs& a, const T* z, T* out, int32_t token, double coef,
                                         const Stats& st, int v0, int v1) {
  const double part = 1.0 / st.s;
#pragma unroll 1
  for (int v = v0 + threadIdx.x; v < v1; v += kThreads) {
    const double q = exp_of((static_cast<double>(one(z + v)) - st.m) * a.inverse_tau) * part;
    put_one(out + v, static_cast<float>(coef * (q - (v == token ? 1.0 : 0.0))));
  }
}

// Every store of this workgroup so far has reached memory before any after it.
__device__ __forceinline__ void stores_done() {
  __builtin_amdgcn_s_waitcnt(0x0f70);   // vmcnt(0)
  __syncthreads();
}

// The statistics of a row with logits far out, taken again from memory by all of
// the workgroup.
template <typename T, int kThreads>
__device__ __forceinline__ Stats far_stats(const LossArgs& a, const T* z, Stats* wave) {
  Stats st = kNoStats;
#pragma unroll 1
  for (int v = threadIdx.x; v < a.vocab; v += kThreads) {
    const float x = one(z + v);
    st = joined(st, Stats{x, exp2_fast((x - base(x)) * a.c)}, a.c);
  }
  st = over_wave(st, a.c);
  __syncthreads();             // all have read what was there
  if ((threadIdx.x & 63) == 0) wave[threadIdx.x / 64] = st;
  __syncthreads();
  return over_waves<kThreads / 64>(wave, a.c);
}

// ------------------------------------------------------ a row in a workgroup

// A row a workgroup, the first kVecs vectors of a lane in registers between the
// two passes, so that HBM is read once; what is behind them is read twice.  While
// a row's gradient is written the next one's logits are on their way into the
// registers that get free, and wave 0 works out its entries.  A workgroup's next
// row comes from a counter, where there are many: rows that do not count take a
// third of the others' time.
template <typename T, bool kTeacher, int kThreads, int kVecs>
__global__ __launch_bounds__(kThreads, 4) void loss_row_kernel(const LossArgs a) {
  constexpr int kWaves = kThreads / 64;
  __shared__ __align__(16) Shared<kTeacher, kWaves> sh;
  const int tid = threadIdx.x, lane = tid & 63, w = uniform(tid >> 6);
  const int rows = static_cast<int>(a.rows);
  const int vecs = a.vocab / kPer<T>, left = a.vocab % kPer<T>;
  const int64_t end = static_cast<int64_t>(vecs) * kPer<T> + tid;   // a lane's of the elements behind the vectors
  auto take = [&](int row) { return static_cast<int>(gridDim.x) + (a.counter ? atomicAdd(a.counter, 1) : row); };
  auto vec = [&](int i) { return i * kThreads + tid; };
  // A lane's i-th vector of a row: a uniform address and 32 bits of the lane's,
  // not their sums kept for every i.
  auto place = [&](auto* of_row, int i) {
    uint32_t off = 16 * tid;
    ZR_OPAQUE_IN(off, i);
    return reinterpret_cast<decltype(of_row)>(reinterpret_cast<uintptr_t>(of_row) + i * (16 * kThreads) + off);
  };
  int row = blockIdx.x, now = 0;
  Asked of_row{};              // of the row, in wave 0
  if (w == 0) {
    of_row = ask<kTeacher>(a, row, lane);
    if (lane == 0) sh.next = take(row);
    put_asked(a, row, of_row, sh.row[0], lane);
  }
  __syncthreads();
  u32x4 x[kVecs];
  float last = -INFINITY;
  const T* z = static_cast<const T*>(a.logits) + row * a.stride;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) x[i] = filled<T>(-INFINITY);
  Teacher t;
  if (uniform(sh.row[0].used) != kNothing) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
      if (vec(i) < vecs) x[i] = load_at<u32x4, sizeof(T)>(place(z, i));
    if (tid < left) last = one(z + end);
    if (w == 0) t = finish_entries<T, kTeacher, true>(a, row, sh.row[0], lane);
  }
#pragma unroll 1
  for (;;) {
    const int next = uniform(sh.next);
    Asked asked{};
    if (w == 0 && next < rows) asked = ask<kTeacher>(a, next, lane);
    const int asks = uniform(sh.row[now].used);
    const bool used = asks != kNothing;
    if (used) {
      float top = last;
#pragma unroll
      for (int i = 0; i < kVecs; ++i) top = top_of<T>(top, x[i]);
      for (int v = vec(kVecs); v < vecs; v += kThreads)
        top = top_of<T>(top, load_at<u32x4, sizeof(T)>(z + static_cast<int64_t>(v) * kPer<T>));
      Stats st{uniform(most_of_wave(top)), 0.0f};
      const Powers p = Powers::fast(base(st.m), a.c);
      if (st.m != -INFINITY) st.m = p.m;
      keep_packed(x);
      st.s = p.of<true>(last);
#pragma unroll
      for (int i = 0; i < kVecs; ++i) st.s += sum_of<true, T>(x[i], p);
      for (int v = vec(kVecs); v < vecs; v += kThreads)
        st.s += sum_of<true, T>(load_at<u32x4, sizeof(T)>(z + static_cast<int64_t>(v) * kPer<T>), p);
      st.s = sum_of_wave(st.s) * p.fix;
      if (lane == 0) sh.wave[w] = st;
    }
    __syncthreads();
    Stats st = over_waves<kWaves>(sh.wave, a.c);
    // the maximum's term is 1, and there are fewer than 2^30 of them
    const bool far = used && st.m != -INFINITY && (st.s < 0.5f || st.s > 0x1p31f);
    if (far) st = far_stats<T, kThreads>(a, z, sh.wave);
    const bool some = used && st.s != 0.0f;   // not every logit is -inf
    const bool sloped = some && (kTeacher || asks == kAll);
    if (w == 0) {
      // only the policy's gradient waits for the loss
      double coef = kTeacher ? of_row.weight * a.tau : 0.0;
      if (!kTeacher && some) coef = finish_row(a, row, sh.row[now], of_row, t, st, lane, true);
      if (lane == 0) {
        if (!some) put_nothing<kTeacher>(a, row);
        sh.coef = coef;
      }
      if (next < rows) put_asked(a, next, asked, sh.row[now ^ 1], lane);
    }
    __syncthreads();
    const bool then = next < rows && uniform(sh.row[now ^ 1].used) != kNothing;
    if (w == 0) {
      if (lane == 0) sh.next = take(next);
      if (kTeacher && some) finish_row(a, row, sh.row[now], of_row, t, st, lane, true);
      if (then) t = finish_entries<T, kTeacher, true>(a, next, sh.row[now ^ 1], lane);
      of_row = asked;
    }
    T* out = a.grad ? static_cast<T*>(a.grad) + row * a.grad_stride : nullptr;
    const T* ahead = static_cast<const T*>(a.logits) + next * a.stride;
    const float coef = sloped ? static_cast<float>(sh.coef) : 0.0f;
    const bool wide = !kTeacher && is_wide(coef);
    const Powers p = Powers::fast(sloped ? uniform(base(st.m)) : 0.0f, a.c);
    const float scale = sloped ? coef / st.s * p.fix : 0.0f;
    const bool plain = sloped && !far && !wide && out;
    keep_packed(x);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      if (vec(i) < vecs) {
        if (plain) store_at<sizeof(T)>(place(out, i), gradient<true, T>(x[i], p, scale));
        if (then) x[i] = load_at<u32x4, sizeof(T)>(place(ahead, i));
      }
    }
    if (plain) {
      for (int v = vec(kVecs); v < vecs; v += kThreads)
        store_at<sizeof(T)>(
            out + static_cast<int64_t>(v) * kPer<T>,
            gradient<true, T>(load_at<u32x4, sizeof(T)>(z + static_cast<int64_t>(v) * kPer<T>), p, scale));
      if (tid < left) put_one(out + end, p.of<true>(last) * scale);
    } else if (wide && out) {
      put_wide<T, kThreads>(a, z, out, sh.row[now].id[0], sh.coef, st, 0, a.vocab);
    } else if (out) {
      const Powers q(base(st.m), a.c);
#pragma unroll 1
      for (int v = tid; v < vecs; v += kThreads) {
        u32x4 g = {0, 0, 0, 0};
        if (sloped)
          g = gradient<false, T>(load_at<u32x4, sizeof(T)>(z + static_cast<int64_t>(v) * kPer<T>), q, coef / st.s);
        store_at<sizeof(T)>(out + static_cast<int64_t>(v) * kPer<T>, g);
      }
      if (tid < left) put_one(out + end, sloped ? q.of<false>(last) * (coef / st.s) : 0.0f);
    }
    if (then && tid < left) last = one(ahead + end);
    stores_done();
    if (out && sloped && !wide) put_entries<T, kThreads>(a, out, sh.row[now], coef, st, 0, a.vocab);
    if (next >= rows) break;
    row = next;
    z = ahead;
    now ^= 1;
  }
}

// The counter of rows, before the rows.
__global__ __launch_bounds__(64) void loss_begin_kernel(const LossArgs a) {
  if (threadIdx.x == 0) *a.counter = 0;
}

// -------------------------------------------------------- a row in pieces

constexpr int kPieceThreads = 256;
constexpr int kPieceVecs = 4;

// A piece's statistics, and the logits of the entries that lie in it.
template <typename T>
__global__ __launch_bounds__(kPieceThreads) void loss_stats_kernel(const LossArgs a) {
  constexpr int kWaves = kPieceThreads / 64;
  __shared__ Stats wave[kWaves];
  const int tid = threadIdx.x, lane = tid & 63, w = uniform(tid >> 6);
  const int64_t row = blockIdx.y;
  const T* z = static_cast<const T*>(a.logits) + row * a.stride;
  const int vecs = a.vocab / kPer<T>, left = a.vocab % kPer<T>;
  const int v0 = blockIdx.x * a.chunk, v1 = v0 + a.chunk < vecs ? v0 + a.chunk : vecs;
  const bool end = static_cast<int>(blockIdx.x) + 1 == a.chunks;
  Stats st = kNoStats;
  // all lanes of a wave go round together
  for (int v = v0 + tid; v - lane < v1; v += kPieceThreads * kPieceVecs) {
    u32x4 x[kPieceVecs];
#pragma unroll
    for (int i = 0; i < kPieceVecs; ++i) {
      x[i] = filled<T>(-INFINITY);
      if (v + i * kPieceThreads < v1)
        x[i] = load_at<u32x4, sizeof(T)>(z + static_cast<int64_t>(v + i * kPieceThreads) * kPer<T>);
    }
    Stats o = kNoStats;
#pragma unroll
    for (int i = 0; i < kPieceVecs; ++i) o.m = top_of<T>(o.m, x[i]);
    o.m = uniform(most_of_wave(o.m));
    const Powers p(base(o.m), a.c);
#pragma unroll
    for (int i = 0; i < kPieceVecs; ++i) o.s += sum_of<false, T>(x[i], p);
    st = joined(st, o, a.c);
  }
  if (end && tid < left) {
    Stats o;
    o.m = one(z + static_cast<int64_t>(vecs) * kPer<T> + tid);
    o.s = exp2_fast((o.m - base(o.m)) * a.c);
    st = joined(st, o, a.c);
  }
  for (int j = tid; j < a.top; j += kPieceThreads) {
    const int32_t id = entry_id(a, row, j);
    if (id >= v0 * kPer<T> && (end || id < v1 * kPer<T>)) a.picked[row * a.top + j] = one(z + id);
  }
  st = over_wave(st, a.c);
  if (lane == 0) wave[w] = st;
  __syncthreads();
  if (tid == 0) {
    for (int k = 1; k < kWaves; ++k) st = joined(st, wave[k], a.c);
    as_global<float>(a.stats)[2 * (row * a.chunks + blockIdx.x)] = st.m;
    as_global<float>(a.stats)[2 * (row * a.chunks + blockIdx.x) + 1] = st.s;
  }
}

// The pieces' statistics put together, by every workgroup of a row in the same
// order, and the piece's gradient; the first one writes the losses.
template <typename T, bool kTeacher>
__global__ __launch_bounds__(kPieceThreads) void loss_piece_kernel(const LossArgs a) {
  constexpr int kWaves = kPieceThreads / 64;
  __shared__ __align__(16) Shared<kTeacher, kWaves> sh;
  const int tid = threadIdx.x, lane = tid & 63, w = uniform(tid >> 6);
  const int64_t row = blockIdx.y;
  const T* z = static_cast<const T*>(a.logits) + row * a.stride;
  T* out = a.grad ? static_cast<T*>(a.grad) + row * a.grad_stride : nullptr;
  const int vecs = a.vocab / kPer<T>, left = a.vocab % kPer<T>;
  const int v0 = blockIdx.x * a.chunk, v1 = v0 + a.chunk < vecs ? v0 + a.chunk : vecs;
  const bool end = static_cast<int>(blockIdx.x) + 1 == a.chunks;
  Stats st = kNoStats;
  if (lane < a.chunks) {
    st.m = as_global<float>(a.stats)[2 * (row * a.chunks + lane)];
    st.s = as_global<float>(a.stats)[2 * (row * a.chunks + lane) + 1];
  }
  st = over_wave(st, a.c);
  const bool empty = st.s == 0.0f;
  if (w == 0) {
    Entries<kTeacher>& e = sh.row[0];
    const Asked of_row = ask<kTeacher>(a, row, lane);
    put_asked(a, row, of_row, e, lane);
    for (int j = lane; j < a.top; j += 64)
      if (e.id[j] >= 0) e.z[j] = as_global<float>(a.picked)[row * a.top + j];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // lane 0's flag
    const bool first = blockIdx.x == 0;
    if (e.used != kNothing && !empty) {
      const Teacher t = finish_entries<T, kTeacher, false>(a, row, e, lane);
      const double coef = finish_row(a, row, e, of_row, t, st, lane, first);
      if (lane == 0) sh.coef = coef;
    } else if (lane == 0) {
      e.used = kNothing;
      if (first) put_nothing<kTeacher>(a, row);
    }
  }
  if (!out) return;
  __syncthreads();
  const bool used = kTeacher ? sh.row[0].used != kNothing : sh.row[0].used == kAll;
  const Powers p(base(st.m), a.c);
  const float coef = used ? static_cast<float>(sh.coef) : 0.0f;
  if (!kTeacher && is_wide(coef)) {
    put_wide<T, kPieceThreads>(a, z, out, sh.row[0].id[0], sh.coef, st, v0 * kPer<T>, end ? a.vocab : v1 * kPer<T>);
    return;
  }
  const float scale = used ? coef / st.s : 0.0f;
  for (int v = v0 + tid; v < v1; v += kPieceThreads * kPieceVecs) {
    u32x4 x[kPieceVecs];
#pragma unroll
    for (int i = 0; i < kPieceVecs; ++i)
      if (used && v + i * kPieceThreads < v1)
        x[i] = load_at<u32x4, sizeof(T)>(z + static_cast<int64_t>(v + i * kPieceThreads) * kPer<T>);
#pragma unroll
    for (int i = 0; i < kPieceVecs; ++i)
      if (v + i * kPieceThreads < v1)
        store_at<sizeof(T)>(out + static_cast<int64_t>(v + i * kPieceThreads) * kPer<T>,
                            used ? gradient<false, T>(x[i], p, scale) : u32x4{0, 0, 0, 0});
  }
  if (end && tid < left) {
    const int64_t v = static_cast<int64_t>(vecs) * kPer<T> + tid;
    put_one(out + v, used ? p.of<false>(one(z + v)) * scale : 0.0f);
  }
  if (!used) return;
  stores_done();
  put_entries<T, kPieceThreads>(a, out, sh.row[0], coef, st, v0 * kPer<T>, end ? a.vocab : v1 * kPer<T>);
}

// ---------------------------------------------------------------------- host

#ifndef ZR_CUS
#define ZR_CUS 256   // the chip's; the kernels run on a smaller one in tests on the CPU
#endif
constexpr int64_t kCus = ZR_CUS;

// How a call's rows are cut.  Few rows in pieces, in two launches; many a row to a
// workgroup, with as many lanes as hold the row in registers (50257 bf16, 1024
// rows: 59 us with 512 lanes, 70 with 1024; 32000: 32 with 256, 39 with 512).  us in
// pieces, and not:
//     rows               32        64        96       128       256
//     128256 bf16    15, 20    18, 21    24, 24    28, 26    48, 32
//     50257 fp32     14, 13    16, 14    19, 15    23, 18    39, 28
//     300000 bf16    19, 43    33, 53    47, 58   (what registers do not hold is
//                                                  read twice by a workgroup)
// Of 1024 lanes a CU holds one workgroup: it takes row after row, the next one's
// logits ahead; from the third row on from a counter, whose own launch costs 2 to 3
// us (losses only, 50257 fp32: 512 rows 31 us with it, 27 without; 777 rows 41 and
// 45, 4096 rows 159 and 171).
struct Shape {
  int32_t chunks = 1, chunk = 0;
  int32_t lanes = 0, grid = 0;       // rows in one piece: a workgroup's lanes, and how many of them
  int64_t stats = 0, bytes = 0;      // workspace: the statistics, all
};
constexpr int64_t kRowVecs = 1024 * 16;   // of a row, in a workgroup's registers
template <typename T>
Shape shape_of(int64_t rows, int64_t vocab, int64_t top) {
  Shape s;
  const int64_t vecs = vocab / kPer<T>;
  const int64_t wanted = rows > 0 ? ceil_div(1024, rows) : 1;
  const int64_t most = std::max<int64_t>(1, vecs / (kPieceThreads * kPieceVecs));
  if (rows <= (vecs > kRowVecs ? 128 : 64) && most > 1) {
    s.chunk = static_cast<int32_t>(ceil_div(vecs, std::min<int64_t>({wanted, most, kMaxChunks})));
    s.chunks = static_cast<int32_t>(ceil_div(vecs, s.chunk));
  }
  if (s.chunks > 1) {
    s.stats = rows * s.chunks * 8;
    s.bytes = ceil_div(s.stats + rows * top * 4, 16) * 16;
    return s;
  }
  s.lanes = vecs <= 256 * 16 ? 256 : vecs <= 512 * 16 ? 512 : 1024;
  s.grid = static_cast<int32_t>(s.lanes == 1024 ? std::min(rows, kCus) : rows);
  if (rows > 2 * s.grid) s.bytes = 16;
  return s;
}
Shape shape_for(zr_dtype dtype, int64_t rows, int64_t vocab, int64_t top) {
  return dtype == ZR_BF16 ? shape_of<uint16_t>(rows, vocab, top) : shape_of<float>(rows, vocab, top);
}

zr_status check_shape(zr_dtype dtype, int64_t rows, int64_t vocab, int64_t top) {
  if (!valid_dtype(dtype)) return fail(ZR_ERR_INVALID, "unsupported element dtype");
  if (rows < 0 || vocab < 1) return fail(ZR_ERR_INVALID, "rows must be >= 0 and vocab >= 1");
  if (top < 1) return fail(ZR_ERR_INVALID, "top must be >= 1");
  if (vocab >= (int64_t(1) << 30)) return fail(ZR_ERR_UNSUPPORTED, "vocab of 2^30 or more");
  if (top > kMaxTop) return fail(ZR_ERR_UNSUPPORTED, "more than " + std::to_string(kMaxTop) + " entries a row");
  if (!fits_launch(rows, 1024)) return fail(ZR_ERR_UNSUPPORTED, "2^22 rows or more");
  return ZR_OK;
}

// What both losses check; `a` has the sizes and pointers.
zr_status check_loss(const LossArgs& a, zr_dtype dtype, int64_t vocab, int64_t top, zr_index ids_type,
                     const char* ids, double temperature) {
  zr_status st = check_shape(dtype, a.rows, vocab, top);
  if (st != ZR_OK) return st;
  if (ids_type != ZR_I32 && ids_type != ZR_I64) return fail(ZR_ERR_INVALID, "unsupported token type");
  // the kernels multiply by log2(e) / temperature in fp32
  if (!(temperature >= 1e-30 && temperature <= 1e30))
    return fail(ZR_ERR_INVALID, "temperature must lie between 1e-30 and 1e30");
  if (a.stride < vocab) return fail(ZR_ERR_INVALID, "logits_stride must be >= vocab");
  if (a.grad && a.grad_stride < vocab) return fail(ZR_ERR_INVALID, "dlogits_stride must be >= vocab");
  if (a.rows == 0) return ZR_OK;
  if (!a.logits || !aligned_to(a.logits, dtype_size(dtype)))
    return fail(ZR_ERR_INVALID, "logits is null or not element-aligned");
  if (!aligned_to(a.grad, dtype_size(dtype))) return fail(ZR_ERR_INVALID, "dlogits is not element-aligned");
  if (!a.ids || !aligned_to(a.ids, ids_type == ZR_I64 ? 8 : 4))
    return fail(ZR_ERR_INVALID, std::string(ids) + " is null or not element-aligned");
  if (!a.loss || !aligned_to(a.loss, 4) || !aligned_to(a.weight, 4))
    return fail(ZR_ERR_INVALID, "loss is null, or loss or weight not element-aligned");
  return ZR_OK;
}

template <typename T, bool kTeacher>
zr_status launch_loss(LossArgs& a, const Shape& s, hipStream_t stream) {
  if (s.chunks > 1) {
    ZR_LAUNCH(dim3(s.chunks, static_cast<uint32_t>(a.rows)), kPieceThreads, stream, a, loss_stats_kernel<T>);
    zr_status st = launched("loss statistics launch");
    if (st != ZR_OK) return st;
    ZR_LAUNCH(dim3(a.grad ? s.chunks : 1, static_cast<uint32_t>(a.rows)), kPieceThreads, stream, a,
              loss_piece_kernel<T, kTeacher>);
    return launched("loss launch");
  }
  if (s.bytes > 0) {
    a.counter = reinterpret_cast<int32_t*>(a.stats);
    ZR_LAUNCH(1, 64, stream, a, loss_begin_kernel);
    const zr_status st = launched("loss counter launch");
    if (st != ZR_OK) return st;
  }
  if (a.vocab / kPer<T> <= 256 * 4) ZR_LAUNCH(s.grid, 256, stream, a, loss_row_kernel<T, kTeacher, 256, 4>);
  else if (s.lanes == 256) ZR_LAUNCH(s.grid, 256, stream, a, loss_row_kernel<T, kTeacher, 256, 16>);
  else if (s.lanes == 512) ZR_LAUNCH(s.grid, 512, stream, a, loss_row_kernel<T, kTeacher, 512, 16>);
  else ZR_LAUNCH(s.grid, 1024, stream, a, loss_row_kernel<T, kTeacher, 1024, 16>);
  return launched("loss launch");
}

template <bool kTeacher>
zr_status run_loss(LossArgs& a, zr_dtype dtype, int64_t vocab, int64_t top, zr_index ids_type,
                   double temperature, void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  const Shape s = shape_for(dtype, a.rows, vocab, top);
  if (s.bytes > 0 && (!workspace || !aligned_to(workspace, 16) || workspace_bytes < s.bytes))
    return fail(ZR_ERR_INVALID, "workspace is null, not 16-byte aligned or smaller than " +
                                    std::to_string(s.bytes) + " bytes");
  if (a.rows == 0) return ZR_OK;
  a.vocab = static_cast<int32_t>(vocab);
  a.top = static_cast<int32_t>(top);
  a.wide = ids_type == ZR_I64;
  a.tau = temperature;
  a.inverse_tau = 1.0 / temperature;
  a.c = static_cast<float>(1.4426950408889634 / temperature);
  a.chunks = s.chunks;
  a.chunk = s.chunk;
  a.stats = static_cast<float*>(workspace);
  a.picked = s.chunks > 1 ? a.stats + s.stats / 4 : nullptr;
  return dtype == ZR_BF16 ? launch_loss<uint16_t, kTeacher>(a, s, stream)
                          : launch_loss<float, kTeacher>(a, s, stream);
}

}  // namespace

extern "C" zr_status zr_loss_workspace(int64_t rows, int64_t vocab, int64_t top, zr_dtype dtype, int64_t* bytes) {
  return guarded([&]() -> zr_status {
    if (!bytes) return fail(ZR_ERR_INVALID, "null output pointer");
    *bytes = 0;
    const zr_status st = check_shape(dtype, rows, vocab, top);
    if (st != ZR_OK) return st;
    *bytes = shape_for(dtype, rows, vocab, top).bytes;
    return ZR_OK;
  });
}

extern "C" zr_status zr_distill_loss(const void* logits, zr_dtype dtype, int64_t rows, int64_t vocab,
                                     int64_t logits_stride, const void* ids, zr_index ids_type,
                                     int64_t ids_stride, const void* teacher, zr_dtype teacher_dtype,
                                     int64_t teacher_stride, int64_t top, const float* weight,
                                     double temperature, float* loss, void* dlogits,
                                     int64_t dlogits_stride, void* workspace, int64_t workspace_bytes,
                                     hipStream_t stream) {
  return guarded([&]() -> zr_status {
    LossArgs a{};
    a.logits = logits;
    a.grad = dlogits;
    a.stride = logits_stride;
    a.grad_stride = dlogits_stride;
    a.ids = ids;
    a.ids_stride = ids_stride;
    a.teacher = teacher;
    a.teacher_stride = teacher_stride;
    a.teacher_bf16 = teacher_dtype == ZR_BF16;
    a.weight = weight;
    a.loss = loss;
    a.rows = rows;
    zr_status st = check_loss(a, dtype, vocab, top, ids_type, "ids", temperature);
    if (st != ZR_OK) return st;
    if (!valid_dtype(teacher_dtype)) return fail(ZR_ERR_INVALID, "unsupported teacher dtype");
    if (ids_stride < top || teacher_stride < top)
      return fail(ZR_ERR_INVALID, "ids_stride and teacher_stride must be >= top");
    if (rows > 0 && (!teacher || !aligned_to(teacher, dtype_size(teacher_dtype))))
      return fail(ZR_ERR_INVALID, "teacher is null or not element-aligned");
    return run_loss<true>(a, dtype, vocab, top, ids_type, temperature, workspace, workspace_bytes, stream);
  });
}

extern "C" zr_status zr_policy_loss(const void* logits, zr_dtype dtype, int64_t rows, int64_t vocab,
                                    int64_t logits_stride, const void* tokens, zr_index token_type,
                                    const float* old_logp, const float* ref_logp, const float* advantage,
                                    const float* weight, double clip_low, double clip_high, double kl,
                                    double temperature, float* loss, float* logp, void* dlogits,
                                    int64_t dlogits_stride, void* workspace, int64_t workspace_bytes,
                                    hipStream_t stream) {
  return guarded([&]() -> zr_status {
    LossArgs a{};
    a.logits = logits;
    a.grad = dlogits;
    a.stride = logits_stride;
    a.grad_stride = dlogits_stride;
    a.ids = tokens;
    a.ids_stride = 1;
    a.old_logp = old_logp;
    a.ref_logp = kl != 0.0 ? ref_logp : nullptr;
    a.advantage = advantage;
    a.weight = weight;
    a.loss = loss;
    a.logp = logp;
    a.clip_low = static_cast<float>(1.0 - clip_low);
    a.clip_high = static_cast<float>(1.0 + clip_high);
    a.log_low = std::log(1.0 - clip_low);
    a.log_high = std::log(1.0 + clip_high);
    a.kl = static_cast<float>(kl);
    a.rows = rows;
    zr_status st = check_loss(a, dtype, vocab, 1, token_type, "tokens", temperature);
    if (st != ZR_OK) return st;
    if (!(clip_low >= 0.0 && clip_low <= 1.0 && clip_high >= 0.0) || !std::isfinite(clip_high))
      return fail(ZR_ERR_INVALID, "clip_low must lie in [0, 1] and clip_high be finite and >= 0");
    if (!(std::fabs(kl) <= 0x1.fffffep127)) return fail(ZR_ERR_INVALID, "kl must be finite in fp32");
    if (rows > 0) {
      if (!old_logp || !advantage || !logp) return fail(ZR_ERR_INVALID, "old_logp, advantage or logp is null");
      if (kl != 0.0 && !ref_logp) return fail(ZR_ERR_INVALID, "kl needs ref_logp, which is null");
      if (!aligned_to(old_logp, 4) || !aligned_to(ref_logp, 4) || !aligned_to(advantage, 4) || !aligned_to(logp, 4))
        return fail(ZR_ERR_INVALID, "old_logp, ref_logp, advantage or logp is not element-aligned");
    }
    return run_loss<false>(a, dtype, vocab, 1, token_type, temperature, workspace, workspace_bytes, stream);
  });
}
