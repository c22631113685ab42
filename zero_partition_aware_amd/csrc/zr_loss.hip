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
// written.  Maxima are exact, exponentials and a lane's sums fp32; what is
// computed once a row (logarithms, ratios, the loss) is 64-bit, since a ratio
// next to the clip's border decides between a gradient and none.

#include <cmath>

#include "zr_layers.h"

using namespace zr;

namespace {

constexpr int kMaxTop = 1024;      // a row's entries, kept in LDS
constexpr int kMaxChunks = 64;     // pieces of a row, one a lane

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
  double tau, clip_low, clip_high, kl;
  float c;                         // log2(e) / tau
  int32_t wide, teacher_bf16;
  int64_t rows;
  int32_t vocab, top;
  // a row in pieces
  int32_t chunks, chunk;           // how many, of how many vectors each
  float* stats;                    // [row][chunk] maximum and sum
  float* picked;                   // [row][entry] its logit
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

// The maximum of some logits and the sum of 2^(c (z - maximum)) over them.  The
// difference is taken before the product: logits of the type's lowest value,
// all of a row's perhaps, stay finite.  A NaN is in the sum, not the maximum.
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
template <typename T>
__device__ __forceinline__ float top_of(float m, const u32x4& v) {
#pragma unroll
  for (int k = 0; k < kPer<T>; ++k) {
    const float x = element<T>(v, k);
    m = x > m ? x : m;
  }
  return m;
}
template <typename T>
__device__ __forceinline__ float sum_of(const u32x4& v, float at, float c) {
  float s = 0.0f;
#pragma unroll
  for (int k = 0; k < kPer<T>; ++k) s += exp2_fast((element<T>(v, k) - at) * c);
  return s;
}
template <typename T>
__device__ __forceinline__ void add_to(Stats& r, const u32x4& v, float c) {
  const float m = top_of<T>(r.m, v), at = base(m);
  r.s = r.s * exp2_fast((r.m - at) * c) + sum_of<T>(v, at, c);
  r.m = m;
}
template <typename T>
__device__ __forceinline__ u32x4 gradient(const u32x4& v, float m, float c, float scale) {
  u32x4 g;
  float x[kPer<T>];
#pragma unroll
  for (int k = 0; k < kPer<T>; ++k) x[k] = exp2_fast((element<T>(v, k) - m) * c) * scale;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (sizeof(T) == 2) g[k] = pack_bf16(x[2 * k], x[2 * k + 1]);
    else g[k] = float_bits(x[k]);
  }
  return g;
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
__device__ __forceinline__ double sum_of_wave(double x) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) x += __shfl_xor(x, d);
  return x;
}

// ------------------------------------------------------------- a row's entries

// In LDS: the entries' columns (-1: none), their probabilities and logits, and
// what wave 0 works out for all.
template <bool kTeacher, int kWaves>
struct Shared {
  static constexpr int kTop = kTeacher ? kMaxTop : 1;
  int32_t id[kTop];
  float p[kTop];
  float z[kTop];
  Stats wave[kWaves];
  float coef;
  int32_t used;
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

// Wave 0: reads the row's entries into LDS and finds out whether the row counts:
// it has an entry in the vocabulary (and, for the teacher's, one above -inf),
// and the teacher's a weight.  kLogits: their logits too.
template <typename T, bool kTeacher, int kWaves, bool kLogits>
__device__ __forceinline__ Teacher read_entries(const LossArgs& a, int64_t row, Shared<kTeacher, kWaves>& sh, int lane) {
  Teacher t;
  const T* z = static_cast<const T*>(a.logits) + row * a.stride;
  if constexpr (kTeacher) {
    float m = -INFINITY, bad = 0.0f;
    for (int j = lane; j < a.top; j += 64) {
      int32_t id = entry_id(a, row, j);
      const float x = id < 0 ? -INFINITY : teacher_logit(a, row, j);
      if (x != x) bad = x;
      if (x == -INFINITY) id = -1;   // no probability, no matter what q is
      m = x > m ? x : m;
      sh.id[j] = id;
      sh.p[j] = x;
      if constexpr (kLogits) sh.z[j] = id < 0 ? 0.0f : one(z + id);
    }
    m = most_of_wave(m);
    const bool some = __ballot(m > -INFINITY || bad != bad) != 0;
    const float w = weight_of(a, row);
    double s = 0.0, mean = 0.0;
    for (int j = lane; j < a.top; j += 64) {
      if (sh.id[j] < 0) continue;
      const double d = (static_cast<double>(sh.p[j]) - m) / a.tau, e = exp(d);
      s += e;
      if (e > 0.0) mean += e * d;
    }
    s = sum_of_wave(s);
    mean = sum_of_wave(mean);
    for (int j = lane; j < a.top; j += 64)
      sh.p[j] = sh.id[j] < 0 ? 0.0f
                             : static_cast<float>(exp((static_cast<double>(sh.p[j]) - m) / a.tau) / s);
    // both less m / tau
    t.lse = log(s);
    t.mean = mean / s;
    if (lane == 0) {
      sh.used = some && w != 0.0f;
      sh.coef = static_cast<float>(w * a.tau);
    }
  } else {
    const int32_t id = entry_id(a, row, 0);
    if (lane == 0) {
      sh.id[0] = id;
      sh.p[0] = 1.0f;
      if constexpr (kLogits) sh.z[0] = id < 0 ? 0.0f : one(z + id);
      sh.used = id >= 0;
    }
  }
  return t;
}

// Wave 0, with the row's statistics and the entries' logits: the loss, and the
// multiple of q in the gradient.
template <bool kTeacher, int kWaves>
__device__ __forceinline__ void finish_row(const LossArgs& a, int64_t row, Shared<kTeacher, kWaves>& sh,
                                           const Teacher& t, const Stats& st, int lane, bool store) {
  const double log_s = log(static_cast<double>(st.s));
  if constexpr (kTeacher) {
    // log q[id] = (z - m) / tau - log s
    double cross = 0.0;
    for (int j = lane; j < a.top; j += 64)
      if (sh.id[j] >= 0 && sh.p[j] != 0.0f)
        cross += sh.p[j] * ((static_cast<double>(sh.z[j]) - st.m) / a.tau - log_s);
    cross = sum_of_wave(cross);
    if (lane == 0 && store)
      a.loss[row] = static_cast<float>(weight_of(a, row) * a.tau * a.tau * ((t.mean - t.lse) - cross));
  } else {
    const double lp = (static_cast<double>(sh.z[0]) - st.m) / a.tau - log_s;
    const double w = weight_of(a, row), adv = a.advantage[row];
    const double r = exp(lp - a.old_logp[row]);
    const double lo = 1.0 - a.clip_low, hi = 1.0 + a.clip_high;
    const double held = r < lo ? lo : r > hi ? hi : r;   // NaN stays
    const bool cut = (adv > 0.0 && r > hi) || (adv < 0.0 && r < lo);
    double loss = cut ? -held * adv : -r * adv, slope = cut ? 0.0 : -r * adv;
    if (a.ref_logp) {
      const double d = a.ref_logp[row] - lp, e = expm1(d);
      loss += a.kl * (e == INFINITY ? e : e - d);
      slope -= a.kl * e;
    }
    if (lane == 0) {
      sh.coef = w == 0.0 ? 0.0f : static_cast<float>(-w * slope / a.tau);
      if (store) {
        a.loss[row] = w == 0.0 ? 0.0f : static_cast<float>(w * loss);
        a.logp[row] = static_cast<float>(lp);
      }
    }
  }
}

// The gradient at the entries' columns inside [v0, v1), over what the row's
// pass wrote there.  Entries of one column write one value.
template <typename T, int kThreads, bool kTeacher, int kWaves>
__device__ __forceinline__ void put_entries(const LossArgs& a, T* out, const Shared<kTeacher, kWaves>& sh,
                                            const Stats& st, int v0, int v1) {
  const float coef = sh.coef, part = 1.0f / st.s;
  for (int j = threadIdx.x; j < a.top; j += kThreads) {
    const int32_t id = sh.id[j];
    if (id < v0 || id >= v1) continue;
    float p = 0.0f;
    for (int i = 0; i < a.top; ++i) p += sh.id[i] == id ? sh.p[i] : 0.0f;
    put_one(out + id, coef * (exp2_fast((sh.z[j] - st.m) * a.c) * part - p));
  }
}

// Every store of this workgroup so far has reached memory before any after it.
__device__ __forceinline__ void stores_done() {
  __builtin_amdgcn_s_waitcnt(0x0f70);   // vmcnt(0)
  __syncthreads();
}

// ------------------------------------------------------ a row in a workgroup

// A row a workgroup, the first kVecs vectors of a lane in registers between
// the two passes, so that HBM is read once; what is behind them is read twice.
template <typename T, bool kTeacher, int kThreads, int kVecs>
__global__ __launch_bounds__(kThreads) void loss_row_kernel(const LossArgs a) {
  constexpr int kWaves = kThreads / 64;
  __shared__ Shared<kTeacher, kWaves> sh;
  const int tid = threadIdx.x, lane = tid & 63, w = uniform(tid >> 6);
  const int64_t row = blockIdx.x;
  const T* z = static_cast<const T*>(a.logits) + row * a.stride;
  const int vecs = a.vocab / kPer<T>, left = a.vocab % kPer<T>;
  Teacher t;
  if (w == 0) t = read_entries<T, kTeacher, kWaves, true>(a, row, sh, lane);
  __syncthreads();
  const bool used = sh.used != 0;
  T* out = a.grad ? static_cast<T*>(a.grad) + row * a.grad_stride : nullptr;
  if (!used) {
    if (tid == 0) {
      a.loss[row] = 0.0f;
      if constexpr (!kTeacher) a.logp[row] = 0.0f;
    }
    if (out) {
      for (int v = tid; v < vecs; v += kThreads) store_at<sizeof(T)>(out + static_cast<int64_t>(v) * kPer<T>, u32x4{0, 0, 0, 0});
      if (tid < left) put_one(out + static_cast<int64_t>(vecs) * kPer<T> + tid, 0.0f);
    }
    return;
  }
  u32x4 x[kVecs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int v = i * kThreads + tid;
    x[i] = filled<T>(-INFINITY);
    if (v < vecs) x[i] = load_at<u32x4, sizeof(T)>(z + static_cast<int64_t>(v) * kPer<T>);
  }
  float last = -INFINITY;
  if (tid < left) last = one(z + static_cast<int64_t>(vecs) * kPer<T> + tid);
  Stats st;
  st.m = last;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) st.m = top_of<T>(st.m, x[i]);
  const float at = base(st.m);
  st.s = exp2_fast((last - at) * a.c);
  keep_packed(x);
#pragma unroll
  for (int i = 0; i < kVecs; ++i) st.s += sum_of<T>(x[i], at, a.c);
  for (int v = kVecs * kThreads + tid; v < vecs; v += kThreads)
    add_to<T>(st, load_at<u32x4, sizeof(T)>(z + static_cast<int64_t>(v) * kPer<T>), a.c);
  st = over_wave(st, a.c);
  if (lane == 0) sh.wave[w] = st;
  __syncthreads();
  st = sh.wave[0];
  for (int k = 1; k < kWaves; ++k) st = joined(st, sh.wave[k], a.c);
  const bool empty = st.s == 0.0f;   // every logit -inf
  if (w == 0) {
    if (empty) {
      if (lane == 0) {
        a.loss[row] = 0.0f;
        if constexpr (!kTeacher) a.logp[row] = 0.0f;
      }
    } else {
      finish_row<kTeacher>(a, row, sh, t, st, lane, true);
    }
  }
  if (!out) return;
  __syncthreads();
  const float scale = empty ? 0.0f : sh.coef / st.s;
  const float m = base(st.m);
  keep_packed(x);
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int v = i * kThreads + tid;
    if (v < vecs)
      store_at<sizeof(T)>(out + static_cast<int64_t>(v) * kPer<T>, gradient<T>(x[i], m, a.c, scale));
  }
  for (int v = kVecs * kThreads + tid; v < vecs; v += kThreads)
    store_at<sizeof(T)>(out + static_cast<int64_t>(v) * kPer<T>,
                        gradient<T>(load_at<u32x4, sizeof(T)>(z + static_cast<int64_t>(v) * kPer<T>), m, a.c, scale));
  if (tid < left)
    put_one(out + static_cast<int64_t>(vecs) * kPer<T> + tid, exp2_fast((last - m) * a.c) * scale);
  if (empty) return;
  stores_done();
  put_entries<T, kThreads>(a, out, sh, st, 0, a.vocab);
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
  for (int v = v0 + tid; v < v1; v += kPieceThreads * kPieceVecs) {
    u32x4 x[kPieceVecs];
#pragma unroll
    for (int i = 0; i < kPieceVecs; ++i) {
      x[i] = filled<T>(-INFINITY);
      if (v + i * kPieceThreads < v1)
        x[i] = load_at<u32x4, sizeof(T)>(z + static_cast<int64_t>(v + i * kPieceThreads) * kPer<T>);
    }
    float m = st.m;
#pragma unroll
    for (int i = 0; i < kPieceVecs; ++i) m = top_of<T>(m, x[i]);
    const float at = base(m);
    st.s *= exp2_fast((st.m - at) * a.c);
    st.m = m;
#pragma unroll
    for (int i = 0; i < kPieceVecs; ++i) st.s += sum_of<T>(x[i], at, a.c);
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
  __shared__ Shared<kTeacher, kWaves> sh;
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
    const Teacher t = read_entries<T, kTeacher, kWaves, false>(a, row, sh, lane);
    for (int j = lane; j < a.top; j += 64)
      if (sh.id[j] >= 0) sh.z[j] = as_global<float>(a.picked)[row * a.top + j];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // lane 0's flag
    const bool first = blockIdx.x == 0;
    if (sh.used != 0 && !empty) {
      finish_row<kTeacher>(a, row, sh, t, st, lane, first);
    } else if (lane == 0) {
      sh.used = 0;
      if (first) {
        a.loss[row] = 0.0f;
        if constexpr (!kTeacher) a.logp[row] = 0.0f;
      }
    }
  }
  if (!out) return;
  __syncthreads();
  const bool used = sh.used != 0;
  const float scale = used ? sh.coef / st.s : 0.0f, m = base(st.m);
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
                            used ? gradient<T>(x[i], m, a.c, scale) : u32x4{0, 0, 0, 0});
  }
  if (end && tid < left) {
    const int64_t v = static_cast<int64_t>(vecs) * kPer<T> + tid;
    put_one(out + v, used ? exp2_fast((one(z + v) - m) * a.c) * scale : 0.0f);
  }
  if (!used) return;
  stores_done();
  put_entries<T, kPieceThreads>(a, out, sh, st, v0 * kPer<T>, end ? a.vocab : v1 * kPer<T>);
}

// ---------------------------------------------------------------------- host

// How a call's rows are cut.
struct Shape {
  int32_t chunks = 1, chunk = 0;
  int64_t stats = 0, bytes = 0;      // workspace: the statistics, all
};
template <typename T>
Shape shape_of(int64_t rows, int64_t vocab, int64_t top) {
  Shape s;
  const int64_t vecs = vocab / kPer<T>;
  const int64_t wanted = rows > 0 ? ceil_div(1024, rows) : 1;
  const int64_t most = std::max<int64_t>(1, vecs / (kPieceThreads * kPieceVecs));
  if (rows <= 128 && most > 1) {
    s.chunk = static_cast<int32_t>(ceil_div(vecs, std::min<int64_t>({wanted, most, kMaxChunks})));
    s.chunks = static_cast<int32_t>(ceil_div(vecs, s.chunk));
  }
  if (s.chunks > 1) {
    s.stats = rows * s.chunks * 8;
    s.bytes = ceil_div(s.stats + rows * top * 4, 16) * 16;
  }
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
  const int64_t vecs = a.vocab / kPer<T>;
  const uint32_t rows = static_cast<uint32_t>(a.rows);
  if (vecs <= 256 * 4) ZR_LAUNCH(rows, 256, stream, a, loss_row_kernel<T, kTeacher, 256, 4>);
  else if (vecs <= 256 * 16) ZR_LAUNCH(rows, 256, stream, a, loss_row_kernel<T, kTeacher, 256, 16>);
  else if (vecs <= 512 * 16) ZR_LAUNCH(rows, 512, stream, a, loss_row_kernel<T, kTeacher, 512, 16>);
  else ZR_LAUNCH(rows, 1024, stream, a, loss_row_kernel<T, kTeacher, 1024, 16>);
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
  a.c = static_cast<float>(1.4426950408889634 / temperature);
  a.chunks = s.chunks;
  a.chunk = s.chunk;
  a.stats = static_cast<float*>(workspace);
  a.picked = s.bytes > 0 ? a.stats + s.stats / 4 : nullptr;
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
    a.clip_low = clip_low;
    a.clip_high = clip_high;
    a.kl = kl;
    a.rows = rows;
    zr_status st = check_loss(a, dtype, vocab, 1, token_type, "tokens", temperature);
    if (st != ZR_OK) return st;
    if (!(clip_low >= 0.0 && clip_low <= 1.0 && clip_high >= 0.0) || !std::isfinite(clip_high))
      return fail(ZR_ERR_INVALID, "clip_low must lie in [0, 1] and clip_high be finite and >= 0");
    if (!std::isfinite(kl)) return fail(ZR_ERR_INVALID, "kl must be finite");
    if (rows > 0) {
      if (!old_logp || !advantage || !logp) return fail(ZR_ERR_INVALID, "old_logp, advantage or logp is null");
      if (kl != 0.0 && !ref_logp) return fail(ZR_ERR_INVALID, "kl needs ref_logp, which is null");
      if (!aligned_to(old_logp, 4) || !aligned_to(ref_logp, 4) || !aligned_to(advantage, 4) || !aligned_to(logp, 4))
        return fail(ZR_ERR_INVALID, "old_logp, ref_logp, advantage or logp is not element-aligned");
    }
    return run_loss<false>(a, dtype, vocab, 1, token_type, temperature, workspace, workspace_bytes, stream);
  });
}
