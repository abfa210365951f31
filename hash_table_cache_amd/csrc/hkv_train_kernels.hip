// gfx950 kernels of the training operators (include/hkv_train.h).
//
// Row mathematics. With k = log2(e) / tau, M the maximum of a row without its
// label and S = sum over v != y of 2^((x_v - M) k), everything a row needs
// follows from (M, S, x_y):
//   d = (x_y - M) / tau
//   d >= 0: logp = -log1p(S e^-d)    d < 0: logp = d - log(S + e^d)
// The label's own term stays out of the sum because a row that is nearly
// certain has logp = -log1p(S e^-d) and 1 - softmax_y = S e^-d / (1 + S e^-d):
// with the label inside, 1 + (something small) would round both away.
// S is summed in 64 bits, of 16-bit elements up to 32 at a time in 32 (kFloats).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <limits>
#include <type_traits>

#include "hkv_train_internal.h"
#include "hkv_train_rows.h"

namespace hkvt {
namespace {

// Running maximum and sum of the elements a thread has seen.
struct Running {
  float m = -kInf;
  double s = 0.0;

  // N elements: their maximum first, so that the sum is rescaled at most once
  // for all of them and, after the first few, by hardly any wave. Up to
  // F at a time are added in 32 bits.
  template <int N, int F>
  __device__ __forceinline__ void add(const float* f, const Scale& c) {
    float mx = f[0];
#pragma unroll
    for (int i = 1; i < N; ++i) mx = fmaxf(mx, f[i]);
    raise(mx, c);
    sum<N, F>(f, c);
  }

  __device__ __forceinline__ void raise(float mx, const Scale& c) {
    if (__any(mx > m)) {
      const float top = fmaxf(m, mx);
      const float t = top == -kInf ? 0.0f : m - top;
      s *= (double)exp2_fast(fmaf(t, c.k_hi, t * c.k_lo));
      m = top;
    }
  }

  template <int N, int F>
  __device__ __forceinline__ void sum(const float* f, const Scale& c) {
    const float base = m == -kInf ? 0.0f : m;
    float e[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float t = f[i] - base;
      e[i] = exp2_fast(fmaf(t, c.k_hi, t * c.k_lo));
    }
    constexpr int G = N < F ? N : F, D = N / G;
    double d[D];
#pragma unroll
    for (int i = 0; i < D; ++i) {
#pragma unroll
      for (int w = G / 2; w > 0; w /= 2)
#pragma unroll
        for (int j = 0; j < w; ++j) e[i * G + j] += e[i * G + j + w];
      d[i] = (double)e[i * G];
    }
#pragma unroll
    for (int w = D / 2; w > 0; w /= 2)
#pragma unroll
      for (int i = 0; i < w; ++i) d[i] += d[i + w];
    s += d[0];
  }
};

// Joins the threads' running values; every thread of the team gets them all.
template <int NT>
__device__ __forceinline__ void join(Running& r, const Scale& c, typename Team<NT>::Shared& sh) {
  constexpr int W = NT < 64 ? NT : 64;
  float top = r.m;
#pragma unroll
  for (int w = W / 2; w > 0; w /= 2) top = fmaxf(top, __shfl_xor(top, w));
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (NT > 64) {
    if (lane == 0) sh.m[wave] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < Team<NT>::kWaves; ++w) top = fmaxf(top, sh.m[w]);
  }
  const float base = top == -kInf ? 0.0f : top;
  const float t = r.m - base;
  double s = r.s * (double)exp2_fast(fmaf(t, c.k_hi, t * c.k_lo));
#pragma unroll
  for (int w = W / 2; w > 0; w /= 2) s += __shfl_xor(s, w);
  if (NT > 64) {
    if (lane == 0) sh.s[wave] = s;
    __syncthreads();
    s = 0.0;
#pragma unroll
    for (int w = 0; w < Team<NT>::kWaves; ++w) s += sh.s[w];
  }
  r.m = top;
  r.s = s;
}

struct RowEnd {
  double logp, lse;
  RowState state;
};

// (M, S, x_y) -> log-probability, normaliser and what the gradient needs.
__device__ __forceinline__ RowEnd finish_row(float m, double s, float xy, double inv_tau) {
  RowEnd r;
  if (m == -kInf && xy == -kInf && s == 0.0) {
    r.logp = 0.0;
    r.lse = -(double)kInf;
    r.state = RowState{0.0, 0.0f, 1.0f, 0.0f, 0};
    return r;
  }
  double d = ((double)xy - (double)m) * inv_tau;
  if (xy == kInf) d = __builtin_nan("");
  if (d >= 0.0) {
    const double er = s * exp_of(-d);
    r.logp = -log1p_of(er);
    r.lse = (double)xy * inv_tau - r.logp;
    r.state = RowState{r.logp, xy, (float)(1.0 + er), (float)er / (float)(1.0 + er), 1};
  } else {
    const double total = s + exp_of(d);
    const double lt = log_of(total);
    r.logp = d - lt;
    r.lse = (double)m * inv_tau + lt;
    r.state = RowState{r.logp, m, (float)total, (float)s / (float)total, 1};
  }
  return r;
}

// A label past the vocabulary: NaN throughout.
__device__ RowEnd nan_row() {
  const double q = __builtin_nan("");
  return RowEnd{q, q, RowState{q, (float)q, (float)q, (float)q, 1}};
}

// Adds N vectors of a row, of which vector `at` holds the label in this thread
// (N or more: none does) as its element `el`. The label stays out.
template <typename T, int N>
__device__ __forceinline__ void add_vecs(Running& r, const u32x4* raw, uint32_t at, uint32_t el, const Scale& c) {
  constexpr int K = Io<T>::K;
  float f[N * K];
#pragma unroll
  for (int i = 0; i < N; ++i) Io<T>::unpack(raw[i], f + i * K);
  if (__any(at < N)) {
#pragma unroll
    for (int i = 0; i < N * K; ++i)
      if (at == i / K && el == i % K) f[i] = -kInf;
  }
  r.add<N * K, Io<T>::kFloats>(f, c);
}

template <typename T, int NT>
__device__ __forceinline__ void add_singles(Running& r, const T* row, const Cut<T, NT>& cut, uint32_t y, uint32_t tid,
                                            const Scale& c) {
  for (uint32_t j0 = 0; j0 < cut.singles(); j0 += NT) {
    const uint32_t j = j0 + tid, i = cut.single(j);
    float f = -kInf;
    if (j < cut.singles() && i != y) f = (float)row[i];
    r.add<1, 1>(&f, c);
  }
}

// One vector of the gradient: -coef * 2^((x - top) k).
template <typename T>
__device__ __forceinline__ u32x4 grad_vec(u32x4 raw, float top, float k, float coef) {
  constexpr int K = Io<T>::K;
  float f[K];
  Io<T>::unpack(raw, f);
#pragma unroll
  for (int i = 0; i < K; ++i) f[i] = -coef * exp2_fast((f[i] - top) * k);
  return Io<T>::pack(f);
}

template <typename T, int NT>
__device__ __forceinline__ void grad_singles(const T* row, T* out, const Cut<T, NT>& cut, uint32_t tid, float top, float k,
                                             float coef) {
  for (uint32_t j = tid; j < cut.singles(); j += NT) {
    const uint32_t i = cut.single(j);
    out[i] = (T)(-coef * exp2_fast(((float)row[i] - top) * k));
  }
}

// The vectors from `first` of a row's gradient, the row read again. (In place,
// every vector is read by the thread that writes it.)
template <typename T, int NT, int U>
__device__ __forceinline__ void grad_vecs(const T* row, T* out, uint32_t first, uint32_t nv, uint32_t tid, float top,
                                          float k, float coef) {
  for_vecs<T, NT, U>(row, first, nv, tid,
                     [&](u32x4 raw, uint32_t v) { store_vec(out, v, grad_vec<T>(raw, top, k, coef)); });
}

// Value and slope of one row of the policy loss.
struct PolicyRow {
  double loss;
  float kl, g;
};

// What it takes beside the logits, loaded before them.
struct PolicyIn {
  float old_logp, advantage, weight, ref;
};

__device__ __forceinline__ PolicyIn policy_in(const Policy& p, uint32_t t) {
  return PolicyIn{p.old_logp[t], p.advantages[t], p.weights[t], p.ref ? p.ref[t] : 0.0f};
}

__device__ __forceinline__ PolicyRow policy_row(const Policy& p, const PolicyIn& in, double logp) {
  const double shift = logp - (double)in.old_logp, a = in.advantage;
  const double r = exp_of(shift);
  const double free = r * a, bound = (r < p.low ? p.low : r > p.high ? p.high : r) * a;
  double loss = -(free <= bound ? free : bound);
  double g = free <= bound ? -free : 0.0;
  if (!(free == free)) loss = g = free;
  double kl = 0.0;
  if (p.ref) {
    const double d = (double)in.ref - logp;
    double slope;  // e^d - 1
    if (fabs(d) < 0.5) {
      // d^2 (1/2 + d/6 + ...): the difference itself would lose what is small
      const float f = (float)d;
      const float q = fmaf(f, fmaf(f, fmaf(f, fmaf(f, fmaf(f, fmaf(f, 1.0f / 362880, 1.0f / 40320), 1.0f / 5040),
                                                 1.0f / 720), 1.0f / 120), 1.0f / 24), 1.0f / 6);
      kl = d * d * (0.5 + d * (double)q);
      slope = kl + d;
    } else {
      slope = exp_of(d) - 1.0;
      kl = slope - d;
    }
    if (p.kl_coef != 0.0) {
      loss += p.kl_coef * kl;
      g -= p.kl_coef * slope;
    }
  }
  return PolicyRow{loss, (float)kl, (float)(g * (double)in.weight * p.grad_scale)};
}

enum Mode { kLogp, kPairs, kPolicy };

struct RowsArgs {
  Logits l;
  Scale c;
  float* logp;
  float* lse;        // kLogp
  RowState* states;  // kPairs, and kPolicy where rows are shared
  float* g;          // the rows' coefficients; kPairs: cleared here
  Policy p;          // kPolicy
  double* weighted;  // kPolicy: the rows' terms of the loss
  uint32_t first;    // row of the first team
};

// The last step of a policy row, by one thread: its outputs and its slope.
__device__ __forceinline__ Slope end_policy_row(const RowsArgs& a, uint32_t t, const PolicyIn& in, const RowEnd& e) {
  PolicyRow p{0.0, 0.0f, 0.0f};
  if (e.state.counts) p = policy_row(a.p, in, e.logp);
  a.p.token_loss[t] = (float)p.loss;
  a.weighted[t] = e.state.counts ? p.loss * (double)in.weight : 0.0;
  a.p.kl[t] = p.kl;
  const float gt = (float)(p.g * a.c.inv_tau);
  return Slope{p.g, e.state.top, gt / e.state.total, gt * e.state.rest};
}

// Statistics of rows, by a team of NT threads each, and for the policy loss,
// whose coefficient needs its own row alone, the gradient in the same kernel:
// the first NV vectors of every thread stay in registers from the one to the
// other, so that a row of up to 16 * NT * NV bytes is read once. Without a
// gradient the same registers hold what is in flight.
template <typename T, int NT, int NV, Mode MODE, bool kKeep>
__global__ __launch_bounds__(Team<NT>::kBlock) void rows_kernel(const RowsArgs a) {
  using Tm = Team<NT>;
  constexpr int K = Io<T>::K;
  constexpr int U = 4;  // vectors summed at a time
  __shared__ typename Tm::Shared sh;
  const uint32_t tid = Tm::thread(), vocab = a.l.vocab;
  const uint32_t t = Tm::row(a.first, blockIdx.x);
  if (t >= a.l.rows) return;  // a whole team
  const bool write = MODE == kPolicy && a.l.dx;
  const T* row = static_cast<const T*>(a.l.x) + (uint64_t)t * a.l.x_stride;
  T* out = static_cast<T*>(a.l.dx) + (uint64_t)t * a.l.dx_stride;
  const Cut<T, NT> cut(write ? out : row, vocab);
  const T* vecs = row + cut.head;
  const uint32_t nv = cut.nv;
  const int64_t y64 = a.l.labels[t];
  const uint32_t y = y64 < 0 || y64 >= (int64_t)vocab ? 0u : (uint32_t)y64;
  PolicyIn in{};
  if (MODE == kPolicy && tid == 0) in = policy_in(a.p, t);
  RowEnd e;
  u32x4 kept[NV];
  if (y64 < 0) {
    e.logp = e.lse = 0.0;
    e.state = RowState{0.0, 0.0f, 1.0f, 0.0f, 0};
  } else if (y64 >= (int64_t)vocab) {
    e = nan_row();
  } else {
    const float xy = (float)row[y];
    Running r;
    const uint32_t yv = cut.vec_of(y);
    // chunks of NT * NV vectors, the first last: it is the one kept
    const uint32_t chunks = nv ? (nv - 1) / (NT * NV) + 1 : 0;
    for (uint32_t ch = chunks; ch-- > 0;) {
      const uint32_t v0 = ch * (NT * NV) + tid;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        kept[i] = no_vec<T>();
        if (v0 + i * NT < nv) kept[i] = load_vec<T, kKeep>(vecs + (ch * NV + i) * (NT * K), tid);
      }
      const uint32_t at = yv >= v0 && (yv - v0) % NT == 0 ? (yv - v0) / NT : ~0u;
#pragma unroll
      for (int i = 0; i < NV; i += U)
        if (ch * (NT * NV) + i * NT < nv) add_vecs<T, U>(r, kept + i, at - i, (y - cut.head) % K, a.c);
    }
    add_singles<T, NT>(r, row, cut, y, tid, a.c);
    join<NT>(r, a.c, sh);
    if (tid == 0) e = finish_row(r.m, r.s, xy, a.c.inv_tau);
  }
  Slope k{};
  if (tid == 0) {
    a.logp[t] = (float)e.logp;
    if (MODE == kLogp && a.lse) a.lse[t] = (float)e.lse;
    if (MODE == kPairs) {
      a.states[t] = e.state;
      a.g[t] = 0.0f;
    }
    if (MODE == kPolicy) k = end_policy_row(a, t, in, e);
  }
  if (write) {
    if (NT > 64) {
      if (tid == 0) sh.got = k;
      __syncthreads();
      k = sh.got;
    } else {
      k.g = __shfl(k.g, 0, NT);
      k.top = __shfl(k.top, 0, NT);
      k.coef = __shfl(k.coef, 0, NT);
      k.at_label = __shfl(k.at_label, 0, NT);
    }
    if (k.g == 0.0f) {
      zero_row<T, NT>(out, cut, tid);
    } else {
      if (y64 >= (int64_t)vocab) {
#pragma unroll
        for (int i = 0; i < NV; ++i) kept[i] = u32x4{0, 0, 0, 0};  // NaN comes from the coefficient
      }
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (tid + i * NT < nv)
          store_vec(out + cut.head + i * (NT * K), tid, grad_vec<T>(kept[i], k.top, a.c.k_hi, k.coef));
      if (nv > NT * NV) grad_vecs<T, NT, 4>(vecs, out + cut.head, NT * NV, nv, tid, k.top, a.c.k_hi, k.coef);
      grad_singles<T, NT>(row, out, cut, tid, k.top, a.c.k_hi, k.coef);
      if (tid == cut.owner(y)) out[y] = (T)k.at_label;  // after its neighbours, by the same thread
    }
  }
}

// Few long rows: a row is shared by workgroups, whose running values a wave
// joins. One workgroup a row reads at what one compute unit can.
struct Partial {
  double s;
  float m;
};

constexpr uint32_t kMostParts = 64;  // a lane each

template <typename T>
__global__ __launch_bounds__(256) void part_kernel(const RowsArgs a, uint32_t parts, uint32_t size, Partial* partial) {
  constexpr int NT = 256, NV = 8, U = 4, K = Io<T>::K;
  __shared__ typename Team<NT>::Shared sh;
  const uint32_t tid = threadIdx.x, t = blockIdx.x / parts;
  const int64_t y64 = a.l.labels[t];
  if (y64 < 0 || y64 >= (int64_t)a.l.vocab) return;
  const T* row = static_cast<const T*>(a.l.x) + (uint64_t)t * a.l.x_stride;
  const Cut<T, NT> cut(row, a.l.vocab, blockIdx.x % parts, size);
  const T* vecs = row + cut.head;
  const uint32_t y = (uint32_t)y64, yv = cut.vec_of(y);
  Running r;
  for (uint32_t first = cut.begin; first < cut.end; first += NT * NV) {
    const uint32_t v0 = first + tid;
    u32x4 raw[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      raw[i] = no_vec<T>();
      if (v0 + i * NT < cut.end) raw[i] = load_vec<T, true>(vecs, v0 + i * NT);
    }
    const uint32_t at = yv >= v0 && (yv - v0) % NT == 0 ? (yv - v0) / NT : ~0u;
#pragma unroll
    for (int i = 0; i < NV; i += U)
      if (first + i * NT < cut.end) add_vecs<T, U>(r, raw + i, at - i, (y - cut.head) % K, a.c);
  }
  add_singles<T, NT>(r, row, cut, y, tid, a.c);
  join<NT>(r, a.c, sh);
  if (tid == 0) partial[blockIdx.x] = Partial{r.s, r.m};
}

template <typename T, Mode MODE>
__global__ __launch_bounds__(64) void join_kernel(const RowsArgs a, uint32_t parts, const Partial* partial) {
  __shared__ typename Team<64>::Shared sh;
  const uint32_t t = blockIdx.x, lane = threadIdx.x;
  const int64_t y64 = a.l.labels[t];
  PolicyIn in{};
  if (MODE == kPolicy && lane == 0) in = policy_in(a.p, t);
  RowEnd e;
  if (y64 < 0) {
    e.logp = e.lse = 0.0;
    e.state = RowState{0.0, 0.0f, 1.0f, 0.0f, 0};
  } else if (y64 >= (int64_t)a.l.vocab) {
    e = nan_row();
  } else {
    const float xy = (float)(static_cast<const T*>(a.l.x) + (uint64_t)t * a.l.x_stride)[y64];
    Running r;
    if (lane < parts) {
      const Partial p = partial[t * parts + lane];
      r.s = p.s;
      r.m = p.m;
    }
    join<64>(r, a.c, sh);
    if (lane == 0) e = finish_row(r.m, r.s, xy, a.c.inv_tau);
  }
  if (lane == 0) {
    a.logp[t] = (float)e.logp;
    if (MODE == kLogp && a.lse) a.lse[t] = (float)e.lse;
    if (MODE != kLogp) a.states[t] = e.state;
    if (MODE == kPairs) a.g[t] = 0.0f;
    if (MODE == kPolicy) a.g[t] = end_policy_row(a, t, in, e).g;
  }
}

// The policy loss of rows past 128 KiB, value and gradient. One workgroup of
// such a row fills a compute unit's registers if they are to hold it, and then
// nothing is read while it joins, and nothing written while it reads. So half
// as many threads keep RV vectors each in registers and LV in LDS, two rows to
// a compute unit, and what is past 16 * NT * (RV + LV) bytes is read a second
// time. 12822 x 131072 fp16: 1172 us (5.45 TB/s) against 1208 us with 1024
// threads of 16 vectors, 6100 x 100000 bf16: 353 us against 394 us; 4 or 8
// vectors in LDS 1172 and 1174, 362 and 359 us.
// All maxima of a chunk come before its sums; the label may be among them, for
// a sum is taken from any value near the row's maximum.
template <typename T, int NT, int RV, int LV>
__global__ __launch_bounds__(NT, NT / 128) void long_policy_kernel(const RowsArgs a) {
  constexpr int K = Io<T>::K;
  __shared__ typename Team<NT>::Shared sh;
  __shared__ u32x4 held[LV][NT];
  const uint32_t tid = threadIdx.x, vocab = a.l.vocab, t = a.first + blockIdx.x;
  const T* row = static_cast<const T*>(a.l.x) + (uint64_t)t * a.l.x_stride;
  T* out = static_cast<T*>(a.l.dx) + (uint64_t)t * a.l.dx_stride;
  const Cut<T, NT> cut(out, vocab);
  const T* vecs = row + cut.head;
  const uint32_t nv = cut.nv;
  const int64_t y64 = a.l.labels[t];
  const bool bad = y64 >= (int64_t)vocab;
  const uint32_t y = y64 < 0 || bad ? 0u : (uint32_t)y64, yv = cut.vec_of(y), el = (y - cut.head) % K;
  PolicyIn in{};
  if (tid == 0) in = policy_in(a.p, t);
  RowEnd e;
  u32x4 kept[RV];
  if (y64 < 0) {
    e.logp = e.lse = 0.0;
    e.state = RowState{0.0, 0.0f, 1.0f, 0.0f, 0};
  } else {
    const float xy = (float)row[y];
    Running r;
    auto sum = [&](u32x4 raw, uint32_t v) {
      float f[K];
      Io<T>::unpack(raw, f);
      if (__any(v == yv)) {
#pragma unroll
        for (int i = 0; i < K; ++i)
          if (v == yv && el == (uint32_t)i) f[i] = -kInf;
      }
      r.sum<K, Io<T>::kFloats>(f, a.c);
    };
    for (uint32_t v0 = (RV + LV) * NT; v0 < nv; v0 += LV * NT) {
      u32x4 raw[LV];
      float mx = -kInf;
#pragma unroll
      for (int i = 0; i < LV; ++i) {
        raw[i] = no_vec<T>();
        if (v0 + tid + i * NT < nv) raw[i] = load_vec<T, true>(vecs, v0 + tid + i * NT);
      }
#pragma unroll
      for (int i = 0; i < LV; ++i) mx = fmaxf(mx, vec_max<T>(raw[i]));
      r.raise(mx, a.c);
#pragma unroll
      for (int i = 0; i < LV; ++i) {
        opaque(raw[i]);
        if (v0 + i * NT < nv) sum(raw[i], v0 + tid + i * NT);
      }
    }
    {
      const uint32_t v0 = RV * NT;
      u32x4 raw[LV];
      float mx = -kInf;
#pragma unroll
      for (int i = 0; i < LV; ++i) {
        raw[i] = no_vec<T>();
        if (v0 + tid + i * NT < nv) raw[i] = load_vec(vecs + v0 * K + i * (NT * K), tid);
      }
#pragma unroll
      for (int i = 0; i < LV; ++i) mx = fmaxf(mx, vec_max<T>(raw[i]));
      r.raise(mx, a.c);
#pragma unroll
      for (int i = 0; i < LV; ++i) {
        opaque(raw[i]);
        held[i][tid] = raw[i];
        if (v0 + i * NT < nv) sum(raw[i], v0 + tid + i * NT);
      }
    }
    float mx = -kInf;
#pragma unroll
    for (int i = 0; i < RV; ++i) {
      kept[i] = no_vec<T>();
      if (tid + i * NT < nv) kept[i] = load_vec(vecs + i * (NT * K), tid);
    }
#pragma unroll
    for (int i = 0; i < RV; ++i) mx = fmaxf(mx, vec_max<T>(kept[i]));
    r.raise(mx, a.c);
#pragma unroll
    for (int i = 0; i < RV; ++i) {
      opaque(kept[i]);
      if (i * NT < nv) sum(kept[i], tid + i * NT);
    }
    add_singles<T, NT>(r, row, cut, y, tid, a.c);
    join<NT>(r, a.c, sh);
    if (tid == 0) e = bad ? nan_row() : finish_row(r.m, r.s, xy, a.c.inv_tau);
  }
  if (tid == 0) {
    a.logp[t] = (float)e.logp;
    sh.got = end_policy_row(a, t, in, e);
  }
  __syncthreads();
  const Slope k = sh.got;
  if (k.g == 0.0f) {
    zero_row<T, NT>(out, cut, tid);
    return;
  }
#pragma unroll
  for (int i = 0; i < RV; ++i) {
    opaque(kept[i]);
    if (tid + i * NT < nv)
      store_vec(out + cut.head + i * (NT * K), tid, grad_vec<T>(kept[i], k.top, a.c.k_hi, k.coef));
  }
#pragma unroll
  for (int i = 0; i < LV; ++i)
    if (tid + (RV + i) * NT < nv)
      store_vec(out + cut.head + (RV + i) * (NT * K), tid, grad_vec<T>(held[i][tid], k.top, a.c.k_hi, k.coef));
  if (nv > (RV + LV) * NT)
    grad_vecs<T, NT, 2>(vecs, out + cut.head, (RV + LV) * NT, nv, tid, k.top, a.c.k_hi, k.coef);
  grad_singles<T, NT>(row, out, cut, tid, k.top, a.c.k_hi, k.coef);
  if (tid == cut.owner(y)) out[y] = (T)k.at_label;  // after its neighbours, by the same thread
}

template <typename T>
__device__ __forceinline__ u32x4 backward_vec(u32x4 raw, const Scale& c, float lse, float g) {
  constexpr int K = Io<T>::K;
  float f[K];
  Io<T>::unpack(raw, f);
#pragma unroll
  for (int i = 0; i < K; ++i) f[i] = -g * exp2_fast(exponent(f[i], c, lse) * kLog2e);
  return Io<T>::pack(f);
}

// The gradient of the log-probabilities from the normalisers.
template <typename T, int NT>
__global__ __launch_bounds__(Team<NT>::kBlock) void backward_kernel(const Logits l, const Scale c, const float* lse,
                                                                    const float* g_rows, uint32_t parts, uint32_t first) {
  using Tm = Team<NT>;
  const uint32_t tid = Tm::thread();
  const uint32_t t = Tm::row(first, blockIdx.x / parts);
  if (t >= l.rows) return;
  const T* row = static_cast<const T*>(l.x) + (uint64_t)t * l.x_stride;
  T* out = static_cast<T*>(l.dx) + (uint64_t)t * l.dx_stride;
  const Cut<T, NT> cut(out, l.vocab, blockIdx.x % parts, Part<NT>::kVecs);
  const int64_t y64 = l.labels[t];
  const float z = lse[t];
  float g = (float)(g_rows[t] * c.inv_tau);
  if (y64 < 0 || z == -kInf || g == 0.0f) {
    zero_row<T, NT>(out, cut, tid);
    return;
  }
  if (y64 >= (int64_t)l.vocab) g = __builtin_nanf("");
  const uint32_t y = y64 >= (int64_t)l.vocab ? 0u : (uint32_t)y64;
  // the label's thread, the only one that writes its place, reads it first
  const uint32_t owner = cut.owner(y);
  const float fy = tid == owner ? (float)row[y] : 0.0f;
  for_vecs<T, NT, Part<NT>::kRounds>(row + cut.head, cut.begin, cut.end, tid, [&](u32x4 raw, uint32_t v) {
    store_vec(out + cut.head, v, backward_vec<T>(raw, c, z, g));
  });
  for (uint32_t j = tid; j < cut.singles(); j += NT) {
    const uint32_t i = cut.single(j);
    out[i] = (T)(-g * exp2_fast(exponent((float)row[i], c, z) * kLog2e));
  }
  if (tid == owner) out[y] = (T)(float)((double)g * rest_of_label(fy, c, z));
}

__device__ __forceinline__ void sequence(const Pairs& p, uint64_t s, uint32_t rows, uint32_t* begin, uint32_t* end) {
  const int64_t a = min(max(p.cu[s], (int64_t)0), (int64_t)rows);
  const int64_t b = min(max(p.cu[s + 1], (int64_t)0), (int64_t)rows);
  *begin = (uint32_t)a;
  *end = (uint32_t)(b < a ? a : b);
}

// One workgroup a pair: the rewards of its sequences, its loss, its rows'
// coefficients. Half of the threads take each sequence.
template <int NT>
__global__ __launch_bounds__(NT) void pairs_kernel(const Pairs p, uint32_t rows, const RowState* states, float* g,
                                                   double* losses) {
  __shared__ double sh[NT / 64];
  const uint32_t side = threadIdx.x / (NT / 2), tid = threadIdx.x % (NT / 2);
  for (uint32_t i = blockIdx.x; i < p.pairs; i += gridDim.x) {
    uint32_t begin, end;
    sequence(p, 2ull * i + side, rows, &begin, &end);
    double sum = 0.0;
    for (uint32_t t = begin + tid; t < end; t += NT / 2) {
      const RowState st = states[t];
      const double ref = p.ref ? (double)p.ref[t] : 0.0;
      if (st.counts) sum += st.logp - ref;
    }
#pragma unroll
    for (int w = 32; w > 0; w /= 2) sum += __shfl_xor(sum, w);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = sum;
    __syncthreads();
    double reward[2] = {0.0, 0.0};
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) reward[w / (NT / 128)] += sh[w];
    reward[0] *= p.beta;
    reward[1] *= p.beta;
    const double m = reward[0] - reward[1];
    // log(1 + e^-m), log(1 + e^m) and sigma(m) - 1 from e^-|m|
    const double e = exp_of(-fabs(m)), tail = log1p_of(e);
    const double below = (m >= 0.0 ? -e : -1.0) / (1.0 + e);
    const double c = p.beta * (below + p.smoothing) / p.pairs * p.grad_scale;
    for (uint32_t t = begin + tid; t < end; t += NT / 2) g[t] = (float)(side ? -c : c);
    if (threadIdx.x == 0) {
      const double down = fmax(-m, 0.0) + tail, up = fmax(m, 0.0) + tail;
      double loss = m == m ? 0.0 : m;
      if (p.smoothing != 1.0) loss += (1.0 - p.smoothing) * down;
      if (p.smoothing != 0.0) loss += p.smoothing * up;
      p.rewards[2ull * i] = (float)reward[0];
      p.rewards[2ull * i + 1] = (float)reward[1];
      p.losses[i] = (float)loss;
      losses[i] = loss;
    }
  }
}

// The mean of the pairs' losses, by one workgroup in a fixed order.
template <int NT>
__device__ __forceinline__ void mean_loss(const double* losses, uint32_t n, float* out, double* sh) {
  double sum = 0.0;
  for (uint32_t i = threadIdx.x; i < n; i += NT) sum += losses[i];
  sum = block_sum<NT>(sum, sh);
  if (threadIdx.x == 0) *out = n ? (float)(sum / n) : 0.0f;
}

template <int NT>
__global__ __launch_bounds__(NT) void mean_kernel(const double* losses, uint32_t n, float* out) {
  __shared__ double sh[NT / 64];
  mean_loss<NT>(losses, n, out, sh);
}

// The gradient of rows whose coefficients and statistics are known. The last
// workgroup of the launch has no rows: it takes the mean of the losses, which
// as a kernel of its own cost 5 us.
template <typename T, int NT>
__global__ __launch_bounds__(Team<NT>::kBlock) void grad_kernel(const Logits l, const Scale c, const RowState* states,
                                                                const float* g_rows, const double* losses,
                                                                uint32_t pairs, float* loss, uint32_t parts, uint32_t first) {
  using Tm = Team<NT>;
  if (loss && blockIdx.x == gridDim.x - 1) {
    __shared__ double sh[Tm::kBlock / 64];
    mean_loss<Tm::kBlock>(losses, pairs, loss, sh);
    return;
  }
  const uint32_t tid = Tm::thread();
  const uint32_t t = Tm::row(first, blockIdx.x / parts);
  if (t >= l.rows) return;
  const T* row = static_cast<const T*>(l.x) + (uint64_t)t * l.x_stride;
  T* out = static_cast<T*>(l.dx) + (uint64_t)t * l.dx_stride;
  const Cut<T, NT> cut(out, l.vocab, blockIdx.x % parts, Part<NT>::kVecs);
  const RowState st = states[t];
  const float gt = g_rows[t];
  const float g = st.counts ? gt : 0.0f;
  const int64_t y64 = l.labels[t];
  if (g == 0.0f) {
    zero_row<T, NT>(out, cut, tid);
    return;
  }
  const uint32_t y = y64 >= (int64_t)l.vocab ? 0u : (uint32_t)y64;
  const float coef = (float)(g * c.inv_tau) / st.total;
  grad_vecs<T, NT, Part<NT>::kRounds>(row + cut.head, out + cut.head, cut.begin, cut.end, tid, st.top, c.k_hi, coef);
  grad_singles<T, NT>(row, out, cut, tid, st.top, c.k_hi, coef);
  if (tid == cut.owner(y)) out[y] = (T)(float)(g * c.inv_tau * st.rest);
}

// The sum of the rows' terms, in 64 bits until the end: rewards of both signs
// leave little of it, and rounded terms would leave that wrong.
template <int NT>
__global__ __launch_bounds__(NT) void sum_kernel(const double* terms, uint32_t n, float* out) {
  __shared__ double sh[NT / 64];
  constexpr uint32_t U = 8;
  double sum = 0.0;
  for (uint64_t i = threadIdx.x; i < n; i += U * NT) {
    double v[U];
#pragma unroll
    for (uint32_t u = 0; u < U; ++u) v[u] = i + u * NT < n ? terms[i + u * NT] : 0.0;
#pragma unroll
    for (uint32_t u = 0; u < U; ++u) sum += v[u];
  }
  sum = block_sum<NT>(sum, sh);
  if (threadIdx.x == 0) *out = (float)sum;
}

// Whether logits are of a size that the caches hold a good part of.
bool cached(const Logits& l, uint64_t size) { return (uint64_t)l.rows * l.vocab * size <= (768ull << 20); }

template <typename T, int NT, int NV, Mode MODE, bool kKeep = MODE == kPairs>
hipError_t rows_n(RowsArgs a, hipStream_t s) {
  return for_rows<NT>(a.l.rows, 1, [&](uint32_t first, uint32_t grid) {
    a.first = first;
    rows_kernel<T, NT, NV, MODE, kKeep><<<grid, Team<NT>::kBlock, 0, s>>>(a);
  });
}

// The smallest team whose registers hold a row, or the largest where there are
// fewer rows than compute units; rows that no team holds twice over in a
// compute unit go by long_policy_kernel. With rows enough to fill the chip by
// waves of their own, teams are as small as their registers allow: more rows
// are on the way in a compute unit, and a wave waits for no other (bf16, larger
// team / smaller: log-probabilities of 30000 x 5000 79 / 59 us, of 20000 x
// 12000 124 / 77 us, of 60000 x 600 45 / 21 us; policy loss of 30000 x 2500
// 115 / 68 us, of 20000 x 12000 246 / 170 us).
template <typename T, Mode MODE>
hipError_t rows_t(const RowsArgs& a, hipStream_t s) {
  const uint32_t nv = a.l.vocab / Io<T>::K;
  if (nv <= 16 * 4) return rows_n<T, 16, 4, MODE>(a, s);
  if (a.l.rows >= kManyRows) {
    if (nv <= 16 * 8) return rows_n<T, 16, 8, MODE>(a, s);
    if (nv > 64 * 4 && nv <= 64 * 8) return rows_n<T, 64, 8, MODE>(a, s);
    if constexpr (MODE == kPolicy) {
      if (nv > 64 * 8 && nv <= 64 * 16) return rows_n<T, 64, 16, MODE>(a, s);
      if (nv > 64 * 16 && nv <= 128 * 16) return rows_n<T, 128, 16, MODE>(a, s);
      if (nv > 128 * 16 && nv <= 256 * 16) return rows_n<T, 256, 16, MODE>(a, s);
    } else {
      if (nv > 64 * 8 && nv <= 64 * 16) return rows_n<T, 64, 8, MODE>(a, s);
      if (nv > 64 * 16 && nv <= 128 * 16) return rows_n<T, 128, 8, MODE>(a, s);
    }
  }
  if (nv <= 64 * 4) return rows_n<T, 64, 4, MODE>(a, s);
  if (nv <= 256 * 4) return rows_n<T, 256, 4, MODE>(a, s);
  if constexpr (MODE == kPolicy) {
    if (nv > 512 * 16 && a.l.rows >= kFewRows && a.l.dx)
      return for_rows<512>(a.l.rows, 1, [&](uint32_t first, uint32_t grid) {
        RowsArgs slice = a;
        slice.first = first;
        long_policy_kernel<T, 512, 16, 6><<<grid, 512, 0, s>>>(slice);
      });
    if (nv > 512 * 16 || a.l.rows < kFewRows) return rows_n<T, 1024, 16, MODE>(a, s);
    if (nv > 512 * 8) return rows_n<T, 512, 16, MODE>(a, s);
  }
  if constexpr (MODE != kPolicy) {
    if (a.l.rows < kFewRows) return rows_n<T, 1024, 8, MODE>(a, s);
  }
  if constexpr (MODE == kPairs) {
    // far more than the caches hold is not left in them: 15251 x 131072 bf16
    // is read in 450 us against 500 us
    if (!cached(a.l, sizeof(T))) return rows_n<T, 512, 8, MODE, false>(a, s);
  }
  return rows_n<T, 512, 8, MODE>(a, s);
}

// Whether rows are shared by workgroups: so few that one to a row leaves most of
// the chip idle, and longer than one takes in a round. Calls, shared against
// not: log-probability of 1 x 262144 fp32 13.5 us against 21.3 us, policy loss
// 26.7 us against 54 us, of 32 x 200001 bf16 27.4 us against 33.6 us, but of 128 x
// 100000 fp32 33.8 us against 28.4 us.
bool shared_rows(const Logits& l) {
  return l.rows < kSharedRows && l.vocab / (l.kind == kF32 ? 4 : 8) > 1024 * 16;
}

template <typename T, Mode MODE>
hipError_t shared_t(const RowsArgs& a, Partial* partial, hipStream_t s) {
  const uint32_t nv = a.l.vocab / Io<T>::K, parts = std::min(nv / 2048, kMostParts), size = (nv - 1) / parts + 1;
  part_kernel<T><<<a.l.rows * parts, 256, 0, s>>>(a, parts, size, partial);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  join_kernel<T, MODE><<<a.l.rows, 64, 0, s>>>(a, parts, partial);
  return hipGetLastError();
}

template <Mode MODE>
hipError_t rows_d(const RowsArgs& a, Partial* partial, hipStream_t s) {
  if (shared_rows(a.l)) {
    if (a.l.kind == kF32) return shared_t<float, MODE>(a, partial, s);
    if (a.l.kind == kBF16) return shared_t<__bf16, MODE>(a, partial, s);
    return shared_t<_Float16, MODE>(a, partial, s);
  }
  if (a.l.kind == kF32) return rows_t<float, MODE>(a, s);
  if (a.l.kind == kBF16) return rows_t<__bf16, MODE>(a, s);
  return rows_t<_Float16, MODE>(a, s);
}

struct GradArgs {
  Logits l;
  Scale c;
  const RowState* states;
  const float* g;
  const double* losses;
  uint32_t pairs;
  float* loss;
};

template <typename T, int NT>
hipError_t grad_n(const GradArgs& a, hipStream_t s) {
  const uint32_t parts = Part<NT>::parts(a.l.vocab / Io<T>::K);
  return for_rows<NT>(a.l.rows, parts, [&](uint32_t first, uint32_t grid) {
    float* loss = first ? nullptr : a.loss;  // the first slice takes the mean
    grad_kernel<T, NT><<<grid + (loss ? 1 : 0), Team<NT>::kBlock, 0, s>>>(a.l, a.c, a.states, a.g, a.losses, a.pairs,
                                                                          loss, parts, first);
  });
}

template <typename T>
hipError_t grad_t(const GradArgs& a, hipStream_t s) {
  const uint32_t nv = a.l.vocab / Io<T>::K;
  if (nv <= 16 * 4) return grad_n<T, 16>(a, s);
  if (nv <= 64 * 8) return grad_n<T, 64>(a, s);
  if (nv <= 64 * 16) return grad_n<T, 128>(a, s);
  // Logits of which the caches still hold a good part after their first reading
  // come faster than memory gives them, and the smaller parts' number shows:
  // 4493 x 40009 fp16 (0.36 GB) 158 us against 151 us; far above, 15251 x
  // 131072 bf16 (4 GB), it is 1601 us against 1638 us.
  if (cached(a.l, sizeof(T))) return grad_n<T, 256>(a, s);
  return grad_n<T, 128>(a, s);
}

hipError_t grad_d(const GradArgs& a, hipStream_t s) {
  if (a.l.kind == kF32) return grad_t<float>(a, s);
  if (a.l.kind == kBF16) return grad_t<__bf16>(a, s);
  return grad_t<_Float16>(a, s);
}

template <typename T, int NT>
hipError_t backward_n(const Logits& l, const Scale& c, const float* lse, const float* g, hipStream_t s) {
  const uint32_t parts = Part<NT>::parts(l.vocab / Io<T>::K);
  return for_rows<NT>(l.rows, parts, [&](uint32_t first, uint32_t grid) {
    backward_kernel<T, NT><<<grid, Team<NT>::kBlock, 0, s>>>(l, c, lse, g, parts, first);
  });
}

template <typename T>
hipError_t backward_t(const Logits& l, const Scale& c, const float* lse, const float* g, hipStream_t s) {
  const uint32_t nv = l.vocab / Io<T>::K;
  if (nv <= 16 * 4) return backward_n<T, 16>(l, c, lse, g, s);
  if (nv <= 64 * 8) return backward_n<T, 64>(l, c, lse, g, s);
  return backward_n<T, 128>(l, c, lse, g, s);
}

// Gradient clipping.

constexpr int kClipThreads = 512;
constexpr uint32_t kClipBlocks = 1024;  // partial sums, and workgroups of a launch
constexpr uint64_t kKeepBytes = 192ull << 20;
constexpr uint32_t kDirect = 140;       // tensors that a launch's arguments hold (4 KB at most)
constexpr uint32_t kScaleBlocks = 8192;

// The list of tensors, in the kernel's arguments where it fits there. A longer
// one is carried to the workspace by upload_kernel, kDirect at a time: through
// arguments, not a copy, so that a captured call owns what it needs.
struct DirectList {
  uint64_t in[kDirect], out[kDirect], n[kDirect];  // n: the kind in the top byte
  uint32_t first[kDirect];

  void set(uint32_t i, const Tensor& t) {
    in[i] = reinterpret_cast<uint64_t>(t.in);
    out[i] = reinterpret_cast<uint64_t>(t.out);
    n[i] = t.n | (uint64_t)t.kind << 56;
    first[i] = t.first;
  }
  __device__ __forceinline__ Tensor at(uint32_t i) const {
    return Tensor{reinterpret_cast<const void*>(in[i]), reinterpret_cast<void*>(out[i]), n[i] & ((1ull << 56) - 1),
                  (uint32_t)(n[i] >> 56), first[i]};
  }
};

struct StoredList {
  const Tensor* t;
};

__global__ void upload_kernel(const DirectList list, Tensor* to, uint32_t n) {
  if (threadIdx.x < n) to[threadIdx.x] = list.at(threadIdx.x);
}

// The last of n tensors whose first chunk is `chunk` or an earlier one.
template <typename F>
__device__ __forceinline__ uint32_t find_tensor(uint32_t n, uint32_t chunk, F&& first) {
  uint32_t lo = 0, hi = n;
  while (hi - lo > 1) {
    const uint32_t mid = (lo + hi) / 2;
    if (first(mid) <= chunk)
      lo = mid;
    else
      hi = mid;
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

// Finds the tensor that holds a chunk. A workgroup keeps what the search reads
// in LDS: the whole list from the arguments, the first chunks of a stored list
// where they fit.
template <typename L>
struct Finder;

template <>
struct Finder<DirectList> {
  typedef Tensor Held[kDirect];
  const Tensor* held;
  uint32_t tensors;
  __device__ __forceinline__ Finder(const DirectList& list, uint32_t n, Held& lds) : held(lds), tensors(n) {
    if (threadIdx.x < n) lds[threadIdx.x] = list.at(threadIdx.x);
    __syncthreads();
  }
  __device__ __forceinline__ Tensor at(uint32_t chunk) const {
    return held[find_tensor(tensors, chunk, [&](uint32_t i) { return held[i].first; })];
  }
};

template <>
struct Finder<StoredList> {
  static constexpr uint32_t kHeld = 2048;
  typedef uint32_t Held[kHeld];
  const Tensor* list;
  const uint32_t* held;
  uint32_t tensors;
  __device__ __forceinline__ Finder(const StoredList& l, uint32_t n, Held& lds) : list(l.t), held(lds), tensors(n) {
    if (n <= kHeld)
      for (uint32_t i = threadIdx.x; i < n; i += kClipThreads) lds[i] = list[i].first;
    __syncthreads();
  }
  __device__ __forceinline__ Tensor at(uint32_t chunk) const {
    return list[find_tensor(tensors, chunk, [&](uint32_t i) { return tensors <= kHeld ? held[i] : list[i].first; })];
  }
};

// Squares are added in 64 bits: those of fp32 and bf16 gradients pass the range
// of 32 on both sides.
template <typename T, bool kKeep>
__device__ __forceinline__ double chunk_squares(const T* p, uint32_t n) {
  constexpr int K = Io<T>::K;
  double s = 0.0, s2 = 0.0;
  const Cut<T, kClipThreads> cut(p, n);
  for_vecs<T, kClipThreads, 4, kKeep>(p + cut.head, 0, cut.nv, threadIdx.x, [&](u32x4 raw, uint32_t) {
    float f[K];
    Io<T>::unpack(raw, f);
#pragma unroll
    for (int i = 0; i < K; i += 2) {
      s += (double)f[i] * (double)f[i];
      s2 += (double)f[i + 1] * (double)f[i + 1];
    }
  });
  if (threadIdx.x < cut.singles()) {
    const double f = (float)p[cut.single(threadIdx.x)];
    s += f * f;
  }
  return s + s2;
}

template <typename T>
__device__ __forceinline__ void chunk_scale(const T* p, T* q, uint32_t n, float c) {
  constexpr int K = Io<T>::K;
  const Cut<T, kClipThreads> cut(q, n);
  for_vecs<T, kClipThreads, 2>(p + cut.head, 0, cut.nv, threadIdx.x, [&](u32x4 raw, uint32_t v) {
    float f[K];
    Io<T>::unpack(raw, f);
#pragma unroll
    for (int i = 0; i < K; ++i) f[i] *= c;
    store_vec(q + cut.head, v, Io<T>::pack(f));
  });
  if (threadIdx.x < cut.singles()) {
    const uint32_t i = cut.single(threadIdx.x);
    q[i] = (T)((float)p[i] * c);
  }
}

// Chunks from `keep` on are left in the caches: the second pass begins there.
template <typename L>
__global__ __launch_bounds__(kClipThreads) void squares_kernel(const L list, uint32_t tensors, uint32_t chunks,
                                                               uint32_t keep, double* partial) {
  __shared__ double sh[kClipThreads / 64];
  __shared__ typename Finder<L>::Held held;
  const Finder<L> find(list, tensors, held);
  double s = 0.0;
  for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const Tensor x = find.at(c);
    const uint64_t at = (c - x.first) * chunk_elems(x.kind);
    const uint32_t n = (uint32_t)min(x.n - at, chunk_elems(x.kind));
    auto squares = [&](auto* p) {
      using T = std::remove_const_t<std::remove_pointer_t<decltype(p)>>;
      return c >= keep ? chunk_squares<T, true>(p + at, n) : chunk_squares<T, false>(p + at, n);
    };
    if (x.kind == kF32)
      s += squares(static_cast<const float*>(x.in));
    else if (x.kind == kBF16)
      s += squares(static_cast<const __bf16*>(x.in));
    else
      s += squares(static_cast<const _Float16*>(x.in));
  }
  s = block_sum<kClipThreads>(s, sh);
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

// Every workgroup adds the partial sums again, in the same order, which costs
// less than a launch between the two passes; then the chunks, last first.
template <typename L>
__global__ __launch_bounds__(kClipThreads) void scale_kernel(const L list, uint32_t tensors, uint32_t chunks,
                                                             uint32_t blocks, const double* partial, double max_norm,
                                                             float* norm) {
  __shared__ double sh[kClipThreads / 64];
  __shared__ typename Finder<L>::Held held;
  double s = 0.0;
  for (uint32_t i = threadIdx.x; i < blocks; i += kClipThreads) s += partial[i];
  const double total = sqrt(block_sum<kClipThreads>(s, sh));
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)total;
  const float k = (float)(total <= max_norm ? 1.0 : max_norm / total);
  const Finder<L> find(list, tensors, held);
  for (uint32_t r = blockIdx.x; r < chunks; r += gridDim.x) {
    const uint32_t c = chunks - 1 - r;
    const Tensor x = find.at(c);
    if (k == 1.0f && x.in == x.out) continue;
    const uint64_t at = (c - x.first) * chunk_elems(x.kind);
    const uint32_t n = (uint32_t)min(x.n - at, chunk_elems(x.kind));
    if (x.kind == kF32)
      chunk_scale(static_cast<const float*>(x.in) + at, static_cast<float*>(x.out) + at, n, k);
    else if (x.kind == kBF16)
      chunk_scale(static_cast<const __bf16*>(x.in) + at, static_cast<__bf16*>(x.out) + at, n, k);
    else
      chunk_scale(static_cast<const _Float16*>(x.in) + at, static_cast<_Float16*>(x.out) + at, n, k);
  }
}

template <typename L>
hipError_t clip_list(const L& list, uint32_t tensors, uint32_t chunks, uint32_t keep, double max_norm, float* norm,
                     double* partial, hipStream_t s) {
  const uint32_t blocks = std::min(chunks, kClipBlocks);
  if (blocks) {
    squares_kernel<<<blocks, kClipThreads, 0, s>>>(list, tensors, chunks, keep, partial);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  scale_kernel<<<std::max(std::min(chunks, kScaleBlocks), 1u), kClipThreads, 0, s>>>(list, tensors, chunks, blocks, partial, max_norm, norm);
  return hipGetLastError();
}

uint64_t partials(uint64_t rows) { return rows < kSharedRows ? rows * kMostParts : 0; }

}  // namespace

uint64_t workspace_bytes(uint64_t rows, uint64_t pairs, uint64_t tensors) {
  return up16(partials(rows) * sizeof(Partial)) + up16(rows * sizeof(RowState)) + up16(rows * 4) + up16(rows * 8) +
         up16(pairs * 8) + up16(tensors * sizeof(Tensor)) + kClipBlocks * 8;
}

uint64_t logprobs_workspace_bytes(const Logits& l) { return shared_rows(l) ? workspace_bytes(l.rows, 0, 0) : 0; }

hipError_t launch_logprobs(const Logits& l, float* logp, float* lse, void* ws, hipStream_t s) {
  Workspace w{static_cast<char*>(ws)};
  RowsArgs a{};
  a.l = l;
  a.c = make_scale(l.tau);
  a.logp = logp;
  a.lse = lse;
  return rows_d<kLogp>(a, w.take<Partial>(partials(l.rows)), s);
}

hipError_t launch_backward(const Logits& l, const float* lse, const float* g, hipStream_t s) {
  const Scale c = make_scale(l.tau);
  if (l.kind == kF32) return backward_t<float>(l, c, lse, g, s);
  if (l.kind == kBF16) return backward_t<__bf16>(l, c, lse, g, s);
  return backward_t<_Float16>(l, c, lse, g, s);
}

hipError_t launch_preference(const Logits& l, const Pairs& p, void* ws, hipStream_t s) {
  Workspace w{static_cast<char*>(ws)};
  Partial* partial = w.take<Partial>(partials(l.rows));
  RowState* states = w.take<RowState>(l.rows);
  float* g = w.take<float>(l.rows);
  double* losses = w.take<double>(p.pairs);
  hipError_t e = hipSuccess;
  if (l.rows) {
    RowsArgs a{};
    a.l = l;
    a.c = make_scale(l.tau);
    a.logp = p.logp;
    a.states = states;
    a.g = g;
    e = rows_d<kPairs>(a, partial, s);
    if (e != hipSuccess) return e;
  }
  if (p.pairs) {
    pairs_kernel<256><<<std::min<uint32_t>(p.pairs, 1u << 20), 256, 0, s>>>(p, l.rows, states, g, losses);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (!l.rows || !l.dx) {
    mean_kernel<256><<<1, 256, 0, s>>>(losses, p.pairs, p.loss);
    return hipGetLastError();
  }
  return grad_d(GradArgs{l, make_scale(l.tau), states, g, losses, p.pairs, p.loss}, s);
}

hipError_t launch_policy(const Logits& l, const Policy& p, void* ws, hipStream_t s) {
  Workspace w{static_cast<char*>(ws)};
  double* weighted = w.take<double>(l.rows);
  if (l.rows) {
    RowsArgs a{};
    a.l = l;
    a.c = make_scale(l.tau);
    a.logp = p.logp;
    a.p = p;
    a.weighted = weighted;
    Partial* partial = w.take<Partial>(partials(l.rows));
    a.states = w.take<RowState>(l.rows);
    a.g = w.take<float>(l.rows);
    hipError_t e = rows_d<kPolicy>(a, partial, s);
    if (e == hipSuccess && l.dx && shared_rows(l)) e = grad_d(GradArgs{l, a.c, a.states, a.g, nullptr, 0, nullptr}, s);
    if (e != hipSuccess) return e;
  }
  sum_kernel<1024><<<1, 1024, 0, s>>>(weighted, l.rows, p.loss);
  return hipGetLastError();
}

hipError_t launch_clip(Tensor* t, uint32_t tensors, double max_norm, float* norm, void* ws, hipStream_t s) {
  Workspace w{static_cast<char*>(ws)};
  Tensor* stored = w.take<Tensor>(tensors);
  double* partial = w.take<double>(kClipBlocks);
  uint32_t chunks = 0;
  for (uint32_t i = 0; i < tensors; ++i) {
    t[i].first = chunks;
    chunks += (uint32_t)((t[i].n - 1) / chunk_elems(t[i].kind) + 1);
  }
  // the last chunks that the memory-side cache can hold for the second pass
  const uint32_t keep = chunks - std::min<uint32_t>(chunks, kKeepBytes / kChunkBytes);
  DirectList direct{};
  for (uint32_t i = 0; i < tensors; i += kDirect) {
    const uint32_t n = std::min(kDirect, tensors - i);
    for (uint32_t j = 0; j < n; ++j) direct.set(j, t[i + j]);
    if (tensors <= kDirect) break;
    upload_kernel<<<1, 256, 0, s>>>(direct, stored + i, n);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (tensors <= kDirect) return clip_list(direct, tensors, chunks, keep, max_norm, norm, partial, s);
  return clip_list(StoredList{stored}, tensors, chunks, keep, max_norm, norm, partial, s);
}

}  // namespace hkvt
