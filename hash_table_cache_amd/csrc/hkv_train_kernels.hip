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
// S is summed eight (four) neighbours at a time in 32 bits, those sums in 64.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "hkv_train_internal.h"

namespace hkvt {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

constexpr float kInf = __builtin_inff();
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// The bits of a word as another type. Takes a value: a bit cast applied to an
// element of a vector itself reads the vector's first element.
__device__ __forceinline__ float as_float(uint32_t u) { return __builtin_bit_cast(float, u); }
__device__ __forceinline__ f16x2 as_halves(uint32_t u) { return __builtin_bit_cast(f16x2, u); }

// 16 bytes of a row as floats and back. Rows begin at any element, so the
// 16-byte accesses are declared with the element's alignment: gfx950 takes
// them as single loads and stores at any such address.
template <typename T>
struct Io;

template <>
struct Io<float> {
  static constexpr int K = 4;
  typedef u32x4 V __attribute__((aligned(4)));
  static __device__ __forceinline__ void unpack(u32x4 v, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = as_float(v[i]);
  }
  static __device__ __forceinline__ u32x4 pack(const float* f) {
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __builtin_bit_cast(uint32_t, f[i]);
    return v;
  }
};

template <>
struct Io<__bf16> {
  static constexpr int K = 8;
  typedef u32x4 V __attribute__((aligned(2)));
  static __device__ __forceinline__ void unpack(u32x4 v, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = as_float(v[i] << 16);
      f[2 * i + 1] = as_float(v[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ u32x4 pack(const float* f) {
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x2 two = {f[2 * i], f[2 * i + 1]};
      v[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(two, bf16x2));
    }
    return v;
  }
};

template <>
struct Io<_Float16> {
  static constexpr int K = 8;
  typedef u32x4 V __attribute__((aligned(2)));
  static __device__ __forceinline__ void unpack(u32x4 v, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f16x2 two = as_halves(v[i]);
      f[2 * i] = (float)two[0];
      f[2 * i + 1] = (float)two[1];
    }
  }
  static __device__ __forceinline__ u32x4 pack(const float* f) {
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x2 two = {f[2 * i], f[2 * i + 1]};
      v[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(two, f16x2));
    }
    return v;
  }
};

// The constants of a call's exponentials, each as a float below the number and
// a second one for what is missing: a float alone is off by up to 2^-24 of the
// exponent, the same way in every element, which over the rows of a sequence
// adds up. The second part is above 0, so that an exponent of -inf stays one.
struct Scale {
  double tau, inv_tau;
  float k_hi, k_lo;    // log2(e) / tau
  float it_hi, it_lo;  // 1 / tau
};

void split(double v, float* hi, float* lo) {
  *hi = (float)v;
  if ((double)*hi >= v) *hi = std::nextafterf(*hi, 0.0f);
  *lo = (float)(v - (double)*hi);
}

Scale make_scale(double tau) {
  const double inv_tau = 1.0 / tau;
  Scale c;
  c.tau = tau;
  c.inv_tau = inv_tau;
  split(inv_tau * 1.4426950408889634074, &c.k_hi, &c.k_lo);
  split(inv_tau, &c.it_hi, &c.it_lo);
  return c;
}

// How a row of `vocab` elements is cut: single elements up to the first 128-byte
// line of the array it is written to (of the one it is read from where nothing
// is written), whole vectors, single elements after the last. Wave-wide stores
// then fill whole lines: with rows of an odd length cut from their own first
// element, lines that two waves share halves of cost a fifth of the rate
// (4514 x 40009 fp16, gradient: 148 us against 117 us).
// A team smaller than a wave, whose rows are short, cuts at the first element.
template <typename T, int NT>
struct Cut {
  static constexpr uint32_t K = Io<T>::K;
  uint32_t head, nv, vocab;
  __device__ __forceinline__ Cut(const T* lines, uint32_t vocab_) : vocab(vocab_) {
    const uint32_t off = (uint32_t)(0 - reinterpret_cast<uintptr_t>(lines)) & 127u;
    head = NT < 64 ? 0 : min(off / (uint32_t)sizeof(T), vocab);
    nv = (vocab - head) / K;
  }
  __device__ __forceinline__ uint32_t singles() const { return vocab - nv * K; }
  // Element of the j-th single one.
  __device__ __forceinline__ uint32_t single(uint32_t j) const { return j < head ? j : j + nv * K; }
  // Vector that holds element y; nv or more: y is a single one.
  __device__ __forceinline__ uint32_t vec_of(uint32_t y) const { return y < head ? ~0u : (y - head) / K; }
  // Thread that reads and writes element y.
  __device__ __forceinline__ uint32_t owner(uint32_t y) const {
    const uint32_t v = vec_of(y);
    return (v < nv ? v : y < head ? y : y - nv * K) % NT;
  }
};

// Vectors of a row, read once and not needed again by this kernel. A row's
// bytes are counted in 32 bits: a scalar base and one register of offset.
template <typename T>
__device__ __forceinline__ u32x4 load_vec(const T* row, uint32_t v) {
  return __builtin_nontemporal_load(
      reinterpret_cast<const typename Io<T>::V*>(reinterpret_cast<const char*>(row) + v * 16u));
}

template <typename T>
__device__ __forceinline__ void store_vec(T* row, uint32_t v, u32x4 x) {
  __builtin_nontemporal_store(x, reinterpret_cast<typename Io<T>::V*>(reinterpret_cast<char*>(row) + v * 16u));
}

// Running maximum and sum of the elements a thread has seen.
struct Running {
  float m = -kInf;
  double s = 0.0;

  // N elements: their maximum first, so that the sum is rescaled at most once
  // for all of them and, after the first few, by hardly any wave.
  template <int N>
  __device__ __forceinline__ void add(const float* f, const Scale& c) {
    float mx = f[0];
#pragma unroll
    for (int i = 1; i < N; ++i) mx = fmaxf(mx, f[i]);
    if (__any(mx > m)) {
      const float top = fmaxf(m, mx);
      const float t = top == -kInf ? 0.0f : m - top;
      s *= (double)exp2_fast(fmaf(t, c.k_hi, t * c.k_lo));
      m = top;
    }
    const float base = m == -kInf ? 0.0f : m;
    float e[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float t = f[i] - base;
      e[i] = exp2_fast(fmaf(t, c.k_hi, t * c.k_lo));
    }
#pragma unroll
    for (int w = N / 2; w > 0; w /= 2)
#pragma unroll
      for (int i = 0; i < w; ++i) e[i] += e[i + w];
    s += (double)e[0];
  }
};

// The threads that serve a row: a part of a wave, a wave, or a workgroup.
template <int NT>
struct Team {
  static constexpr int kBlock = NT < 256 ? 256 : NT;  // threads of the workgroup
  static constexpr int kRows = kBlock / NT;           // rows it works on at a time
  static constexpr int kWaves = NT > 64 ? NT / 64 : 1;
  struct Shared {
    float m[kWaves];
    double s[kWaves];
    float got[4];
  };
  static __device__ __forceinline__ uint32_t thread() { return threadIdx.x % NT; }
  // This team's row; the same in every lane where a wave has one row, and then
  // told to the compiler, which keeps addresses in scalar registers.
  static __device__ __forceinline__ uint32_t row(uint32_t first) {
    const uint32_t r = first + blockIdx.x * kRows + threadIdx.x / NT;
    return NT >= 64 ? __builtin_amdgcn_readfirstlane(r) : r;
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
__device__ RowEnd finish_row(float m, double s, float xy, double inv_tau) {
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
    const double er = s * exp(-d);
    r.logp = -log1p(er);
    r.lse = (double)xy * inv_tau - r.logp;
    r.state = RowState{r.logp, xy, (float)(1.0 + er), (float)(er / (1.0 + er)), 1};
  } else {
    const double total = s + exp(d);
    const double lt = log(total);
    r.logp = d - lt;
    r.lse = (double)m * inv_tau + lt;
    r.state = RowState{r.logp, m, (float)total, (float)(s / total), 1};
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
  r.add<N * K>(f, c);
}

// A vector of -inf, where a row has no more.
template <typename T>
__device__ __forceinline__ u32x4 no_vec() {
  float f[Io<T>::K];
#pragma unroll
  for (int i = 0; i < Io<T>::K; ++i) f[i] = -kInf;
  return Io<T>::pack(f);
}

template <typename T, int NT>
__device__ __forceinline__ void add_singles(Running& r, const T* row, const Cut<T, NT>& cut, uint32_t y, uint32_t tid,
                                            const Scale& c) {
  for (uint32_t j0 = 0; j0 < cut.singles(); j0 += NT) {
    const uint32_t j = j0 + tid, i = cut.single(j);
    float f = -kInf;
    if (j < cut.singles() && i != y) f = (float)row[i];
    r.add<1>(&f, c);
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
  uint32_t v = first + tid;
  for (; v + (U - 1) * NT < nv; v += U * NT) {
    u32x4 raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) raw[u] = load_vec(row, v + u * NT);
#pragma unroll
    for (int u = 0; u < U; ++u) store_vec(out, v + u * NT, grad_vec<T>(raw[u], top, k, coef));
  }
  for (; v < nv; v += NT) store_vec(out, v, grad_vec<T>(load_vec(row, v), top, k, coef));
}

template <typename T, int NT>
__device__ __forceinline__ void zero_row(T* out, const Cut<T, NT>& cut, uint32_t tid) {
  for (uint32_t v = tid; v < cut.nv; v += NT) store_vec(out + cut.head, v, u32x4{0, 0, 0, 0});
  for (uint32_t j = tid; j < cut.singles(); j += NT) out[cut.single(j)] = (T)0.0f;
}

// Value and slope of one row of the policy loss.
struct PolicyRow {
  float loss, kl, g;
};

// What it takes beside the logits, loaded before them.
struct PolicyIn {
  float old_logp, advantage, weight, ref;
};

__device__ PolicyRow policy_row(const Policy& p, const PolicyIn& in, double logp) {
  const double r = exp(logp - (double)in.old_logp), a = in.advantage;
  const double free = r * a, bound = fmin(fmax(r, p.low), p.high) * a;
  double loss = -(free <= bound ? free : bound);
  double g = free <= bound ? -free : 0.0;
  if (!(free == free)) loss = g = free;
  double kl = 0.0;
  if (p.ref) {
    const double d = (double)in.ref - logp, e = expm1(d);
    kl = e - d;
    if (p.kl_coef != 0.0) {
      loss += p.kl_coef * kl;
      g -= p.kl_coef * e;
    }
  }
  return PolicyRow{(float)loss, (float)kl, (float)(g * (double)in.weight * p.grad_scale)};
}

enum Mode { kLogp, kPairs, kPolicy };

struct RowsArgs {
  Logits l;
  Scale c;
  float* logp;
  float* lse;        // kLogp
  RowState* states;  // kPairs
  float* g;          // kPairs: the rows' coefficients, cleared here
  Policy p;          // kPolicy
  uint32_t first;    // row of the first team
};

// Statistics of rows, by a team of NT threads each, and for the policy loss,
// whose coefficient needs its own row alone, the gradient in the same kernel:
// the first NV vectors of every thread stay in registers from the one to the
// other, so that a row of up to 16 * NT * NV bytes is read once. Without a
// gradient the same registers hold what is in flight.
template <typename T, int NT, int NV, Mode MODE>
__global__ __launch_bounds__(Team<NT>::kBlock) void rows_kernel(const RowsArgs a) {
  using Tm = Team<NT>;
  constexpr int K = Io<T>::K;
  constexpr int U = NV > 8 ? 2 : 4;  // vectors summed at a time
  __shared__ typename Tm::Shared sh;
  const uint32_t tid = Tm::thread(), vocab = a.l.vocab;
  const uint32_t t = Tm::row(a.first);
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
  if (MODE == kPolicy && tid == 0) {
    in.old_logp = a.p.old_logp[t];
    in.advantage = a.p.advantages[t];
    in.weight = a.p.weights[t];
    if (a.p.ref) in.ref = a.p.ref[t];
  }
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
        if (v0 + i * NT < nv) kept[i] = load_vec(vecs, v0 + i * NT);
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
  PolicyRow p{0.0f, 0.0f, 0.0f};
  if (tid == 0) {
    a.logp[t] = (float)e.logp;
    if (MODE == kLogp && a.lse) a.lse[t] = (float)e.lse;
    if (MODE == kPairs) {
      a.states[t] = e.state;
      a.g[t] = 0.0f;
    }
    if (MODE == kPolicy) {
      if (e.state.counts) p = policy_row(a.p, in, e.logp);
      a.p.token_loss[t] = p.loss;
      a.p.kl[t] = p.kl;
    }
  }
  if (write) {
    float g = p.g, top = e.state.top;
    float coef = (float)(g * a.c.inv_tau / e.state.total), at_label = (float)(g * a.c.inv_tau * e.state.rest);
    if (NT > 64) {
      if (tid == 0) {
        sh.got[0] = g;
        sh.got[1] = top;
        sh.got[2] = coef;
        sh.got[3] = at_label;
      }
      __syncthreads();
      g = sh.got[0];
      top = sh.got[1];
      coef = sh.got[2];
      at_label = sh.got[3];
    } else {
      g = __shfl(g, 0, NT);
      top = __shfl(top, 0, NT);
      coef = __shfl(coef, 0, NT);
      at_label = __shfl(at_label, 0, NT);
    }
    if (g == 0.0f) {
      zero_row<T, NT>(out, cut, tid);
    } else {
      if (y64 >= (int64_t)vocab) {
#pragma unroll
        for (int i = 0; i < NV; ++i) kept[i] = u32x4{0, 0, 0, 0};  // NaN comes from the coefficient
      }
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (tid + i * NT < nv) store_vec(out + cut.head, tid + i * NT, grad_vec<T>(kept[i], top, a.c.k_hi, coef));
      if (nv > NT * NV) grad_vecs<T, NT, 4>(vecs, out + cut.head, NT * NV, nv, tid, top, a.c.k_hi, coef);
      grad_singles<T, NT>(row, out, cut, tid, top, a.c.k_hi, coef);
      if (tid == cut.owner(y)) out[y] = (T)at_label;  // after its neighbours, by the same thread
    }
  }
}

// The gradient of rows whose coefficients and statistics are known.
template <typename T, int NT>
__global__ __launch_bounds__(Team<NT>::kBlock) void grad_kernel(const Logits l, const Scale c, const RowState* states,
                                                                const float* g_rows, uint32_t first) {
  using Tm = Team<NT>;
  const uint32_t tid = Tm::thread();
  const uint32_t t = Tm::row(first);
  if (t >= l.rows) return;
  const T* row = static_cast<const T*>(l.x) + (uint64_t)t * l.x_stride;
  T* out = static_cast<T*>(l.dx) + (uint64_t)t * l.dx_stride;
  const Cut<T, NT> cut(out, l.vocab);
  const RowState st = states[t];
  const float g = st.counts ? g_rows[t] : 0.0f;
  const int64_t y64 = l.labels[t];
  if (g == 0.0f) {
    zero_row<T, NT>(out, cut, tid);
    return;
  }
  const uint32_t y = y64 >= (int64_t)l.vocab ? 0u : (uint32_t)y64;
  const float coef = (float)(g * c.inv_tau / st.total);
  grad_vecs<T, NT, 4>(row + cut.head, out + cut.head, 0, cut.nv, tid, st.top, c.k_hi, coef);
  grad_singles<T, NT>(row, out, cut, tid, st.top, c.k_hi, coef);
  if (tid == cut.owner(y)) out[y] = (T)(float)(g * c.inv_tau * st.rest);
}

// x / tau - lse: the first step cancels what the two have in common exactly,
// the second adds what 1 / tau lacks in a float. The exponent is at most the
// rounding of lse; where logits are so large (a row of the type's lowest value)
// that lse as a float does not tell their exponents any more, it is held to 1,
// so that no gradient becomes infinite. NaN stays.
__device__ __forceinline__ float exponent(float x, const Scale& c, float lse) {
  const float z = fmaf(x, c.it_lo, fmaf(x, c.it_hi, -lse));
  return z > 1.0f ? 1.0f : z;
}

// 1 - softmax at the label, from the same difference in 64 bits.
__device__ __forceinline__ double rest_of_label(float x, const Scale& c, float lse) {
  const double z = (double)x / c.tau - (double)lse;
  return -expm1(z > 1.0 ? 1.0 : z);
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
                                                                    const float* g_rows, uint32_t first) {
  using Tm = Team<NT>;
  constexpr int U = 4;
  const uint32_t tid = Tm::thread();
  const uint32_t t = Tm::row(first);
  if (t >= l.rows) return;
  const T* row = static_cast<const T*>(l.x) + (uint64_t)t * l.x_stride;
  T* out = static_cast<T*>(l.dx) + (uint64_t)t * l.dx_stride;
  const Cut<T, NT> cut(out, l.vocab);
  const uint32_t nv = cut.nv;
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
  const T* vecs = row + cut.head;
  uint32_t v = tid;
  for (; v + (U - 1) * NT < nv; v += U * NT) {
    u32x4 raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) raw[u] = load_vec(vecs, v + u * NT);
#pragma unroll
    for (int u = 0; u < U; ++u) store_vec(out + cut.head, v + u * NT, backward_vec<T>(raw[u], c, z, g));
  }
  for (; v < nv; v += NT) store_vec(out + cut.head, v, backward_vec<T>(load_vec(vecs, v), c, z, g));
  for (uint32_t j = tid; j < cut.singles(); j += NT) {
    const uint32_t i = cut.single(j);
    out[i] = (T)(-g * exp2_fast(exponent((float)row[i], c, z) * kLog2e));
  }
  if (tid == owner) out[y] = (T)(float)((double)g * rest_of_label(fy, c, z));
}

// Sum over a workgroup, in a fixed order; every thread gets it.
template <int NT>
__device__ __forceinline__ double block_sum(double v, double* sh) {
#pragma unroll
  for (int w = 32; w > 0; w /= 2) v += __shfl_xor(v, w);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
  __syncthreads();
  double all = 0.0;
#pragma unroll
  for (int w = 0; w < NT / 64; ++w) all += sh[w];
  return all;
}

__device__ __forceinline__ void sequence(const Pairs& p, uint64_t s, uint32_t rows, uint32_t* begin, uint32_t* end) {
  const int64_t a = min(max(p.cu[s], (int64_t)0), (int64_t)rows);
  const int64_t b = min(max(p.cu[s + 1], (int64_t)0), (int64_t)rows);
  *begin = (uint32_t)a;
  *end = (uint32_t)(b < a ? a : b);
}

// One workgroup a pair: the rewards of its sequences, its loss, its rows' coefficients.
template <int NT>
__global__ __launch_bounds__(NT) void pairs_kernel(const Pairs p, uint32_t rows, const RowState* states, float* g,
                                                   double* losses) {
  __shared__ double sh[NT / 64];
  for (uint32_t i = blockIdx.x; i < p.pairs; i += gridDim.x) {
    double reward[2];
    uint32_t begin[2], end[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      sequence(p, 2ull * i + s, rows, &begin[s], &end[s]);
      double sum = 0.0;
      for (uint32_t t = begin[s] + threadIdx.x; t < end[s]; t += NT)
        if (states[t].counts) sum += states[t].logp - (p.ref ? (double)p.ref[t] : 0.0);
      reward[s] = p.beta * block_sum<NT>(sum, sh);
    }
    const double m = reward[0] - reward[1];
    // log(1 + e^-m) and log(1 + e^m), sigma(m)
    const double tail = log1p(exp(-fabs(m)));
    const double down = fmax(-m, 0.0) + tail, up = fmax(m, 0.0) + tail;
    double loss = m == m ? 0.0 : m;
    if (p.smoothing != 1.0) loss += (1.0 - p.smoothing) * down;
    if (p.smoothing != 0.0) loss += p.smoothing * up;
    const double slope = 1.0 / (1.0 + exp(-m)) - 1.0 + p.smoothing;
    const double c = p.beta * slope / p.pairs * p.grad_scale;
    if (threadIdx.x == 0) {
      p.rewards[2ull * i] = (float)reward[0];
      p.rewards[2ull * i + 1] = (float)reward[1];
      p.losses[i] = (float)loss;
      losses[i] = loss;
    }
#pragma unroll
    for (int s = 0; s < 2; ++s)
      for (uint32_t t = begin[s] + threadIdx.x; t < end[s]; t += NT) g[t] = (float)(s ? -c : c);
  }
}

// loss = scale * sum of losses, by one workgroup in a fixed order.
template <int NT>
__global__ __launch_bounds__(NT) void mean_kernel(const double* losses, uint32_t n, float* out) {
  __shared__ double sh[NT / 64];
  double sum = 0.0;
  for (uint32_t i = threadIdx.x; i < n; i += NT) sum += losses[i];
  sum = block_sum<NT>(sum, sh);
  if (threadIdx.x == 0) *out = n ? (float)(sum / n) : 0.0f;
}

template <int NT>
__global__ __launch_bounds__(NT) void weighted_sum_kernel(const float* loss, const float* weights, uint32_t n,
                                                          float* out) {
  __shared__ double sh[NT / 64];
  constexpr uint32_t U = 8;
  double sum = 0.0;
  for (uint64_t i = threadIdx.x; i < n; i += U * NT) {
    float l[U], w[U];
#pragma unroll
    for (uint32_t u = 0; u < U; ++u) {
      l[u] = w[u] = 0.0f;
      if (i + u * NT < n) {
        l[u] = loss[i + u * NT];
        w[u] = weights[i + u * NT];
      }
    }
#pragma unroll
    for (uint32_t u = 0; u < U; ++u)
      if (l[u] != 0.0f) sum += (double)l[u] * (double)w[u];  // rows left out have 0, whatever their weight
  }
  sum = block_sum<NT>(sum, sh);
  if (threadIdx.x == 0) *out = (float)sum;
}

// One team a row: launch(first row, workgroups) for slices of rows that keep a
// launch's threads under 2^32.
template <int NT, typename F>
hipError_t for_rows(uint32_t rows, F&& launch) {
  constexpr uint32_t kSlice = (1u << 21) * Team<NT>::kRows;
  for (uint64_t first = 0; first < rows; first += kSlice) {
    const uint32_t n = (uint32_t)std::min<uint64_t>(rows - first, kSlice);
    launch((uint32_t)first, (n - 1) / Team<NT>::kRows + 1);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename T, int NT, int NV, Mode MODE>
hipError_t rows_n(RowsArgs a, hipStream_t s) {
  return for_rows<NT>(a.l.rows, [&](uint32_t first, uint32_t grid) {
    a.first = first;
    rows_kernel<T, NT, NV, MODE><<<grid, Team<NT>::kBlock, 0, s>>>(a);
  });
}

// The smallest team whose registers hold a row.
template <typename T, Mode MODE>
hipError_t rows_t(const RowsArgs& a, hipStream_t s) {
  const uint32_t nv = a.l.vocab / Io<T>::K;
  if (nv <= 16 * 4) return rows_n<T, 16, 4, MODE>(a, s);
  if (nv <= 64 * 4) return rows_n<T, 64, 4, MODE>(a, s);
  if (nv <= 256 * 4) return rows_n<T, 256, 4, MODE>(a, s);
  if constexpr (MODE == kPolicy) {
    if (nv > 512 * 16) return rows_n<T, 1024, 16, MODE>(a, s);
    if (nv > 512 * 8) return rows_n<T, 512, 16, MODE>(a, s);
  }
  return rows_n<T, 512, 8, MODE>(a, s);
}

template <Mode MODE>
hipError_t rows_d(const RowsArgs& a, hipStream_t s) {
  if (a.l.kind == kF32) return rows_t<float, MODE>(a, s);
  if (a.l.kind == kBF16) return rows_t<__bf16, MODE>(a, s);
  return rows_t<_Float16, MODE>(a, s);
}

template <typename T, int NT>
hipError_t grad_n(const Logits& l, const Scale& c, const RowState* states, const float* g, hipStream_t s) {
  return for_rows<NT>(l.rows, [&](uint32_t first, uint32_t grid) {
    grad_kernel<T, NT><<<grid, Team<NT>::kBlock, 0, s>>>(l, c, states, g, first);
  });
}

template <typename T>
hipError_t grad_t(const Logits& l, const Scale& c, const RowState* states, const float* g, hipStream_t s) {
  const uint32_t nv = l.vocab / Io<T>::K;
  if (nv <= 16 * 4) return grad_n<T, 16>(l, c, states, g, s);
  if (nv <= 64 * 4) return grad_n<T, 64>(l, c, states, g, s);
  return grad_n<T, 512>(l, c, states, g, s);
}

template <typename T, int NT>
hipError_t backward_n(const Logits& l, const Scale& c, const float* lse, const float* g, hipStream_t s) {
  return for_rows<NT>(l.rows, [&](uint32_t first, uint32_t grid) {
    backward_kernel<T, NT><<<grid, Team<NT>::kBlock, 0, s>>>(l, c, lse, g, first);
  });
}

template <typename T>
hipError_t backward_t(const Logits& l, const Scale& c, const float* lse, const float* g, hipStream_t s) {
  const uint32_t nv = l.vocab / Io<T>::K;
  if (nv <= 16 * 4) return backward_n<T, 16>(l, c, lse, g, s);
  if (nv <= 64 * 4) return backward_n<T, 64>(l, c, lse, g, s);
  return backward_n<T, 512>(l, c, lse, g, s);
}

// Gradient clipping.

constexpr int kClipThreads = 512;
constexpr uint32_t kClipBlocks = 1024;
constexpr int kUpload = 100;  // tensors a launch's arguments carry

struct Upload {
  Tensor t[kUpload];
};

__global__ void upload_kernel(const Upload u, Tensor* to, uint32_t n) {
  if (threadIdx.x < n) to[threadIdx.x] = u.t[threadIdx.x];
}

// The tensor that holds chunk c.
__device__ __forceinline__ uint32_t find_tensor(const Tensor* t, uint32_t tensors, uint32_t c) {
  uint32_t lo = 0, hi = tensors;
  while (hi - lo > 1) {
    const uint32_t mid = (lo + hi) / 2;
    if (t[mid].first <= c)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// Squares in 64 bits: those of fp32 and bf16 gradients pass the range of 32.
template <typename T>
__device__ __forceinline__ double chunk_squares(const T* p, uint32_t n) {
  constexpr int K = Io<T>::K;
  double s = 0.0;
  const uint32_t nv = n / K;
  for (uint32_t v = threadIdx.x; v < nv; v += kClipThreads) {
    float f[K];
    Io<T>::unpack(*reinterpret_cast<const typename Io<T>::V*>(p + v * K), f);
#pragma unroll
    for (int i = 0; i < K; ++i) s += (double)f[i] * (double)f[i];
  }
  const uint32_t i = nv * K + threadIdx.x;
  if (i < n) s += (double)(float)p[i] * (double)(float)p[i];
  return s;
}

template <typename T>
__device__ __forceinline__ void chunk_scale(const T* p, T* q, uint32_t n, float c) {
  constexpr int K = Io<T>::K;
  const uint32_t nv = n / K;
  for (uint32_t v = threadIdx.x; v < nv; v += kClipThreads) {
    float f[K];
    Io<T>::unpack(*reinterpret_cast<const typename Io<T>::V*>(p + v * K), f);
#pragma unroll
    for (int i = 0; i < K; ++i) f[i] *= c;
    *reinterpret_cast<typename Io<T>::V*>(q + v * K) = Io<T>::pack(f);
  }
  const uint32_t i = nv * K + threadIdx.x;
  if (i < n) q[i] = (T)((float)p[i] * c);
}

__global__ __launch_bounds__(kClipThreads) void squares_kernel(const Tensor* t, uint32_t tensors, uint32_t chunks,
                                                               double* partial) {
  __shared__ double sh[kClipThreads / 64];
  double s = 0.0;
  for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const Tensor x = t[find_tensor(t, tensors, c)];
    const uint64_t at = (uint64_t)(c - x.first) * kChunkElems;
    const uint32_t n = (uint32_t)min(x.n - at, kChunkElems);
    if (x.kind == kF32)
      s += chunk_squares(static_cast<const float*>(x.in) + at, n);
    else if (x.kind == kBF16)
      s += chunk_squares(static_cast<const __bf16*>(x.in) + at, n);
    else
      s += chunk_squares(static_cast<const _Float16*>(x.in) + at, n);
  }
  s = block_sum<kClipThreads>(s, sh);
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

__global__ __launch_bounds__(kClipThreads) void norm_kernel(const double* partial, uint32_t blocks, double max_norm,
                                                            float* norm, double* coef) {
  __shared__ double sh[kClipThreads / 64];
  double s = 0.0;
  for (uint32_t i = threadIdx.x; i < blocks; i += kClipThreads) s += partial[i];
  s = block_sum<kClipThreads>(s, sh);
  if (threadIdx.x == 0) {
    const double n = sqrt(s);
    *norm = (float)n;
    *coef = n <= max_norm ? 1.0 : max_norm / n;
  }
}

__global__ __launch_bounds__(kClipThreads) void scale_kernel(const Tensor* t, uint32_t tensors, uint32_t chunks,
                                                             const double* coef) {
  const float k = (float)*coef;
  for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const Tensor x = t[find_tensor(t, tensors, c)];
    if (k == 1.0f && x.in == x.out) continue;
    const uint64_t at = (uint64_t)(c - x.first) * kChunkElems;
    const uint32_t n = (uint32_t)min(x.n - at, kChunkElems);
    if (x.kind == kF32)
      chunk_scale(static_cast<const float*>(x.in) + at, static_cast<float*>(x.out) + at, n, k);
    else if (x.kind == kBF16)
      chunk_scale(static_cast<const __bf16*>(x.in) + at, static_cast<__bf16*>(x.out) + at, n, k);
    else
      chunk_scale(static_cast<const _Float16*>(x.in) + at, static_cast<_Float16*>(x.out) + at, n, k);
  }
}

uint64_t up16(uint64_t b) { return (b + 15) & ~15ull; }

}  // namespace

uint64_t workspace_bytes(uint64_t rows, uint64_t pairs, uint64_t tensors) {
  return up16(rows * sizeof(RowState)) + up16(rows * 4) + up16(pairs * 8) + up16(tensors * sizeof(Tensor)) +
         kClipBlocks * 8 + 16;
}

hipError_t launch_logprobs(const Logits& l, float* logp, float* lse, void*, hipStream_t s) {
  RowsArgs a{};
  a.l = l;
  a.c = make_scale(l.tau);
  a.logp = logp;
  a.lse = lse;
  return rows_d<kLogp>(a, s);
}

hipError_t launch_backward(const Logits& l, const float* lse, const float* g, hipStream_t s) {
  const Scale c = make_scale(l.tau);
  if (l.kind == kF32) return backward_t<float>(l, c, lse, g, s);
  if (l.kind == kBF16) return backward_t<__bf16>(l, c, lse, g, s);
  return backward_t<_Float16>(l, c, lse, g, s);
}

hipError_t launch_preference(const Logits& l, const Pairs& p, void* ws, hipStream_t s) {
  char* at = static_cast<char*>(ws);
  RowState* states = reinterpret_cast<RowState*>(at);
  at += up16((uint64_t)l.rows * sizeof(RowState));
  float* g = reinterpret_cast<float*>(at);
  at += up16((uint64_t)l.rows * 4);
  double* losses = reinterpret_cast<double*>(at);
  hipError_t e = hipSuccess;
  if (l.rows) {
    RowsArgs a{};
    a.l = l;
    a.c = make_scale(l.tau);
    a.logp = p.logp;
    a.states = states;
    a.g = g;
    e = rows_d<kPairs>(a, s);
    if (e != hipSuccess) return e;
  }
  if (p.pairs) {
    pairs_kernel<256><<<std::min<uint32_t>(p.pairs, 1u << 20), 256, 0, s>>>(p, l.rows, states, g, losses);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  mean_kernel<256><<<1, 256, 0, s>>>(losses, p.pairs, p.loss);
  if ((e = hipGetLastError()) != hipSuccess || !l.rows || !l.dx) return e;
  const Scale c = make_scale(l.tau);
  if (l.kind == kF32) return grad_t<float>(l, c, states, g, s);
  if (l.kind == kBF16) return grad_t<__bf16>(l, c, states, g, s);
  return grad_t<_Float16>(l, c, states, g, s);
}

hipError_t launch_policy(const Logits& l, const Policy& p, void*, hipStream_t s) {
  if (l.rows) {
    RowsArgs a{};
    a.l = l;
    a.c = make_scale(l.tau);
    a.logp = p.logp;
    a.p = p;
    const hipError_t e = rows_d<kPolicy>(a, s);
    if (e != hipSuccess) return e;
  }
  weighted_sum_kernel<1024><<<1, 1024, 0, s>>>(p.token_loss, p.weights, l.rows, p.loss);
  return hipGetLastError();
}

hipError_t launch_clip(Tensor* t, uint32_t tensors, double max_norm, float* norm, void* ws, hipStream_t s) {
  char* at = static_cast<char*>(ws);
  Tensor* list = reinterpret_cast<Tensor*>(at);
  at += up16((uint64_t)tensors * sizeof(Tensor));
  double* partial = reinterpret_cast<double*>(at);
  double* coef = partial + kClipBlocks;
  uint32_t chunks = 0;
  for (uint32_t i = 0; i < tensors; ++i) {
    t[i].first = chunks;
    chunks += (uint32_t)((t[i].n + kChunkElems - 1) / kChunkElems);
  }
  hipError_t e = hipSuccess;
  for (uint32_t i = 0; i < tensors; i += kUpload) {
    const uint32_t n = std::min<uint32_t>(kUpload, tensors - i);
    Upload u{};
    std::copy(t + i, t + i + n, u.t);
    upload_kernel<<<1, 128, 0, s>>>(u, list + i, n);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  const uint32_t blocks = std::min(chunks, kClipBlocks);
  if (blocks) {
    squares_kernel<<<blocks, kClipThreads, 0, s>>>(list, tensors, chunks, partial);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  norm_kernel<<<1, kClipThreads, 0, s>>>(partial, blocks, max_norm, norm, coef);
  if ((e = hipGetLastError()) != hipSuccess || !blocks) return e;
  scale_kernel<<<blocks, kClipThreads, 0, s>>>(list, tensors, chunks, coef);
  return hipGetLastError();
}

}  // namespace hkvt
