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

// Running maximum and sum of the elements a thread has seen.
struct Running {
  float m = -kInf;
  double s = 0.0;

  template <int K>
  __device__ __forceinline__ void add(const float* f, const Scale& c) {
    float mx = f[0];
#pragma unroll
    for (int i = 1; i < K; ++i) mx = fmaxf(mx, f[i]);
    if (mx > m) {
      const float t = m - mx;
      s *= (double)exp2_fast(fmaf(t, c.k_hi, t * c.k_lo));
      m = mx;
    }
    const float base = m == -kInf ? 0.0f : m;
    float e[K];
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const float t = f[i] - base;
      e[i] = exp2_fast(fmaf(t, c.k_hi, t * c.k_lo));
    }
#pragma unroll
    for (int w = K / 2; w > 0; w /= 2)
#pragma unroll
      for (int i = 0; i < w; ++i) e[i] += e[i + w];
    s += (double)e[0];
  }
};

template <int NT>
struct Shared {
  float m[NT / 64];
  double s[NT / 64];
};

__device__ __forceinline__ double shfl_xor(double v, int mask) { return __shfl_xor(v, mask); }

// Joins the threads' running values; every thread gets the workgroup's.
template <int NT>
__device__ __forceinline__ void join(Running& r, const Scale& c, Shared<NT>& sh) {
  float m = r.m;
#pragma unroll
  for (int w = 32; w > 0; w /= 2) m = fmaxf(m, __shfl_xor(m, w));
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  __syncthreads();  // the last use of `sh` is over
  if (lane == 0) sh.m[wave] = m;
  __syncthreads();
  float top = -kInf;
#pragma unroll
  for (int w = 0; w < NT / 64; ++w) top = fmaxf(top, sh.m[w]);
  const float base = top == -kInf ? 0.0f : top;
  const float t = r.m - base;
  double s = r.s * (double)exp2_fast(fmaf(t, c.k_hi, t * c.k_lo));
#pragma unroll
  for (int w = 32; w > 0; w /= 2) s += shfl_xor(s, w);
  if (lane == 0) sh.s[wave] = s;
  __syncthreads();
  double all = 0.0;
#pragma unroll
  for (int w = 0; w < NT / 64; ++w) all += sh.s[w];
  r.m = top;
  r.s = all;
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

// Running values of one row, the label left out.
template <typename T, int NT>
__device__ __forceinline__ Running read_row(const T* row, uint32_t vocab, uint32_t y, const Scale& c) {
  constexpr int K = Io<T>::K;
  const uint32_t nv = vocab / K, yv = y / K;
  Running r;
  for (uint32_t v = threadIdx.x; v < nv; v += NT) {
    float f[K];
    Io<T>::unpack(*reinterpret_cast<const typename Io<T>::V*>(row + (uint64_t)v * K), f);
    if (v == yv) {
#pragma unroll
      for (int i = 0; i < K; ++i)
        if (i == (int)(y % K)) f[i] = -kInf;
    }
    r.add<K>(f, c);
  }
  const uint32_t i = nv * K + threadIdx.x;
  if (i < vocab && i != y) {
    const float f = (float)row[i];
    r.add<1>(&f, c);
  }
  return r;
}

// The row of the gradient: coef = g / (tau * total); at the label g * rest / tau.
template <typename T, int NT>
__device__ __forceinline__ void write_row(const T* row, T* out, uint32_t vocab, uint32_t y, float top, float k,
                                          float coef, float at_label) {
  constexpr int K = Io<T>::K;
  const uint32_t nv = vocab / K, yv = y / K;
  for (uint32_t v = threadIdx.x; v < nv; v += NT) {
    float f[K];
    Io<T>::unpack(*reinterpret_cast<const typename Io<T>::V*>(row + (uint64_t)v * K), f);
#pragma unroll
    for (int i = 0; i < K; ++i) f[i] = -coef * exp2_fast((f[i] - top) * k);
    if (v == yv) {
#pragma unroll
      for (int i = 0; i < K; ++i)
        if (i == (int)(y % K)) f[i] = at_label;
    }
    *reinterpret_cast<typename Io<T>::V*>(out + (uint64_t)v * K) = Io<T>::pack(f);
  }
  const uint32_t i = nv * K + threadIdx.x;
  if (i < vocab) out[i] = (T)(i == y ? at_label : -coef * exp2_fast(((float)row[i] - top) * k));
}

template <typename T, int NT>
__device__ __forceinline__ void zero_row(T* out, uint32_t vocab) {
  constexpr int K = Io<T>::K;
  const uint32_t nv = vocab / K;
  for (uint32_t v = threadIdx.x; v < nv; v += NT)
    *reinterpret_cast<typename Io<T>::V*>(out + (uint64_t)v * K) = u32x4{0, 0, 0, 0};
  const uint32_t i = nv * K + threadIdx.x;
  if (i < vocab) out[i] = (T)0.0f;
}

// Value and slope of one row of the policy loss.
struct PolicyRow {
  float loss, kl, g;
};

__device__ PolicyRow policy_row(const Policy& p, uint32_t t, double logp) {
  const double r = exp(logp - (double)p.old_logp[t]), a = p.advantages[t];
  const double free = r * a, bound = fmin(fmax(r, p.low), p.high) * a;
  double loss = -(free <= bound ? free : bound);
  double g = free <= bound ? -free : 0.0;
  if (!(free == free)) loss = g = free;
  double kl = 0.0;
  if (p.ref) {
    const double d = (double)p.ref[t] - logp, e = expm1(d);
    kl = e - d;
    if (p.kl_coef != 0.0) {
      loss += p.kl_coef * kl;
      g -= p.kl_coef * e;
    }
  }
  return PolicyRow{(float)loss, (float)kl, (float)(g * (double)p.weights[t] * p.grad_scale)};
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
};

// One workgroup a row: statistics, and for the policy loss, whose coefficient
// needs its own row alone, the gradient in the same kernel.
template <typename T, int NT, Mode MODE>
__global__ __launch_bounds__(NT) void rows_kernel(const RowsArgs a) {
  __shared__ Shared<NT> sh;
  __shared__ float got[4];
  for (uint32_t t = blockIdx.x; t < a.l.rows; t += gridDim.x) {
    const T* row = static_cast<const T*>(a.l.x) + (uint64_t)t * a.l.x_stride;
    const int64_t y = a.l.labels[t];
    RowEnd e;
    if (y < 0) {
      e.logp = e.lse = 0.0;
      e.state = RowState{0.0, 0.0f, 1.0f, 0.0f, 0};
    } else if (y >= (int64_t)a.l.vocab) {
      e = nan_row();
    } else {
      Running r = read_row<T, NT>(row, a.l.vocab, (uint32_t)y, a.c);
      join<NT>(r, a.c, sh);
      if (threadIdx.x == 0) e = finish_row(r.m, r.s, (float)row[y], a.c.inv_tau);
    }
    if (threadIdx.x == 0) {
      a.logp[t] = (float)e.logp;
      if (MODE == kLogp && a.lse) a.lse[t] = (float)e.lse;
      if (MODE == kPairs) {
        a.states[t] = e.state;
        a.g[t] = 0.0f;
      }
      if (MODE == kPolicy) {
        PolicyRow p{0.0f, 0.0f, 0.0f};
        if (e.state.counts) p = policy_row(a.p, t, e.logp);
        a.p.token_loss[t] = p.loss;
        a.p.kl[t] = p.kl;
        got[0] = p.g;
        got[1] = e.state.top;
        got[2] = (float)(p.g * a.c.inv_tau / e.state.total);
        got[3] = (float)(p.g * a.c.inv_tau * e.state.rest);
      }
    }
    if (MODE == kPolicy && a.l.dx) {
      __syncthreads();
      const float g = got[0], top = got[1], coef = got[2], at_label = got[3];
      T* out = static_cast<T*>(a.l.dx) + (uint64_t)t * a.l.dx_stride;
      if (g == 0.0f)
        zero_row<T, NT>(out, a.l.vocab);
      else
        write_row<T, NT>(row, out, a.l.vocab, y >= (int64_t)a.l.vocab ? 0u : (uint32_t)y, top, a.c.k_hi, coef,
                         at_label);
      __syncthreads();
    }
  }
}

// The gradient of rows whose coefficients and statistics are known.
template <typename T, int NT>
__global__ __launch_bounds__(NT) void grad_kernel(const Logits l, const Scale c, const RowState* states,
                                                  const float* g_rows) {
  for (uint32_t t = blockIdx.x; t < l.rows; t += gridDim.x) {
    const T* row = static_cast<const T*>(l.x) + (uint64_t)t * l.x_stride;
    T* out = static_cast<T*>(l.dx) + (uint64_t)t * l.dx_stride;
    const RowState st = states[t];
    const float g = st.counts ? g_rows[t] : 0.0f;
    const int64_t y = l.labels[t];
    if (g == 0.0f)
      zero_row<T, NT>(out, l.vocab);
    else
      write_row<T, NT>(row, out, l.vocab, y >= (int64_t)l.vocab ? 0u : (uint32_t)y, st.top, c.k_hi,
                       (float)(g * c.inv_tau / st.total), (float)(g * c.inv_tau * st.rest));
  }
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

// The gradient of the log-probabilities from the normalisers.
template <typename T, int NT>
__global__ __launch_bounds__(NT) void backward_kernel(const Logits l, const Scale c, const float* lse,
                                                      const float* g_rows) {
  constexpr int K = Io<T>::K;
  constexpr float kLog2e = 1.4426950408889634f;
  for (uint32_t t = blockIdx.x; t < l.rows; t += gridDim.x) {
    const T* row = static_cast<const T*>(l.x) + (uint64_t)t * l.x_stride;
    T* out = static_cast<T*>(l.dx) + (uint64_t)t * l.dx_stride;
    const int64_t yy = l.labels[t];
    const float z = lse[t];
    float g = (float)(g_rows[t] * c.inv_tau);
    if (yy < 0 || z == -kInf || g == 0.0f) {
      zero_row<T, NT>(out, l.vocab);
      continue;
    }
    if (yy >= (int64_t)l.vocab) g = __builtin_nanf("");
    const uint32_t y = yy >= (int64_t)l.vocab ? 0u : (uint32_t)yy;
    const uint32_t nv = l.vocab / K;
    for (uint32_t v = threadIdx.x; v < nv; v += NT) {
      float f[K];
      Io<T>::unpack(*reinterpret_cast<const typename Io<T>::V*>(row + (uint64_t)v * K), f);
      float fy = 0.0f;
      if (v == y / K) {
#pragma unroll
        for (int i = 0; i < K; ++i)
          if (i == (int)(y % K)) fy = f[i];
      }
#pragma unroll
      for (int i = 0; i < K; ++i) f[i] = -g * exp2_fast(exponent(f[i], c, z) * kLog2e);
      if (v == y / K) {
        const float at_label = (float)((double)g * rest_of_label(fy, c, z));
#pragma unroll
        for (int i = 0; i < K; ++i)
          if (i == (int)(y % K)) f[i] = at_label;
      }
      *reinterpret_cast<typename Io<T>::V*>(out + (uint64_t)v * K) = Io<T>::pack(f);
    }
    const uint32_t i = nv * K + threadIdx.x;
    if (i < l.vocab) {
      const float f = (float)row[i];
      out[i] = (T)(i == y ? (float)((double)g * rest_of_label(f, c, z))
                          : -g * exp2_fast(exponent(f, c, z) * kLog2e));
    }
  }
}

// Sum over a workgroup, in a fixed order; every thread gets it.
template <int NT>
__device__ __forceinline__ double block_sum(double v, double* sh) {
#pragma unroll
  for (int w = 32; w > 0; w /= 2) v += shfl_xor(v, w);
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
  double sum = 0.0;
  for (uint32_t i = threadIdx.x; i < n; i += NT) {
    const float l = loss[i];
    if (l != 0.0f) sum += (double)l * (double)weights[i];  // rows left out have 0, whatever their weight
  }
  sum = block_sum<NT>(sum, sh);
  if (threadIdx.x == 0) *out = (float)sum;
}

uint32_t row_grid(uint32_t rows) { return std::min<uint32_t>(rows, 1u << 20); }

template <typename T, Mode MODE>
hipError_t rows_t(const RowsArgs& a, hipStream_t s) {
  rows_kernel<T, 512, MODE><<<row_grid(a.l.rows), 512, 0, s>>>(a);
  return hipGetLastError();
}

template <Mode MODE>
hipError_t rows_d(const RowsArgs& a, hipStream_t s) {
  if (a.l.kind == kF32) return rows_t<float, MODE>(a, s);
  if (a.l.kind == kBF16) return rows_t<__bf16, MODE>(a, s);
  return rows_t<_Float16, MODE>(a, s);
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
  const uint32_t grid = row_grid(l.rows);
  if (l.kind == kF32)
    backward_kernel<float, 512><<<grid, 512, 0, s>>>(l, c, lse, g);
  else if (l.kind == kBF16)
    backward_kernel<__bf16, 512><<<grid, 512, 0, s>>>(l, c, lse, g);
  else
    backward_kernel<_Float16, 512><<<grid, 512, 0, s>>>(l, c, lse, g);
  return hipGetLastError();
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
  const uint32_t grid = row_grid(l.rows);
  if (l.kind == kF32)
    grad_kernel<float, 512><<<grid, 512, 0, s>>>(l, c, states, g);
  else if (l.kind == kBF16)
    grad_kernel<__bf16, 512><<<grid, 512, 0, s>>>(l, c, states, g);
  else
    grad_kernel<_Float16, 512><<<grid, 512, 0, s>>>(l, c, states, g);
  return hipGetLastError();
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
