// Device code that the kernels of the training operators share: elements of
// rows, how rows are cut and which threads serve them, exponentials and
// logarithms. For .hip files only; everything here is local to the file.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <limits>
#include <type_traits>

#include "hkv_train_internal.h"

namespace hkvt {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

constexpr float kInf = __builtin_inff();
constexpr float kLog2e = 1.4426950408889634f;
constexpr uint32_t kFewRows = 256;    // as many as there are compute units
constexpr uint32_t kSharedRows = 64;
constexpr uint32_t kManyRows = 4096;  // as many as there are places for waves of 128 registers

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// The bits of a word as another type. Takes a value: a bit cast applied to an
// element of a vector itself reads the vector's first element.
__device__ __forceinline__ float as_float(uint32_t u) { return __builtin_bit_cast(float, u); }
__device__ __forceinline__ f16x2 as_halves(uint32_t u) { return __builtin_bit_cast(f16x2, u); }

// 16 bytes of a row as floats and back. Rows begin at any element, so the
// 16-byte accesses are declared with the element's alignment: gfx950 takes
// them as single loads and stores at any such address.
// kFloats: how many exponentials at most are added in 32 bits before their sum
// goes on in 64. With fp32 elements memory leaves the time to add each of them
// in 64 bits (2047 x 50021: 47.8 us against 47.4 us), and log-probabilities
// before their last rounding are off (rms, in 2^-24, 8192 x 1000) by 0.16
// instead of 0.35 with sums of 16; the divergence of the policy loss, a
// difference of them, by 1.1e-7 of its size instead of 2.4e-7 (534 x 1000).
// 16-bit elements come twice as fast, and one by one would cost up to a third
// (3643 x 50021 bf16, policy loss: 145 us against 111 us); they are themselves
// rounded in their ninth or twelfth bit, which is far more than what the sums of
// 32 lose (0.40 instead of 0.20).
template <typename T>
struct Io;

template <>
struct Io<float> {
  static constexpr int K = 4, kFloats = 1;
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
  static constexpr int K = 8, kFloats = 32;
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
  static constexpr int K = 8, kFloats = 32;
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

inline void split(double v, float* hi, float* lo) {
  *hi = (float)v;
  if ((double)*hi >= v) *hi = std::nextafterf(*hi, 0.0f);
  *lo = std::max((float)(v - (double)*hi), std::numeric_limits<float>::denorm_min());
}

inline Scale make_scale(double tau) {
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
// (4493 x 40009 fp16, gradient: 148 us against 120 us).
// A team smaller than a wave, whose rows are short, cuts at the first element.
template <typename T, int NT>
struct Cut {
  static constexpr uint32_t K = Io<T>::K;
  uint32_t head, nv, vocab;
  uint32_t begin, end;  // the vectors of this part of the row
  bool first;           // the part that has the single elements
  // `part`: the vectors [part * size, (part + 1) * size) of the row alone.
  __device__ __forceinline__ Cut(const T* lines, uint32_t vocab_, uint32_t part = 0, uint32_t size = ~0u)
      : vocab(vocab_) {
    const uint32_t off = (uint32_t)(0 - reinterpret_cast<uintptr_t>(lines)) & 127u;
    head = NT < 64 ? 0 : min(off / (uint32_t)sizeof(T), vocab);
    nv = (vocab - head) / K;
    begin = min(part * size, nv);
    end = begin + min(size, nv - begin);
    first = part == 0;
  }
  // Single elements: the first part's.
  __device__ __forceinline__ uint32_t singles() const { return first ? vocab - nv * K : 0; }
  // Element of the j-th single one.
  __device__ __forceinline__ uint32_t single(uint32_t j) const { return j < head ? j : j + nv * K; }
  // Vector that holds element y; nv or more: y is a single one.
  __device__ __forceinline__ uint32_t vec_of(uint32_t y) const { return y < head ? ~0u : (y - head) / K; }
  // Thread that reads and writes element y; none of this part where it lies in another.
  __device__ __forceinline__ uint32_t owner(uint32_t y) const {
    const uint32_t v = vec_of(y);
    if (v < nv) return v >= begin && v < end ? (v - begin) % NT : ~0u;
    return first ? (y < head ? y : y - nv * K) % NT : ~0u;
  }
};

// Vectors of a row. A row's bytes are counted in 32 bits: a scalar base and one
// register of offset. What is read for the last time and what is written go
// past the caches (2047 x 50021 fp32: 49 us against 55 us); kKeep is for what a
// later kernel reads again: the preference loss's second reading finds up to
// 256 MB of it in the memory-side cache (7448 x 32768 bf16, 40% of the rows left
// out: 166 us against 195 us without, 191 us with both readings kept).
template <typename T, bool kKeep = false>
__device__ __forceinline__ u32x4 load_vec(const T* row, uint32_t v) {
  const auto* p = reinterpret_cast<const typename Io<T>::V*>(reinterpret_cast<const char*>(row) + v * 16u);
  if (kKeep) return *p;
  return __builtin_nontemporal_load(p);
}

template <typename T>
__device__ __forceinline__ void store_vec(T* row, uint32_t v, u32x4 x) {
  __builtin_nontemporal_store(x, reinterpret_cast<typename Io<T>::V*>(reinterpret_cast<char*>(row) + v * 16u));
}

// Calls use(vector, its number) for a thread's share of vectors first .. nv of
// a row, U of which are on the way at a time, in the last round too.
template <typename T, int NT, int U, bool kKeep = false, typename F>
__device__ __forceinline__ void for_vecs(const T* row, uint32_t first, uint32_t nv, uint32_t tid, F&& use) {
  for (uint32_t v = first + tid; v < nv; v += U * NT) {
    u32x4 raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (v + u * NT < nv) raw[u] = load_vec<T, kKeep>(row, v + u * NT);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (v + u * NT < nv) use(raw[u], v + u * NT);
  }
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

// What a row's gradient is written from: -coef 2^((x - top) k), at_label at the
// label; zeros where g is 0.
struct Slope {
  float g, top, coef, at_label;
};

// The threads that serve a row: a part of a wave, a wave, or a workgroup.
template <int NT>
struct Team {
  static constexpr int kBlock = NT < 128 ? 256 : NT;  // threads of the workgroup
  static constexpr int kRows = kBlock / NT;           // rows it works on at a time
  static constexpr int kWaves = NT > 64 ? NT / 64 : 1;
  struct Shared {
    float m[kWaves];
    double s[kWaves];
    Slope got;
  };
  static __device__ __forceinline__ uint32_t thread() { return threadIdx.x % NT; }
  // This team's row; the same in every lane where a wave has one row, and then
  // told to the compiler, which keeps addresses in scalar registers.
  static __device__ __forceinline__ uint32_t row(uint32_t first, uint32_t block) {
    const uint32_t r = first + block * kRows + threadIdx.x / NT;
    return NT >= 64 ? __builtin_amdgcn_readfirstlane(r) : r;
  }
};

// e^x to 1e-11: 2^n times the series of the rest, |u| < 0.35. What is left of a
// sum of losses of both signs may be a hundredth of them, and a ratio to a
// float's precision would then be wrong in its fifth digit.
__device__ __forceinline__ double exp_of(double x) {
  if (x > 709.0) return (double)kInf;
  if (x < -745.0) return 0.0;
  const double n = rint(x * 1.4426950408889634074);
  const double u = fma(n, -0.69314718055994530942, x);
  double s = 1.0 / 362880;
  s = fma(s, u, 1.0 / 40320);
  s = fma(s, u, 1.0 / 5040);
  s = fma(s, u, 1.0 / 720);
  s = fma(s, u, 1.0 / 120);
  s = fma(s, u, 1.0 / 24);
  s = fma(s, u, 1.0 / 6);
  s = fma(s, u, 0.5);
  s = fma(s, u, 1.0);
  s = fma(s, u, 1.0);
  return __builtin_ldexp(s, (int)n);
}

// The logarithm to 5e-10, as the row's end takes it: log m = 2 atanh z with
// z = (m - 1) / (m + 1), |z| < 0.172, whose series after its first term is taken
// in floats: it is at most 3.4e-3, and their roundings of it are what the bound
// is. (Of log(1 + u) for small u, 1.4e-9 of its size.) A row's sum is off by
// 1e-8. (The library's functions in 64 bits cost a row 2 us of one thread and
// more than a hundred registers of constants.)
__device__ __forceinline__ double log_from(int exponent, double z) {
  const float w = (float)(z * z);
  const float q = fmaf(w, fmaf(w, fmaf(w, fmaf(w, 1.0f / 11, 1.0f / 9), 1.0f / 7), 1.0f / 5), 1.0f / 3);
  return (double)exponent * 0.69314718055994530942 + 2.0 * (z + z * (double)(w * q));
}

__device__ __forceinline__ double log_of(double u) {
  double m = __builtin_amdgcn_frexp_mant(u);
  int e = __builtin_amdgcn_frexp_exp(u);
  if (m < 0.70710678) {
    m *= 2.0;
    e -= 1;
  }
  return log_from(e, (m - 1.0) / (m + 1.0));
}

// log(1 + u), u >= 0: of a small u every digit stays.
__device__ __forceinline__ double log1p_of(double u) { return u < 0.41 ? log_from(0, u / (2.0 + u)) : log_of(1.0 + u); }

// A vector of -inf, where a row has no more.
template <typename T>
__device__ __forceinline__ u32x4 no_vec() {
  float f[Io<T>::K];
#pragma unroll
  for (int i = 0; i < Io<T>::K; ++i) f[i] = -kInf;
  return Io<T>::pack(f);
}

template <typename T, int NT>
__device__ __forceinline__ void zero_row(T* out, const Cut<T, NT>& cut, uint32_t tid) {
  for (uint32_t v = cut.begin + tid; v < cut.end; v += NT) store_vec(out + cut.head, v, u32x4{0, 0, 0, 0});
  for (uint32_t j = tid; j < cut.singles(); j += NT) out[cut.single(j)] = (T)0.0f;
}

// The largest element of a vector.
template <typename T>
__device__ __forceinline__ float vec_max(u32x4 raw) {
  constexpr int K = Io<T>::K;
  if constexpr (std::is_same_v<T, _Float16>) {
    const f16x2 a = __builtin_elementwise_max(as_halves(raw[0]), as_halves(raw[1]));
    const f16x2 b = __builtin_elementwise_max(as_halves(raw[2]), as_halves(raw[3]));
    const f16x2 m = __builtin_elementwise_max(a, b);
    return fmaxf((float)m[0], (float)m[1]);
  } else {
    float f[K];
    Io<T>::unpack(raw, f);
    float m = f[0];
#pragma unroll
    for (int i = 1; i < K; ++i) m = fmaxf(m, f[i]);
    return m;
  }
}

// Keeps the compiler from holding on to a vector's unpacked elements, twice its
// size, between its uses.
__device__ __forceinline__ void opaque(u32x4& v) { asm volatile("" : "+v"(v)); }

// A row's gradient from known statistics is written by several workgroups, two
// vectors a thread each, next to each other in the launch: what is on the way
// at a time then lies close together in memory. 8192 x 65536 bf16: 298 us (6.3
// TB/s) in parts of 128 threads, 310 us of 256, 316 us of 512, 341 us with a
// workgroup a row, 339 us with the parts of a row far apart in the launch; 307
// and 323 us with one or four vectors a thread. Rows of up to 512 vectors have
// one part, a wave's or less (30000 x 2500 bf16: 54 us against 66 us).
template <int NT>
struct Part {
  static constexpr int kRounds = NT > 64 ? 2 : 4;
  static constexpr uint32_t kVecs = NT > 64 ? NT * kRounds : ~0u;
  static uint32_t parts(uint32_t nv) { return nv ? (nv - 1) / kVecs + 1 : 1; }
};

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

// launch(first row, workgroups) for slices of rows, of `parts` workgroups a
// team's rows, that keep a launch's threads under 2^32.
template <int NT, typename F>
hipError_t for_rows(uint32_t rows, uint32_t parts, F&& launch) {
  const uint64_t slice = std::max(1u, (1u << 21) / parts) * (uint64_t)Team<NT>::kRows;
  for (uint64_t first = 0; first < rows; first += slice) {
    const uint32_t n = (uint32_t)std::min<uint64_t>(rows - first, slice);
    launch((uint32_t)first, ((n - 1) / Team<NT>::kRows + 1) * parts);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

inline uint64_t up16(uint64_t b) { return (b + 15) & ~15ull; }

// A call's workspace, handed out from its beginning.
struct Workspace {
  char* at;
  template <typename T>
  T* take(uint64_t n) {
    T* p = reinterpret_cast<T*>(at);
    at += up16(n * sizeof(T));
    return p;
  }
};

}  // namespace
}  // namespace hkvt
