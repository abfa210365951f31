// Device code that the kernels of matrices share: elements of any type, the update
// and its norm. For .hip files only; everything here is local to the file.
#pragma once

#include "hkv_train_rows.h"

namespace hkvt {
namespace {

typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr float kUnit = 4096.0f;  // what 1 is held as
constexpr int kPolarThreads = 256;
constexpr uint32_t kNormParts = 1024;  // partial sums of a matrix at most
constexpr uint32_t kNormRows = 16, kNormCols = 256;
// The last of n items whose first workgroup is `block` or an earlier one.
template <typename Item>
__device__ __forceinline__ const Item& find_item(const Item* items, uint32_t n, uint32_t block, uint32_t Item::* first) {
  uint32_t lo = 0, hi = n;
  while (hi - lo > 1) {
    const uint32_t mid = (lo + hi) / 2;
    if (items[mid].*first <= block)
      lo = mid;
    else
      hi = mid;
  }
  return items[__builtin_amdgcn_readfirstlane(lo)];
}

// Up to four elements next to each other, of a matrix of any type, as floats and
// back. Rows begin at any element: single accesses of 16 or 8 bytes at such
// addresses are gfx950's.
typedef u32x4 Quad32 __attribute__((aligned(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 Quad16 __attribute__((aligned(2)));

template <typename T>
__device__ __forceinline__ void load_few(const T* p, uint32_t n, float* v) {
  if (n == 4) {
    if constexpr (sizeof(T) == 4) {
      const u32x4 x = *reinterpret_cast<const Quad32*>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = as_float(x[i]);
    } else {
      const u32x2 x = *reinterpret_cast<const Quad16*>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint16_t h = (uint16_t)(x[i / 2] >> (i % 2 * 16));
        v[i] = (float)__builtin_bit_cast(T, h);
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = (uint32_t)i < n ? (float)p[i] : 0.0f;
}

template <typename T>
__device__ __forceinline__ void store_few(T* p, uint32_t n, const float* v) {
  if (n == 4) {
    if constexpr (sizeof(T) == 4) {
      u32x4 x;
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = __builtin_bit_cast(uint32_t, v[i]);
      *reinterpret_cast<Quad32*>(p) = x;
    } else {
      u32x2 x{0, 0};
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i / 2] |= (uint32_t)__builtin_bit_cast(uint16_t, (T)v[i]) << (i % 2 * 16);
      *reinterpret_cast<Quad16*>(p) = x;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if ((uint32_t)i < n) p[i] = (T)v[i];
}

__device__ __forceinline__ void load_kind(const void* p, uint32_t kind, uint64_t i, uint32_t n, float* v) {
  if (kind == kF32)
    load_few(static_cast<const float*>(p) + i, n, v);
  else if (kind == kBF16)
    load_few(static_cast<const __bf16*>(p) + i, n, v);
  else
    load_few(static_cast<const _Float16*>(p) + i, n, v);
}

__device__ __forceinline__ void store_kind(void* p, uint32_t kind, uint64_t i, uint32_t n, const float* v) {
  if (kind == kF32)
    store_few(static_cast<float*>(p) + i, n, v);
  else if (kind == kBF16)
    store_few(static_cast<__bf16*>(p) + i, n, v);
  else
    store_few(static_cast<_Float16*>(p) + i, n, v);
}

// The float next to v, of two the odd one, where v is none: rounded to 16 bits it gives
// what v would at once. (By way of the nearest float, what lies within 2^-25 of the
// middle between two of 16 bits would be taken for the middle.)
__device__ __forceinline__ float odd_float(double v) {
  const float f = (float)v;
  const double g = (double)f;
  uint32_t bits = __builtin_bit_cast(uint32_t, f);
  if (fabs(g) > fabs(v)) --bits;
  if (g < v || g > v) bits |= 1;
  return as_float(bits);
}

// The update that is orthogonalised, n elements of a row, in 64 bits. MOVE: the
// momentum takes the gradient in first.
template <bool MOVE>
__device__ __forceinline__ void update_few(const PolarMatrix& m, const PolarRule& r, uint64_t row, uint64_t col, uint32_t n,
                                           double* u) {
  float g[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (MOVE || !m.momentum || r.nesterov) load_kind(m.in, m.in_kind, row * m.in_stride + col, n, g);
  if (!m.momentum) {
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = g[i];
    return;
  }
  float s[4];
  float* at = m.momentum + row * m.momentum_stride + col;
  load_few(at, n, s);
  if (MOVE) {
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = (float)(r.momentum * (double)s[i] + (1.0 - r.momentum) * (double)g[i]);
    store_few(at, n, s);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) u[i] = r.nesterov ? (1.0 - r.momentum) * (double)g[i] + r.momentum * (double)s[i] : (double)s[i];
}

// The momentum, and partial sums of the squares of the update, in 64 bits: a wave
// takes 256 elements of a row at a time.
template <typename Item>
__global__ __launch_bounds__(kPolarThreads) void polar_norm_kernel(const Item* items, uint32_t n, const PolarRule r) {
  __shared__ double sh[kPolarThreads / 64];
  const Item& it = find_item(items, n, blockIdx.x, &Item::first_part);
  const PolarMatrix m = it.m;
  const uint32_t part = blockIdx.x - it.first_part, across = (m.cols - 1) / kNormCols + 1;
  const uint32_t tiles = across * ((m.rows - 1) / kNormRows + 1);
  const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  double sum = 0.0;
  for (uint32_t k = 0; k < it.part_tiles; ++k) {
    const uint32_t tile = part * it.part_tiles + k;
    if (tile >= tiles) break;
    const uint32_t c0 = tile % across * kNormCols + lane * 4;
    const uint32_t r0 = tile / across * kNormRows, r1 = min(r0 + kNormRows, m.rows);
    if (c0 >= m.cols) continue;
    const uint32_t few = min(m.cols - c0, 4u);
#pragma unroll 4
    for (uint32_t row = r0 + wave; row < r1; row += kPolarThreads / 64) {
      double u[4];
      update_few<true>(m, r, row, c0, few, u);
#pragma unroll
      for (int i = 0; i < 4; ++i) sum += (uint32_t)i < few ? u[i] * u[i] : 0.0;
    }
  }
  sum = block_sum<kPolarThreads>(sum, sh);
  if (threadIdx.x == 0) it.partial[part] = sum;
}

// What a float is held as: the nearest half, and the half nearest to the rest.
__device__ __forceinline__ f16x4 upper_halves(const float* v) {
  f16x4 h;
#pragma unroll
  for (int k = 0; k < 4; ++k) h[k] = (_Float16)v[k];
  return h;
}

__device__ __forceinline__ f16x4 lower_halves(const float* v) {
  f16x4 h;
#pragma unroll
  for (int k = 0; k < 4; ++k) h[k] = (_Float16)(v[k] - (float)(_Float16)v[k]);
  return h;
}

// How a matrix's squares are summed: tiles of kNormRows x kNormCols, in at most
// kNormParts partial sums.
inline void norm_parts(const PolarMatrix& m, uint32_t* parts, uint32_t* part_tiles) {
  const uint64_t tiles = (uint64_t)((m.cols - 1) / kNormCols + 1) * ((m.rows - 1) / kNormRows + 1);
  *part_tiles = (uint32_t)((tiles - 1) / kNormParts + 1);
  *parts = (uint32_t)((tiles - 1) / *part_tiles + 1);
}

inline uint64_t up256(uint64_t b) { return (b + 255) & ~255ull; }

}  // namespace
}  // namespace hkvt
