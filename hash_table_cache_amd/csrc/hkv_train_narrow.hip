// gfx950 kernels that orthogonalise matrices whose shorter side is at most 64
// (include/hkv_train.h): the dense layers beside rows of 16 to 64 floats.
//
// The steps are those of the general kernels, which would take three launches for
// each, of a few workgroups that wait for memory most of their time. With p <= 64
// rows, A and B fit one workgroup's LDS, and the columns of X need each other only
// in A: a wave keeps 64 columns of X in registers, in 32 bits, from step to step,
//   A = sum over the waves of X_w X_w^T,   X_w <- a X_w + B X_w.
// Up to 256 columns are one workgroup's: all steps in one launch (64 x 64 bf16: 23
// us against 87 us of 18 launches). Longer rows are blocks of 256 columns. A launch
// takes all blocks through the end of one step and the beginning of the next, A's
// partial sums go through memory, and every workgroup squares A for itself; from
// kManyBlocks blocks on the partial sums are added by a launch of their own before.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <vector>

#include "hkv_train_internal.h"
#include "hkv_train_matrix.h"

namespace hkvt {
namespace {

constexpr uint32_t kBlockCols = 256;
constexpr uint32_t kManyBlocks = 4;
constexpr uint32_t kMostBlocks = 256;
constexpr uint32_t kDirectItems = 16;
constexpr uint32_t kElems = 64 * 64;  // of A

struct NarrowItem {
  PolarMatrix m;
  float* image;   // X between launches, as the threads hold it
  float* sums;    // [2][blocks][64][64]: partial sums of A, of this step and of the next
  float* joined;  // [64][64]: A
  double* partial;
  uint32_t flip;  // rows > cols: X is the transpose
  uint32_t blocks;
  uint32_t parts, part_tiles;
  uint32_t first_part, first_block;
};

// Items in a kernel's arguments, as its first one: read where the arguments lie,
// for indexing the parameter itself would copy all of them to scratch memory.
struct DirectItems {
  NarrowItem item[kDirectItems];
  static __device__ __forceinline__ NarrowItem at(uint32_t i) {
    struct Words {
      uint32_t w[sizeof(NarrowItem) / 4];
    } words;
    const auto* from = (const __attribute__((address_space(4))) uint32_t*)__builtin_amdgcn_kernarg_segment_ptr() +
                       i * (sizeof(NarrowItem) / 4);
#pragma unroll
    for (uint32_t k = 0; k < sizeof(NarrowItem) / 4; ++k) words.w[k] = from[k];
    return __builtin_bit_cast(NarrowItem, words);
  }
};

struct StoredItems {
  const NarrowItem* item;
  __device__ __forceinline__ NarrowItem at(uint32_t i) const { return item[i]; }
};

struct NarrowSteps {
  float c[3 * kMostSteps];
  uint32_t steps;
};

__global__ void narrow_upload_kernel(const DirectItems u, NarrowItem* to, uint32_t n) {
  const uint32_t words = n * sizeof(NarrowItem) / 4;
  for (uint32_t i = threadIdx.x; i < words; i += kPolarThreads)
    reinterpret_cast<uint32_t*>(to)[i] = reinterpret_cast<const uint32_t*>(&u)[i];
}

// A workgroup's block: 4 waves of 64 columns, R * 32 rows. A thread holds, of each
// fragment (i, j) of 32 x 32, column j * 32 + lane % 32 and four rows at a time.
template <int R, bool SPLIT>
struct Narrow {
  static constexpr int P = R * 32;
  static constexpr int KS = P / 16;  // sixteens of rows
  static constexpr int planes = SPLIT ? 2 : 1;
  struct Shared {
    f16x8 wave[4][2][64 * 8];  // halves of a wave's X, by rows or by columns; or its part of A
    f16x8 a[2][64 * 8], b[2][64 * 8];
    float d[64], e[64];
    double sum[4];
  };
  f32x16 x[R][2];
  Shared& sh;
  uint32_t lane, wave, n0;

  __device__ __forceinline__ Narrow(Shared& sh_, uint32_t block)
      : sh(sh_), lane(threadIdx.x & 63), wave(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) {
    n0 = block * kBlockCols + wave * 64;
  }

  // use(row, column of the wave, fragment, quad) for a thread's quads.
  template <typename Use>
  __device__ __forceinline__ void quads(Use&& use) const {
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g) use(i * 32 + g * 8 + (lane >> 5) * 4, j * 32 + (lane & 31), i, j, g);
  }

  // The block's elements of a matrix of X's shape (or, flip, its transpose's).
  template <typename T>
  __device__ __forceinline__ void gather(const T* p, uint64_t stride, const PolarMatrix& m, bool flip, f32x16 (&to)[R][2]) const {
    quads([&](uint32_t r, uint32_t c, int i, int j, int g) {
      const uint32_t n = n0 + c;
      float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      if (flip) {
        if (n < m.rows && r < m.cols) load_few(p + n * stride + r, min(m.cols - r, 4u), v);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (r + k < m.rows && n < m.cols) v[k] = (float)p[(r + k) * stride + n];
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) to[i][j][g * 4 + k] = v[k];
    });
  }

  template <typename T>
  __device__ __forceinline__ void scatter(T* p, uint64_t stride, const PolarMatrix& m, bool flip, const f32x16 (&from)[R][2]) const {
    quads([&](uint32_t r, uint32_t c, int i, int j, int g) {
      const uint32_t n = n0 + c;
      float v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = from[i][j][g * 4 + k];
      if (flip) {
        if (n < m.rows && r < m.cols) store_few(p + n * stride + r, min(m.cols - r, 4u), v);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (r + k < m.rows && n < m.cols) p[(r + k) * stride + n] = (T)v[k];
      }
    });
  }

  __device__ __forceinline__ void gather_kind(const void* p, uint32_t kind, uint64_t stride, const PolarMatrix& m, bool flip,
                                              f32x16 (&to)[R][2]) const {
    if (kind == kF32)
      gather(static_cast<const float*>(p), stride, m, flip, to);
    else if (kind == kBF16)
      gather(static_cast<const __bf16*>(p), stride, m, flip, to);
    else
      gather(static_cast<const _Float16*>(p), stride, m, flip, to);
  }

  // The update, and the sum of its squares over the workgroup. MOVE: the momentum
  // takes the gradient in.
  template <bool MOVE>
  __device__ __forceinline__ double update(const NarrowItem& it, const PolarRule& r) {
    const PolarMatrix& m = it.m;
    if (MOVE || !m.momentum || r.nesterov) gather_kind(m.in, m.in_kind, m.in_stride, m, it.flip, x);
    double sum = 0.0;
    if (m.momentum) {
      f32x16 s[R][2];
      gather(m.momentum, m.momentum_stride, m, it.flip, s);
      if (MOVE) {
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int k = 0; k < 16; ++k)
              s[i][j][k] = (float)(r.momentum * (double)s[i][j][k] + (1.0 - r.momentum) * (double)x[i][j][k]);
        scatter(m.momentum, m.momentum_stride, m, it.flip, s);
      }
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const double u = r.nesterov ? (1.0 - r.momentum) * (double)x[i][j][k] + r.momentum * (double)s[i][j][k] : (double)s[i][j][k];
            sum += u * u;
            x[i][j][k] = (float)u;
          }
    } else {
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int k = 0; k < 16; ++k) sum += (double)x[i][j][k] * (double)x[i][j][k];
    }
    return sum;
  }

  // A matrix whose norm is not finite becomes NaN.
  __device__ __forceinline__ void scale(double squares, double eps) {
    const double norm = sqrt(squares);
    const double f = norm < (double)kInf ? kUnit / fmax(norm, eps) : __builtin_nan("");
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int k = 0; k < 16; ++k) x[i][j][k] = (float)((double)x[i][j][k] * f);
  }

  // 16 bytes of halves `piece` of row r of an array of 64 halves a row: shuffled so
  // that reading one piece of 32 rows meets all banks.
  static __device__ __forceinline__ uint32_t place(uint32_t r, uint32_t piece) { return r * 8 + (piece ^ ((r >> 1) & 7)); }
  static __device__ __forceinline__ _Float16& half_at(f16x8* to, uint32_t r, uint32_t c) {
    return reinterpret_cast<_Float16*>(to + place(r, c >> 3))[c & 7];
  }
  static __device__ __forceinline__ f16x4& quad_at(f16x8* to, uint32_t r, uint32_t c) {
    return *reinterpret_cast<f16x4*>(reinterpret_cast<_Float16*>(to + place(r, c >> 3)) + (c & 7));
  }

  static __device__ __forceinline__ f32x16 product(f32x16 acc, const f16x8* a, const f16x8* b) {
    if (SPLIT) {
      acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(a[1], b[0], acc, 0, 0, 0);
      acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(a[0], b[1], acc, 0, 0, 0);
    }
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a[0], b[0], acc, 0, 0, 0);
  }

  static __device__ __forceinline__ void read(const f16x8 (*from)[64 * 8], uint32_t r, uint32_t piece, f16x8* to) {
#pragma unroll
    for (int p = 0; p < planes; ++p) to[p] = from[p][place(r, piece)];
  }

  static __device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }

  // The wave's part of A, into its LDS: the fragments on and above the diagonal.
  __device__ __forceinline__ void gram() {
    f16x8(*own)[64 * 8] = sh.wave[wave];
    wave_sync();
    quads([&](uint32_t r, uint32_t c, int i, int j, int g) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float v = x[i][j][g * 4 + k];
        const _Float16 hi = (_Float16)v;
        half_at(own[0], r + k, c) = hi;
        if (SPLIT) half_at(own[1], r + k, c) = (_Float16)(v - (float)hi);
      }
    });
    wave_sync();
    f32x16 s[R][R] = {};
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      f16x8 f[R][2];
#pragma unroll
      for (int i = 0; i < R; ++i) read(own, i * 32 + (lane & 31), ks * 2 + (lane >> 5), f[i]);
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = i; j < R; ++j) s[i][j] = product(s[i][j], f[i], f[j]);
    }
    wave_sync();
    float* part = reinterpret_cast<float*>(own);
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = i; j < R; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            part[(i * 32 + g * 8 + (lane >> 5) * 4 + k) * P + j * 32 + (lane & 31)] = s[i][j][g * 4 + k];
  }

  // use(row, column, sum over the waves) for a thread's elements of A.
  template <typename Use>
  __device__ __forceinline__ void join(Use&& use) {
    __syncthreads();
#pragma unroll 4
    for (uint32_t e = threadIdx.x; e < P * P; e += kPolarThreads) {
      const uint32_t r = e / P, c = e % P;
      const uint32_t at = r / 32 > c / 32 ? c * P + r : e;
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < 4; ++w) v += reinterpret_cast<const float*>(sh.wave[w])[at];
      use(r, c, v);
    }
  }

  // An element of A goes to LDS as halves, the diagonal apart.
  __device__ __forceinline__ void take(uint32_t r, uint32_t c, float sum) {
    float v = sum * (1.0f / kUnit);
    if (r == c) {
      sh.d[r] = v * (1.0f / kUnit);
      v = 0.0f;
    }
    const _Float16 hi = (_Float16)v;
    half_at(sh.a[0], r, c) = hi;
    if (SPLIT) half_at(sh.a[1], r, c) = (_Float16)(v - (float)hi);
  }

  // B without its diagonal, and E, from A: a fragment a wave.
  __device__ __forceinline__ void square(float b, float c2) {
    __syncthreads();
    if (wave < R * R) {
      const uint32_t i = wave / R, j = wave % R;
      f32x16 s = {};
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        f16x8 fa[2], fb[2];
        read(sh.a, i * 32 + (lane & 31), ks * 2 + (lane >> 5), fa);
        read(sh.a, j * 32 + (lane & 31), ks * 2 + (lane >> 5), fb);
        s = product(s, fa, fb);
      }
      const uint32_t col = j * 32 + (lane & 31);
      const float dc = sh.d[col];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const uint32_t row = i * 32 + g * 8 + (lane >> 5) * 4;
        const f16x4 hi = quad_at(sh.a[0], col, row);  // A is symmetric
        f16x4 lo = {};
        if (SPLIT) lo = quad_at(sh.a[1], col, row);
        float v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float a = (float)hi[k] + (float)lo[k];
          v[k] = fmaf(fmaf(c2, sh.d[row + k] + dc, b), a, s[g * 4 + k] * (c2 / kUnit));
          if (row + k == col) {
            sh.e[col] = fmaf(c2, dc * dc, fmaf(b, dc, v[k] * (1.0f / kUnit)));
            v[k] = 0.0f;
          }
        }
        quad_at(sh.b[0], col, row) = upper_halves(v);
        if (SPLIT) quad_at(sh.b[1], col, row) = lower_halves(v);
      }
    }
    __syncthreads();
  }

  // X <- a X + B X.
  __device__ __forceinline__ void next(float a) {
    f16x8(*own)[64 * 8] = sh.wave[wave];
    wave_sync();
    quads([&](uint32_t r, uint32_t c, int i, int j, int g) {
      float v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = x[i][j][g * 4 + k];
      quad_at(own[0], c, r) = upper_halves(v);
      if (SPLIT) quad_at(own[1], c, r) = lower_halves(v);
    });
    wave_sync();
    f32x16 s[R][2] = {};
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      f16x8 fb[R][2], fx[2][2];
#pragma unroll
      for (int i = 0; i < R; ++i) read(sh.b, i * 32 + (lane & 31), ks * 2 + (lane >> 5), fb[i]);
#pragma unroll
      for (int j = 0; j < 2; ++j) read(own, j * 32 + (lane & 31), ks * 2 + (lane >> 5), fx[j]);
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) s[i][j] = product(s[i][j], fb[i], fx[j]);
    }
    quads([&](uint32_t r, uint32_t, int i, int j, int g) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int e = g * 4 + k;
        x[i][j][e] = fmaf(a + sh.e[r + k], x[i][j][e], s[i][j][e] * (1.0f / kUnit));
      }
    });
  }

  // The result, to the matrix or into the weights.
  __device__ __forceinline__ void write(const NarrowItem& it) {
    const PolarMatrix& m = it.m;
    f32x16 old[R][2];
    if (m.momentum) gather_kind(m.out, m.out_kind, m.out_stride, m, it.flip, old);
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const float o = x[i][j][k] * (1.0f / kUnit);
          x[i][j][k] = m.momentum ? (float)(m.keep * (double)old[i][j][k] + m.step * (double)o) : o;
        }
    if (m.out_kind == kF32)
      scatter(static_cast<float*>(m.out), m.out_stride, m, it.flip, x);
    else if (m.out_kind == kBF16)
      scatter(static_cast<__bf16*>(m.out), m.out_stride, m, it.flip, x);
    else
      scatter(static_cast<_Float16*>(m.out), m.out_stride, m, it.flip, x);
  }

  __device__ __forceinline__ u32x4* image(const NarrowItem& it, uint32_t block) const {
    return reinterpret_cast<u32x4*>(it.image) + ((uint64_t)block * 4 + wave) * (R * 2 * 4 * 64) + lane;
  }
  __device__ __forceinline__ void keep(const NarrowItem& it, uint32_t block) const {
    u32x4* to = image(it, block);
    quads([&](uint32_t, uint32_t, int i, int j, int g) {
      u32x4 v;
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = __builtin_bit_cast(uint32_t, (float)x[i][j][g * 4 + k]);
      to[((i * 2 + j) * 4 + g) * 64] = v;
    });
  }
  __device__ __forceinline__ void recall(const NarrowItem& it, uint32_t block) {
    const u32x4* from = image(it, block);
    quads([&](uint32_t, uint32_t, int i, int j, int g) {
      const u32x4 v = from[((i * 2 + j) * 4 + g) * 64];
#pragma unroll
      for (int k = 0; k < 4; ++k) x[i][j][g * 4 + k] = as_float(v[k]);
    });
  }
};

// All steps of matrices of one block.
template <int R, bool SPLIT, typename List>
__global__ __launch_bounds__(kPolarThreads) void narrow_whole_kernel(const List list, const PolarRule r, const NarrowSteps c) {
  using N = Narrow<R, SPLIT>;
  __shared__ typename N::Shared sh;
  const NarrowItem it = list.at(blockIdx.x);
  N w(sh, 0);
  const double sum = w.template update<true>(it, r);
  w.scale(block_sum<kPolarThreads>(sum, sh.sum), r.eps);
  for (uint32_t k = 0; k < c.steps; ++k) {
    w.gram();
    w.join([&](uint32_t row, uint32_t col, float v) { w.take(row, col, v); });
    w.square(c.c[3 * k + 1], c.c[3 * k + 2]);
    w.next(c.c[3 * k]);
  }
  w.write(it);
}

// The beginning of the first step: X, and the blocks' parts of A.
template <int R, bool SPLIT>
__global__ __launch_bounds__(kPolarThreads) void narrow_first_kernel(const NarrowItem* items, uint32_t n, const PolarRule r) {
  using N = Narrow<R, SPLIT>;
  __shared__ typename N::Shared sh;
  const NarrowItem& it = find_item(items, n, blockIdx.x, &NarrowItem::first_block);
  const uint32_t block = blockIdx.x - it.first_block;
  N w(sh, block);
  w.template update<false>(it, r);
  double sum = 0.0;
  for (uint32_t i = threadIdx.x; i < it.parts; i += kPolarThreads) sum += it.partial[i];
  w.scale(block_sum<kPolarThreads>(sum, sh.sum), r.eps);
  w.keep(it, block);
  w.gram();
  float* to = it.sums + (uint64_t)block * kElems;
  w.join([&](uint32_t row, uint32_t col, float v) { to[row * N::P + col] = v; });
}

// A of matrices of many blocks, from the blocks' parts for a step: 256 elements a
// workgroup.
__global__ __launch_bounds__(kPolarThreads) void narrow_join_kernel(const NarrowItem* items, uint32_t elems, uint32_t step) {
  const NarrowItem& it = items[blockIdx.y];
  const uint32_t e = blockIdx.x * kPolarThreads + threadIdx.x;
  if (e >= elems) return;
  const float* from = it.sums + (uint64_t)(step & 1) * it.blocks * kElems + e;
  float v = 0.0f;
#pragma unroll 8
  for (uint32_t b = 0; b < it.blocks; ++b) v += from[(uint64_t)b * kElems];
  it.joined[e] = v;
}

// The end of a step, and the beginning of the next unless it is the last.
// `joined`: A is there whole.
template <int R, bool SPLIT>
__global__ __launch_bounds__(kPolarThreads) void narrow_step_kernel(const NarrowItem* items, uint32_t n, float a, float b,
                                                                    float c, uint32_t step, bool joined, bool last) {
  using N = Narrow<R, SPLIT>;
  __shared__ typename N::Shared sh;
  const NarrowItem& it = find_item(items, n, blockIdx.x, &NarrowItem::first_block);
  const uint32_t block = blockIdx.x - it.first_block;
  N w(sh, block);
  w.recall(it, block);
  const float* from = joined ? it.joined : it.sums + (uint64_t)(step & 1) * it.blocks * kElems;
  const uint32_t parts = joined ? 1 : it.blocks;
#pragma unroll 4
  for (uint32_t e = threadIdx.x; e < N::P * N::P; e += kPolarThreads) {
    float v = 0.0f;
    for (uint32_t k = 0; k < parts; ++k) v += from[(uint64_t)k * kElems + e];
    w.take(e / N::P, e % N::P, v);
  }
  w.square(b, c);
  w.next(a);
  if (last) {
    w.write(it);
    return;
  }
  w.keep(it, block);
  w.gram();
  float* to = it.sums + ((uint64_t)(~step & 1) * it.blocks + block) * kElems;
  w.join([&](uint32_t row, uint32_t col, float v) { to[row * N::P + col] = v; });
}

// The matrices of a launch: of one precision, number of fragments, and one block
// or more each.
constexpr uint64_t kNarrowBytes = 4ull << 30;
constexpr uint32_t kNarrowBlocks = 1u << 20;

struct NarrowGroup {
  std::vector<uint32_t> list;  // of the call's matrices
  bool split, one, many;       // many: blocks' parts are added by a launch of their own
  int fragments;
  uint64_t bytes = 0;
};

uint32_t blocks_of(const PolarMatrix& m) { return (std::max(m.rows, m.cols) - 1) / kBlockCols + 1; }

// Takes an item's scratch, from `at` on where that is memory; returns its bytes.
uint64_t lay_out(const PolarMatrix& m, int fragments, char* at, NarrowItem* it) {
  uint64_t used = 0;
  auto take = [&](uint64_t bytes) {
    char* p = at ? at + used : nullptr;
    used += up256(bytes);
    return p;
  };
  *it = NarrowItem{};
  it->m = m;
  it->flip = m.rows > m.cols;
  it->blocks = blocks_of(m);
  norm_parts(m, &it->parts, &it->part_tiles);
  if (it->blocks == 1) return 0;
  it->image = reinterpret_cast<float*>(take((uint64_t)it->blocks * kBlockCols * fragments * 32 * 4));
  it->sums = reinterpret_cast<float*>(take((uint64_t)it->blocks * kElems * 4 * 2));
  it->joined = reinterpret_cast<float*>(take(kElems * 4));
  it->partial = reinterpret_cast<double*>(take(it->parts * 8ull));
  return used;
}

std::vector<NarrowGroup> make_groups(const PolarMatrix* m, uint32_t n) {
  std::vector<NarrowGroup> groups;
  for (int kind = 0; kind < 12; ++kind) {
    NarrowGroup g;
    g.split = kind & 1;
    g.fragments = kind & 2 ? 2 : 1;
    g.one = kind / 4 == 0;
    g.many = kind / 4 == 2;
    uint64_t blocks = 0;
    auto close = [&]() {
      if (!g.list.empty()) groups.push_back(g);
      g.list.clear();
      g.bytes = blocks = 0;
    };
    for (uint32_t i = 0; i < n; ++i) {
      const uint32_t b = blocks_of(m[i]), fragments = std::min(m[i].rows, m[i].cols) > 32 ? 2 : 1;
      if (splits(m[i]) != g.split || (int)fragments != g.fragments || (b == 1) != g.one || (b > kManyBlocks) != g.many) continue;
      NarrowItem it;
      const uint64_t bytes = lay_out(m[i], g.fragments, nullptr, &it) + sizeof(NarrowItem);
      if (!g.list.empty() && (g.bytes + bytes > kNarrowBytes || blocks + b > kNarrowBlocks || g.list.size() >= 65535)) close();
      g.list.push_back(i);
      g.bytes += bytes;
      blocks += b;
    }
    close();
  }
  return groups;
}

template <int R, bool SPLIT>
hipError_t run_group(const PolarMatrix* m, const NarrowGroup& g, const PolarRule& r, const double* c, uint32_t steps,
                     char* ws, hipStream_t s) {
  const uint32_t n = (uint32_t)g.list.size();
  NarrowItem* stored = reinterpret_cast<NarrowItem*>(ws);
  char* at = ws + up256((uint64_t)n * sizeof(NarrowItem));
  uint32_t parts = 0, blocks = 0;
  DirectItems direct{};
  hipError_t e = hipSuccess;
  for (uint32_t i = 0; i < n; i += kDirectItems) {
    const uint32_t many = std::min(kDirectItems, n - i);
    for (uint32_t j = 0; j < many; ++j) {
      NarrowItem& it = direct.item[j];
      at += lay_out(m[g.list[i + j]], g.fragments, at, &it);
      it.first_part = parts;
      it.first_block = blocks;
      parts += it.parts;
      blocks += it.blocks;
    }
    if (g.one && n <= kDirectItems) break;
    narrow_upload_kernel<<<1, kPolarThreads, 0, s>>>(direct, stored + i, many);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (g.one) {
    NarrowSteps all{};
    all.steps = steps;
    for (uint32_t k = 0; k < 3 * steps; ++k) all.c[k] = (float)c[k];
    if (n <= kDirectItems)
      narrow_whole_kernel<R, SPLIT><<<n, kPolarThreads, 0, s>>>(direct, r, all);
    else
      narrow_whole_kernel<R, SPLIT><<<n, kPolarThreads, 0, s>>>(StoredItems{stored}, r, all);
    return hipGetLastError();
  }
  polar_norm_kernel<<<parts, kPolarThreads, 0, s>>>(stored, n, r);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  narrow_first_kernel<R, SPLIT><<<blocks, kPolarThreads, 0, s>>>(stored, n, r);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  for (uint32_t k = 0; k < steps; ++k, c += 3) {
    if (g.many) {
      constexpr uint32_t elems = R * 32 * R * 32;
      narrow_join_kernel<<<dim3(elems / kPolarThreads, n), kPolarThreads, 0, s>>>(stored, elems, k);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    narrow_step_kernel<R, SPLIT><<<blocks, kPolarThreads, 0, s>>>(stored, n, (float)c[0], (float)c[1], (float)c[2], k, g.many,
                                                                   k + 1 == steps);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

bool is_narrow(const PolarMatrix& m) { return std::min(m.rows, m.cols) <= 64 && blocks_of(m) <= kMostBlocks; }

uint64_t narrow_workspace_bytes(const PolarMatrix* m, uint32_t n) {
  uint64_t most = 0;
  for (const NarrowGroup& g : make_groups(m, n)) most = std::max(most, g.bytes + 256);
  return most;
}

hipError_t launch_narrow(const PolarMatrix* m, uint32_t n, const PolarRule& r, const double* coefficients,
                         uint32_t steps, void* ws, hipStream_t s) {
  char* at = static_cast<char*>(ws);
  for (const NarrowGroup& g : make_groups(m, n)) {
    hipError_t e;
    if (g.fragments == 1)
      e = g.split ? run_group<1, true>(m, g, r, coefficients, steps, at, s) : run_group<1, false>(m, g, r, coefficients, steps, at, s);
    else
      e = g.split ? run_group<2, true>(m, g, r, coefficients, steps, at, s) : run_group<2, false>(m, g, r, coefficients, steps, at, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace hkvt
