// gfx950 kernels that orthogonalise matrices whose shorter side is at most 64
// (include/hkv_train.h): the dense layers beside rows of 16 to 64 floats.
//
// The steps are those of the general kernels, which would take three launches for
// each, of a few workgroups that wait for memory most of their time. With p <= 64
// rows, A and B fit one workgroup's LDS, and the columns of X need each other only
// in A: a wave keeps 16 columns of X in registers, in 32 bits, from step to step.
// Up to 256 columns are one workgroup's: all steps in one launch (64 x 64 bf16: 18
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
constexpr int kNarrowThreads = 1024;
constexpr uint32_t kFragments = 10 * 64;  // A's fragments on and above the diagonal, four elements a lane

struct NarrowItem {
  PolarMatrix m;
  float* image;   // X between launches, as the threads hold it
  f32x4* sums;    // [2][blocks][kFragments]: partial sums of A, of this step and of the next
  f32x4* joined;  // [kFragments]: A
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

// A workgroup's block: 16 waves of 16 columns, F * 16 rows. A thread holds, of each
// fragment of 16 x 16, column lane % 16 and rows 4 (lane / 16) .. + 3. (4 waves of
// 64 columns, with a part of A from each, took three times as long: a wave alone on
// its SIMD issues an instruction every four cycles, and most of a step is bringing
// X into halves. 64 x 64: 6.5 us a step.)
template <int F, bool SPLIT>
struct Narrow {
  static constexpr int P = F * 16;
  static constexpr int kUpper = F * (F + 1) / 2;  // fragments of A on and above the diagonal
  static constexpr int planes = SPLIT ? 2 : 1;
  struct Shared {
    union {
      float cells[64 * kBlockCols];        // X on its way from or to memory
      f16x8 rows[2][64 * kBlockCols / 8];  // halves of X by rows, for A
      f16x8 cols[2][64 * kBlockCols / 8];  // by columns, for B X
    };
    f16x8 a[2][64 * 8], b[2][64 * 8];
    float d[64], e[64];
    double sum[kNarrowThreads / 64];
  };
  f32x4 x[F];
  Shared& sh;
  uint32_t lane, wave, block, cols;  // cols: of this block

  __device__ __forceinline__ Narrow(Shared& sh_, const NarrowItem& it, uint32_t block_)
      : sh(sh_), lane(threadIdx.x & 63), wave(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)), block(block_) {
    cols = min((it.flip ? it.m.rows : it.m.cols) - block * kBlockCols, kBlockCols);
  }
  __device__ __forceinline__ uint32_t row(int i) const { return i * 16 + (lane >> 4) * 4; }
  __device__ __forceinline__ uint32_t col() const { return wave * 16 + (lane & 15); }

  // use(row and column of the matrix, cell of X) for a thread's elements of the
  // block: lanes go along rows of memory, which are rows or, flip, columns of X.
  static __device__ __forceinline__ uint32_t cell(uint32_t r, uint32_t c) { return r * kBlockCols + (c ^ (r & 31)); }

  template <typename Use>
  __device__ __forceinline__ void cells(const PolarMatrix& m, bool flip, Use&& use) const {
    const uint32_t across = flip ? P : kBlockCols;
#pragma unroll 8
    for (uint32_t e = threadIdx.x; e < P * kBlockCols; e += kNarrowThreads) {
      const uint32_t a = e / across, b = e % across, r = flip ? b : a, c = flip ? a : b;
      if (c < cols && r < (flip ? m.cols : m.rows))
        use(flip ? (uint64_t)block * kBlockCols + c : r, flip ? r : block * kBlockCols + c, cell(r, c));
    }
  }

  // X from the update, and the sum of its squares over the thread's elements. MOVE:
  // the momentum takes the gradient in.
  template <bool MOVE, typename T>
  __device__ __forceinline__ double update_of(const NarrowItem& it, const PolarRule& r, const T* in) {
    const PolarMatrix& m = it.m;
    double sum = 0.0;
    if (!m.momentum) {
      cells(m, it.flip, [&](uint64_t row, uint32_t col, uint32_t at) {
        const double u = (float)in[row * m.in_stride + col];
        sum += u * u;
        sh.cells[at] = (float)u;
      });
    } else if (MOVE || r.nesterov) {
      cells(m, it.flip, [&](uint64_t row, uint32_t col, uint32_t at) {
        const double g = (float)in[row * m.in_stride + col];
        float* s = m.momentum + row * m.momentum_stride + col;
        float v = *s;
        if (MOVE) *s = v = (float)(r.momentum * (double)v + (1.0 - r.momentum) * g);
        const double u = r.nesterov ? (1.0 - r.momentum) * g + r.momentum * (double)v : (double)v;
        sum += u * u;
        sh.cells[at] = (float)u;
      });
    } else {
      cells(m, it.flip, [&](uint64_t row, uint32_t col, uint32_t at) { sh.cells[at] = m.momentum[row * m.momentum_stride + col]; });
    }
    return sum;
  }

  template <bool MOVE>
  __device__ __forceinline__ double update(const NarrowItem& it, const PolarRule& r) {
    for (uint32_t e = threadIdx.x; e < P * kBlockCols; e += kNarrowThreads) sh.cells[e] = 0.0f;
    __syncthreads();
    const void* in = it.m.in;
    double sum;
    if (it.m.in_kind == kF32)
      sum = update_of<MOVE>(it, r, static_cast<const float*>(in));
    else if (it.m.in_kind == kBF16)
      sum = update_of<MOVE>(it, r, static_cast<const __bf16*>(in));
    else
      sum = update_of<MOVE>(it, r, static_cast<const _Float16*>(in));
    __syncthreads();
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) x[i][k] = sh.cells[cell(row(i) + k, col())];
    return sum;
  }

  // A matrix whose norm is not finite becomes NaN.
  __device__ __forceinline__ void scale(double squares, double eps) {
    const double norm = sqrt(squares);
    const double f = norm < (double)kInf ? kUnit / fmax(norm, eps) : __builtin_nan("");
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) x[i][k] = (float)((double)x[i][k] * f);
  }

  // Pieces of 16 bytes of rows of halves, shuffled so that reading a piece of each of
  // 16 rows meets all banks: rows of 256 halves, and of 64.
  static __device__ __forceinline__ uint32_t wide(uint32_t r, uint32_t piece) { return r * 32 + (piece ^ (r & 15)); }
  static __device__ __forceinline__ uint32_t slim(uint32_t r, uint32_t piece) { return r * 8 + (piece ^ ((r >> 1) & 7)); }
  static __device__ __forceinline__ _Float16& half_at(f16x8* to, uint32_t place, uint32_t c) {
    return reinterpret_cast<_Float16*>(to + place)[c & 7];
  }
  static __device__ __forceinline__ f16x4& quad_at(f16x8* to, uint32_t r, uint32_t c) {
    return *reinterpret_cast<f16x4*>(reinterpret_cast<_Float16*>(to + slim(r, c >> 3)) + (c & 7));
  }

  static __device__ __forceinline__ f32x4 product(f32x4 acc, const f16x8* a, const f16x8* b) {
    if (SPLIT) {
      acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[1], b[0], acc, 0, 0, 0);
      acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[0], b[1], acc, 0, 0, 0);
    }
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a[0], b[0], acc, 0, 0, 0);
  }

  // Fragment f of A on or above the diagonal.
  __device__ __forceinline__ void upper(uint32_t f, uint32_t* i, uint32_t* j) const {
    uint32_t c = 0;
#pragma unroll
    for (uint32_t k = 1; k < F; ++k) c = f >= k * (k + 1) / 2 ? k : c;
    *j = c;
    *i = f - c * (c + 1) / 2;
  }

  // The block's part of A: a fragment a wave, of all columns. The first waves have one.
  __device__ __forceinline__ f32x4 gram() {
    __syncthreads();
    if (wave * 16 < cols) {
#pragma unroll
      for (int i = 0; i < F; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const _Float16 hi = (_Float16)x[i][k];
          const uint32_t place = wide(row(i) + k, col() >> 3);
          half_at(sh.rows[0], place, col()) = hi;
          if (SPLIT) half_at(sh.rows[1], place, col()) = (_Float16)(x[i][k] - (float)hi);
        }
    } else if (wave % 2 && wave * 16 < cols + 16) {  // the rest of 32 columns
#pragma unroll
      for (int i = 0; i < F; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t place = wide(row(i) + k, col() >> 3);
          half_at(sh.rows[0], place, col()) = (_Float16)0.0f;
          if (SPLIT) half_at(sh.rows[1], place, col()) = (_Float16)0.0f;
        }
    }
    __syncthreads();
    f32x4 s = {};
    if (wave < kUpper) {
      uint32_t i, j;
      upper(wave, &i, &j);
      const uint32_t ra = i * 16 + (lane & 15), rb = j * 16 + (lane & 15), end = (cols + 31) / 32;
#pragma unroll 2
      for (uint32_t ks = 0; ks < end; ++ks) {
        f16x8 fa[2], fb[2];
#pragma unroll
        for (int p = 0; p < planes; ++p) {
          fa[p] = sh.rows[p][wide(ra, ks * 4 + (lane >> 4))];
          fb[p] = sh.rows[p][wide(rb, ks * 4 + (lane >> 4))];
        }
        s = product(s, fa, fb);
      }
    }
    return s;
  }

  // The wave's fragment of A, summed over the blocks, goes to LDS as halves, the
  // diagonal apart.
  __device__ __forceinline__ void take(f32x4 s) {
    if (wave >= kUpper) return;
    uint32_t i, j;
    upper(wave, &i, &j);
    const uint32_t r = i * 16 + (lane >> 4) * 4, c = j * 16 + (lane & 15);
    float v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[k] = s[k] * (1.0f / kUnit);
      if (r + k == c) {
        sh.d[c] = v[k] * (1.0f / kUnit);
        v[k] = 0.0f;
      }
    }
    const f16x4 hi = upper_halves(v), lo = lower_halves(v);
    quad_at(sh.a[0], c, r) = hi;
    if (SPLIT) quad_at(sh.a[1], c, r) = lo;
    if (i == j) return;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      half_at(sh.a[0], slim(r + k, c >> 3), c) = hi[k];
      if (SPLIT) half_at(sh.a[1], slim(r + k, c >> 3), c) = lo[k];
    }
  }

  // B without its diagonal, and E, from A: a fragment a wave.
  __device__ __forceinline__ void square(float b, float c2) {
    __syncthreads();
    if (wave < F * F) {
      const uint32_t i = wave / F, j = wave % F;
      f32x4 s = {};
#pragma unroll
      for (int ks = 0; ks < P / 32; ++ks) {
        f16x8 fa[2], fb[2];
#pragma unroll
        for (int p = 0; p < planes; ++p) {
          fa[p] = sh.a[p][slim(i * 16 + (lane & 15), ks * 4 + (lane >> 4))];
          fb[p] = sh.a[p][slim(j * 16 + (lane & 15), ks * 4 + (lane >> 4))];
        }
        s = product(s, fa, fb);
      }
      const uint32_t r = i * 16 + (lane >> 4) * 4, c = j * 16 + (lane & 15);
      const float dc = sh.d[c];
      const f16x4 hi = quad_at(sh.a[0], c, r);  // A is symmetric
      f16x4 lo = {};
      if (SPLIT) lo = quad_at(sh.a[1], c, r);
      float v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[k] = fmaf(fmaf(c2, sh.d[r + k] + dc, b), (float)hi[k] + (float)lo[k], s[k] * (c2 / kUnit));
        if (r + k == c) {
          sh.e[c] = fmaf(c2, dc * dc, fmaf(b, dc, v[k] * (1.0f / kUnit)));
          v[k] = 0.0f;
        }
      }
      quad_at(sh.b[0], c, r) = upper_halves(v);
      if (SPLIT) quad_at(sh.b[1], c, r) = lower_halves(v);
    }
    __syncthreads();
  }

  // X <- a X + B X: every wave its own columns. Both halves of X in either precision
  // (with the upper one alone directions that X does not have would come in), here in
  // the last steps too: 64 x 64 bf16 19.5 us, with the upper half alone 18.3 us.
  __device__ __forceinline__ void next(float a) {
    if (wave * 16 >= cols) return;
#pragma unroll
    for (int i = 0; i < F; ++i) {
      float v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = x[i][k];
      quad_at(sh.cols[0], col(), row(i)) = upper_halves(v);
      quad_at(sh.cols[1], col(), row(i)) = lower_halves(v);
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    f32x4 s[F] = {};
#pragma unroll
    for (int ks = 0; ks < P / 32; ++ks) {
      f16x8 fx[2];
#pragma unroll
      for (int p = 0; p < 2; ++p) fx[p] = sh.cols[p][slim(col(), ks * 4 + (lane >> 4))];
#pragma unroll
      for (int i = 0; i < F; ++i) {
        f16x8 fb[2];
#pragma unroll
        for (int p = 0; p < planes; ++p) fb[p] = sh.b[p][slim(i * 16 + (lane & 15), ks * 4 + (lane >> 4))];
        if (!SPLIT) s[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(fb[0], fx[1], s[i], 0, 0, 0);
        s[i] = product(s[i], fb, fx);
      }
    }
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) x[i][k] = fmaf(a + sh.e[row(i) + k], x[i][k], s[i][k] * (1.0f / kUnit));
  }

  // The result, to the matrix or into the weights.
  template <typename T>
  __device__ __forceinline__ void write_to(const NarrowItem& it, T* out) const {
    const PolarMatrix& m = it.m;
    if (m.momentum)
      cells(m, it.flip, [&](uint64_t row, uint32_t col, uint32_t at) {
        T* w = out + row * m.out_stride + col;
        const double v = m.keep * (double)(float)*w + m.step * (double)(sh.cells[at] * (1.0f / kUnit));
        *w = (T)(sizeof(T) == 4 ? (float)v : odd_float(v));
      });
    else
      cells(m, it.flip, [&](uint64_t row, uint32_t col, uint32_t at) {
        out[row * m.out_stride + col] = (T)(sh.cells[at] * (1.0f / kUnit));
      });
  }

  __device__ __forceinline__ void write(const NarrowItem& it) const {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) sh.cells[cell(row(i) + k, col())] = x[i][k];
    __syncthreads();
    if (it.m.out_kind == kF32)
      write_to(it, static_cast<float*>(it.m.out));
    else if (it.m.out_kind == kBF16)
      write_to(it, static_cast<__bf16*>(it.m.out));
    else
      write_to(it, static_cast<_Float16*>(it.m.out));
  }

  __device__ __forceinline__ f32x4* image(const NarrowItem& it) const {
    return reinterpret_cast<f32x4*>(it.image) + (uint64_t)block * F * kNarrowThreads + threadIdx.x;
  }
  __device__ __forceinline__ void keep(const NarrowItem& it) const {
#pragma unroll
    for (int i = 0; i < F; ++i) image(it)[i * kNarrowThreads] = x[i];
  }
  __device__ __forceinline__ void recall(const NarrowItem& it) {
#pragma unroll
    for (int i = 0; i < F; ++i) x[i] = image(it)[i * kNarrowThreads];
  }
  // Where the wave's fragment of a block's part of A lies.
  __device__ __forceinline__ uint32_t fragment() const { return wave * 64 + lane; }
};

// All steps of matrices of one block.
template <int F, bool SPLIT, typename List>
__global__ __launch_bounds__(kNarrowThreads) void narrow_whole_kernel(const List list, const PolarRule r, const NarrowSteps c) {
  using N = Narrow<F, SPLIT>;
  __shared__ typename N::Shared sh;
  const NarrowItem it = list.at(blockIdx.x);
  N w(sh, it, 0);
  const double sum = w.template update<true>(it, r);
  w.scale(block_sum<kNarrowThreads>(sum, sh.sum), r.eps);
  for (uint32_t k = 0; k < c.steps; ++k) {
    w.take(w.gram());
    w.square(c.c[3 * k + 1], c.c[3 * k + 2]);
    w.next(c.c[3 * k]);
  }
  w.write(it);
}

// The beginning of the first step: X, and the blocks' parts of A.
template <int F, bool SPLIT>
__global__ __launch_bounds__(kNarrowThreads) void narrow_first_kernel(const NarrowItem* items, uint32_t n, const PolarRule r) {
  using N = Narrow<F, SPLIT>;
  __shared__ typename N::Shared sh;
  const NarrowItem& it = find_item(items, n, blockIdx.x, &NarrowItem::first_block);
  const uint32_t block = blockIdx.x - it.first_block;
  N w(sh, it, block);
  w.template update<false>(it, r);
  double sum = 0.0;
  for (uint32_t i = threadIdx.x; i < it.parts; i += kNarrowThreads) sum += it.partial[i];
  w.scale(block_sum<kNarrowThreads>(sum, sh.sum), r.eps);
  w.keep(it);
  const f32x4 s = w.gram();
  if (w.wave < N::kUpper) it.sums[(uint64_t)block * kFragments + w.fragment()] = s;
}

// A of matrices of many blocks, from the blocks' parts for a step: a fragment a
// wave.
__global__ __launch_bounds__(64) void narrow_join_kernel(const NarrowItem* items, uint32_t step) {
  const NarrowItem& it = items[blockIdx.y];
  const uint32_t at = blockIdx.x * 64 + threadIdx.x;
  const f32x4* from = it.sums + (uint64_t)(step & 1) * it.blocks * kFragments + at;
  f32x4 v = {};
#pragma unroll 8
  for (uint32_t b = 0; b < it.blocks; ++b) v += from[(uint64_t)b * kFragments];
  it.joined[at] = v;
}

// The end of a step, and the beginning of the next unless it is the last.
// `joined`: A is there whole.
template <int F, bool SPLIT>
__global__ __launch_bounds__(kNarrowThreads) void narrow_step_kernel(const NarrowItem* items, uint32_t n, float a, float b,
                                                                     float c, uint32_t step, bool joined, bool last) {
  using N = Narrow<F, SPLIT>;
  __shared__ typename N::Shared sh;
  const NarrowItem& it = find_item(items, n, blockIdx.x, &NarrowItem::first_block);
  const uint32_t block = blockIdx.x - it.first_block;
  N w(sh, it, block);
  w.recall(it);
  f32x4 s = {};
  if (w.wave < N::kUpper) {
    const f32x4* from = joined ? it.joined : it.sums + (uint64_t)(step & 1) * it.blocks * kFragments;
    for (uint32_t k = 0; k < (joined ? 1 : it.blocks); ++k) s += from[(uint64_t)k * kFragments + w.fragment()];
  }
  w.take(s);
  w.square(b, c);
  w.next(a);
  if (last) {
    w.write(it);
    return;
  }
  w.keep(it);
  s = w.gram();
  if (w.wave < N::kUpper) it.sums[((uint64_t)(~step & 1) * it.blocks + block) * kFragments + w.fragment()] = s;
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
  it->image = reinterpret_cast<float*>(take((uint64_t)it->blocks * kBlockCols * fragments * 16 * 4));
  it->sums = reinterpret_cast<f32x4*>(take((uint64_t)it->blocks * kFragments * 16 * 2));
  it->joined = reinterpret_cast<f32x4*>(take(kFragments * 16));
  it->partial = reinterpret_cast<double*>(take(it->parts * 8ull));
  return used;
}

std::vector<NarrowGroup> make_groups(const PolarMatrix* m, uint32_t n) {
  std::vector<NarrowGroup> groups;
  for (int kind = 0; kind < 12; ++kind) {
    NarrowGroup g;
    g.split = kind & 1;
    g.fragments = kind & 2 ? 4 : 2;
    g.one = kind / 4 == 0;
    g.many = kind / 4 == 2;
    uint64_t blocks = 0;
    auto close = [&]() {
      if (!g.list.empty()) groups.push_back(g);
      g.list.clear();
      g.bytes = blocks = 0;
    };
    for (uint32_t i = 0; i < n; ++i) {
      const uint32_t b = blocks_of(m[i]), fragments = std::min(m[i].rows, m[i].cols) > 32 ? 4 : 2;
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

template <int F, bool SPLIT>
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
      narrow_whole_kernel<F, SPLIT><<<n, kNarrowThreads, 0, s>>>(direct, r, all);
    else
      narrow_whole_kernel<F, SPLIT><<<n, kNarrowThreads, 0, s>>>(StoredItems{stored}, r, all);
    return hipGetLastError();
  }
  polar_norm_kernel<<<parts, kPolarThreads, 0, s>>>(stored, n, r);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  narrow_first_kernel<F, SPLIT><<<blocks, kNarrowThreads, 0, s>>>(stored, n, r);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  for (uint32_t k = 0; k < steps; ++k, c += 3) {
    if (g.many) {
      narrow_join_kernel<<<dim3(F * (F + 1) / 2, n), 64, 0, s>>>(stored, k);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    narrow_step_kernel<F, SPLIT><<<blocks, kNarrowThreads, 0, s>>>(stored, n, (float)c[0], (float)c[1], (float)c[2], k, g.many,
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
    if (g.fragments == 2)
      e = g.split ? run_group<2, true>(m, g, r, coefficients, steps, at, s) : run_group<2, false>(m, g, r, coefficients, steps, at, s);
    else
      e = g.split ? run_group<4, true>(m, g, r, coefficients, steps, at, s) : run_group<4, false>(m, g, r, coefficients, steps, at, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace hkvt
