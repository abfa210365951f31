// gfx950 kernels that orthogonalise matrices, and the momentum update that uses
// it (include/hkv_train.h).
//
// With X = u / |u|, oriented so that its rows are its shorter side (p rows of q),
// a step is
//   A = X X^T,  B = b A + c A A,  X <- a X + B X.
// All three are products of matrices whose rows are read along the inner
// dimension once X is also held transposed: A from rows of X, A A from rows of A
// (A is symmetric), and (B X)^T = X^T B from rows of X^T and rows of B. Of the
// first two only the tiles on and above the diagonal are computed.
//
// The matrix cores multiply halves and add in 32 bits. Everything is held scaled
// by 2^12: |X| <= 2, |A| < 16, |B| < 16 (the host checks it for the coefficients)
// keep halves finite, and elements down to 2^-26 of |X| keep their digits. Two
// precisions:
//   - split: a number is the sum of two halves, and a product three products of
//     halves (what is left out is 2^-22 of it): as precise as float32.
//   - single: one product of halves. Rounding would still cost most where it
//     counts: in X, whose small singular values a X carries, and on the
//     diagonals of A and B, which near the end are nearly all of them. So X
//     keeps both halves, the diagonals are kept out of the halves in 32 bits,
//     D = diag A, E = diag B:
//       B X = E X + (B - E) X,  A A = (A - D)(A - D) + D (A - D) + (A - D) D + D D.
//     (B - E) X takes both halves of X too, in two products. Then a step is a
//     product M X of the X that is held, and what A's and B's roundings do to M
//     turns X's directions without adding any. With the upper half alone, E times
//     its rounding stays behind in directions that X does not have, where only a
//     and E act, and every step multiplies it by a: 64 x 64 of rank 1, 5 steps,
//     would be off by 7e-3, of rank 16 after 10 steps by 1.2 (2-norm). In the last
//     two steps, after which it is multiplied once at most, the upper half is
//     enough: 16 of about 2048 x 4096 9.0 ms (7.5 ms with it alone throughout, 10.0
//     ms with both throughout), two of 10007 x 321 275 us (247, 291). Results are off
//     by 2e-4 to 1.6e-3, less than their rounding to bf16 (1.7e-3), for full,
//     decaying and low-rank spectra and up to 6 steps. A is off by X's rounding, 2^-12
//     of it; where all elements are rounded alike (a multiple of the identity) that
//     moves all singular values alike, by up to 7e-3.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <vector>

#include "hkv_train_internal.h"
#include "hkv_train_matrix.h"

namespace hkvt {
namespace {

constexpr uint32_t kUploads = 15;
constexpr uint32_t kDies = 8;

// 16 bytes a lane from memory to LDS, to where the wave's first lane points and on.
__device__ __forceinline__ void bring(const _Float16* from, f16x8* to) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)from,
                                   (__attribute__((address_space(3))) void*)to, 16, 0, 0);
}

// One matrix of a launch, as the kernels see it. Halves lie in planes: the
// upper halves, then the lower ones.
struct PolarItem {
  PolarMatrix m;
  _Float16* x;     // [p][q]
  _Float16* t[2];  // [q][p], both halves: of this step and of the next
  _Float16* a;     // [p][p]
  _Float16* b;     // [p][p]
  float* d;        // [p]: diagonal of A
  float* e;        // [p]: diagonal of B
  double* partial;
  f32x4* cut;           // [cuts][tiles on and above A's diagonal][1024]
  uint32_t p, q;        // padded to the tile
  uint32_t rows, cols;  // of X itself, not padded
  uint32_t flip;        // rows > cols: X is the transpose
  uint32_t parts;       // partial sums
  uint32_t part_tiles;  // tiles that each has
  uint32_t first_part, first_pack;  // numbers among all items' workgroups
  uint32_t first_sum;
  uint32_t first_gram, first_cut, first_next;  // numbers among all items' tiles
  uint32_t cuts;                               // workgroups that share a tile of A
};

struct PolarUpload {
  PolarItem item[kUploads];
};
static_assert(sizeof(PolarUpload) <= 4064, "kernel arguments");

__global__ void polar_upload_kernel(const PolarUpload u, PolarItem* to, uint32_t n) {
  const uint32_t words = n * sizeof(PolarItem) / 4;
  for (uint32_t i = threadIdx.x; i < words; i += kPolarThreads)
    reinterpret_cast<uint32_t*>(to)[i] = reinterpret_cast<const uint32_t*>(&u)[i];
}

// X and its transpose from the update, 64 x 64 elements a workgroup, zeros where
// the tiles reach past the matrix. A matrix whose norm is not finite becomes NaN.
template <bool SPLIT>
__global__ __launch_bounds__(kPolarThreads) void polar_pack_kernel(const PolarItem* items, uint32_t n, const PolarRule r) {
  __shared__ double sh[kPolarThreads / 64];
  __shared__ float tile[64][65];  // of the matrix
  const PolarItem& it = find_item(items, n, blockIdx.x, &PolarItem::first_pack);
  const PolarMatrix m = it.m;
  const uint32_t block = blockIdx.x - it.first_pack, across = it.q / 64;
  const uint32_t i0 = block / across * 64, j0 = block % across * 64;  // of X
  const uint32_t row0 = it.flip ? j0 : i0, col0 = it.flip ? i0 : j0;  // of the matrix
  const uint32_t c = threadIdx.x % 16 * 4, r0 = threadIdx.x / 16;
  double u[4][4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t row = row0 + r0 + k * 16, col = col0 + c;
    if (row < m.rows && col < m.cols) {
      update_few<false>(m, r, row, col, min(m.cols - col, 4u), u[k]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) u[k][i] = 0.0;
    }
  }
  double sum = 0.0;
  for (uint32_t i = threadIdx.x; i < it.parts; i += kPolarThreads) sum += it.partial[i];
  const double norm = sqrt(block_sum<kPolarThreads>(sum, sh));
  const double scale = norm < (double)kInf ? kUnit / fmax(norm, r.eps) : __builtin_nan("");
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool in = row0 + r0 + k * 16 < m.rows && col0 + c + i < m.cols;
      tile[r0 + k * 16][c + i] = in ? (float)(u[k][i] * scale) : 0.0f;
    }
  __syncthreads();
  const uint64_t plane = (uint64_t)it.p * it.q;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t a = r0 + k * 16;
    float v[4], w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = tile[a][c + i];
      w[i] = tile[c + i][a];
    }
    const float *x = it.flip ? w : v, *t = it.flip ? v : w;
    const uint64_t ix = (uint64_t)(i0 + a) * it.q + j0 + c, tx = (uint64_t)(j0 + a) * it.p + i0 + c;
    *reinterpret_cast<f16x4*>(it.x + ix) = upper_halves(x);
    if (SPLIT) *reinterpret_cast<f16x4*>(it.x + plane + ix) = lower_halves(x);
    *reinterpret_cast<f16x4*>(it.t[0] + tx) = upper_halves(t);
    *reinterpret_cast<f16x4*>(it.t[0] + plane + tx) = lower_halves(t);
  }
}

// A tile of T x T of a product of rows, acc[i][j] = sum over k of a[i][k] b[j][k],
// by WM x WN waves of FM x FN fragments of 32 x 32 each. BOTH: both halves of a
// number come together and meet in three products; where two buffers of them do
// not fit (T = 256), the halves' products are passes, one after the other. kWaves: on
// a SIMD, which registers have to leave room for; with 256 threads that is as many
// workgroups, with 512 half as many.
template <int T, bool SPLIT>
struct Shape;
template <>
struct Shape<64, false> {
  static constexpr int WM = 2, WN = 2, FM = 1, FN = 1, kBuffers = 3, kWaves = 3;
  static constexpr bool BOTH = false;
};
template <>
struct Shape<64, true> {
  static constexpr int WM = 2, WN = 2, FM = 1, FN = 1, kBuffers = 2, kWaves = 2;
  static constexpr bool BOTH = true;
};
template <>
struct Shape<128, false> {
  static constexpr int WM = 2, WN = 2, FM = 2, FN = 2, kBuffers = 2, kWaves = 2;
  static constexpr bool BOTH = false;
};
template <>
struct Shape<128, true> {
  static constexpr int WM = 2, WN = 4, FM = 2, FN = 1, kBuffers = 2, kWaves = 2;
  static constexpr bool BOTH = true;
};
template <bool SPLIT>
struct Shape<256, SPLIT> {
  static constexpr int WM = 2, WN = 4, FM = 4, FN = 2, kBuffers = 2, kWaves = 2;
  static constexpr bool BOTH = false;
};

// 64 inner elements at a time go through LDS, in buffers that memory itself
// writes, 16 bytes a lane. A row of a buffer is 8 pieces of 16 bytes, and their
// order is shuffled by the row: a wave reads one piece of 32 rows at once, 16 rows
// at a time, and two rows of 128 bytes share the 64 banks, so that rows 2 i and 2 i
// + 1 have piece k at k ^ (i % 8). (By the row itself, half of LDS's cycles were
// conflicts.) The next buffer's loads are issued between the products, a quarter
// with each sixteen inner elements: all at once they hold the waves up for as long
// as half of the products take (4096 x 4096 x 2048, T = 256: 1008 TFLOP/s against
// 950; T = 128: 854 against 830; more buffers, or fragments read one step ahead,
// were no faster).
template <int T, bool SPLIT>
struct Product {
  using S = Shape<T, SPLIT>;
  static constexpr int FM = S::FM, FN = S::FN, B = S::kBuffers, H = S::BOTH ? 2 : 1;
  static constexpr int kThreads = S::WM * S::WN * 64;
  static constexpr int L = T * 8 / kThreads;  // pieces that a thread brings, of each side and half
  static constexpr int kPlane = T * 8;
  static constexpr int kStage = 2 * H * kPlane;
  typedef f16x8 Shared[B * kStage];
  f32x16 acc[FM][FN];

  // The i-th piece that a thread brings of a round: first side a's halves, then b's.
  static __device__ __forceinline__ void bring_piece(int i, const _Float16* a, const _Float16* b, uint64_t plane_a,
                                                     uint64_t plane_b, uint32_t off, uint64_t hop, f16x8* to, uint32_t wave) {
    const int side = i / (H * L), half = i / L % H, k = i % L;
    const _Float16* from = side ? b + half * plane_b : a + half * plane_a;
    bring(from + k * hop + off, to + (side * H + half) * kPlane + k * kThreads + wave * 64);
  }

  // `to` and `from` are buffers apart, which the compiler has to know: it would
  // otherwise wait for the loads before it reads.
  __device__ __forceinline__ void stage(f16x8* __restrict to, const f16x8* __restrict from, const _Float16* a,
                                        const _Float16* b, uint64_t plane_a, uint64_t plane_b, uint32_t off, uint64_t hop,
                                        bool more, uint32_t wave, uint32_t ar, uint32_t br, uint32_t key) {
    constexpr int N = 2 * H * L;
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      f16x8 fa[H][FM], fb[H][FN];
      const uint32_t pc = (ks * 2) ^ key;
#pragma unroll
      for (int h = 0; h < H; ++h) {
#pragma unroll
        for (int i = 0; i < FM; ++i) fa[h][i] = from[h * kPlane + ar + i * 256 + pc];
#pragma unroll
        for (int i = 0; i < FN; ++i) fb[h][i] = from[(H + h) * kPlane + br + i * 256 + pc];
      }
      if (more) {
#pragma unroll
        for (int i = ks * N / 4; i < (ks + 1) * N / 4; ++i) bring_piece(i, a, b, plane_a, plane_b, off, hop, to, wave);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int pass = H == 2 ? 0 : 2; pass < 3; ++pass)  // lower x upper, upper x lower, upper x upper
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fa[pass == 0 ? H - 1 : 0][i], fb[pass == 1 ? H - 1 : 0][j],
                                                               acc[i][j], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  // Rows `stride` apart, K inner elements from the first one; the lower halves lie
  // plane_a and plane_b elements behind the upper ones. PRODUCTS of halves: upper x
  // upper, before it (2) upper x lower, before that (3) lower x upper.
  template <int PRODUCTS = SPLIT ? 3 : 1>
  __device__ __forceinline__ void run(const _Float16* a, const _Float16* b, uint32_t stride, uint32_t K, uint64_t plane_a,
                                      uint64_t plane_b, Shared& sh) {
    constexpr uint32_t kPasses = H == 2 ? 1 : PRODUCTS;
    static_assert(H == 1 || PRODUCTS == 3, "stage() takes both halves");
    const uint32_t tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = f32x16{};
    const uint32_t row = tid >> 3, off = row * stride + ((tid & 7) ^ ((row >> 1) & 7)) * 8;
    const uint64_t hop = (uint64_t)(kThreads / 8) * stride;
    const uint32_t fr = lane & 31, key = (lane >> 5) ^ ((fr >> 1) & 7);
    const uint32_t ar = (wave / S::WN * FM * 32 + fr) * 8, br = (wave % S::WN * FN * 32 + fr) * 8;
    const uint32_t blocks = (K + 63) / 64, rounds = kPasses * blocks;
    const _Float16 *pa = kPasses == 3 ? a + plane_a : a, *pb = kPasses == 2 ? b + plane_b : b;
    uint32_t left = blocks, passes = kPasses;  // this one included
    auto advance = [&]() {
      pa += 64;
      pb += 64;
      if (kPasses > 1 && --left == 0) {
        --passes;
        pa = a;
        pb = passes == 2 ? b + plane_b : b;
        left = blocks;
      }
    };
#pragma unroll
    for (int s = 0; s < B - 1; ++s) {
      if ((uint32_t)s < rounds) {
#pragma unroll
        for (int i = 0; i < 2 * H * L; ++i) bring_piece(i, pa, pb, plane_a, plane_b, off, hop, sh + s * kStage, wave);
        advance();
      }
    }
    uint32_t at = 0, to = B - 1;
#pragma unroll 1
    for (uint32_t r = 0; r < rounds; ++r) {
      // This wave's loads of this round's buffer are there, those of later ones may
      // be on their way; behind the barrier the others' are there too, and nobody
      // reads the buffer of the round before any more.
      if (r + B - 2 < rounds)
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((B - 2) * 2 * H * L) : "memory");
      else
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      stage(sh + to * kStage, sh + at * kStage, pa, pb, plane_a, plane_b, off, hop, r + B - 1 < rounds, wave, ar, br, key);
      advance();
      at = at + 1 == B ? 0 : at + 1;
      to = to + 1 == B ? 0 : to + 1;
    }
  }

  // use(row, column, four values of rows row .. row + 3) for each of a thread's
  // quads, few of them at a time: registers are full.
  template <typename Use>
  __device__ __forceinline__ void each(Use&& use) {
    uint32_t lane = threadIdx.x & 63;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    asm volatile("" : "+v"(lane));  // neither addresses nor halves are kept from one use to the next
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) asm volatile("" : "+v"(acc[i][j]));
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          if (T == 256 && g % 2 == 0) __builtin_amdgcn_sched_barrier(0);
          float v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) v[k] = acc[i][j][g * 4 + k];
          const uint32_t r = wave / S::WN * FM * 32 + i * 32 + g * 8 + (lane >> 5) * 4;
          const uint32_t c = wave % S::WN * FN * 32 + j * 32 + (lane & 31);
          use(r, c, v);
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[i][j][g * 4 + k] = v[k];
        }
  }

  // Tiles of halves in LDS, T columns of T, on their way from or to memory by 16
  // bytes a lane; a quad of a column is 8 bytes of it. Pieces are shuffled by the
  // column as above. kFit of them have room at a time.
  static constexpr int kTile = T * T / 8, kFit = B * kStage / kTile;

  static __device__ __forceinline__ f16x4& quad(f16x8* tile, uint32_t r, uint32_t c) {
    return *reinterpret_cast<f16x4*>(reinterpret_cast<_Float16*>(tile) + c * T + (((r >> 3) ^ c) % (T / 8)) * 8 + (r & 7));
  }

  // Brings N tiles `plane` apart, of columns `stride` apart in memory.
  template <int N>
  static __device__ __forceinline__ void load_tiles(const _Float16* from, uint64_t stride, uint64_t plane, Shared& sh) {
    static_assert(N <= kFit, "LDS");
    const uint32_t tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (uint32_t i = 0; i < kTile / kThreads; ++i) {
        const uint32_t at = i * kThreads + tid, c = at / (T / 8), piece = (at ^ c) % (T / 8);
        bring(from + n * plane + c * stride + piece * 8, sh + n * kTile + i * kThreads + wave * 64);
      }
    __syncthreads();
  }

  // A tile that is written: upper or lower halves, by columns or, `rows`, by rows,
  // which are `stride` apart in memory; not where to is NULL.
  struct Out {
    _Float16* to;
    uint64_t stride;
    bool rows, lower;
  };

  template <int N>
  __device__ __forceinline__ void store_tiles(const Out (&out)[N], Shared& sh) {
#pragma unroll
    for (int first = 0; first < N; first += kFit) {
      __syncthreads();
#pragma unroll
      for (int n = first; n < first + kFit && n < N; ++n) {
        const Out& o = out[n];
        f16x8* tile = sh + (n - first) * kTile;
        if (!o.to) continue;
        each([&](uint32_t r, uint32_t c, float* v) {
          const f16x4 h = o.lower ? lower_halves(v) : upper_halves(v);
          if (o.rows) {
#pragma unroll
            for (int k = 0; k < 4; ++k) reinterpret_cast<_Float16*>(tile)[(r + k) * T + c] = h[k];
          } else {
            quad(tile, r, c) = h;
          }
        });
      }
      __syncthreads();
#pragma unroll
      for (int n = first; n < first + kFit && n < N; ++n) {
        const Out& o = out[n];
        const f16x8* tile = sh + (n - first) * kTile;
        if (!o.to) continue;
#pragma unroll 4
        for (uint32_t i = 0; i < kTile / kThreads; ++i) {
          const uint32_t at = i * kThreads + threadIdx.x, line = at / (T / 8), piece = (o.rows ? at : at ^ line) % (T / 8);
          *reinterpret_cast<f16x8*>(o.to + line * o.stride + piece * 8) = tile[at];
        }
      }
    }
  }
};

// Consecutive workgroups go to the 8 dies in turn. Each die takes an eighth of the
// work, of tiles next to each other, so that what they share is in its cache (16 of
// 2048 x 4096 bf16, all steps: 6.78 ms against 7.14 ms with an eighth of each matrix's
// tiles to every die; 12 of 500 x 1300: 275 us against 310 us; both with one product for
// B X in every step). Tiles of 256 are few rounds of the chip, and a die with long
// products alone ends late: of many matrices their work is cut into `rows` times 8
// pieces, about half a matrix each, which go to the dies forth and back, so that each
// has long products and, last, short ones (16 of 1100 x 3400 to 3005 x 5005: 9.89 ms
// against 10.20 ms; smaller tiles lose by it, 40 of 128 x 512: 178 us against 169 us).
// `first`: each piece's first tile, and their number.
constexpr uint32_t kMostRows = 4;

struct Dies {
  uint32_t rows;
  uint32_t first[kMostRows * kDies + 1];
};

// The workgroup's matrix and its tile of it; false where its die has no more.
__device__ __forceinline__ bool find_tile(const PolarItem* items, uint32_t n, const Dies& dies, uint32_t PolarItem::* first,
                                          const PolarItem** item, uint32_t* tile) {
  const uint32_t die = blockIdx.x % kDies;
  uint32_t at = blockIdx.x / kDies;
  for (uint32_t r = 0; r < dies.rows; ++r) {
    const uint32_t piece = r * kDies + (r % 2 ? kDies - 1 - die : die);
    const uint32_t begin = dies.first[piece], tiles = dies.first[piece + 1] - begin;
    if (at < tiles) {
      const PolarItem& it = find_item(items, n, begin + at, first);
      *item = &it;
      *tile = begin + at - it.*first;
      return true;
    }
    at -= tiles;
  }
  return false;
}

// Number of a tile on or above the diagonal -> its place: 0 (0,0), 1 (0,1), 2 (1,1), 3 (0,2) ...
__device__ __forceinline__ void upper_tile(uint32_t tile, uint32_t* i, uint32_t* j) {
  uint32_t c = (uint32_t)((__builtin_sqrtf(8.0f * (float)tile + 1.0f) - 1.0f) * 0.5f);
  while (c * (c + 1) / 2 > tile) --c;
  while ((c + 1) * (c + 2) / 2 <= tile) ++c;
  *j = c;
  *i = tile - c * (c + 1) / 2;
}

// Writes a tile of a symmetric matrix at both its places, as halves.
template <int T, bool SPLIT>
__device__ __forceinline__ void store_both(Product<T, SPLIT>& m, _Float16* to, uint64_t p, uint32_t ti, uint32_t tj,
                                           typename Product<T, SPLIT>::Shared& sh) {
  using Out = typename Product<T, SPLIT>::Out;
  _Float16* col = to + (uint64_t)tj * T * p + ti * T;
  _Float16* row = ti == tj ? nullptr : to + (uint64_t)ti * T * p + tj * T;
  if constexpr (SPLIT) {
    const Out out[4] = {{col, p, false, false}, {row, p, true, false}, {col + p * p, p, false, true}, {row ? row + p * p : nullptr, p, true, true}};
    m.store_tiles(out, sh);
  } else {
    const Out out[2] = {{col, p, false, false}, {row, p, true, false}};
    m.store_tiles(out, sh);
  }
}

// A without its diagonal, and D, from a tile of X X^T.
template <int T, bool SPLIT>
__device__ __forceinline__ void write_gram(Product<T, SPLIT>& m, const PolarItem& it, uint32_t ti, uint32_t tj,
                                           typename Product<T, SPLIT>::Shared& sh) {
  m.each([&](uint32_t r, uint32_t c, float* v) {
    const uint32_t row = ti * T + r, col = tj * T + c;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[k] *= 1.0f / kUnit;
      if (row + k == col) {
        it.d[col] = v[k] * (1.0f / kUnit);
        v[k] = 0.0f;
      }
    }
  });
  store_both<T, SPLIT>(m, it.a, it.p, ti, tj, sh);
}

template <int T, bool SPLIT>
__global__ __launch_bounds__((Product<T, SPLIT>::kThreads), (Shape<T, SPLIT>::kWaves)) void polar_gram_kernel(const PolarItem* items, uint32_t n,
                                                                                         const Dies dies) {
  __shared__ typename Product<T, SPLIT>::Shared sh;
  const PolarItem* item;
  uint32_t tile, ti, tj;
  if (!find_tile(items, n, dies, &PolarItem::first_gram, &item, &tile)) return;
  const PolarItem& it = *item;
  upper_tile(tile, &ti, &tj);
  const uint64_t p = it.p, q = it.q;
  Product<T, SPLIT> m;
  m.run(it.x + ti * T * q, it.x + tj * T * q, it.q, it.cols, p * q, p * q, sh);
  write_gram<T, SPLIT>(m, it, ti, tj, sh);
}

// Few tiles of long rows: a tile is shared by `cuts` workgroups, each a range of
// the inner elements; what they have is added in a fixed order by a launch of its
// own (two of 10007 x 321 bf16: 42 us a step by 21 tiles, 9 us by 240 workgroups and
// the sums; 200 x 60000: 590 us against 26 us).
template <bool SPLIT>
__global__ __launch_bounds__((Product<64, SPLIT>::kThreads), (Shape<64, SPLIT>::kWaves)) void polar_cut_kernel(const PolarItem* items, uint32_t n,
                                                                                        const Dies dies) {
  using M = Product<64, SPLIT>;
  __shared__ typename M::Shared sh;
  const PolarItem* item;
  uint32_t part;
  if (!find_tile(items, n, dies, &PolarItem::first_cut, &item, &part)) return;
  const PolarItem& it = *item;
  const uint32_t across = it.p / 64, tiles = across * (across + 1) / 2, cut = part / tiles, tile = part % tiles;
  uint32_t ti, tj;
  upper_tile(tile, &ti, &tj);
  const uint64_t p = it.p, q = it.q;
  const uint32_t blocks = (it.cols + 63) / 64, begin = cut * blocks / it.cuts, end = (cut + 1) * blocks / it.cuts;
  M m;
  m.run(it.x + ti * 64 * q + begin * 64, it.x + tj * 64 * q + begin * 64, it.q, (end - begin) * 64, p * q, p * q, sh);
  f32x4* to = it.cut + ((uint64_t)cut * tiles + tile) * 1024 + threadIdx.x;
#pragma unroll
  for (int g = 0; g < 4; ++g)
    to[g * 256] = f32x4{m.acc[0][0][4 * g], m.acc[0][0][4 * g + 1], m.acc[0][0][4 * g + 2], m.acc[0][0][4 * g + 3]};
}

template <bool SPLIT>
__global__ __launch_bounds__((Product<64, SPLIT>::kThreads)) void polar_sum_kernel(const PolarItem* items, uint32_t n) {
  using M = Product<64, SPLIT>;
  __shared__ typename M::Shared sh;
  const PolarItem& it = find_item(items, n, blockIdx.x, &PolarItem::first_sum);
  const uint32_t across = it.p / 64, tiles = across * (across + 1) / 2, tile = blockIdx.x - it.first_sum;
  uint32_t ti, tj;
  upper_tile(tile, &ti, &tj);
  M m;
  m.acc[0][0] = f32x16{};
  const f32x4* from = it.cut + (uint64_t)tile * 1024 + threadIdx.x;
#pragma unroll 4
  for (uint32_t cut = 0; cut < it.cuts; ++cut, from += (uint64_t)tiles * 1024)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const f32x4 v = from[g * 256];
#pragma unroll
      for (int k = 0; k < 4; ++k) m.acc[0][0][4 * g + k] += v[k];
    }
  write_gram<64, SPLIT>(m, it, ti, tj, sh);
}

// B without its diagonal, and E.
template <int T, bool SPLIT>
__global__ __launch_bounds__((Product<T, SPLIT>::kThreads), (Shape<T, SPLIT>::kWaves)) void polar_square_kernel(const PolarItem* items, uint32_t n,
                                                                                           const Dies dies, float b, float c2) {
  __shared__ typename Product<T, SPLIT>::Shared sh;
  const PolarItem* item;
  uint32_t number, ti, tj;
  if (!find_tile(items, n, dies, &PolarItem::first_gram, &item, &number)) return;
  const PolarItem& it = *item;
  upper_tile(number, &ti, &tj);
  const uint64_t p = it.p;
  using M = Product<T, SPLIT>;
  M m;
  const _Float16* tile = it.a + (uint64_t)tj * T * p + ti * T;  // A is symmetric
  const float *dr = it.d + ti * T, *dc = it.d + tj * T;
  constexpr int H = SPLIT ? 2 : 1;
  auto add = [&](float* v, f32x4 d, float dcol, f16x4 x, bool first) {  // what A - D adds
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = fmaf(fmaf(c2, d[k] + dcol, b), (float)x[k], first ? v[k] * (c2 / kUnit) : v[k]);
  };
  m.run(it.a + ti * T * p, it.a + tj * T * p, it.p, it.rows, p * p, p * p, sh);
  constexpr int N = H <= M::kFit ? H : 1;
  for (int plane = H - N; plane >= 0; plane -= N) {
    m.template load_tiles<N>(tile + plane * p * p, p, p * p, sh);
    m.each([&](uint32_t r, uint32_t c, float* v) {
      const f32x4 d = *reinterpret_cast<const f32x4*>(dr + r);
#pragma unroll
      for (int h = N - 1; h >= 0; --h) add(v, d, dc[c], m.quad(sh + h * M::kTile, r, c), plane + h == H - 1);
    });
  }
  m.each([&](uint32_t r, uint32_t c, float* v) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (ti * T + r + k == tj * T + c) {
        const float d = dc[c];
        it.e[tj * T + c] = fmaf(c2, d * d, fmaf(b, d, v[k] * (1.0f / kUnit)));
        v[k] = 0.0f;
      }
    }
  });
  store_both<T, SPLIT>(m, it.b, p, ti, tj, sh);
}

// The tile (ti, tj) of the result, to the matrix or into the weights: by way of
// LDS, 32 columns of every wave at a time, so that lanes lie next to each other
// in memory.
template <int T, bool SPLIT>
__device__ __forceinline__ void write_out(Product<T, SPLIT>& m, const PolarItem& it, uint32_t ti, uint32_t tj,
                                          typename Product<T, SPLIT>::Shared& sh) {
  using S = Shape<T, SPLIT>;
  constexpr uint32_t W = S::WN * 32;  // columns at a time
  float* lds = reinterpret_cast<float*>(sh);
  const PolarMatrix w = it.m;
  const bool flip = it.flip;
#pragma unroll
  for (int j = 0; j < S::FN; ++j) {
    __syncthreads();
    m.each([&](uint32_t r, uint32_t c, float* v) {
      if (c / 32 % S::FN != (uint32_t)j) return;
      const uint32_t cc = c / 32 / S::FN * 32 + c % 32;
#pragma unroll
      for (int k = 0; k < 4; ++k) lds[flip ? cc * T + ((r + k) ^ (cc * 4 % T)) : (r + k) * W + cc] = v[k];
    });
    __syncthreads();
    for (uint32_t i = threadIdx.x * 4; i < T * W; i += Product<T, SPLIT>::kThreads * 4) {
      const uint32_t cc = flip ? i / T : i % W, r = flip ? (i % T) ^ (cc * 4 % T) : i / W;
      const uint32_t row = ti * T + r, col = tj * T + (cc / 32 * S::FN + j) * 32 + cc % 32;  // of X
      const uint32_t wr = flip ? col : row, wc = flip ? row : col;
      if (wr >= w.rows || wc >= w.cols) continue;
      const uint32_t few = min(w.cols - wc, 4u);
      const uint64_t at = wr * w.out_stride + wc;
      float o[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) o[k] = lds[i + k] * (1.0f / kUnit);
      if (w.momentum) {
        float old[4];
        load_kind(w.out, w.out_kind, at, few, old);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const double v = w.keep * (double)old[k] + w.step * (double)o[k];
          o[k] = w.out_kind == kF32 ? (float)v : odd_float(v);
        }
      }
      store_kind(w.out, w.out_kind, at, few, o);
    }
  }
}

// a X + B X of step `k`; the last one's goes to its destination. Columns of the
// tile are rows of X^T. PRODUCTS of halves make B X.
template <int T, bool SPLIT, bool LAST, int PRODUCTS>
__global__ __launch_bounds__((Product<T, SPLIT>::kThreads), (Shape<T, SPLIT>::kWaves)) void polar_next_kernel(const PolarItem* items, uint32_t n,
                                                                                         const Dies dies, float a, uint32_t step) {
  __shared__ typename Product<T, SPLIT>::Shared sh;
  const PolarItem* item;
  uint32_t tile;
  if (!find_tile(items, n, dies, &PolarItem::first_next, &item, &tile)) return;
  const PolarItem& it = *item;
  const uint64_t p = it.p, q = it.q;
  const uint32_t across = it.p / T, ti = tile % across, tj = tile / across;
  const _Float16* from = it.t[step & 1];
  using M = Product<T, SPLIT>;
  M m;
  const uint64_t at = (uint64_t)tj * T * p + ti * T;
  const float* e = it.e + ti * T;
  auto add = [&](float* v, f32x4 d, f16x4 x, bool first) {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = fmaf(a + d[k], (float)x[k], first ? v[k] * (1.0f / kUnit) : v[k]);
  };
  m.template run<PRODUCTS>(it.b + ti * T * p, from + tj * T * p, it.p, it.rows, p * p, p * q, sh);
  constexpr int N = M::kFit >= 2 ? 2 : 1;
  for (int plane = 2 - N; plane >= 0; plane -= N) {
    m.template load_tiles<N>(from + plane * p * q + at, p, p * q, sh);
    m.each([&](uint32_t r, uint32_t c, float* v) {
      const f32x4 d = *reinterpret_cast<const f32x4*>(e + r);
#pragma unroll
      for (int h = N - 1; h >= 0; --h) add(v, d, m.quad(sh + h * M::kTile, r, c), plane + h == 1);
    });
  }
  if (LAST) {
    write_out(m, it, ti, tj, sh);
    return;
  }
  _Float16 *to = it.t[~step & 1] + at, *x = it.x + (uint64_t)ti * T * q + tj * T;
  using Out = typename M::Out;
  if constexpr (SPLIT) {
    const Out out[4] = {{to, p, false, false}, {to + p * q, p, false, true}, {x, q, true, false}, {x + p * q, q, true, true}};
    m.store_tiles(out, sh);
  } else {
    const Out out[3] = {{to, p, false, false}, {to + p * q, p, false, true}, {x, q, true, false}};
    m.store_tiles(out, sh);
  }
}

// How a call's matrices are worked on: in groups whose scratch fits into
// kGroupBytes, of one precision and tile each.
constexpr uint64_t kGroupBytes = 4ull << 30;
constexpr uint32_t kGroupTiles = 1u << 22;

struct Group {
  uint32_t begin, end;  // of the order
  uint32_t tile, gram_tile;  // of the third product, whose sides X is padded to; of the other two
  bool split;
  uint32_t cuts;  // workgroups that may share a tile of A
  uint64_t bytes;
};

uint64_t up(uint64_t v, uint64_t to) { return (v + to - 1) / to * to; }

// Takes an item's scratch, from `at` on where that is memory; returns its bytes.
uint64_t lay_out(const PolarMatrix& m, uint32_t tile, bool split, uint32_t cuts, char* at, PolarItem* it) {
  uint64_t used = 0;
  auto take = [&](uint64_t bytes) {
    char* p = at ? at + used : nullptr;
    used += up256(bytes);
    return p;
  };
  const uint64_t p = up(std::min(m.rows, m.cols), tile), q = up(std::max(m.rows, m.cols), tile), planes = split ? 2 : 1;
  it->x = reinterpret_cast<_Float16*>(take(p * q * 2 * planes));
  for (auto& t : it->t) t = reinterpret_cast<_Float16*>(take(p * q * 4));
  it->a = reinterpret_cast<_Float16*>(take(p * p * 2 * planes));
  it->b = reinterpret_cast<_Float16*>(take(p * p * 2 * planes));
  it->d = reinterpret_cast<float*>(take(p * 4));
  it->e = reinterpret_cast<float*>(take(p * 4));
  norm_parts(m, &it->parts, &it->part_tiles);
  it->partial = reinterpret_cast<double*>(take(it->parts * 8));
  // more cuts make sums longer: 0.25 us a round of 64 inner elements against 0.2 us a cut
  const uint32_t rounds = (uint32_t)(q / 64) * (split ? 3 : 1), best = (uint32_t)std::sqrt(1.25 * rounds);
  it->cuts = std::max(1u, std::min({cuts, best, (uint32_t)(q / 64)}));
  it->cut = cuts > 1 ? reinterpret_cast<f32x4*>(take(p / 64 * (p / 64 + 1) / 2 * it->cuts * 64 * 64 * 4)) : nullptr;
  it->p = (uint32_t)p;
  it->q = (uint32_t)q;
  it->rows = std::min(m.rows, m.cols);
  it->cols = std::max(m.rows, m.cols);
  it->flip = m.rows > m.cols;
  it->m = m;
  return used;
}

// Large tiles feed the matrix cores better, small ones are more workgroups and less
// padding. A third product of 256 tiles of 256 has them (16 matrices of 2048 x 4096:
// 797 us against 1041 us with 128; 4096 x 4096, all steps: 2129 against 2445 us); of
// 256 tiles of 128 those (all steps: 2500 x 2500 bf16 814 us against 1088 us with 64,
// 2048 x 2048 501 and 535 us, of float32 761 and 916 us; 800 x 5000 bf16 302 and 279 us)
// unless its rounds are few and its ends most of it (12 of 500 x 1300: 361 and 309 us).
// A has half as many tiles: they are taken of that size from 256 tiles on, or 128 of
// 256 or where both halves meet (4 of 1024 x 2048 float32, all steps: 753 us against
// 809, but bf16 480 against 414; 12 of 500 x 1300 bf16: 23 us with 64 against 29 us
// with 128).
//
// Tiles of 256 have to be worth their padding and their last round of the chip. A
// matrix counts for them if they pad it to at most 5/4 of what tiles of 64 do (32 of
// 192 x 4096 bf16: 761 us, 571 us with 64; 16 of 300 x 8192: 1689 and 1163; 640 x
// 4096, padded to 6/5, still 1670 against 1696), and they are taken where their
// rounds of 256 take no longer than those of 512 tiles of 128, two of which a compute
// unit has at a time, at 23/20 of the rate (16 of 1024 x 4096, 4 rounds each: 2641 us
// against 2955 us with 128; 8 of 1500 x 1500, 2 rounds against 3: 1461 against 1348 us;
// 11 of 1100 x 1100: 1199 against 782 us). What does not count goes apart from what
// does: 4096 x 4096 with 100 of 70 x 70 2478 us, 3157 us in one group of 256.
constexpr uint64_t kManyBig = 256, kManyTiles = 256, kManyUpper = 256, kManyUpperPairs = 128;

struct Plan {
  std::vector<uint32_t> order;
  std::vector<Group> groups;
  std::vector<PolarMatrix> narrow;
  uint64_t bytes = 0;  // of the largest group, the items' list included
};

Plan make_plan(const PolarMatrix* m, uint32_t n) {
  Plan plan;
  plan.order.reserve(n);
  for (uint32_t i = 0; i < n; ++i)
    if (is_narrow(m[i])) plan.narrow.push_back(m[i]);
  plan.bytes = narrow_workspace_bytes(plan.narrow.data(), (uint32_t)plan.narrow.size());
  const auto area = [&](uint32_t i, uint64_t tile) { return up(m[i].rows, tile) * up(m[i].cols, tile); };
  // Adds the groups of matrices of one precision, in tiles of 256 or of what they are enough for.
  const auto add = [&](const std::vector<uint32_t>& list, bool split, bool small, bool whole) {
    const uint32_t begin = (uint32_t)plan.order.size();
    uint64_t tiles = 0, upper[3] = {}, rounds = 0;  // upper: of 64, 128 and 256
    uint32_t longest = 0;
    for (const uint32_t i : list) {
      plan.order.push_back(i);
      tiles += area(i, 128) / (128 * 128);
      for (int k = 0; k < 3; ++k) {
        const uint64_t side = up(std::min(m[i].rows, m[i].cols), 64 << k) / (64 << k);
        upper[k] += side * (side + 1) / 2;
      }
      rounds += up(std::min(m[i].rows, m[i].cols), 64) / 64 * (split ? 3 : 1);
      longest = std::max({longest, m[i].rows, m[i].cols});
    }
    // long products first, so that the last ones to end are short
    std::stable_sort(plan.order.begin() + begin, plan.order.end(), [&](uint32_t a, uint32_t b) {
      return std::min(m[a].rows, m[a].cols) > std::min(m[b].rows, m[b].cols);
    });
    const uint64_t many = plan.order.size() - begin;
    const uint32_t tile = whole ? 256 : !small && tiles >= kManyTiles && rounds >= 12 * many ? 128 : 64;
    const uint64_t most = split ? kManyUpperPairs : kManyUpper;
    const uint32_t gram_tile = tile == 256 && upper[2] >= kManyUpperPairs ? 256 : tile >= 128 && upper[1] >= most ? 128 : 64;
    if (tile < 256) {  // long and short ones by turns: every die has both
      const std::vector<uint32_t> sorted(plan.order.begin() + begin, plan.order.end());
      for (uint64_t k = 0; k < many; ++k) plan.order[begin + k] = sorted[k % 2 ? many - 1 - k / 2 : k / 2];
    }
    // A's few tiles are shared where rows are long enough to pay for the sums
    const bool shared = gram_tile == 64 && upper[0] <= 256 && up(longest, 64) / 64 * (split ? 3 : 1) >= 32;
    const uint32_t cuts = shared ? (uint32_t)(512 / std::max<uint64_t>(upper[0], 1)) : 1;
    for (uint32_t at = begin; at < plan.order.size();) {
      Group g{at, at, tile, gram_tile, split, cuts, 0};
      uint64_t count = 0;
      while (g.end < plan.order.size()) {
        PolarItem it;
        const PolarMatrix& x = m[plan.order[g.end]];
        const uint64_t bytes = lay_out(x, tile, split, cuts, nullptr, &it) + up256(sizeof(PolarItem));
        const uint64_t more = (uint64_t)(it.p / 64) * (it.q / 64);
        if (g.end > at && (g.bytes + bytes > kGroupBytes || count + more > kGroupTiles)) break;
        g.bytes += bytes;
        count += more;
        ++g.end;
      }
      plan.bytes = std::max(plan.bytes, g.bytes);
      plan.groups.push_back(g);
      at = g.end;
    }
  };
  for (const bool split : {false, true}) {
    std::vector<uint32_t> small, large, others;
    uint64_t big = 0, tiles = 0;  // large's tiles of 256 and of 128
    for (uint32_t i = 0; i < n; ++i) {
      if (is_narrow(m[i]) || splits(m[i]) != split) continue;
      if (std::min(m[i].rows, m[i].cols) <= 64) {
        small.push_back(i);
      } else if (4 * area(i, 256) <= 5 * area(i, 64)) {
        large.push_back(i);
        big += area(i, 256) / (256 * 256);
        tiles += area(i, 128) / (128 * 128);
      } else {
        others.push_back(i);
      }
    }
    const bool whole = big >= kManyBig && 40 * up(big, 256) / 256 <= 23 * up(tiles, 512) / 512;
    if (!whole) {
      large.insert(large.end(), others.begin(), others.end());
      std::sort(large.begin(), large.end());
      others.clear();
    }
    add(large, split, false, whole);
    add(others, split, false, false);
    add(small, split, true, false);
  }
  return plan;
}

// The tiles of a launch: how many each matrix has, and how long one takes, in
// rounds of 64 inner elements and about as many as its ends are.
class Tiles {
 public:
  // Returns the first one's number.
  uint32_t add(uint32_t tiles, uint32_t inner, bool split) {
    list_.push_back({tiles, (inner + 63) / 64 * (split ? 3 : 1) + 16});
    count_ += tiles;
    return count_ - tiles;
  }
  void share(uint32_t tile) {
    dies_.rows = tile == 256 ? std::max(1u, std::min(kMostRows, (uint32_t)list_.size() / 4)) : 1;
    const uint32_t pieces = dies_.rows * kDies;
    uint64_t whole = 0, before = 0;
    for (const Some& s : list_) whole += (uint64_t)s.tiles * s.each;
    uint32_t first = 0, piece = 1;
    for (const Some& s : list_) {
      const uint64_t after = before + (uint64_t)s.tiles * s.each;
      for (; piece < pieces && after >= whole * piece / pieces; ++piece)
        dies_.first[piece] = first + (uint32_t)((whole * piece / pieces - before + s.each - 1) / s.each);
      before = after;
      first += s.tiles;
    }
    dies_.first[pieces] = count_;
    uint32_t most = 0;
    for (uint32_t d = 0; d < kDies; ++d) {
      uint32_t tiles = 0;
      for (uint32_t r = 0; r < dies_.rows; ++r) {
        const uint32_t p = r * kDies + (r % 2 ? kDies - 1 - d : d);
        tiles += dies_.first[p + 1] - dies_.first[p];
      }
      most = std::max(most, tiles);
    }
    grid_ = most * kDies;
  }
  const Dies& dies() const { return dies_; }
  uint32_t grid() const { return grid_; }
  bool empty() const { return list_.empty(); }

 private:
  struct Some {
    uint32_t tiles, each;
  };
  std::vector<Some> list_;
  uint32_t count_ = 0, grid_ = 0;
  Dies dies_{};
};

// Workgroups of a group's launches.
struct Launches {
  uint32_t parts = 0, packs = 0, sums = 0;
  Tiles cut, gram, square, next;
};

template <bool SPLIT>
hipError_t gram_t(const PolarItem* items, uint32_t n, const Launches& l, uint32_t tile, hipStream_t s) {
  if (!l.cut.empty()) {
    polar_cut_kernel<SPLIT><<<l.cut.grid(), Product<64, SPLIT>::kThreads, 0, s>>>(items, n, l.cut.dies());
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    polar_sum_kernel<SPLIT><<<l.sums, Product<64, SPLIT>::kThreads, 0, s>>>(items, n);
  } else if (tile == 64) {
    polar_gram_kernel<64, SPLIT><<<l.gram.grid(), Product<64, SPLIT>::kThreads, 0, s>>>(items, n, l.gram.dies());
  } else if (tile == 128) {
    polar_gram_kernel<128, SPLIT><<<l.gram.grid(), Product<128, SPLIT>::kThreads, 0, s>>>(items, n, l.gram.dies());
  } else {
    polar_gram_kernel<256, SPLIT><<<l.gram.grid(), Product<256, SPLIT>::kThreads, 0, s>>>(items, n, l.gram.dies());
  }
  return hipGetLastError();
}

template <bool SPLIT>
hipError_t square_t(const PolarItem* items, uint32_t n, const Launches& l, uint32_t tile, float b, float c, hipStream_t s) {
  if (tile == 64)
    polar_square_kernel<64, SPLIT><<<l.square.grid(), Product<64, SPLIT>::kThreads, 0, s>>>(items, n, l.square.dies(), b, c);
  else if (tile == 128)
    polar_square_kernel<128, SPLIT><<<l.square.grid(), Product<128, SPLIT>::kThreads, 0, s>>>(items, n, l.square.dies(), b, c);
  else
    polar_square_kernel<256, SPLIT><<<l.square.grid(), Product<256, SPLIT>::kThreads, 0, s>>>(items, n, l.square.dies(), b, c);
  return hipGetLastError();
}

template <int T, bool SPLIT, bool LAST, int PRODUCTS>
void launch_next(const PolarItem* items, uint32_t n, const Launches& l, float a, uint32_t step, hipStream_t s) {
  polar_next_kernel<T, SPLIT, LAST, PRODUCTS><<<l.next.grid(), Product<T, SPLIT>::kThreads, 0, s>>>(items, n, l.next.dies(), a, step);
}

template <int T, bool SPLIT>
hipError_t next_t(const PolarItem* items, uint32_t n, const Launches& l, float a, uint32_t step, uint32_t steps, hipStream_t s) {
  if constexpr (SPLIT) {
    if (step + 1 == steps)
      launch_next<T, true, true, 3>(items, n, l, a, step, s);
    else
      launch_next<T, true, false, 3>(items, n, l, a, step, s);
  } else {
    if (step + 1 == steps)
      launch_next<T, false, true, 1>(items, n, l, a, step, s);
    else if (step + 2 == steps)  // what X's rounding leaves is multiplied by `a` once more
      launch_next<T, false, false, 1>(items, n, l, a, step, s);
    else
      launch_next<T, false, false, 2>(items, n, l, a, step, s);
  }
  return hipGetLastError();
}

template <bool SPLIT>
hipError_t steps_t(const PolarItem* items, uint32_t n, const Launches& l, const Group& g, const double* c, uint32_t steps,
                   hipStream_t s) {
  for (uint32_t k = 0; k < steps; ++k, c += 3) {
    hipError_t e = gram_t<SPLIT>(items, n, l, g.gram_tile, s);
    if (e != hipSuccess) return e;
    if ((e = square_t<SPLIT>(items, n, l, g.gram_tile, (float)c[1], (float)c[2], s)) != hipSuccess) return e;
    const float a = (float)c[0];
    if (g.tile == 256)
      e = next_t<256, SPLIT>(items, n, l, a, k, steps, s);
    else if (g.tile == 128)
      e = next_t<128, SPLIT>(items, n, l, a, k, steps, s);
    else
      e = next_t<64, SPLIT>(items, n, l, a, k, steps, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t run_group(const PolarMatrix* m, const uint32_t* order, const Group& g, const PolarRule& r, const double* c,
                     uint32_t steps, char* ws, hipStream_t s) {
  const uint32_t n = g.end - g.begin;
  PolarItem* items = reinterpret_cast<PolarItem*>(ws);
  char* at = ws + up256((uint64_t)n * sizeof(PolarItem));
  Launches l;
  for (uint32_t i = 0; i < n; i += kUploads) {
    PolarUpload u;
    const uint32_t many = std::min(kUploads, n - i);
    for (uint32_t j = 0; j < many; ++j) {
      PolarItem& it = u.item[j];
      at += lay_out(m[order[g.begin + i + j]], g.tile, g.split, g.cuts, at, &it);
      const uint32_t pt = it.p / g.tile, qt = it.q / g.tile, side = it.p / g.gram_tile, upper = side * (side + 1) / 2;
      it.first_part = l.parts;
      it.first_pack = l.packs;
      it.first_sum = l.sums;
      it.first_gram = l.gram.add(upper, it.cols, g.split);
      l.square.add(upper, it.rows, g.split);
      if (g.cuts > 1) it.first_cut = l.cut.add(upper * it.cuts, it.cols / it.cuts, g.split);
      it.first_next = l.next.add(pt * qt, it.rows, g.split);
      l.parts += it.parts;
      l.packs += it.p / 64 * (it.q / 64);
      l.sums += upper;
    }
    polar_upload_kernel<<<1, kPolarThreads, 0, s>>>(u, items + i, many);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  for (Tiles* tiles : {&l.cut, &l.gram, &l.square, &l.next}) tiles->share(g.tile);
  polar_norm_kernel<<<l.parts, kPolarThreads, 0, s>>>(items, n, r);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (g.split)
    polar_pack_kernel<true><<<l.packs, kPolarThreads, 0, s>>>(items, n, r);
  else
    polar_pack_kernel<false><<<l.packs, kPolarThreads, 0, s>>>(items, n, r);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  return g.split ? steps_t<true>(items, n, l, g, c, steps, s) : steps_t<false>(items, n, l, g, c, steps, s);
}

}  // namespace

uint64_t polar_workspace_bytes(const PolarMatrix* m, uint32_t n) { return make_plan(m, n).bytes; }

hipError_t launch_polar(const PolarMatrix* m, uint32_t n, const PolarRule& r, const double* coefficients,
                        uint32_t steps, void* ws, hipStream_t s) {
  const Plan plan = make_plan(m, n);
  if (!plan.narrow.empty()) {
    const hipError_t e = launch_narrow(plan.narrow.data(), (uint32_t)plan.narrow.size(), r, coefficients, steps, ws, s);
    if (e != hipSuccess) return e;
  }
  for (const Group& g : plan.groups) {
    const hipError_t e = run_group(m, plan.order.data(), g, r, coefficients, steps, static_cast<char*>(ws), s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace hkvt
