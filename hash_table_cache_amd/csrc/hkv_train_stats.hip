// gfx950 kernels of the token statistics (include/hkv_train.h): log-probability,
// entropy and the k largest logits of each row, and the gradient through the
// first two.
//
// Row mathematics. With M the row's maximum, a_v = (M - x_v) / tau >= 0,
// S = sum over v != y of e^-a_v and W = sum over v != y of a_v e^-a_v:
//   T = S + e^-a_y,  logp = -a_y - log T,  H = log T + (W + a_y e^-a_y) / T.
// Both terms of H are sums of what is not negative, so nothing cancels where a
// row is nearly certain; the label stays out of the sums for the same reason as
// in token_logprobs. A row is read once: S and W are rescaled when a larger
// maximum comes, and the k largest elements are kept beside them.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "hkv_train_internal.h"
#include "hkv_train_rows.h"

namespace hkvt {
namespace {

constexpr float kLn2 = 0.69314718055994530942f;

// The value of the lane whose number differs in bit W: by the ways that lanes of a
// wave have to each other's registers, a third of the time of one through LDS.
template <int W>
__device__ __forceinline__ uint32_t lane_xor(uint32_t v) {
  if constexpr (W == 1) return __builtin_amdgcn_update_dpp(0, v, 0xB1, 0xF, 0xF, true);  // quad_perm 1 0 3 2
  if constexpr (W == 2) return __builtin_amdgcn_update_dpp(0, v, 0x4E, 0xF, 0xF, true);  // quad_perm 2 3 0 1
  if constexpr (W == 4) {  // the mirror of 8 lanes, then of 4
    const uint32_t m = __builtin_amdgcn_update_dpp(0, v, 0x141, 0xF, 0xF, true);
    return __builtin_amdgcn_update_dpp(0, m, 0x1B, 0xF, 0xF, true);
  }
  if constexpr (W == 8) return __builtin_amdgcn_update_dpp(0, v, 0x128, 0xF, 0xF, true);  // 16 lanes turned by 8
  if constexpr (W == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return threadIdx.x & 16 ? r[0] : r[1];
  }
  const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return threadIdx.x & 32 ? r[0] : r[1];
}

template <int W>
__device__ __forceinline__ float lane_xor(float v) {
  return as_float(lane_xor<W>(__builtin_bit_cast(uint32_t, v)));
}

template <int W>
__device__ __forceinline__ unsigned long long lane_xor(unsigned long long v) {
  return (unsigned long long)lane_xor<W>((uint32_t)(v >> 32)) << 32 | lane_xor<W>((uint32_t)v);
}

template <int W>
__device__ __forceinline__ double lane_xor(double v) {
  return __builtin_bit_cast(double, lane_xor<W>(__builtin_bit_cast(unsigned long long, v)));
}

// Running maximum and sums of the elements a thread has seen; w is in units of
// log 2, as the exponents are.
struct Spread {
  float m = -kInf;
  double s = 0.0, w = 0.0;

  // Takes the sums to a new base, `t` = (old - new) / tau in units of log 2.
  __device__ __forceinline__ void rescale(float t) {
    const double f = exp2_fast(t);
    w = f == 0.0 ? 0.0 : f * (w - s * (double)t);
    s *= f;
  }

  __device__ __forceinline__ void raise(float mx, const Scale& c) {
    if (__any(mx > m)) {
      const float top = fmaxf(m, mx);
      const float t = top == -kInf ? 0.0f : m - top;
      rescale(fmaf(t, c.k_hi, t * c.k_lo));
      m = top;
    }
  }

  // What distances are taken from.
  __device__ __forceinline__ float base() const { return m == -kInf ? 0.0f : m; }

  // Up to F elements are added in 32 bits before 64, in es and as.
  __device__ __forceinline__ void flush(float* es, float* as) {
    s += (double)*es;
    w += (double)*as;
    *es = *as = 0.0f;
  }

  // N elements' distances from base(), none above it.
  template <int N, int F>
  __device__ __forceinline__ void add(const float* t, const Scale& c, float* es, float* as) {
    float e[N], a[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float z = fmaf(t[i], c.k_hi, t[i] * c.k_lo);
      e[i] = exp2_fast(z);
      a[i] = e[i] * fminf(-z, 1024.0f);  // a masked element has no weight, nor an infinite distance
    }
    constexpr int G = N < F ? N : F;
#pragma unroll
    for (int i = 0; i < N; i += G) {
#pragma unroll
      for (int w = G / 2; w > 0; w /= 2)
#pragma unroll
        for (int j = 0; j < w; ++j) {
          e[i + j] += e[i + j + w];
          a[i + j] += a[i + j + w];
        }
      *es += e[i];
      *as += a[i];
      if (N >= F) flush(es, as);
    }
  }
};

// The elements of a vector less `base`. Halves are subtracted as they are: their
// conversion takes as long as four subtractions (4096 x 131072 fp16: 195 us
// against 245 us, with four vectors' sums in 32 bits before 64 and no alternatives).
template <typename T>
__device__ __forceinline__ void distances(u32x4 raw, float base, float* t) {
  constexpr int K = Io<T>::K;
  if constexpr (std::is_same_v<T, _Float16>) {
    float one = 1.0f;
    asm("" : "+s"(one));  // a multiplication by it would be left out, and with it the mixed instruction
#pragma unroll
    for (int i = 0; i < K; ++i) t[i] = fmaf((float)as_halves(raw[i / 2])[i % 2], one, -base);
  } else {
    Io<T>::unpack(raw, t);
#pragma unroll
    for (int i = 0; i < K; ++i) t[i] -= base;
  }
}

template <typename V>
__device__ __forceinline__ V sum_lanes(V v) {
  v += lane_xor<1>(v);
  v += lane_xor<2>(v);
  v += lane_xor<4>(v);
  v += lane_xor<8>(v);
  v += lane_xor<16>(v);
  return v + lane_xor<32>(v);
}

__device__ __forceinline__ float max_lanes(float v) {
  v = fmaxf(v, lane_xor<1>(v));
  v = fmaxf(v, lane_xor<2>(v));
  v = fmaxf(v, lane_xor<4>(v));
  v = fmaxf(v, lane_xor<8>(v));
  v = fmaxf(v, lane_xor<16>(v));
  return fmaxf(v, lane_xor<32>(v));
}

// Joins a wave's lanes; every lane gets the sums.
__device__ __forceinline__ void join_lanes(Spread& r, const Scale& c) {
  const float top = max_lanes(r.m), base = top == -kInf ? 0.0f : top;
  const float t = r.m - base;
  r.rescale(fmaf(t, c.k_hi, t * c.k_lo));
  r.m = top;
  r.s = sum_lanes(r.s);
  r.w = sum_lanes(r.w);
}

struct StatsEnd {
  double logp, lse, entropy;
  bool counts;  // false: the row is left out
};

// (M, S, W, x_y) -> log-probability, normaliser and entropy.
__device__ __forceinline__ StatsEnd finish_stats(const Spread& r, float xy, double inv_tau) {
  if (r.m == -kInf && xy == -kInf && r.s == 0.0) return StatsEnd{0.0, -(double)kInf, 0.0, false};
  StatsEnd e;
  e.counts = true;
  double d = ((double)xy - (double)r.m) * inv_tau;
  if (xy == kInf) d = __builtin_nan("");
  const double w = r.w * 0.69314718055994530942;
  if (d >= 0.0) {
    const double f = exp_of(-d), er = r.s * f, lt = log1p_of(er);
    e.logp = -lt;
    e.lse = (double)xy * inv_tau + lt;
    e.entropy = lt + (f == 0.0 ? 0.0 : f * (w + r.s * d)) / (1.0 + er);
  } else {
    const double f = exp_of(d), total = r.s + f, lt = log_of(total);
    e.logp = d - lt;
    e.lse = (double)r.m * inv_tau + lt;
    e.entropy = lt + (f == 0.0 ? w : w - f * d) / total;
  }
  if (e.entropy < 0.0) e.entropy = 0.0;
  return e;
}

__device__ __forceinline__ StatsEnd nan_stats() {
  const double q = __builtin_nan("");
  return StatsEnd{q, q, q, true};
}

// The largest elements. An element is a key of 64 bits that sorts as they do:
// its value in order, and under it the index, lower ones above. 0 is no element.
typedef unsigned long long Key;

__device__ __forceinline__ Key key_of(float f, uint32_t i) {
  const uint32_t u = __builtin_bit_cast(uint32_t, f + 0.0f);  // -0 is 0
  return (Key)(u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u)) << 32 | (uint32_t)~i;
}

__device__ __forceinline__ float value_of(Key k) {
  const uint32_t u = (uint32_t)(k >> 32);
  return as_float(u & 0x80000000u ? u ^ 0x80000000u : ~u);
}

__device__ __forceinline__ uint32_t index_of(Key k) { return ~(uint32_t)k; }

// A step of a bitonic sort: the larger of two lanes' values goes to the lower one
// where `down`.
template <int W, typename V>
__device__ __forceinline__ V sort_step(V v, bool down) {
  const V o = lane_xor<W>(v);
  return (((threadIdx.x & W) == 0) == down) == (v > o) ? v : o;
}

// Blocks of SIZE lanes that go up and then down, sorted.
template <int SIZE, typename V>
__device__ __forceinline__ V sort_blocks(V v, bool down) {
  if constexpr (SIZE >= 64) v = sort_step<32>(v, down);
  if constexpr (SIZE >= 32) v = sort_step<16>(v, down);
  if constexpr (SIZE >= 16) v = sort_step<8>(v, down);
  if constexpr (SIZE >= 8) v = sort_step<4>(v, down);
  if constexpr (SIZE >= 4) v = sort_step<2>(v, down);
  return sort_step<1>(v, down);
}

// The lanes' values, falling.
template <typename V>
__device__ __forceinline__ V sort_lanes(V v) {
  const uint32_t lane = threadIdx.x;
  v = sort_blocks<2>(v, (lane & 2) == 0);
  v = sort_blocks<4>(v, (lane & 4) == 0);
  v = sort_blocks<8>(v, (lane & 8) == 0);
  v = sort_blocks<16>(v, (lane & 16) == 0);
  v = sort_blocks<32>(v, (lane & 32) == 0);
  return sort_blocks<64>(v, true);
}

// The 64 largest of two sorted lists. `other` comes in reverse.
__device__ __forceinline__ Key merge_lanes(Key v, Key other) { return sort_blocks<64>(v > other ? v : other, true); }

__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// What the W waves of a team share while they look for the k <= 64 largest
// elements: what each has gathered, H elements at most, and the bounds that
// they found.
template <int W, int H>
struct TopsShared {
  Key held[W][H];
  u32x4 vecs[W][H];  // vectors with elements that may pass, and the first one's index
  uint32_t at[W][H];
  float bound[W];
  uint32_t count[W];
};

// Takes the first element off a vector.
template <typename T>
__device__ __forceinline__ float first_of(u32x4& x) {
  const uint32_t w = x[0];
  if constexpr (sizeof(T) == 4) {
    x = u32x4{x[1], x[2], x[3], 0};
    return as_float(w);
  } else {
    x = u32x4{w >> 16 | x[1] << 16, x[1] >> 16 | x[2] << 16, x[2] >> 16 | x[3] << 16, x[3] >> 16};
    return (float)__builtin_bit_cast(T, (uint16_t)w);
  }
}

// The k largest elements that a wave has seen, sorted, one a lane, and a bound
// under which no element comes among the team's. Vectors of which an element passes
// the bound are gathered in LDS and looked through 64 at a time, a lane each, for
// they come one or two at a time; their elements that pass are gathered again and
// join the list 64 at a time (4096 x 131072 fp16, 64 alternatives: 211 us against
// 283 us with vectors looked through as they come).
// The bound: a wave knows j = ceil(k / W) lanes that have seen an element of at
// least b_w; then k elements are at least the ceil(k / j)-th largest of the b_w. Of a row of
// random order few more than k elements pass it (64 of 131072 by 8 waves: about
// 270, where each wave's own 64th lane lets 4000 pass), and waves need not wait for
// each other's bounds but in the first round: an old one is only lower.
template <int W, int H>
struct Tops {
  using Shared = TopsShared<W, H>;
  Key list = 0;
  float bound = -kInf;    // an element of this value passes
  uint32_t bound_at = 0;  // if its index is lower
  uint32_t count = 0;     // gathered
  uint32_t vecs = 0;      // vectors
  float seen = -kInf;     // by this lane
  bool first = true, taken = false;
  Shared& sh;
  uint32_t k, wave;
  int lane;

  __device__ __forceinline__ Tops(Shared& sh_, uint32_t k_, uint32_t wave_)
      : sh(sh_), k(k_), wave(wave_), lane(threadIdx.x & 63) {}

  // The bound that lanes of largest elements `mx` in the next round give.
  __device__ __forceinline__ void expect(float mx) {
    seen = fmaxf(seen, mx);
    if (!first && __popcll(__ballot(mx > bound)) < 4) return;
    const uint32_t j = (k + W - 1) / W, m = (k + j - 1) / j;
    const float own = j == 1 ? max_lanes(seen) : __shfl(sort_lanes(seen), (int)j - 1);
    float least = own;
    if (W > 1) {
      if (lane == 0) sh.bound[wave] = own;
      if (first)
        __syncthreads();
      else
        wave_sync();
      const float mine = *(volatile float*)&sh.bound[lane % W];
      uint32_t above = 0;  // of the others' bounds
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float o = __shfl(mine, w);
        above += o > mine || (o == mine && w < lane % W) ? 1 : 0;
      }
      least = __shfl(mine, __builtin_ctzll(__ballot(above == m - 1) | 1ull << 63));
    }
    first = false;
    if (least == -kInf && W > 1) least = __shfl(sort_lanes(seen), (int)k - 1);  // a wave without candidates
    if (least > bound) {
      bound = least;
      bound_at = ~0u;
    }
  }

  __device__ __forceinline__ bool passes(float f, uint32_t i) const {
    return f > bound || (f == bound && i < bound_at);
  }

  __device__ __forceinline__ void add(float f, uint32_t i, bool live) {
    const bool in = live && passes(f, i);
    const uint64_t who = __ballot(in);
    if (who == 0) return;
    const uint32_t below = __builtin_amdgcn_mbcnt_hi((uint32_t)(who >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)who, 0));
    if (in) sh.held[wave][count + below] = key_of(f, i);
    count += __popcll(who);
    if (count >= 64) take();
  }

  // Gathers the vectors of lanes whose largest element `mx` may pass; `i` is the
  // index of their first element.
  template <typename T>
  __device__ __forceinline__ void gather(u32x4 raw, float mx, uint32_t i) {
    const bool in = mx >= fmaxf(bound, -__FLT_MAX__);
    const uint64_t who = __ballot(in);
    if (who == 0) return;
    const uint32_t below = __builtin_amdgcn_mbcnt_hi((uint32_t)(who >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)who, 0));
    if (in) {
      sh.vecs[wave][vecs + below] = raw;
      sh.at[wave][vecs + below] = i;
    }
    vecs += __popcll(who);
    if (vecs >= 64) look<T>();
  }

  // Looks through the last 64 vectors, or all of fewer.
  template <typename T>
  __device__ __forceinline__ void look() {
    constexpr int K = Io<T>::K;
    const uint32_t n = min(vecs, 64u);
    vecs -= n;
    wave_sync();
    const bool mine = (uint32_t)lane < n;
    u32x4 x = sh.vecs[wave][vecs + (mine ? lane : 0)];
    const uint32_t i = sh.at[wave][vecs + (mine ? lane : 0)];
    wave_sync();
#pragma unroll 1
    for (int j = 0; j < K; ++j) {
      const float f = first_of<T>(x);
      add(f, i + j, mine && f >= -__FLT_MAX__);
    }
  }

  // Joins the last 64 gathered ones, or all of fewer.
  __device__ __forceinline__ void take() {
    const uint32_t n = min(count, 64u);
    count -= n;
    wave_sync();
    const Key v = sort_lanes((uint32_t)lane < n ? sh.held[wave][count + lane] : 0);
    list = taken ? merge_lanes(list, __shfl(v, 63 - lane)) : v;
    taken = true;
    const Key last = __shfl(list, (int)k - 1);
    if (last) {
      const float at = value_of(last);
      if (at >= bound) {  // not below what expect() found
        bound_at = at > bound ? index_of(last) : min(bound_at, index_of(last));
        bound = at;
      }
    }
    wave_sync();
  }

  // The team's list, in its first wave. Few elements are that wave's to sort;
  // of many, every wave sorts its own, and pairs of lists are merged.
  __device__ __forceinline__ void join() {
    if (W == 1) {
      while (count) take();
      return;
    }
    if (lane == 0) sh.count[wave] = taken ? 1u << 16 : count;
    __syncthreads();
    uint32_t total = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) total += sh.count[w];
    if (total <= 128) {
      if (wave) return;
      for (uint32_t from = 0; from < total; from += 64) {
        uint32_t at = from + lane;
        Key v = 0;
        bool found = false;
#pragma unroll
        for (int w = 0; w < W; ++w) {
          if (!found && at < sh.count[w]) {
            v = sh.held[w][at];
            found = true;
          }
          if (!found) at -= sh.count[w];
        }
        v = sort_lanes(v);
        list = from ? merge_lanes(list, __shfl(v, 63 - lane)) : v;
      }
      return;
    }
    while (count) take();
    sh.held[wave][lane] = list;
    __syncthreads();
#pragma unroll
    for (int n = W / 2; n > 0; n /= 2) {
      if (wave < n) {
        list = merge_lanes(list, sh.held[wave + n][63 - lane]);
        if (n > 1) sh.held[wave][lane] = list;
      }
      if (n > 1) __syncthreads();
    }
  }
};

struct StatsArgs {
  Logits l;
  Scale c;
  Stats out;
  uint32_t first;  // row of the first team
};

// Writes a row's results: `lane` of its first wave, with the row's list.
__device__ __forceinline__ void write_stats(const StatsArgs& a, uint32_t t, const StatsEnd& e, Key list, int lane) {
  if (lane == 0) {
    a.out.logp[t] = (float)e.logp;
    if (a.out.lse) a.out.lse[t] = (float)e.lse;
    a.out.entropy[t] = (float)e.entropy;
  }
  if ((uint32_t)lane < a.out.k) {
    const bool lives = list != 0 && e.lse == e.lse;
    const double v = lives ? (double)value_of(list) * a.c.inv_tau - e.lse : e.lse == e.lse ? -(double)kInf : e.lse;
    a.out.top_logp[(uint64_t)t * a.out.k + lane] = (float)v;
    a.out.top_ids[(uint64_t)t * a.out.k + lane] = lives ? (int64_t)index_of(list) : -1;
  }
}

template <int NT, bool TOP>
using TopsOf = Tops<NT / 64, TOP ? 128 : 1>;

// One row, or a part of it, by a team: sums in r, the largest in the waves' lists.
template <typename T, int NT, int NV, bool TOP>
__device__ __forceinline__ void scan_row(const T* row, const Cut<T, NT>& cut, uint32_t y, uint32_t tid, const Scale& c,
                                         Spread& r, TopsOf<NT, TOP>& tops) {
  constexpr int K = Io<T>::K;
  const T* vecs = row + cut.head;
  const uint32_t yv = cut.vec_of(y), el = (y - cut.head) % K;
  for (uint32_t c0 = cut.begin; c0 < cut.end; c0 += NT * NV) {
    u32x4 raw[NV];
    float mx[NV], most = -kInf;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      raw[i] = no_vec<T>();
      if (c0 + i * NT + tid < cut.end) raw[i] = load_vec(vecs, c0 + i * NT + tid);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      mx[i] = vec_max<T>(raw[i]);
      most = fmaxf(most, mx[i]);
    }
    r.raise(most, c);
    if (TOP) tops.expect(most);
    const float base = r.base();
    float es = 0.0f, as = 0.0f;  // of up to kFloats elements
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      opaque(raw[i]);
      const uint32_t v = c0 + i * NT + tid;
      if (c0 + i * NT < cut.end) {
        float t[K];
        distances<T>(raw[i], base, t);
        if (__any(v == yv)) {
#pragma unroll
          for (int j = 0; j < K; ++j)
            if (v == yv && el == (uint32_t)j) t[j] = -kInf;
        }
        r.template add<K, Io<T>::kFloats>(t, c, &es, &as);
      }
      if (K < Io<T>::kFloats && ((i + 1) * K % Io<T>::kFloats == 0 || i + 1 == NV)) r.flush(&es, &as);
    }
    if (TOP) {
#pragma unroll
      for (int i = 0; i < NV; ++i) tops.template gather<T>(raw[i], mx[i], cut.head + (c0 + i * NT + tid) * K);
    }
  }
  if (TOP)
    while (tops.vecs) tops.template look<T>();
  for (uint32_t j0 = 0; j0 < cut.singles(); j0 += NT) {
    const uint32_t j = j0 + tid, i = cut.single(j);
    float f = j < cut.singles() ? (float)row[i] : -kInf;
    if (TOP) {
      tops.add(f, i, j < cut.singles());
    }
    if (i == y) f = -kInf;
    r.raise(f, c);
    f -= r.base();
    float es = 0.0f, as = 0.0f;
    r.template add<1, 1>(&f, c, &es, &as);
  }
  if (TOP) tops.join();
}

template <int W>
struct StatsShared {
  float m[W];
  double s[W], w[W];
};

// Joins the waves of a team; the first wave gets it all.
template <int NT>
__device__ __forceinline__ void join_waves(Spread& r, const Scale& c, StatsShared<NT / 64>& sh) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  join_lanes(r, c);
  if (NT == 64) return;
  constexpr int W = NT / 64;
  if (lane == 0) {
    sh.m[wave] = r.m;
    sh.s[wave] = r.s;
    sh.w[wave] = r.w;
  }
  __syncthreads();
  if (wave == 0) {
    r.m = lane < W ? sh.m[lane] : -kInf;
    r.s = lane < W ? sh.s[lane] : 0.0;
    r.w = lane < W ? sh.w[lane] : 0.0;
    join_lanes(r, c);  // every lane gets it
  }
}

// The teams' waves' LDS; without alternatives there is no list.
template <int NT, bool TOP>
struct StatsLds {
  static constexpr int kTeams = NT == 64 ? Team<NT>::kBlock / 64 : 1;
  StatsShared<NT / 64> sums;
  typename TopsOf<NT, TOP>::Shared tops[TOP ? kTeams : 1];
};

template <typename T, int NT, int NV, bool TOP>
__global__ __launch_bounds__(Team<NT>::kBlock) void stats_kernel(const StatsArgs a) {
  using Tm = Team<NT>;
  __shared__ StatsLds<NT, TOP> sh;
  const uint32_t tid = Tm::thread(), t = Tm::row(a.first, blockIdx.x);
  const int lane = threadIdx.x & 63;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (t >= a.l.rows) return;  // a whole team
  const T* row = static_cast<const T*>(a.l.x) + (uint64_t)t * a.l.x_stride;
  const int64_t y64 = a.l.labels[t];
  StatsEnd e;
  Key list = 0;
  if (y64 < 0) {
    e = StatsEnd{0.0, 0.0, 0.0, false};
  } else if (y64 >= (int64_t)a.l.vocab) {
    e = nan_stats();
  } else {
    const float xy = (float)row[y64];
    const Cut<T, NT> cut(row, a.l.vocab);
    Spread r;
    TopsOf<NT, TOP> tops(sh.tops[NT == 64 && TOP ? wave : 0], a.out.k, NT == 64 ? 0 : wave);
    scan_row<T, NT, NV, TOP>(row, cut, (uint32_t)y64, tid, a.c, r, tops);
    list = tops.list;
    join_waves<NT>(r, a.c, sh.sums);
    e = finish_stats(r, xy, a.c.inv_tau);
  }
  if (tid < 64) write_stats(a, t, e, list, lane);
}

// Few long rows: a row is shared by workgroups, whose sums and lists one joins.
struct StatsPartial {
  double s, w;
  float m;
};

constexpr uint32_t kStatsParts = 64;

template <typename T, bool TOP>
__global__ __launch_bounds__(256) void stats_part_kernel(const StatsArgs a, uint32_t parts, uint32_t size,
                                                         StatsPartial* partial, Key* lists) {
  constexpr int NT = 256, NV = 4;
  __shared__ StatsLds<NT, TOP> sh;
  const uint32_t tid = threadIdx.x, t = blockIdx.x / parts;
  const int64_t y64 = a.l.labels[t];
  if (y64 < 0 || y64 >= (int64_t)a.l.vocab) return;
  const T* row = static_cast<const T*>(a.l.x) + (uint64_t)t * a.l.x_stride;
  const Cut<T, NT> cut(row, a.l.vocab, blockIdx.x % parts, size);
  Spread r;
  TopsOf<NT, TOP> tops(sh.tops[0], a.out.k, __builtin_amdgcn_readfirstlane(tid >> 6));
  scan_row<T, NT, NV, TOP>(row, cut, (uint32_t)y64, tid, a.c, r, tops);
  join_waves<NT>(r, a.c, sh.sums);
  if (tid == 0) partial[blockIdx.x] = StatsPartial{r.s, r.w, r.m};
  if (TOP && tid < 64) lists[(uint64_t)blockIdx.x * 64 + tid] = tops.list;
}

template <typename T, bool TOP>
__global__ __launch_bounds__(512) void stats_join_kernel(const StatsArgs a, uint32_t parts, const StatsPartial* partial,
                                                         const Key* lists) {
  constexpr int W = 8;
  __shared__ Key held[W][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t t = blockIdx.x;
  const int64_t y64 = a.l.labels[t];
  const bool reads = y64 >= 0 && y64 < (int64_t)a.l.vocab;
  Key list = 0;
  if (TOP && reads) {
    for (uint32_t p = wave; p < parts; p += W)
      list = merge_lanes(list, lists[((uint64_t)t * parts + p) * 64 + 63 - lane]);
    held[wave][lane] = list;
    __syncthreads();
#pragma unroll
    for (int n = W / 2; n > 0; n /= 2) {
      if (wave < n) {
        list = merge_lanes(list, held[wave + n][63 - lane]);
        held[wave][lane] = list;
      }
      __syncthreads();
    }
  }
  if (wave) return;
  StatsEnd e;
  if (y64 < 0) {
    e = StatsEnd{0.0, 0.0, 0.0, false};
  } else if (!reads) {
    e = nan_stats();
  } else {
    Spread r;
    if ((uint32_t)lane < parts) {
      const StatsPartial p = partial[t * parts + lane];
      r.s = p.s;
      r.w = p.w;
      r.m = p.m;
    }
    join_lanes(r, a.c);
    e = finish_stats(r, (float)(static_cast<const T*>(a.l.x) + (uint64_t)t * a.l.x_stride)[y64], a.c.inv_tau);
  }
  write_stats(a, t, e, list, lane);
}

// The gradient: -p / tau (g + h (log p + H)), and g / tau more at the label.
struct StatsBack {
  Logits l;
  Scale c;
  const float* lse;
  const float* entropy;
  const float* g;
  const float* ge;
};

__device__ __forceinline__ float back_of(float x, const Scale& c, float lse, float h, float g, float ge) {
  float z = exponent(x, c, lse);
  z = z < -1024.0f ? -1024.0f : z;  // a masked element has no weight, nor an infinite distance
  return exp2_fast(z * kLog2e) * fmaf(-ge, z + h, -g);
}

template <typename T>
__device__ __forceinline__ u32x4 back_vec(u32x4 raw, const Scale& c, float lse, float h, float g, float ge) {
  constexpr int K = Io<T>::K;
  float f[K];
  Io<T>::unpack(raw, f);
#pragma unroll
  for (int i = 0; i < K; ++i) f[i] = back_of(f[i], c, lse, h, g, ge);
  return Io<T>::pack(f);
}

template <typename T, int NT>
__global__ __launch_bounds__(Team<NT>::kBlock) void stats_backward_kernel(const StatsBack a, uint32_t parts, uint32_t first) {
  using Tm = Team<NT>;
  const uint32_t tid = Tm::thread(), t = Tm::row(first, blockIdx.x / parts);
  if (t >= a.l.rows) return;
  const T* row = static_cast<const T*>(a.l.x) + (uint64_t)t * a.l.x_stride;
  T* out = static_cast<T*>(a.l.dx) + (uint64_t)t * a.l.dx_stride;
  const Cut<T, NT> cut(out, a.l.vocab, blockIdx.x % parts, Part<NT>::kVecs);
  const int64_t y64 = a.l.labels[t];
  const float lse = a.lse[t];
  float g = a.g ? (float)(a.g[t] * a.c.inv_tau) : 0.0f;
  const float ge = a.ge ? (float)(a.ge[t] * a.c.inv_tau) : 0.0f;
  const float h = ge == 0.0f ? 0.0f : a.entropy[t];
  if (y64 < 0 || lse == -kInf || (g == 0.0f && ge == 0.0f)) {
    zero_row<T, NT>(out, cut, tid);
    return;
  }
  if (y64 >= (int64_t)a.l.vocab) g = __builtin_nanf("");
  const uint32_t y = y64 >= (int64_t)a.l.vocab ? 0u : (uint32_t)y64;
  // the label's thread, the only one that writes its place, reads it first
  const uint32_t owner = cut.owner(y);
  const float fy = tid == owner ? (float)row[y] : 0.0f;
  for_vecs<T, NT, Part<NT>::kRounds>(row + cut.head, cut.begin, cut.end, tid, [&](u32x4 raw, uint32_t v) {
    store_vec(out + cut.head, v, back_vec<T>(raw, a.c, lse, h, g, ge));
  });
  for (uint32_t j = tid; j < cut.singles(); j += NT) {
    const uint32_t i = cut.single(j);
    float d = back_of((float)row[i], a.c, lse, h, g, ge);
    asm("" : "+v"(d));  // rounded to 32 bits first, as a vector's elements are, not once with the product
    out[i] = (T)d;
  }
  if (tid == owner)
    out[y] = (T)(float)((double)g * rest_of_label(fy, a.c, lse) + (double)back_of(fy, a.c, lse, h, 0.0f, ge));
}

template <typename T, int NT, int NV>
hipError_t stats_n(const StatsArgs& a, hipStream_t s) {
  return for_rows<NT>(a.l.rows, 1, [&](uint32_t first, uint32_t grid) {
    StatsArgs slice = a;
    slice.first = first;
    if (a.out.k)
      stats_kernel<T, NT, NV, true><<<grid, Team<NT>::kBlock, 0, s>>>(slice);
    else
      stats_kernel<T, NT, NV, false><<<grid, Team<NT>::kBlock, 0, s>>>(slice);
  });
}

// Whether rows are shared by workgroups: so few that one to a row leaves much of
// the chip idle, and longer than one of 1024 threads takes in a round (1 x 32768
// bf16: 15.5 us by one workgroup, 18.5 us shared). Calls with 20 alternatives,
// shared against not: 64 x 131072 bf16 21.5 us against 32.5 us, 100 rows 24.8
// against 32.8, but 200 rows 34.2 against 32.6.
constexpr uint32_t kStatsShared = 128;
constexpr uint32_t kUnits = 256;      // compute units
constexpr uint32_t kOneRound = 4096;  // vectors

bool shared_stats(const Logits& l) {
  return l.rows < kStatsShared && l.vocab / (l.kind == kF32 ? 4 : 8) > kOneRound;
}

uint32_t stats_parts(const Logits& l) {
  return std::min({l.vocab / (l.kind == kF32 ? 4 : 8) / 512, kStatsParts, 2048 / std::max(l.rows, 1u)});
}

template <typename T>
hipError_t stats_t(const StatsArgs& a, void* ws, hipStream_t s) {
  const uint32_t nv = a.l.vocab / Io<T>::K;
  if (shared_stats(a.l)) {
    const uint32_t parts = stats_parts(a.l), size = (nv - 1) / parts + 1;
    Workspace w{static_cast<char*>(ws)};
    StatsPartial* partial = w.take<StatsPartial>((uint64_t)a.l.rows * parts);
    Key* lists = w.take<Key>(a.out.k ? (uint64_t)a.l.rows * parts * 64 : 0);
    const uint32_t grid = a.l.rows * parts;
    if (a.out.k)
      stats_part_kernel<T, true><<<grid, 256, 0, s>>>(a, parts, size, partial, lists);
    else
      stats_part_kernel<T, false><<<grid, 256, 0, s>>>(a, parts, size, partial, lists);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (a.out.k)
      stats_join_kernel<T, true><<<a.l.rows, 512, 0, s>>>(a, parts, partial, lists);
    else
      stats_join_kernel<T, false><<<a.l.rows, 512, 0, s>>>(a, parts, partial, lists);
    return hipGetLastError();
  }
  if (nv <= 64 * 4) return stats_n<T, 64, 4>(a, s);
  // Small teams where rows are many, as for log-probabilities: more of them are in
  // a compute unit while others sort (20 alternatives, teams of 64 threads against
  // 256: 30000 x 2500 bf16 71 us against 219 us, 8000 x 8000 40 against 69; of 256
  // against 512: 4096 x 131072 fp16 210 against 247, 1000 x 60000 bf16 37 against
  // 45, but 512 x 131072, of which teams of 512 are all there at once, 43 against 40).
  if (nv <= 64 * 16) return a.l.rows >= 1024 ? stats_n<T, 64, 8>(a, s) : stats_n<T, 256, 4>(a, s);
  if (a.l.rows > 2 * kUnits) return stats_n<T, 256, 8>(a, s);
  if (a.l.rows < kFewRows && nv <= kOneRound) return stats_n<T, 1024, 4>(a, s);
  return stats_n<T, 512, 8>(a, s);
}

template <typename T, int NT>
hipError_t stats_backward_n(const StatsBack& a, hipStream_t s) {
  const uint32_t parts = Part<NT>::parts(a.l.vocab / Io<T>::K);
  return for_rows<NT>(a.l.rows, parts, [&](uint32_t first, uint32_t grid) {
    stats_backward_kernel<T, NT><<<grid, Team<NT>::kBlock, 0, s>>>(a, parts, first);
  });
}

// Teams as in the gradient of the log-probabilities, which moves the same bytes.
template <typename T>
hipError_t stats_backward_t(const StatsBack& a, hipStream_t s) {
  const uint32_t nv = a.l.vocab / Io<T>::K;
  if (nv <= 16 * 4) return stats_backward_n<T, 16>(a, s);
  if (nv <= 64 * 8) return stats_backward_n<T, 64>(a, s);
  return stats_backward_n<T, 128>(a, s);
}

}  // namespace

uint64_t stats_workspace_bytes(const Logits& l, uint32_t k) {
  if (!shared_stats(l)) return 0;
  const uint64_t n = (uint64_t)l.rows * stats_parts(l);
  return up16(n * sizeof(StatsPartial)) + (k ? n * 64 * sizeof(Key) : 0);
}

hipError_t launch_stats(const Logits& l, const Stats& out, void* ws, hipStream_t s) {
  const StatsArgs a{l, make_scale(l.tau), out, 0};
  if (l.kind == kF32) return stats_t<float>(a, ws, s);
  if (l.kind == kBF16) return stats_t<__bf16>(a, ws, s);
  return stats_t<_Float16>(a, ws, s);
}

hipError_t launch_stats_backward(const Logits& l, const float* lse, const float* entropy, const float* g,
                                 const float* ge, hipStream_t s) {
  const StatsBack a{l, make_scale(l.tau), lse, entropy, g, ge};
  if (l.kind == kF32) return stats_backward_t<float>(a, s);
  if (l.kind == kBF16) return stats_backward_t<__bf16>(a, s);
  return stats_backward_t<_Float16>(a, s);
}

}  // namespace hkvt
