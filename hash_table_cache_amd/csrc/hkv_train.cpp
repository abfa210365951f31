// Host side of the C ABI declared in include/hkv_train.h: argument checks and
// launches. The calls keep no state and allocate nothing on the device.
#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <exception>
#include <numeric>
#include <string>
#include <vector>

#include "hkv_train.h"
#include "hkv_train_internal.h"

#define HKV_API extern "C" __attribute__((visibility("default")))

namespace {

thread_local std::string g_error;

hkv_status fail(hkv_status code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_error = buf;
  return code;
}

hkv_status fail_hip(hipError_t e, const char* what) {
  (void)hipGetLastError();
  return fail(HKV_EHIP, "%s: %s", what, hipGetErrorString(e));
}

// Runs a call's body; what it throws (out of host memory) becomes a status.
template <typename F>
hkv_status guarded(F&& body) {
  try {
    return body();
  } catch (const std::exception& e) {
    return fail(HKV_ENOMEM, "%s", e.what());
  } catch (...) {
    return fail(HKV_ENOMEM, "unknown exception");
  }
}

class DeviceGuard {
 public:
  explicit DeviceGuard(int device) : target_(device) {
    err_ = hipGetDevice(&prev_);
    if (err_ == hipSuccess && prev_ != target_) err_ = hipSetDevice(target_);
  }
  ~DeviceGuard() {
    if (err_ == hipSuccess && prev_ != target_) (void)hipSetDevice(prev_);
  }
  hipError_t error() const { return err_; }

 private:
  int prev_ = -1;
  int target_;
  hipError_t err_;
};

#define HKV_TRY(expr)                    \
  do {                                   \
    const hkv_status st_ = (expr);       \
    if (st_ != HKV_OK) return st_;       \
  } while (0)

// The buffers of one call. The first one checked decides the GPU and has to be
// device memory; the others have to be memory that this GPU can access (its
// own, or pinned host memory). Each lies inside one allocation. Allocations are
// remembered while the call lasts: a call's small tensors mostly share one, and
// a lookup costs 0.1 us.
class Buffers {
 public:
  int device() const { return device_; }

  hkv_status check(const void* p, uint64_t bytes, const char* what, int64_t index = -1) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    for (const Range& r : known_)
      if (a >= r.begin && a < r.end && bytes <= r.end - a) return HKV_OK;
    char name[48];
    if (index >= 0) {
      std::snprintf(name, sizeof(name), "%s[%lld]", what, (long long)index);
      what = name;
    }
    if (!p) return fail(HKV_EINVAL, "%s is NULL", what);
    hipPointerAttribute_t attr;
    std::memset(&attr, 0, sizeof(attr));
    hipError_t e = hipPointerGetAttributes(&attr, p);
    if (e != hipSuccess || attr.type == hipMemoryTypeUnregistered) {
      (void)hipGetLastError();
      return fail(HKV_EINVAL, "%s (%p) is not device-accessible memory (pageable host memory?)", what, p);
    }
    if (device_ < 0) {
      if (attr.type != hipMemoryTypeDevice) return fail(HKV_EINVAL, "%s (%p) is not device memory", what, p);
      device_ = attr.device;
    } else if (attr.type == hipMemoryTypeDevice && attr.device != device_) {
      return fail(HKV_EINVAL, "%s lives on device %d, the call runs on device %d", what, attr.device, device_);
    }
    hipDeviceptr_t base = nullptr;
    size_t size = 0;
    e = hipMemGetAddressRange(&base, &size, const_cast<void*>(p));
    if (e == hipSuccess && base && size) {
      const uint64_t off = a - reinterpret_cast<uintptr_t>(base);
      if (off > size || bytes > size - off)
        return fail(HKV_EINVAL, "%s holds %llu bytes past %p, call needs %llu", what,
                    static_cast<unsigned long long>(size - off), p, static_cast<unsigned long long>(bytes));
      known_[next_++ % 4] = Range{a - off, a - off + size};
    } else {
      (void)hipGetLastError();
    }
    return HKV_OK;
  }

 private:
  struct Range {
    uintptr_t begin = 0, end = 0;
  };
  int device_ = -1;
  Range known_[4];
  unsigned next_ = 0;
};

bool kind_size(uint32_t kind, uint64_t* size) {
  if (kind > hkvt::kF16) return false;
  *size = kind == hkvt::kF32 ? 4 : 2;
  return true;
}

bool overlap(const void* a, uint64_t an, const void* b, uint64_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return an && bn && x < y + bn && y < x + an;
}

// Whether two [rows][vocab] arrays whose ranges overlap lie in different columns
// of the same wider rows: no row of the one then reaches into a row of the other.
bool beside(const void* a, uint64_t a_stride, const void* b, uint64_t b_stride, uint64_t vocab, uint64_t es) {
  if (a_stride != b_stride) return false;
  const int64_t elems = ((int64_t)reinterpret_cast<uintptr_t>(a) - (int64_t)reinterpret_cast<uintptr_t>(b)) / (int64_t)es;
  const int64_t stride = (int64_t)a_stride, column = ((elems % stride) + stride) % stride;
  return column >= (int64_t)vocab && column <= stride - (int64_t)vocab;
}

// Whether rows this far apart reach past 2^60 elements, whose bytes the checks
// below (and the kernels' addresses) could no longer count in 64 bits.
bool too_far(uint64_t rows, uint64_t stride) { return rows > 1 && stride > (1ull << 60) / (rows - 1); }

// The arguments that every operator on logits has. A call without rows looks
// at no array but its scalar outputs.
hkv_status check_logits(Buffers& buffers, uint64_t rows, uint64_t vocab, uint32_t dtype, const void* logits,
                        uint64_t stride, const int64_t* labels, float temperature, const void* grad,
                        uint64_t grad_stride, hkvt::Logits* out) {
  uint64_t es = 0;
  if (!kind_size(dtype, &es)) return fail(HKV_EINVAL, "dtype %u is none of HKV_F32, HKV_BF16, HKV_F16", dtype);
  if (rows >= (1ull << 31)) return fail(HKV_EINVAL, "rows = %llu, the limit is 2^31 - 1", (unsigned long long)rows);
  if (vocab == 0 || vocab >= (1ull << 29))
    return fail(HKV_EINVAL, "vocab = %llu is outside 1 .. 2^29 - 1", (unsigned long long)vocab);
  if (!(temperature > 0.0f) || !std::isfinite(temperature) || !std::isfinite(1.0f / temperature))
    return fail(HKV_EINVAL, "temperature = %g has to be a positive finite number", (double)temperature);
  if (stride < vocab || stride > (1ull << 40))
    return fail(HKV_EINVAL, "logits_stride = %llu with vocab = %llu", (unsigned long long)stride,
                (unsigned long long)vocab);
  if (grad && (grad_stride < vocab || grad_stride > (1ull << 40)))
    return fail(HKV_EINVAL, "grad_stride = %llu with vocab = %llu", (unsigned long long)grad_stride,
                (unsigned long long)vocab);
  if (too_far(rows, stride) || (grad && too_far(rows, grad_stride)))
    return fail(HKV_EINVAL, "%s = %llu with rows = %llu: an array of more than 2^60 elements",
                too_far(rows, stride) ? "logits_stride" : "grad_stride",
                (unsigned long long)(too_far(rows, stride) ? stride : grad_stride), (unsigned long long)rows);
  *out = hkvt::Logits{logits, stride, const_cast<void*>(grad), grad_stride, labels, (uint32_t)rows, (uint32_t)vocab,
                      dtype, temperature};
  if (rows == 0) return HKV_OK;
  const uint64_t bytes = ((rows - 1) * stride + vocab) * es;
  HKV_TRY(buffers.check(logits, bytes, "logits"));
  if (reinterpret_cast<uintptr_t>(logits) % es) return fail(HKV_EINVAL, "logits is not aligned to its type");
  HKV_TRY(buffers.check(labels, rows * 8, "labels"));
  if (grad) {
    const uint64_t gbytes = ((rows - 1) * grad_stride + vocab) * es;
    HKV_TRY(buffers.check(grad, gbytes, "grad_out"));
    if (reinterpret_cast<uintptr_t>(grad) % es) return fail(HKV_EINVAL, "grad_out is not aligned to its type");
    if (!(grad == logits && grad_stride == stride) && overlap(grad, gbytes, logits, bytes) &&
        !beside(grad, grad_stride, logits, stride, vocab, es))
      return fail(HKV_EINVAL, "grad_out overlaps logits without being the same array");
  }
  return HKV_OK;
}

hkv_status check_workspace(Buffers& buffers, const void* ws, uint64_t bytes, uint64_t need) {
  if (bytes < need)
    return fail(HKV_EINVAL, "workspace_bytes = %llu, the call needs %llu", (unsigned long long)bytes,
                (unsigned long long)need);
  HKV_TRY(buffers.check(ws, need, "workspace"));
  if (reinterpret_cast<uintptr_t>(ws) & 15) return fail(HKV_EINVAL, "workspace is not 16-byte aligned");
  return HKV_OK;
}

// Whether the singular values and what a step makes of them stay in the range
// that the kernels hold: they start in [0, 1], and over the interval that a step
// can reach, |s| < 3.9 (A = s^2 < 16) and |b s^2 + c s^4| < 15.5 are required.
hkv_status check_coefficients(uint32_t steps, const double* c) {
  if (steps == 0 || steps > hkvt::kMostSteps)
    return fail(HKV_EINVAL, "steps = %u is outside 1 .. %u", steps, hkvt::kMostSteps);
  if (!c) return fail(HKV_EINVAL, "coefficients is NULL");
  double most = 1.0;
  for (uint32_t k = 0; k < steps; ++k) {
    const double a = c[3 * k], b = c[3 * k + 1], d = c[3 * k + 2];
    if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(d))
      return fail(HKV_EINVAL, "coefficients of step %u are not finite", k);
    const double s = most * (1.0 + 1.0 / 256), end = s * s;  // rounding included
    double value = 0.0, inner = 0.0;
    const auto at = [&](double square) {
      if (!(square >= 0.0 && square <= end)) return;
      inner = std::max(inner, std::fabs(square * (b + d * square)));
      value = std::max(value, std::fabs(std::sqrt(square) * (a + square * (b + d * square))));
    };
    at(end);
    if (d != 0.0) {
      at(-b / (2.0 * d));
      const double root = std::sqrt(std::max(0.0, 9.0 * b * b - 20.0 * a * d));
      at((-3.0 * b + root) / (10.0 * d));
      at((-3.0 * b - root) / (10.0 * d));
    } else if (b != 0.0) {
      at(-a / (3.0 * b));
    }
    if (!(s < 3.9) || !(inner < 15.5))
      return fail(HKV_EINVAL, "coefficients of step %u take singular values out of range (up to %g, inner part %g)", k,
                  s, inner);
    most = std::max(value, 1e-6);
  }
  if (!(most < 3.9)) return fail(HKV_EINVAL, "coefficients take singular values out of range (up to %g)", most);
  return HKV_OK;
}

// The memory of matrices: no written one may share an element with another. Two
// whose ranges overlap may lie in different columns of the same wider rows, and one
// of them have only some of the rows, or a single one.
class Places {
 public:
  void add(const void* p, uint64_t rows, uint64_t cols, uint64_t stride, uint64_t es, bool written) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    list_.push_back({a, a + ((rows - 1) * stride + cols) * es, rows > 1 ? stride * es : 0, cols * es, written});
  }
  bool clash() {
    std::sort(list_.begin(), list_.end(), [](const Place& a, const Place& b) { return a.begin < b.begin; });
    std::vector<Place> written, read;  // those that may reach further
    for (const Place& p : list_) {
      const auto over = [&](const Place& o) { return o.end <= p.begin; };
      written.erase(std::remove_if(written.begin(), written.end(), over), written.end());
      for (const Place& o : written)
        if (!apart(o, p)) return true;
      if (p.written) {
        read.erase(std::remove_if(read.begin(), read.end(), over), read.end());
        for (const Place& o : read)
          if (!apart(o, p)) return true;
      }
      (p.written ? written : read).push_back(p);
    }
    return false;
  }

 private:
  struct Place {
    uintptr_t begin, end;
    uint64_t stride, width;  // stride: 0 of a single row
    bool written;
  };
  // o begins first and reaches past p's beginning. Rows of both are a multiple of
  // their strides' common divisor apart.
  static bool apart(const Place& o, const Place& p) {
    const uint64_t line = std::gcd(o.stride, p.stride);
    if (line == 0) return false;
    const uint64_t column = (p.begin - o.begin) % line;
    return column >= o.width && column + p.width <= line;
  }
  std::vector<Place> list_;
};

hkv_status check_layout(uint64_t rows, uint64_t cols, uint64_t stride, uint64_t dtype, const char* what, uint64_t i, uint64_t* es) {
  if (dtype > hkvt::kF16 || !kind_size((uint32_t)dtype, es))
    return fail(HKV_EINVAL, "%s[%llu]: dtype %llu", what, (unsigned long long)i, (unsigned long long)dtype);
  if (stride < cols || stride > (1ull << 40))
    return fail(HKV_EINVAL, "%s[%llu]: stride = %llu with %llu columns", what, (unsigned long long)i,
                (unsigned long long)stride, (unsigned long long)cols);
  if (too_far(rows, stride))
    return fail(HKV_EINVAL, "%s[%llu]: stride = %llu with %llu rows reaches past any memory", what, (unsigned long long)i,
                (unsigned long long)stride, (unsigned long long)rows);
  return HKV_OK;
}

hkv_status check_place(Buffers& buffers, const void* p, uint64_t rows, uint64_t cols, uint64_t stride, uint64_t es,
                       const char* what, uint64_t i) {
  HKV_TRY(buffers.check(p, ((rows - 1) * stride + cols) * es, what, (int64_t)i));
  if (reinterpret_cast<uintptr_t>(p) % es)
    return fail(HKV_EINVAL, "%s[%llu] is not aligned to its type", what, (unsigned long long)i);
  return HKV_OK;
}

hkv_status check_sides(uint64_t rows, uint64_t cols, uint64_t i) {
  if (rows > (1ull << 24) || cols > (1ull << 24) || rows * cols > (1ull << 32) || std::min(rows, cols) > (1ull << 15))
    return fail(HKV_EINVAL, "matrix %llu: %llu x %llu is past 2^24 a side, 2^15 for the shorter one or 2^32 elements",
                (unsigned long long)i, (unsigned long long)rows, (unsigned long long)cols);
  return HKV_OK;
}

// Norms are 0 or far above it: no float's square comes near, nor do the momentum's
// shares of one. The kernels divide by eps, which for a smaller one would overflow.
constexpr double kLeastEps = 1e-200;

hkv_status run_polar(Buffers& buffers, const std::vector<hkvt::PolarMatrix>& list, const hkvt::PolarRule& rule,
                     uint32_t steps, const double* coefficients, void* workspace, uint64_t workspace_bytes,
                     hipStream_t stream, const char* what) {
  if (list.empty()) return HKV_OK;
  const uint32_t n = (uint32_t)list.size();
  HKV_TRY(check_workspace(buffers, workspace, workspace_bytes, hkvt::polar_workspace_bytes(list.data(), n)));
  DeviceGuard dg(buffers.device());
  if (dg.error() != hipSuccess) return fail_hip(dg.error(), "hipSetDevice");
  const hipError_t e = hkvt::launch_polar(list.data(), n, rule, coefficients, steps, workspace, stream);
  return e == hipSuccess ? HKV_OK : fail_hip(e, what);
}

}  // namespace

HKV_API uint64_t hkv_train_workspace_bytes(uint64_t rows, uint64_t pairs, uint64_t tensors) {
  return hkvt::workspace_bytes(rows, pairs, tensors);
}

HKV_API hkv_status hkv_token_logprobs(uint64_t rows, uint64_t vocab, uint32_t dtype, const void* logits,
                                      uint64_t logits_stride, const int64_t* labels, float temperature,
                                      float* logp_out, float* lse_out, void* workspace, uint64_t workspace_bytes,
                                      hipStream_t stream) {
  return guarded([&]() -> hkv_status {
    hkvt::Logits l;
    Buffers buffers;
    HKV_TRY(check_logits(buffers, rows, vocab, dtype, logits, logits_stride, labels, temperature, nullptr, 0, &l));
    if (rows == 0) return HKV_OK;
    HKV_TRY(buffers.check(logp_out, rows * 4, "logp_out"));
    if (lse_out) HKV_TRY(buffers.check(lse_out, rows * 4, "lse_out"));
    const uint64_t need = hkvt::logprobs_workspace_bytes(l);
    if (need) HKV_TRY(check_workspace(buffers, workspace, workspace_bytes, need));
    DeviceGuard dg(buffers.device());
    if (dg.error() != hipSuccess) return fail_hip(dg.error(), "hipSetDevice");
    const hipError_t e = hkvt::launch_logprobs(l, logp_out, lse_out, workspace, stream);
    return e == hipSuccess ? HKV_OK : fail_hip(e, "hkv_token_logprobs launch");
  });
}

HKV_API hkv_status hkv_token_logprobs_backward(uint64_t rows, uint64_t vocab, uint32_t dtype, const void* logits,
                                               uint64_t logits_stride, const int64_t* labels, float temperature,
                                               const float* lse, const float* grad_logp, void* grad_out,
                                               uint64_t grad_stride, hipStream_t stream) {
  return guarded([&]() -> hkv_status {
    hkvt::Logits l;
    Buffers buffers;
    if (!grad_out && rows) return fail(HKV_EINVAL, "grad_out is NULL");
    HKV_TRY(check_logits(buffers, rows, vocab, dtype, logits, logits_stride, labels, temperature, grad_out,
                         grad_stride, &l));
    if (rows == 0) return HKV_OK;
    HKV_TRY(buffers.check(lse, rows * 4, "lse"));
    HKV_TRY(buffers.check(grad_logp, rows * 4, "grad_logp"));
    DeviceGuard dg(buffers.device());
    if (dg.error() != hipSuccess) return fail_hip(dg.error(), "hipSetDevice");
    const hipError_t e = hkvt::launch_backward(l, lse, grad_logp, stream);
    return e == hipSuccess ? HKV_OK : fail_hip(e, "hkv_token_logprobs_backward launch");
  });
}

HKV_API uint64_t hkv_token_stats_workspace_bytes(uint64_t rows, uint64_t vocab, uint32_t dtype, uint32_t k) {
  if (rows >= (1ull << 31) || vocab >= (1ull << 29) || dtype > hkvt::kF16 || k > hkvt::kMostTops) return 0;
  hkvt::Logits l{};
  l.rows = (uint32_t)rows;
  l.vocab = (uint32_t)vocab;
  l.kind = dtype;
  return hkvt::stats_workspace_bytes(l, k);
}

HKV_API hkv_status hkv_token_stats(uint64_t rows, uint64_t vocab, uint32_t dtype, const void* logits,
                                   uint64_t logits_stride, const int64_t* labels, float temperature, uint32_t k,
                                   float* logp_out, float* lse_out, float* entropy_out, float* top_logp_out,
                                   int64_t* top_ids_out, void* workspace, uint64_t workspace_bytes,
                                   hipStream_t stream) {
  return guarded([&]() -> hkv_status {
    hkvt::Logits l;
    Buffers buffers;
    if (k > hkvt::kMostTops) return fail(HKV_EINVAL, "k = %u, the limit is %u", k, hkvt::kMostTops);
    HKV_TRY(check_logits(buffers, rows, vocab, dtype, logits, logits_stride, labels, temperature, nullptr, 0, &l));
    if (rows == 0) return HKV_OK;
    HKV_TRY(buffers.check(logp_out, rows * 4, "logp_out"));
    if (lse_out) HKV_TRY(buffers.check(lse_out, rows * 4, "lse_out"));
    HKV_TRY(buffers.check(entropy_out, rows * 4, "entropy_out"));
    if (k) {
      HKV_TRY(buffers.check(top_logp_out, rows * k * 4, "top_logp_out"));
      HKV_TRY(buffers.check(top_ids_out, rows * k * 8, "top_ids_out"));
    }
    const uint64_t need = hkvt::stats_workspace_bytes(l, k);
    if (need) HKV_TRY(check_workspace(buffers, workspace, workspace_bytes, need));
    DeviceGuard dg(buffers.device());
    if (dg.error() != hipSuccess) return fail_hip(dg.error(), "hipSetDevice");
    const hkvt::Stats out{logp_out, lse_out, entropy_out, top_logp_out, top_ids_out, k};
    const hipError_t e = hkvt::launch_stats(l, out, workspace, stream);
    return e == hipSuccess ? HKV_OK : fail_hip(e, "hkv_token_stats launch");
  });
}

HKV_API hkv_status hkv_token_stats_backward(uint64_t rows, uint64_t vocab, uint32_t dtype, const void* logits,
                                            uint64_t logits_stride, const int64_t* labels, float temperature,
                                            const float* lse, const float* entropy, const float* grad_logp,
                                            const float* grad_entropy, void* grad_out, uint64_t grad_stride,
                                            hipStream_t stream) {
  return guarded([&]() -> hkv_status {
    hkvt::Logits l;
    Buffers buffers;
    if (!grad_out && rows) return fail(HKV_EINVAL, "grad_out is NULL");
    if (!grad_logp && !grad_entropy && rows) return fail(HKV_EINVAL, "grad_logp and grad_entropy are NULL");
    HKV_TRY(check_logits(buffers, rows, vocab, dtype, logits, logits_stride, labels, temperature, grad_out,
                         grad_stride, &l));
    if (rows == 0) return HKV_OK;
    HKV_TRY(buffers.check(lse, rows * 4, "lse"));
    if (grad_logp) HKV_TRY(buffers.check(grad_logp, rows * 4, "grad_logp"));
    if (grad_entropy) {
      HKV_TRY(buffers.check(grad_entropy, rows * 4, "grad_entropy"));
      HKV_TRY(buffers.check(entropy, rows * 4, "entropy"));
    }
    DeviceGuard dg(buffers.device());
    if (dg.error() != hipSuccess) return fail_hip(dg.error(), "hipSetDevice");
    const hipError_t e = hkvt::launch_stats_backward(l, lse, entropy, grad_logp, grad_entropy, stream);
    return e == hipSuccess ? HKV_OK : fail_hip(e, "hkv_token_stats_backward launch");
  });
}

HKV_API hkv_status hkv_preference_loss(uint64_t rows, uint64_t vocab, uint32_t dtype, const void* logits,
                                       uint64_t logits_stride, const int64_t* labels, float temperature,
                                       uint64_t pairs, const int64_t* cu_seqlens, const float* ref_logp, float beta,
                                       float label_smoothing, float grad_scale, float* loss_out, float* losses_out,
                                       float* rewards_out, float* logp_out, void* grad_out, uint64_t grad_stride,
                                       void* workspace, uint64_t workspace_bytes, hipStream_t stream) {
  return guarded([&]() -> hkv_status {
    hkvt::Logits l;
    Buffers buffers;
    if (pairs >= (1ull << 30)) return fail(HKV_EINVAL, "pairs = %llu, the limit is 2^30 - 1", (unsigned long long)pairs);
    if (!std::isfinite(beta)) return fail(HKV_EINVAL, "beta = %g is not finite", (double)beta);
    if (!(label_smoothing >= 0.0f && label_smoothing <= 1.0f))
      return fail(HKV_EINVAL, "label_smoothing = %g is outside 0 .. 1", (double)label_smoothing);
    if (!std::isfinite(grad_scale)) return fail(HKV_EINVAL, "grad_scale = %g is not finite", (double)grad_scale);
    HKV_TRY(check_logits(buffers, rows, vocab, dtype, logits, logits_stride, labels, temperature, grad_out,
                         grad_stride, &l));
    HKV_TRY(buffers.check(loss_out, 4, "loss_out"));
    if (rows) {
      if (ref_logp) HKV_TRY(buffers.check(ref_logp, rows * 4, "ref_logp"));
      HKV_TRY(buffers.check(logp_out, rows * 4, "logp_out"));
    }
    if (pairs) {
      HKV_TRY(buffers.check(cu_seqlens, (2 * pairs + 1) * 8, "cu_seqlens"));
      HKV_TRY(buffers.check(losses_out, pairs * 4, "losses_out"));
      HKV_TRY(buffers.check(rewards_out, pairs * 8, "rewards_out"));
    }
    HKV_TRY(check_workspace(buffers, workspace, workspace_bytes, hkvt::workspace_bytes(rows, pairs, 0)));
    DeviceGuard dg(buffers.device());
    if (dg.error() != hipSuccess) return fail_hip(dg.error(), "hipSetDevice");
    const hkvt::Pairs p{(uint32_t)pairs, cu_seqlens, ref_logp, beta, label_smoothing, grad_scale, loss_out, losses_out,
                        rewards_out, logp_out};
    const hipError_t e = hkvt::launch_preference(l, p, workspace, stream);
    return e == hipSuccess ? HKV_OK : fail_hip(e, "hkv_preference_loss launch");
  });
}

HKV_API hkv_status hkv_policy_loss(uint64_t rows, uint64_t vocab, uint32_t dtype, const void* logits,
                                   uint64_t logits_stride, const int64_t* labels, float temperature,
                                   const float* old_logp, const float* advantages, const float* weights,
                                   const float* ref_logp, float clip_low, float clip_high, float kl_coef,
                                   float grad_scale, float* loss_out, float* token_loss_out, float* kl_out,
                                   float* logp_out, void* grad_out, uint64_t grad_stride, void* workspace,
                                   uint64_t workspace_bytes, hipStream_t stream) {
  return guarded([&]() -> hkv_status {
    hkvt::Logits l;
    Buffers buffers;
    if (!(clip_low >= 0.0f && clip_low <= 1.0f))
      return fail(HKV_EINVAL, "clip_low = %g is outside 0 .. 1", (double)clip_low);
    if (!(clip_high >= 0.0f) || !std::isfinite(clip_high))
      return fail(HKV_EINVAL, "clip_high = %g has to be a finite number >= 0", (double)clip_high);
    if (!std::isfinite(kl_coef)) return fail(HKV_EINVAL, "kl_coef = %g is not finite", (double)kl_coef);
    if (kl_coef != 0.0f && !ref_logp && rows) return fail(HKV_EINVAL, "kl_coef = %g without ref_logp", (double)kl_coef);
    if (!std::isfinite(grad_scale)) return fail(HKV_EINVAL, "grad_scale = %g is not finite", (double)grad_scale);
    HKV_TRY(check_logits(buffers, rows, vocab, dtype, logits, logits_stride, labels, temperature, grad_out,
                         grad_stride, &l));
    HKV_TRY(buffers.check(loss_out, 4, "loss_out"));
    if (rows) {
      HKV_TRY(buffers.check(old_logp, rows * 4, "old_logp"));
      HKV_TRY(buffers.check(advantages, rows * 4, "advantages"));
      HKV_TRY(buffers.check(weights, rows * 4, "weights"));
      if (ref_logp) HKV_TRY(buffers.check(ref_logp, rows * 4, "ref_logp"));
      HKV_TRY(buffers.check(token_loss_out, rows * 4, "token_loss_out"));
      HKV_TRY(buffers.check(kl_out, rows * 4, "kl_out"));
      HKV_TRY(buffers.check(logp_out, rows * 4, "logp_out"));
    }
    HKV_TRY(check_workspace(buffers, workspace, workspace_bytes, hkvt::workspace_bytes(rows, 0, 0)));
    DeviceGuard dg(buffers.device());
    if (dg.error() != hipSuccess) return fail_hip(dg.error(), "hipSetDevice");
    const hkvt::Policy p{old_logp, advantages, weights,    ref_logp, 1.0 - (double)clip_low, 1.0 + (double)clip_high,
                         kl_coef,  grad_scale, loss_out, token_loss_out, kl_out, logp_out};
    const hipError_t e = hkvt::launch_policy(l, p, workspace, stream);
    return e == hipSuccess ? HKV_OK : fail_hip(e, "hkv_policy_loss launch");
  });
}

HKV_API hkv_status hkv_clip_grad_norm(uint64_t tensors, void* const* grads, void* const* outs, const uint64_t* numel,
                                      const uint8_t* dtypes, float max_norm, float* norm_out, void* workspace,
                                      uint64_t workspace_bytes, hipStream_t stream) {
  return guarded([&]() -> hkv_status {
    if (tensors >= (1ull << 20))
      return fail(HKV_EINVAL, "tensors = %llu, the limit is 2^20 - 1", (unsigned long long)tensors);
    if (tensors && (!grads || !numel || !dtypes)) return fail(HKV_EINVAL, "grads, numel or dtypes is NULL");
    if (!(max_norm >= 0.0f)) return fail(HKV_EINVAL, "max_norm = %g has to be >= 0", (double)max_norm);
    Buffers buffers;
    // the tensors that hold anything, and the ranges they read and write
    std::vector<hkvt::Tensor> list;
    list.reserve(tensors);
    struct Range {
      uintptr_t begin, end;
      bool written;
    };
    std::vector<Range> ranges, more;  // of the gradients, of outputs elsewhere
    ranges.reserve(outs ? 2 * tensors : tensors);
    if (outs) more.reserve(tensors);
    uint64_t chunks = 0;
    for (uint64_t i = 0; i < tensors; ++i) {
      uint64_t es = 0;
      if (!kind_size(dtypes[i], &es)) return fail(HKV_EINVAL, "tensor %llu: dtype %u", (unsigned long long)i, dtypes[i]);
      const uint64_t n = numel[i];
      if (n == 0) continue;
      if (n > (1ull << 48)) return fail(HKV_EINVAL, "tensor %llu: numel", (unsigned long long)i);
      void* out = outs ? outs[i] : grads[i];
      HKV_TRY(buffers.check(grads[i], n * es, "grads", (int64_t)i));
      if (out != grads[i]) HKV_TRY(buffers.check(out, n * es, "outs", (int64_t)i));
      if (reinterpret_cast<uintptr_t>(grads[i]) % es || reinterpret_cast<uintptr_t>(out) % es)
        return fail(HKV_EINVAL, "tensor %llu is not aligned to its type", (unsigned long long)i);
      list.push_back({grads[i], out, n, dtypes[i], 0});
      chunks += (n - 1) / hkvt::chunk_elems(dtypes[i]) + 1;
      const uintptr_t a = reinterpret_cast<uintptr_t>(grads[i]), b = reinterpret_cast<uintptr_t>(out);
      ranges.push_back({a, a + n * es, out == grads[i]});
      if (out != grads[i]) more.push_back({b, b + n * es, true});
    }
    if (chunks >= (1ull << 31)) return fail(HKV_EINVAL, "more than 2^31 chunks of %llu bytes", (unsigned long long)hkvt::kChunkBytes);
    const auto before = [](const Range& a, const Range& b) { return a.begin < b.begin; };
    for (auto* part : {&ranges, &more})  // mostly in the order of their allocation
      if (!std::is_sorted(part->begin(), part->end(), before)) std::sort(part->begin(), part->end(), before);
    const auto middle = ranges.insert(ranges.end(), more.begin(), more.end());
    std::inplace_merge(ranges.begin(), middle, ranges.end(), before);
    // a range that begins before an earlier one ends, of which one is written
    uintptr_t end = 0, written_end = 0;
    for (const Range& r : ranges) {
      if (r.begin < written_end || (r.written && r.begin < end))
        return fail(HKV_EINVAL, "two tensors overlap, and one of them is written");
      end = std::max(end, r.end);
      if (r.written) written_end = std::max(written_end, r.end);
    }
    HKV_TRY(buffers.check(norm_out, 4, "norm_out"));
    HKV_TRY(check_workspace(buffers, workspace, workspace_bytes, hkvt::workspace_bytes(0, 0, tensors)));
    DeviceGuard dg(buffers.device());
    if (dg.error() != hipSuccess) return fail_hip(dg.error(), "hipSetDevice");
    const hipError_t e = hkvt::launch_clip(list.data(), (uint32_t)list.size(), max_norm, norm_out, workspace, stream);
    return e == hipSuccess ? HKV_OK : fail_hip(e, "hkv_clip_grad_norm launch");
  });
}

HKV_API uint64_t hkv_orthogonalize_workspace_bytes(uint64_t matrices, const uint64_t* rows, const uint64_t* cols,
                                                   const uint8_t* out_dtypes) {
  try {
    if (!rows || !cols || !out_dtypes || matrices >= (1ull << 20)) return 0;
    std::vector<hkvt::PolarMatrix> list;
    for (uint64_t i = 0; i < matrices; ++i) {
      if (rows[i] == 0 || cols[i] == 0) continue;
      if (rows[i] > (1ull << 24) || cols[i] > (1ull << 24)) return 0;
      hkvt::PolarMatrix m{};
      m.rows = (uint32_t)rows[i];
      m.cols = (uint32_t)cols[i];
      m.out_kind = out_dtypes[i];
      list.push_back(m);
    }
    return list.empty() ? 0 : hkvt::polar_workspace_bytes(list.data(), (uint32_t)list.size());
  } catch (...) {
    return 0;
  }
}

HKV_API hkv_status hkv_orthogonalize(uint64_t matrices, const hkv_matrix* list, uint32_t steps,
                                     const double* coefficients, double eps, void* workspace,
                                     uint64_t workspace_bytes, hipStream_t stream) {
  return guarded([&]() -> hkv_status {
    if (matrices >= (1ull << 20))
      return fail(HKV_EINVAL, "matrices = %llu, the limit is 2^20 - 1", (unsigned long long)matrices);
    if (matrices && !list) return fail(HKV_EINVAL, "list is NULL");
    HKV_TRY(check_coefficients(steps, coefficients));
    if (!(eps > 0.0) || !std::isfinite(eps)) return fail(HKV_EINVAL, "eps = %g has to be a positive finite number", eps);
    Buffers buffers;
    Places places;
    std::vector<hkvt::PolarMatrix> todo;
    todo.reserve(matrices);
    for (uint64_t i = 0; i < matrices; ++i) {
      const hkv_matrix& m = list[i];
      if (m.rows == 0 || m.cols == 0) continue;
      HKV_TRY(check_sides(m.rows, m.cols, i));
      uint64_t in_size = 0, out_size = 0;
      HKV_TRY(check_layout(m.rows, m.cols, m.in_stride, m.in_dtype, "in", i, &in_size));
      HKV_TRY(check_layout(m.rows, m.cols, m.out_stride, m.out_dtype, "out", i, &out_size));
      HKV_TRY(check_place(buffers, m.in, m.rows, m.cols, m.in_stride, in_size, "in", i));
      HKV_TRY(check_place(buffers, m.out, m.rows, m.cols, m.out_stride, out_size, "out", i));
      const bool same = m.in == m.out && m.in_stride == m.out_stride && m.in_dtype == m.out_dtype;
      if (!same) places.add(m.in, m.rows, m.cols, m.in_stride, in_size, false);
      places.add(m.out, m.rows, m.cols, m.out_stride, out_size, true);
      todo.push_back({m.in, m.out, nullptr, m.in_stride, m.out_stride, 0, 0.0, 1.0, (uint32_t)m.rows, (uint32_t)m.cols,
                      (uint32_t)m.in_dtype, (uint32_t)m.out_dtype});
    }
    if (places.clash()) return fail(HKV_EINVAL, "two matrices overlap, and one of them is written");
    return run_polar(buffers, todo, hkvt::PolarRule{0.0, std::max(eps, kLeastEps), 0}, steps, coefficients, workspace, workspace_bytes,
                     stream, "hkv_orthogonalize launch");
  });
}

HKV_API hkv_status hkv_muon_update(uint64_t matrices, const hkv_muon_matrix* list, double momentum, uint32_t nesterov,
                                   double weight_decay, uint32_t steps, const double* coefficients, double eps,
                                   void* workspace, uint64_t workspace_bytes, hipStream_t stream) {
  return guarded([&]() -> hkv_status {
    if (matrices >= (1ull << 20))
      return fail(HKV_EINVAL, "matrices = %llu, the limit is 2^20 - 1", (unsigned long long)matrices);
    if (matrices && !list) return fail(HKV_EINVAL, "list is NULL");
    if (!(momentum >= 0.0 && momentum < 1.0)) return fail(HKV_EINVAL, "momentum = %g is outside 0 .. 1", momentum);
    if (nesterov > 1) return fail(HKV_EINVAL, "nesterov = %u is neither 0 nor 1", nesterov);
    if (!std::isfinite(weight_decay)) return fail(HKV_EINVAL, "weight_decay = %g is not finite", weight_decay);
    HKV_TRY(check_coefficients(steps, coefficients));
    if (!(eps > 0.0) || !std::isfinite(eps)) return fail(HKV_EINVAL, "eps = %g has to be a positive finite number", eps);
    Buffers buffers;
    Places places;
    std::vector<hkvt::PolarMatrix> todo;
    todo.reserve(matrices);
    for (uint64_t i = 0; i < matrices; ++i) {
      const hkv_muon_matrix& m = list[i];
      if (m.rows == 0 || m.cols == 0) continue;
      HKV_TRY(check_sides(m.rows, m.cols, i));
      if (!std::isfinite(m.lr) || !std::isfinite(m.scale))
        return fail(HKV_EINVAL, "matrix %llu: lr = %g, scale = %g", (unsigned long long)i, m.lr, m.scale);
      uint64_t ws = 0, gs = 0, ms = 0;
      HKV_TRY(check_layout(m.rows, m.cols, m.weight_stride, m.weight_dtype, "weight", i, &ws));
      HKV_TRY(check_layout(m.rows, m.cols, m.grad_stride, m.grad_dtype, "grad", i, &gs));
      HKV_TRY(check_layout(m.rows, m.cols, m.momentum_stride, HKV_F32, "momentum", i, &ms));
      HKV_TRY(check_place(buffers, m.weight, m.rows, m.cols, m.weight_stride, ws, "weight", i));
      HKV_TRY(check_place(buffers, m.grad, m.rows, m.cols, m.grad_stride, gs, "grad", i));
      HKV_TRY(check_place(buffers, m.momentum, m.rows, m.cols, m.momentum_stride, ms, "momentum", i));
      places.add(m.weight, m.rows, m.cols, m.weight_stride, ws, true);
      places.add(m.grad, m.rows, m.cols, m.grad_stride, gs, false);
      places.add(m.momentum, m.rows, m.cols, m.momentum_stride, ms, true);
      todo.push_back({m.grad, m.weight, m.momentum, m.grad_stride, m.weight_stride, m.momentum_stride,
                      1.0 - m.lr * weight_decay, -m.lr * m.scale, (uint32_t)m.rows, (uint32_t)m.cols,
                      (uint32_t)m.grad_dtype, (uint32_t)m.weight_dtype});
    }
    if (places.clash()) return fail(HKV_EINVAL, "two matrices overlap, and one of them is written");
    return run_polar(buffers, todo, hkvt::PolarRule{momentum, std::max(eps, kLeastEps), nesterov}, steps, coefficients, workspace,
                     workspace_bytes, stream, "hkv_muon_update launch");
  });
}

HKV_API const char* hkv_train_last_error(void) { return g_error.c_str(); }
