// Host side of the C ABI declared in include/hkv_train.h: argument checks and
// launches. The calls keep no state and allocate nothing on the device.
#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <exception>
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

HKV_API const char* hkv_train_last_error(void) { return g_error.c_str(); }
