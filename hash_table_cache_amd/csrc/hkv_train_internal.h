// Internal interface between the host side of the training operators
// (hkv_train.cpp) and their gfx950 kernels (hkv_train_kernels.hip). Not part
// of the public ABI.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace hkvt {

enum Kind : uint32_t { kF32 = 0, kBF16 = 1, kF16 = 2 };

// One [rows][vocab] array of logits, its labels and, where a gradient is
// wanted, the array that takes it.
struct Logits {
  const void* x;
  uint64_t x_stride;  // elements
  void* dx;           // nullptr: no gradient
  uint64_t dx_stride;
  const int64_t* labels;
  uint32_t rows;
  uint32_t vocab;
  uint32_t kind;
  double tau;  // temperature
};

// What the gradient of a row needs, left by the kernel that read it first.
struct RowState {
  double logp;
  float top;    // maximum of the row
  float total;  // sum of exp((x - top) / tau)
  float rest;   // 1 - softmax at the label
  uint32_t counts;  // 0: the row is left out
};

struct Pairs {
  uint32_t pairs;
  const int64_t* cu;
  const float* ref;
  double beta;
  double smoothing;
  double grad_scale;
  float* loss;
  float* losses;
  float* rewards;
  float* logp;
};

struct Policy {
  const float* old_logp;
  const float* advantages;
  const float* weights;
  const float* ref;
  double low, high;  // 1 - clip_low, 1 + clip_high
  double kl_coef;
  double grad_scale;
  float* loss;
  float* token_loss;
  float* kl;
  float* logp;
};

// One gradient tensor: `n` elements of `kind` at `in`, the product goes to `out`.
struct Tensor {
  const void* in;
  void* out;
  uint64_t n;
  uint32_t kind;
  uint32_t first;  // number of its first chunk among all tensors' chunks
};

// Bytes of workspace of a call (every part 16-byte aligned).
uint64_t workspace_bytes(uint64_t rows, uint64_t pairs, uint64_t tensors);
// launch_logprobs: 0 unless workgroups share the rows.
uint64_t logprobs_workspace_bytes(const Logits& l);

hipError_t launch_logprobs(const Logits& l, float* logp, float* lse, void* ws, hipStream_t s);
hipError_t launch_backward(const Logits& l, const float* lse, const float* g, hipStream_t s);
hipError_t launch_preference(const Logits& l, const Pairs& p, void* ws, hipStream_t s);
hipError_t launch_policy(const Logits& l, const Policy& p, void* ws, hipStream_t s);

// A chunk of a tensor's elements.
constexpr uint64_t kChunkBytes = 32768;
__host__ __device__ constexpr uint64_t chunk_elems(uint32_t kind) { return kChunkBytes / (kind == kF32 ? 4 : 2); }
// `first` is filled in here.
hipError_t launch_clip(Tensor* t, uint32_t tensors, double max_norm, float* norm, void* ws, hipStream_t s);

}  // namespace hkvt
