// Definitions shared by the host side and the kernels of the training
// operators (include/xp_train.h).
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstddef>
#include <cstdint>

#include "xp_train.h"

namespace xp {

// A positive number that belongs to a device, asked for once: whoever comes
// first on whatever thread, every call gets the same answer from then on, as a
// workspace's size and the launch that fills it must.
class PerDevice {
  static constexpr int kDevices = 64;
  std::atomic<int> known_[kDevices] = {};

 public:
  template <typename Ask>
  int get(Ask ask) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) {
      (void)cudaGetLastError();
      dev = 0;
    }
    if (dev >= kDevices) return ask(dev);
    int n = known_[dev].load(std::memory_order_acquire);
    if (n > 0) return n;
    const int asked = ask(dev);
    return known_[dev].compare_exchange_strong(n, asked, std::memory_order_acq_rel) ? asked : n;
  }
};

// One tensor of a group, in the group's device table.
struct GroupTensor {
  void* param;
  const void* grad;
  void* m;
  void* v;
  uint8_t* m_scale;
  uint8_t* v_scale;
  void* copy;
  unsigned long long count;
  unsigned long long pos;      // the hash position of element 0
  float decay;
  int aligned;                 // every pointer but grad allows 16-byte (codes: 8-byte) accesses
};
static_assert(sizeof(GroupTensor) == 80, "table layout");

// A piece of a tensor that one CTA works on: elements [start, start + n).
struct GroupUnit {
  unsigned tensor;
  unsigned n;
  unsigned long long start;
};

// Words that live on the device from step to step.  The coefficients belong
// to the coming step; the step that used them writes the next ones.
struct GroupState {
  unsigned long long step;     // steps taken
  double power1, power2;       // beta1^(step + 1), beta2^(step + 1)
  float inv_bias1;             // 1 / (1 - power1)
  float inv_sqrt_bias2;        // 1 / sqrt(1 - power2)
  unsigned arrived_step;       // CTAs of the running step that have read the words above
  unsigned arrived_norm;       // CTAs of the running norm that have written their sums
};

constexpr int kStepThreads = 256;
constexpr int kVec = 8;                  // elements a thread moves at once
constexpr int kDecodeCta = 2 * kStepThreads * kVec;   // codes of one CTA of a decode
constexpr int kNormThreads = 256;
constexpr int kNormMaxCtas = 152 * 5;
constexpr int kSetGradsMax = 448;        // pointers passed in one launch's parameters

struct StepParams {
  const GroupUnit* units;
  const GroupTensor* tensors;
  GroupState* state;
  const xp_grad_report* report;
  const float* lr_dev;
  float lr, grad_scale;
  float beta1, beta2, one_minus_beta1, one_minus_beta2, eps;
  double beta1_d, beta2_d;
  unsigned seed;
  int skip_nonfinite;
};

struct NormParams {
  const GroupUnit* units;
  unsigned nunits;
  const GroupTensor* tensors;
  GroupState* state;
  double* partial;                       // one per CTA
  xp_grad_report* report;
  float grad_scale, max_norm;
  int accumulate;
};

struct SetGradsParams {
  GroupTensor* tensors;
  int first, n;
  const void* grad[kSetGradsMax];
};

struct DecodeParams {
  const uint8_t* code[2];
  const uint8_t* scale[2];
  void* out[2];
  unsigned long long count;
};

struct NormRowsParams {
  const void* x;
  const void* dy;
  const void* gamma;
  const void* beta;
  void* out;                             // y, or dx
  float* mean;
  float* rstd;
  float* partial;                        // backward: per CTA cols sums of dgamma, then of dbeta
  float* dgamma;
  float* dbeta;
  unsigned long long x_stride, dy_stride, out_stride;
  unsigned long long rows;
  unsigned cols;
  int threads;                           // of a row (of one CTA of its cluster)
  unsigned nparts;                       // backward: CTAs (per slice) that leave partial sums
  int stages;                            // rows in flight per group
  float eps;
  int gamma_bf16;
  int accumulate;
};

cudaError_t launch_adamw(const StepParams& p, unsigned nunits, int param_dtype, int grad_dtype, int state_dtype,
                         cudaStream_t st);
cudaError_t launch_grad_norm(const NormParams& p, int grad_dtype, cudaStream_t st);
cudaError_t launch_set_grads(const SetGradsParams& p, cudaStream_t st);
cudaError_t launch_set_step(GroupState* s, unsigned long long step, double beta1, double beta2, cudaStream_t st);
cudaError_t launch_decode(const DecodeParams& p, int out_dtype, cudaStream_t st);

cudaError_t launch_ln_forward(NormRowsParams& p, int dtype, cudaStream_t st);
// How a backward pass over so many rows (1 at least) is laid out: asked for
// once per call, for the workspace (nparts * 2 * cols floats) and the launch.
struct BackwardShape {
  int e, many, threads, groups, csize;   // many: 4 rows a turn (fp32, unaligned: 2), else 1
  unsigned nparts;                       // partial sums per column
};
BackwardShape ln_backward_shape(size_t rows, size_t cols);
cudaError_t launch_ln_backward(NormRowsParams& p, const BackwardShape& s, int dtype, cudaStream_t st);

}  // namespace xp
