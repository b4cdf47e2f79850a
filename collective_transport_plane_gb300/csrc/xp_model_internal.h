// Definitions shared by the host side and the kernels of include/xp_model.h.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "xp_model.h"

namespace xp {

unsigned long long spin_timeout_ns();     // xp_set_spin_timeout_ns's

struct Matmul8Params {
  CUtensorMap p_map, q_map;              // B's and A's codes
  const uint8_t* p_scales;
  const uint8_t* q_scales;
  unsigned long long p_pitch, q_pitch;   // bytes from one row of scales to the next
  int p_shift, q_shift;                  // 7: a row of scales serves 128 rows
  unsigned p_rows, q_rows;               // C's columns and rows
  unsigned kblocks;
  unsigned bn, ctas, split;              // rows of A in a tile; CTAs of a pair; CTAs that share the columns of a tile
  unsigned stages, nsums;
  unsigned tiles_p, tiles_q;
  void* c;
  unsigned long long c_stride;           // elements
  int out_bf16, accumulate;
  unsigned long long limit_ns;           // after which a warp gives up a wait for another
};
cudaError_t launch_matmul8(Matmul8Params& p, int sms, cudaStream_t st);
cudaError_t matmul8_stalls(unsigned* n);

struct Encode8Params {
  const void* x;
  uint8_t* codes;                        // NULL: the transposed ones alone
  uint8_t* scales;
  uint8_t* codes_t;
  uint8_t* scales_t;
  unsigned long long x_stride, codes_stride, scales_stride, codes_t_stride, scales_t_stride;
  unsigned rows, cols, tiles_c, tiles;
  int x_aligned, codes_aligned, codes_t_aligned, all_aligned;   // four elements are one access
};
cudaError_t launch_encode8(const Encode8Params& p, int dtype, int block_rows, int sms, cudaStream_t st);

struct Decode8Params {
  const uint8_t* codes;
  const uint8_t* scales;
  void* out;
  unsigned long long codes_stride, scales_stride, out_stride;
  unsigned rows, cols;
  int shift, aligned;                    // 16 bytes of output are one access, and so are their codes
};
cudaError_t launch_decode8(const Decode8Params& p, int dtype, cudaStream_t st);

struct RmsForwardParams {
  const void* x;
  const void* residual;
  const void* gamma;
  void* added;
  void* y;
  uint8_t* y8;
  uint8_t* y8_scales;
  float* rstd;
  unsigned long long x_stride, residual_stride, added_stride, y_stride, y8_stride, y8_scales_stride;
  unsigned long long rows;
  unsigned cols, threads;                // threads of a row
  float eps;
  int gamma_bf16;
};
// wide: every row and gamma allow 16-byte accesses (codes 8-byte ones).
cudaError_t launch_rms_forward(RmsForwardParams& p, int dtype, bool wide, cudaStream_t st);

struct RmsBackwardParams {
  const void* dy;
  const void* h;
  const void* gamma;
  const void* dadded;
  void* dx;
  const float* rstd;
  float* dgamma;
  float* partial;                        // nparts rows of cols sums; NULL where dgamma is
  float* row_sums;                       // of long rows
  unsigned long long dy_stride, h_stride, dadded_stride, dx_stride;
  unsigned long long rows;
  unsigned cols, threads, nparts;
  int stages;                            // rows in flight per group, and one in work
  int gamma_bf16, accumulate;
};
// How a backward pass is cut: threads of a row with nu units each, rows of a
// CTA at a time, and CTAs (slices of rows, where they are long).
struct RmsBackwardShape {
  unsigned nu, threads, groups, per_sm, nparts;
  bool is_long;
};
RmsBackwardShape rms_backward_shape(size_t rows, size_t cols, int dtype, bool wide, int sms);
cudaError_t launch_rms_backward(RmsBackwardParams& p, const RmsBackwardShape& s, int dtype, bool wide, cudaStream_t st);

struct DistillParams {
  const void* logits;
  const int32_t* ids;
  const float* teacher;
  float* loss;                           // forward
  float* lse;
  const float* dloss;                    // backward
  void* dlogits;
  unsigned long long logits_stride, dlogits_stride;
  unsigned rows, vocab, top;
  float temperature;
};
cudaError_t launch_distill_forward(const DistillParams& p, int dtype, int sms, cudaStream_t st);
cudaError_t launch_distill_backward(const DistillParams& p, int dtype, int sms, cudaStream_t st);

}  // namespace xp
