// train.hpp -- internal interface between the C ABI of the training operators
// (train_abi.hip) and their kernels (norm.hip, ffn.hip). Not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "msamp.h"

namespace msamp {

// A checkpoint as the kernels take it (codes null: none).
struct CkptRef {
  uint8_t* codes = nullptr;
  int64_t ld = 0;
  uint8_t* scales = nullptr;
  int64_t ld_scales = 0;
  int fmt = 0;
};

struct NormArgs {
  int64_t rows, cols;
  const void* x;  // null: ck is read
  int64_t ldx;
  CkptRef ck;
  const void* weight;  // may be null (1)
  const void* bias;    // may be null (0); forward only
  bool weight_f32;
  // forward
  void* y;
  int64_t ldy;
  float* mean;  // null: RMS norm. Read by the backward pass.
  float* rstd;
  float eps;
  CkptRef save;
  // backward (x's statistics in mean and rstd)
  const void* dy;
  int64_t lddy;
  void* dx;
  int64_t lddx;
  float* dweight;
  float* dbias;
  int accumulate;
  float* partial;    // [2][nparts][cols]: each workgroup's sums over its rows (null: nparts <= 1)
  int64_t nparts;
};

hipError_t launch_checkpoint_save(int dtype, int64_t rows, int64_t cols, const void* x, int64_t ldx,
                                  const CkptRef& ck, hipStream_t s);
hipError_t launch_checkpoint_load(int dtype, int64_t rows, int64_t cols, const CkptRef& ck, void* out, int64_t ldout,
                                  hipStream_t s);
hipError_t launch_norm_forward(int dtype, const NormArgs& a, hipStream_t s);
// Workgroups (and partial sums per column) of the backward pass.
int64_t norm_backward_parts(int64_t rows, int64_t cols);
hipError_t launch_norm_backward(int dtype, const NormArgs& a, hipStream_t s);
// dweight and dbias from the partial sums (zeros from none).
hipError_t launch_norm_reduce(const NormArgs& a, hipStream_t s);

}  // namespace msamp
