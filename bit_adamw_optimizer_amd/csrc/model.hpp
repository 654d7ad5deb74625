// model.hpp -- internal interface between the C ABI of the operators at the
// ends of a model and between its tokens (model_abi.hip) and their kernels
// (embedding.hip, recurrence.hip, loss.hip). Not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "msamp.h"

namespace msamp {

// An id or length of a device array.
__device__ __forceinline__ int64_t load_int(const void* p, int bytes, int64_t i) {
  return bytes == 8 ? ((const __attribute__((address_space(1))) int64_t*)p)[i]
                    : (int64_t)((const __attribute__((address_space(1))) int32_t*)p)[i];
}

struct EmbeddingArgs {
  int64_t rows, vocab, cols;
  const void* ids;
  int id_bytes;
  float scale;
  const void* weight;  // forward
  int64_t ldw;
  void* y;
  int64_t ldy;
  const void* dy;  // backward
  int64_t lddy;
  float* dweight;
  int64_t ld_dweight;
  int accumulate;
};

hipError_t launch_embedding_forward(int dtype, const EmbeddingArgs& a, hipStream_t s);
int64_t embedding_workspace(int64_t rows, int64_t vocab, int64_t cols);
// The rows sorted by id into the workspace, then the sums.
hipError_t launch_embedding_sort(const EmbeddingArgs& a, void* ws, hipStream_t s);
hipError_t launch_embedding_backward(int dtype, const EmbeddingArgs& a, void* ws, hipStream_t s);

int64_t recurrence_workspace(const msamp_recurrence& a, bool backward);
hipError_t launch_recurrence_forward(const msamp_recurrence& a, void* ws, hipStream_t s);
hipError_t launch_recurrence_backward(const msamp_recurrence& a, void* ws, hipStream_t s);

int64_t loss_workspace(bool policy, const msamp_vocab_loss& a);
hipError_t launch_loss_forward(bool policy, const msamp_vocab_loss& a, void* ws, hipStream_t s);
hipError_t launch_loss_backward(bool policy, const msamp_vocab_loss& a, hipStream_t s);

}  // namespace msamp
