// train_abi.hip -- the C ABI of the training operators (8-bit activation
// checkpoints, norms, gated feed-forward block): argument checks and the
// launches. Every check comes before the first launch.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cmath>
#include <string>

#include "args.hpp"
#include "ffn.hpp"
#include "host.hpp"
#include "train.hpp"

namespace msamp {
namespace {

CkptRef ref(const msamp_checkpoint* c) {
  CkptRef r;
  if (c != nullptr) r = {c->codes, c->ld, c->scales, c->ld_scales, (int)c->fmt};
  return r;
}

// Exactly one of x and its checkpoint.
msamp_status check_input(const void* x, int64_t ldx, const msamp_checkpoint* ck, int64_t rows, int64_t cols,
                         int dtype) {
  if (ck == nullptr) return check_matrix(x, rows, cols, ldx, elem_size(dtype), false, "x");
  if (x != nullptr) return invalid("both x and x_ckpt are set");
  return check_checkpoint(ck, rows, cols, false, "x_ckpt");
}

msamp_status check_norm(int64_t rows, int64_t cols, int dtype, const void* weight, const void* bias,
                        int weight_dtype) {
  MSAMP_TRY(check_shape(rows, cols));
  if (cols > MSAMP_NORM_MAX_COLS)
    return invalid("cols exceeds " + std::to_string(MSAMP_NORM_MAX_COLS));
  MSAMP_TRY(check_dtype(dtype, "dtype"));
  MSAMP_TRY(check_dtype(weight_dtype, "weight_dtype"));
  if (weight_dtype != dtype && weight_dtype != MSAMP_F32) return invalid("weight_dtype must be dtype or MSAMP_F32");
  if (weight != nullptr) MSAMP_TRY(check_vector(weight, cols, elem_size(weight_dtype), "weight"));
  if (bias != nullptr) MSAMP_TRY(check_vector(bias, cols, elem_size(weight_dtype), "bias"));
  return MSAMP_OK;
}

// The bytes of the partial sums: two sums a column from each workgroup. (One
// alone writes the gradients itself and leaves them unused.)
int64_t norm_workspace(int64_t rows, int64_t cols) { return 2 * norm_backward_parts(rows, cols) * cols * 4; }

msamp_status check_ffn(const msamp_gated_ffn* a, bool backward) {
  if (a == nullptr) return invalid("args is NULL");
  const int64_t T = a->tokens, K = a->hidden, F = a->ffn;
  if (T < 0 || K < 0 || F < 0) return invalid("a size is negative");
  if (T > kMaxCols || K > kMaxCols || F > kMaxCols) return invalid("a size exceeds 2^31 - 1");
  if (T * F > kMaxSpan || T * K > kMaxSpan || F * K > kMaxSpan) return invalid("a matrix has more than 2^58 elements");
  if (a->dtype != MSAMP_F16 && a->dtype != MSAMP_BF16) return invalid("dtype must be MSAMP_F16 or MSAMP_BF16");
  if (a->act != MSAMP_ACT_SILU && a->act != MSAMP_ACT_GELU && a->act != MSAMP_ACT_GELU_TANH)
    return invalid("unknown activation");
  if (a->x_ckpt != nullptr && !backward) return invalid("the forward pass does not take a checkpoint");
  MSAMP_TRY(check_input(a->x, a->ldx, a->x_ckpt, T, K, a->dtype));
  MSAMP_TRY(check_matrix(a->w_gate, F, K, a->ld_gate, 2, false, "w_gate"));
  MSAMP_TRY(check_matrix(a->w_up, F, K, a->ld_up, 2, false, "w_up"));
  if (!backward) return check_matrix(a->h, T, F, a->ldh, 2, true, "h");
  if (a->h != nullptr) MSAMP_TRY(check_matrix(a->h, T, F, a->ldh, 2, true, "h"));
  MSAMP_TRY(check_matrix(a->dh, T, F, a->lddh, 2, false, "dh"));
  MSAMP_TRY(check_matrix(a->dx, T, K, a->lddx, 2, true, "dx"));
  if (a->dw_dtype != a->dtype && a->dw_dtype != MSAMP_F32) return invalid("dw_dtype must be dtype or MSAMP_F32");
  if (a->dw_accumulate && a->dw_dtype != MSAMP_F32) return invalid("dw_accumulate needs dw_dtype MSAMP_F32");
  MSAMP_TRY(check_matrix(a->dw_gate, F, K, a->ld_dw_gate, elem_size(a->dw_dtype), true, "dw_gate"));
  return check_matrix(a->dw_up, F, K, a->ld_dw_up, elem_size(a->dw_dtype), true, "dw_up");
}

msamp_status check_ffn_memory(const msamp_gated_ffn* a, bool backward, const void* workspace, int64_t bytes) {
  const int64_t T = a->tokens, K = a->hidden, F = a->ffn;
  Regions m;
  if (a->x_ckpt == nullptr) m.add(a->x, T, K, a->ldx, 2, false, "x");
  else m.checkpoint(a->x_ckpt, T, K, false, "x_ckpt");
  m.add(a->w_gate, F, K, a->ld_gate, 2, false, "w_gate");
  m.add(a->w_up, F, K, a->ld_up, 2, false, "w_up");
  m.add(a->h, T, F, a->ldh, 2, true, "h");
  if (backward) {
    const int64_t size = elem_size(a->dw_dtype);
    m.add(a->dh, T, F, a->lddh, 2, false, "dh");
    m.add(a->dx, T, K, a->lddx, 2, true, "dx");
    m.add(a->dw_gate, F, K, a->ld_dw_gate, size, true, "dw_gate");
    m.add(a->dw_up, F, K, a->ld_dw_up, size, true, "dw_up");
  }
  m.vector(workspace, bytes, 1, true, "workspace");
  return m.check();
}

}  // namespace
}  // namespace msamp

using namespace msamp;

extern "C" {

msamp_status msamp_checkpoint_save(int64_t rows, int64_t cols, const void* x, int64_t ldx, msamp_dtype dtype,
                                   const msamp_checkpoint* ckpt, void* stream) {
  return guarded([&]() -> msamp_status {
    clear_error();
    MSAMP_TRY(check_shape(rows, cols));
    MSAMP_TRY(check_dtype(dtype, "dtype"));
    MSAMP_TRY(check_checkpoint(ckpt, rows, cols, true, "ckpt"));
    MSAMP_TRY(check_matrix(x, rows, cols, ldx, elem_size(dtype), false, "x"));
    if (rows == 0 || cols == 0) return MSAMP_OK;
    Regions m;
    m.add(x, rows, cols, ldx, elem_size(dtype), false, "x");
    m.checkpoint(ckpt, rows, cols, true, "ckpt");
    MSAMP_TRY(m.check());
    hipStream_t s = (hipStream_t)stream;
    MSAMP_LAUNCH(MSAMP_KERNEL_CHECKPOINT_SAVE, s,
                 launch_checkpoint_save(dtype, rows, cols, x, ldx, ref(ckpt), s));
    return MSAMP_OK;
  });
}

msamp_status msamp_checkpoint_load(int64_t rows, int64_t cols, const msamp_checkpoint* ckpt, void* out,
                                   int64_t ldout, msamp_dtype dtype, void* stream) {
  return guarded([&]() -> msamp_status {
    clear_error();
    MSAMP_TRY(check_shape(rows, cols));
    MSAMP_TRY(check_dtype(dtype, "dtype"));
    MSAMP_TRY(check_checkpoint(ckpt, rows, cols, false, "ckpt"));
    MSAMP_TRY(check_matrix(out, rows, cols, ldout, elem_size(dtype), true, "out"));
    if (rows == 0 || cols == 0) return MSAMP_OK;
    Regions m;
    m.checkpoint(ckpt, rows, cols, false, "ckpt");
    m.add(out, rows, cols, ldout, elem_size(dtype), true, "out");
    MSAMP_TRY(m.check());
    hipStream_t s = (hipStream_t)stream;
    MSAMP_LAUNCH(MSAMP_KERNEL_CHECKPOINT_LOAD, s,
                 launch_checkpoint_load(dtype, rows, cols, ref(ckpt), out, ldout, s));
    return MSAMP_OK;
  });
}

msamp_status msamp_layernorm_forward(int64_t rows, int64_t cols, const void* x, int64_t ldx,
                                     const msamp_checkpoint* x_ckpt, msamp_dtype dtype, const void* weight,
                                     const void* bias, msamp_dtype weight_dtype, void* y, int64_t ldy, float* mean,
                                     float* rstd, double eps, const msamp_checkpoint* save, void* stream) {
  return guarded([&]() -> msamp_status {
    clear_error();
    MSAMP_TRY(check_norm(rows, cols, dtype, weight, bias, weight_dtype));
    MSAMP_TRY(check_input(x, ldx, x_ckpt, rows, cols, dtype));
    MSAMP_TRY(check_matrix(y, rows, cols, ldy, elem_size(dtype), true, "y"));
    if (mean != nullptr) MSAMP_TRY(check_vector(mean, rows, 4, "mean"));
    MSAMP_TRY(check_vector(rstd, rows, 4, "rstd"));
    if (!std::isfinite((float)eps) || eps < 0.0) return invalid("eps must be finite in binary32 and >= 0");
    if (save != nullptr) {
      if (x_ckpt != nullptr) return invalid("save: x is a checkpoint already");
      MSAMP_TRY(check_checkpoint(save, rows, cols, true, "save"));
    }
    if (rows == 0 || cols == 0) return MSAMP_OK;
    const int64_t size = elem_size(dtype), wsize = elem_size(weight_dtype);
    Regions m;
    m.add(x, rows, cols, ldx, size, false, "x", true);
    m.checkpoint(x_ckpt, rows, cols, false, "x_ckpt");
    m.vector(weight, cols, wsize, false, "weight");
    m.vector(bias, cols, wsize, false, "bias");
    m.add(y, rows, cols, ldy, size, true, "y", true);
    m.vector(mean, rows, 4, true, "mean");
    m.vector(rstd, rows, 4, true, "rstd");
    m.checkpoint(save, rows, cols, true, "save");
    MSAMP_TRY(m.check());
    NormArgs a = {};
    a.rows = rows, a.cols = cols;
    a.x = x, a.ldx = ldx, a.ck = ref(x_ckpt);
    a.weight = weight, a.bias = bias, a.weight_f32 = weight_dtype == MSAMP_F32;
    a.y = y, a.ldy = ldy, a.mean = mean, a.rstd = rstd, a.eps = (float)eps;
    a.save = ref(save);
    hipStream_t s = (hipStream_t)stream;
    MSAMP_LAUNCH(MSAMP_KERNEL_NORM_FORWARD, s, launch_norm_forward(dtype, a, s));
    return MSAMP_OK;
  });
}

int64_t msamp_layernorm_backward_workspace(int64_t rows, int64_t cols) {
  return workspace_of([&](int64_t* bytes) -> msamp_status {
    MSAMP_TRY(check_norm(rows, cols, MSAMP_F32, nullptr, nullptr, MSAMP_F32));
    *bytes = norm_workspace(rows, cols);
    return MSAMP_OK;
  });
}

msamp_status msamp_layernorm_backward(int64_t rows, int64_t cols, const void* dy, int64_t lddy, const void* x,
                                      int64_t ldx, const msamp_checkpoint* x_ckpt, msamp_dtype dtype,
                                      const void* weight, msamp_dtype weight_dtype, const float* mean,
                                      const float* rstd, void* dx, int64_t lddx, float* dweight, float* dbias,
                                      int accumulate, void* workspace, int64_t workspace_bytes, void* stream) {
  return guarded([&]() -> msamp_status {
    clear_error();
    MSAMP_TRY(check_norm(rows, cols, dtype, weight, nullptr, weight_dtype));
    MSAMP_TRY(check_matrix(dy, rows, cols, lddy, elem_size(dtype), false, "dy"));
    MSAMP_TRY(check_input(x, ldx, x_ckpt, rows, cols, dtype));
    if (mean != nullptr) MSAMP_TRY(check_vector(mean, rows, 4, "mean"));
    MSAMP_TRY(check_vector(rstd, rows, 4, "rstd"));
    MSAMP_TRY(check_matrix(dx, rows, cols, lddx, elem_size(dtype), true, "dx"));
    if (dweight != nullptr) MSAMP_TRY(check_vector(dweight, cols, 4, "dweight"));
    if (dbias != nullptr) MSAMP_TRY(check_vector(dbias, cols, 4, "dbias"));
    const bool sums = dweight != nullptr || dbias != nullptr;
    if (sums) MSAMP_TRY(check_workspace(workspace, workspace_bytes, norm_workspace(rows, cols)));
    if (cols == 0) return MSAMP_OK;
    const int64_t size = elem_size(dtype);
    Regions m;
    m.add(dy, rows, cols, lddy, size, false, "dy", true);
    m.add(x, rows, cols, ldx, size, false, "x", true);
    m.checkpoint(x_ckpt, rows, cols, false, "x_ckpt");
    m.vector(weight, cols, elem_size(weight_dtype), false, "weight");
    m.vector(mean, rows, 4, false, "mean");
    m.vector(rstd, rows, 4, false, "rstd");
    m.add(dx, rows, cols, lddx, size, true, "dx", true);
    m.vector(dweight, cols, 4, true, "dweight");
    m.vector(dbias, cols, 4, true, "dbias");
    if (sums) m.vector(workspace, norm_workspace(rows, cols), 1, true, "workspace");
    if (rows > 0) MSAMP_TRY(m.check());  // of no rows nothing is read
    NormArgs a = {};
    a.rows = rows, a.cols = cols;
    a.x = x, a.ldx = ldx, a.ck = ref(x_ckpt);
    a.weight = weight, a.weight_f32 = weight_dtype == MSAMP_F32;
    a.mean = const_cast<float*>(mean), a.rstd = const_cast<float*>(rstd);
    a.dy = dy, a.lddy = lddy, a.dx = dx, a.lddx = lddx;
    a.dweight = dweight, a.dbias = dbias, a.accumulate = accumulate;
    a.nparts = norm_backward_parts(rows, cols);
    a.partial = sums && a.nparts > 1 ? (float*)workspace : nullptr;
    hipStream_t s = (hipStream_t)stream;
    if (rows > 0) MSAMP_LAUNCH(MSAMP_KERNEL_NORM_BACKWARD, s, launch_norm_backward(dtype, a, s));
    if (sums && a.nparts != 1) MSAMP_LAUNCH(MSAMP_KERNEL_NORM_REDUCE, s, launch_norm_reduce(a, s));
    return MSAMP_OK;
  });
}

int64_t msamp_gated_ffn_forward_workspace(const msamp_gated_ffn* args) {
  return workspace_of([&](int64_t* bytes) -> msamp_status {
    MSAMP_TRY(check_ffn(args, false));
    return ffn_forward_workspace(*args, bytes);
  });
}

int64_t msamp_gated_ffn_backward_workspace(const msamp_gated_ffn* args) {
  return workspace_of([&](int64_t* bytes) -> msamp_status {
    MSAMP_TRY(check_ffn(args, true));
    return ffn_backward_workspace(*args, bytes);
  });
}

msamp_status msamp_gated_ffn_plan(const msamp_gated_ffn* args, int backward, int32_t* plan) {
  return guarded([&]() -> msamp_status {
    clear_error();
    MSAMP_TRY(check_ffn(args, backward != 0));
    if (plan == nullptr) return invalid("plan is NULL");
    return ffn_plan(*args, backward != 0, plan);
  });
}

msamp_status msamp_gated_ffn_forward(const msamp_gated_ffn* args, void* workspace, int64_t workspace_bytes,
                                     void* stream) {
  return guarded([&]() -> msamp_status {
    clear_error();
    MSAMP_TRY(check_ffn(args, false));
    int64_t need = 0;
    MSAMP_TRY(ffn_forward_workspace(*args, &need));
    MSAMP_TRY(check_workspace(workspace, workspace_bytes, need));
    MSAMP_TRY(check_ffn_memory(args, false, workspace, need));
    return ffn_forward(*args, workspace, (hipStream_t)stream);
  });
}

msamp_status msamp_gated_ffn_backward(const msamp_gated_ffn* args, void* workspace, int64_t workspace_bytes,
                                      void* stream) {
  return guarded([&]() -> msamp_status {
    clear_error();
    MSAMP_TRY(check_ffn(args, true));
    int64_t need = 0;
    MSAMP_TRY(ffn_backward_workspace(*args, &need));
    MSAMP_TRY(check_workspace(workspace, workspace_bytes, need));
    MSAMP_TRY(check_ffn_memory(args, true, workspace, need));
    return ffn_backward(*args, workspace, (hipStream_t)stream);
  });
}

}  // extern "C"
