// model_abi.hip -- the C ABI of the operators at the ends of a model and
// between its tokens (embedding, gated linear recurrence, losses over a
// vocabulary): argument checks and the launches. Every check comes before the
// first launch.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cmath>
#include <string>

#include "args.hpp"
#include "host.hpp"
#include "model.hpp"

namespace msamp {
namespace {

constexpr int64_t kMaxInt = INT32_MAX;

msamp_status check_int_bytes(int bytes, const char* role) {
  if (bytes != 4 && bytes != 8) return invalid(std::string(role) + " must be 4 or 8");
  return MSAMP_OK;
}

// ------------------------------------------------------------- embedding ---

msamp_status check_embedding(int64_t rows, int64_t vocab, int64_t cols) {
  if (rows < 0 || vocab < 0 || cols < 0) return invalid("a size is negative");
  if (rows > kMaxInt) return invalid("rows exceeds 2^31 - 1");
  if (vocab > MSAMP_EMBEDDING_MAX_VOCAB) return invalid("vocab exceeds 2^30");
  if (cols > MSAMP_EMBEDDING_MAX_COLS) return invalid("cols exceeds 2^22");
  return MSAMP_OK;
}

msamp_status check_scale(double scale) {
  if (!std::isfinite((float)scale)) return invalid("scale must be finite in binary32");
  return MSAMP_OK;
}

// ------------------------------------------------------------ recurrence ---

msamp_status check_recurrence(const msamp_recurrence* a, bool backward) {
  if (a == nullptr) return invalid("args is NULL");
  const int64_t B = a->batch, T = a->time, C = a->channels;
  if (B < 0 || T < 0 || C < 0) return invalid("a size is negative");
  if (B > kMaxInt || T > kMaxInt || C > kMaxInt) return invalid("a size exceeds 2^31 - 1");
  // every launch's lanes (two channels each, or 64 channels to a workgroup of at most 1,024) within 32 bits
  if (B * ((C + 63) / 64) > (1 << 22)) return invalid("more than 2^22 sequences of 64 channels");
  MSAMP_TRY(check_dtype(a->dtype, "dtype"));
  const int64_t size = elem_size(a->dtype);
  if (a->lengths != nullptr) {
    MSAMP_TRY(check_int_bytes(a->length_bytes, "length_bytes"));
    MSAMP_TRY(check_vector(a->lengths, B, a->length_bytes, "lengths"));
  }
  MSAMP_TRY(check_cube(a->x, B, T, C, a->x_batch, a->x_time, size, false, "x"));
  MSAMP_TRY(check_cube(a->gate, B, T, C, a->gate_batch, a->gate_time, size, false, "gate"));
  const int64_t chunks = (T + MSAMP_RECURRENCE_CHUNK - 1) / MSAMP_RECURRENCE_CHUNK;
  if (C > 0 && B * chunks > kMaxSpan / C) return invalid("states spans too much memory");
  if (backward || a->states != nullptr)
    MSAMP_TRY(check_matrix(a->states, B * chunks, C, C, 4, !backward, "states"));
  if (!backward) {
    MSAMP_TRY(check_cube(a->y, B, T, C, a->y_batch, a->y_time, size, true, "y"));
    if (a->h0 != nullptr) MSAMP_TRY(check_matrix(a->h0, B, C, a->ld_h0, 4, false, "h0"));
    if (a->h_last != nullptr) MSAMP_TRY(check_matrix(a->h_last, B, C, a->ld_h_last, 4, true, "h_last"));
    return MSAMP_OK;
  }
  MSAMP_TRY(check_cube(a->dy, B, T, C, a->dy_batch, a->dy_time, size, false, "dy"));
  MSAMP_TRY(check_cube(a->dx, B, T, C, a->dx_batch, a->dx_time, size, true, "dx"));
  MSAMP_TRY(check_cube(a->dgate, B, T, C, a->dgate_batch, a->dgate_time, size, true, "dgate"));
  if (a->dh_last != nullptr) MSAMP_TRY(check_matrix(a->dh_last, B, C, a->ld_dh_last, 4, false, "dh_last"));
  if (a->dh0 != nullptr) MSAMP_TRY(check_matrix(a->dh0, B, C, a->ld_dh0, 4, true, "dh0"));
  return MSAMP_OK;
}

// In place: y over x or gate, dx and dgate over dy, x or gate (group 1), the
// last state over the first one and their gradients likewise (group 2).
msamp_status check_recurrence_memory(const msamp_recurrence* a, bool backward, const void* workspace, int64_t bytes) {
  const int64_t B = a->batch, T = a->time, C = a->channels, size = elem_size(a->dtype);
  const int64_t chunks = (T + MSAMP_RECURRENCE_CHUNK - 1) / MSAMP_RECURRENCE_CHUNK;
  Regions m;
  if (a->lengths != nullptr) m.vector(a->lengths, B, a->length_bytes, false, "lengths");
  m.cube(a->x, B, T, C, a->x_batch, a->x_time, size, false, "x", 1);
  m.cube(a->gate, B, T, C, a->gate_batch, a->gate_time, size, false, "gate", 1);
  m.add(a->states, B * chunks, C, C, 4, !backward, "states");
  if (!backward) {
    m.cube(a->y, B, T, C, a->y_batch, a->y_time, size, true, "y", 1);
    m.add(a->h0, B, C, a->ld_h0, 4, false, "h0", 2);
    m.add(a->h_last, B, C, a->ld_h_last, 4, true, "h_last", 2);
  } else {
    m.cube(a->dy, B, T, C, a->dy_batch, a->dy_time, size, false, "dy", 1);
    m.cube(a->dx, B, T, C, a->dx_batch, a->dx_time, size, true, "dx", 1);
    m.cube(a->dgate, B, T, C, a->dgate_batch, a->dgate_time, size, true, "dgate", 1);
    m.add(a->dh_last, B, C, a->ld_dh_last, 4, false, "dh_last", 2);
    m.add(a->dh0, B, C, a->ld_dh0, 4, true, "dh0", 2);
  }
  m.vector(workspace, bytes, 1, true, "workspace");
  return m.check();
}

msamp_status run_recurrence(const msamp_recurrence* args, bool backward, void* workspace, int64_t workspace_bytes,
                            hipStream_t s) {
  MSAMP_TRY(check_recurrence(args, backward));
  msamp_recurrence a = *args;
  if (a.batch == 0 || a.channels == 0) return MSAMP_OK;
  // distances that lead nowhere are not multiplied by anything
  if (a.batch == 1) a.x_batch = a.gate_batch = a.y_batch = a.dy_batch = a.dx_batch = a.dgate_batch = 0;
  if (a.time <= 1) a.x_time = a.gate_time = a.y_time = a.dy_time = a.dx_time = a.dgate_time = 0;
  const int64_t need = recurrence_workspace(a, backward);
  MSAMP_TRY(check_workspace(workspace, workspace_bytes, need));
  MSAMP_TRY(check_recurrence_memory(&a, backward, workspace, need));
  if (backward) MSAMP_LAUNCH(MSAMP_KERNEL_RECURRENCE_BACKWARD, s, launch_recurrence_backward(a, workspace, s));
  else MSAMP_LAUNCH(MSAMP_KERNEL_RECURRENCE_FORWARD, s, launch_recurrence_forward(a, workspace, s));
  return MSAMP_OK;
}

// ---------------------------------------------------------------- losses ---

msamp_status check_loss(const msamp_vocab_loss* a, bool policy, bool backward) {
  if (a == nullptr) return invalid("args is NULL");
  const int64_t R = a->rows, V = a->vocab;
  if (R < 0 || V < 0) return invalid("a size is negative");
  if (R > kMaxInt) return invalid("rows exceeds 2^31 - 1");
  if (V > MSAMP_LOSS_MAX_VOCAB) return invalid("vocab exceeds 2^29");
  MSAMP_TRY(check_dtype(a->dtype, "dtype"));
  MSAMP_TRY(check_int_bytes(a->id_bytes, "id_bytes"));
  const float tau = (float)a->temperature, inv = (float)(1.44269504088896341 / a->temperature);
  if (!(tau > 0.0f) || !std::isfinite(tau) || !(inv > 0.0f) || !std::isfinite(inv))
    return invalid("temperature must be above 0, it and log2(e) / temperature finite in binary32");
  const int64_t size = elem_size(a->dtype);
  MSAMP_TRY(check_matrix(a->logits, R, V, a->ld_logits, size, false, "logits"));
  if (policy) {
    MSAMP_TRY(check_vector(a->ids, R, a->id_bytes, "actions"));
    MSAMP_TRY(check_vector(a->old_logp, R, 4, "old_logp"));
    MSAMP_TRY(check_vector(a->advantages, R, 4, "advantages"));
    if (!(a->clip_low >= 0.0 && a->clip_low <= 1.0)) return invalid("clip_low must be from 0 to 1");
    if (!(a->clip_high >= 0.0)) return invalid("clip_high must be 0 or more");
    if (!std::isfinite((float)a->kl)) return invalid("kl must be finite in binary32");
    if ((float)a->kl != 0.0f || a->ref_logp != nullptr) MSAMP_TRY(check_vector(a->ref_logp, R, 4, "ref_logp"));
    if (!backward && a->logp != nullptr) MSAMP_TRY(check_vector(a->logp, R, 4, "logp"));
  } else {
    if (a->top < 0 || a->top > MSAMP_DISTILL_MAX_TOP)
      return invalid("top must be from 0 to " + std::to_string(MSAMP_DISTILL_MAX_TOP));
    MSAMP_TRY(check_dtype(a->teacher_dtype, "teacher_dtype"));
    MSAMP_TRY(check_matrix(a->ids, R, a->top, a->ld_ids, a->id_bytes, false, "ids"));
    MSAMP_TRY(check_matrix(a->teacher, R, a->top, a->ld_teacher, elem_size(a->teacher_dtype), false, "teacher"));
  }
  if (!backward) MSAMP_TRY(check_vector(a->loss, R, 4, "loss"));
  if (backward || a->stats != nullptr) MSAMP_TRY(check_vector(a->stats, 2 * R, 4, "stats"));
  if (backward || a->dlogits != nullptr) {
    MSAMP_TRY(check_matrix(a->dlogits, R, V, a->ld_dlogits, size, true, "dlogits"));
    if (a->dloss != nullptr) MSAMP_TRY(check_vector(a->dloss, R, 4, "dloss"));
  }
  return MSAMP_OK;
}

msamp_status check_loss_memory(const msamp_vocab_loss* a, bool policy, bool backward, const void* workspace,
                               int64_t bytes) {
  const int64_t R = a->rows, V = a->vocab, size = elem_size(a->dtype);
  Regions m;
  m.add(a->logits, R, V, a->ld_logits, size, false, "logits", 1);
  if (policy) {
    m.vector(a->ids, R, a->id_bytes, false, "actions");
    m.vector(a->old_logp, R, 4, false, "old_logp");
    m.vector(a->ref_logp, R, 4, false, "ref_logp");
    m.vector(a->advantages, R, 4, false, "advantages");
    if (!backward) m.vector(a->logp, R, 4, true, "logp");
  } else {
    m.add(a->ids, R, a->top, a->ld_ids, a->id_bytes, false, "ids");
    m.add(a->teacher, R, a->top, a->ld_teacher, elem_size(a->teacher_dtype), false, "teacher");
  }
  if (!backward) m.vector(a->loss, R, 4, true, "loss");
  m.vector(a->stats, 2 * R, 4, !backward, "stats");
  m.add(a->dlogits, R, V, a->ld_dlogits, size, true, "dlogits", 1);
  if (a->dlogits != nullptr) m.vector(a->dloss, R, 4, false, "dloss");
  m.vector(workspace, bytes, 1, true, "workspace");
  return m.check();
}

msamp_status run_loss_forward(const msamp_vocab_loss* args, bool policy, void* workspace, int64_t workspace_bytes,
                              hipStream_t s) {
  MSAMP_TRY(check_loss(args, policy, false));
  if (args->rows == 0) return MSAMP_OK;
  const int64_t need = loss_workspace(policy, *args);
  MSAMP_TRY(check_workspace(workspace, workspace_bytes, need));
  MSAMP_TRY(check_loss_memory(args, policy, false, workspace, need));
  MSAMP_LAUNCH(MSAMP_KERNEL_LOSS_FORWARD, s, launch_loss_forward(policy, *args, workspace, s));
  return MSAMP_OK;
}

msamp_status run_loss_backward(const msamp_vocab_loss* args, bool policy, hipStream_t s) {
  MSAMP_TRY(check_loss(args, policy, true));
  if (args->rows == 0 || args->vocab == 0) return MSAMP_OK;
  MSAMP_TRY(check_loss_memory(args, policy, true, nullptr, 0));
  MSAMP_LAUNCH(MSAMP_KERNEL_LOSS_BACKWARD, s, launch_loss_backward(policy, *args, s));
  return MSAMP_OK;
}

}  // namespace
}  // namespace msamp

using namespace msamp;

extern "C" {

msamp_status msamp_embedding_forward(int64_t rows, int64_t vocab, int64_t cols, const void* ids, int id_bytes,
                                     const void* weight, int64_t ldw, msamp_dtype dtype, void* y, int64_t ldy,
                                     double scale, void* stream) {
  return guarded([&]() -> msamp_status {
    clear_error();
    MSAMP_TRY(check_embedding(rows, vocab, cols));
    MSAMP_TRY(check_dtype(dtype, "dtype"));
    MSAMP_TRY(check_int_bytes(id_bytes, "id_bytes"));
    MSAMP_TRY(check_scale(scale));
    const int64_t size = elem_size(dtype);
    MSAMP_TRY(check_vector(ids, rows, id_bytes, "ids"));
    MSAMP_TRY(check_matrix(weight, vocab, cols, ldw, size, false, "weight"));
    MSAMP_TRY(check_matrix(y, rows, cols, ldy, size, true, "y"));
    if (rows == 0 || cols == 0) return MSAMP_OK;
    Regions m;
    m.vector(ids, rows, id_bytes, false, "ids");
    m.add(weight, vocab, cols, ldw, size, false, "weight");
    m.add(y, rows, cols, ldy, size, true, "y");
    MSAMP_TRY(m.check());
    EmbeddingArgs a = {};
    a.rows = rows, a.vocab = vocab, a.cols = cols;
    a.ids = ids, a.id_bytes = id_bytes, a.scale = (float)scale;
    a.weight = weight, a.ldw = vocab > 1 ? ldw : 0, a.y = y, a.ldy = rows > 1 ? ldy : 0;
    hipStream_t s = (hipStream_t)stream;
    MSAMP_LAUNCH(MSAMP_KERNEL_EMBEDDING_FORWARD, s, launch_embedding_forward(dtype, a, s));
    return MSAMP_OK;
  });
}

int64_t msamp_embedding_backward_workspace(int64_t rows, int64_t vocab, int64_t cols) {
  return workspace_of([&](int64_t* bytes) -> msamp_status {
    MSAMP_TRY(check_embedding(rows, vocab, cols));
    *bytes = embedding_workspace(rows, vocab, cols);
    return MSAMP_OK;
  });
}

msamp_status msamp_embedding_backward(int64_t rows, int64_t vocab, int64_t cols, const void* dy, int64_t lddy,
                                      msamp_dtype dtype, const void* ids, int id_bytes, float* dweight,
                                      int64_t ld_dweight, double scale, int accumulate, void* workspace,
                                      int64_t workspace_bytes, void* stream) {
  return guarded([&]() -> msamp_status {
    clear_error();
    MSAMP_TRY(check_embedding(rows, vocab, cols));
    MSAMP_TRY(check_dtype(dtype, "dtype"));
    MSAMP_TRY(check_int_bytes(id_bytes, "id_bytes"));
    MSAMP_TRY(check_scale(scale));
    const int64_t size = elem_size(dtype), need = embedding_workspace(rows, vocab, cols);
    MSAMP_TRY(check_vector(ids, rows, id_bytes, "ids"));
    MSAMP_TRY(check_matrix(dy, rows, cols, lddy, size, false, "dy"));
    MSAMP_TRY(check_matrix(dweight, vocab, cols, ld_dweight, 4, true, "dweight"));
    MSAMP_TRY(check_workspace(workspace, workspace_bytes, need));
    if (vocab == 0 || cols == 0) return MSAMP_OK;
    Regions m;
    m.vector(ids, rows, id_bytes, false, "ids");
    m.add(dy, rows, cols, lddy, size, false, "dy");
    m.add(dweight, vocab, cols, ld_dweight, 4, true, "dweight");
    m.vector(workspace, need, 1, true, "workspace");
    MSAMP_TRY(m.check());
    EmbeddingArgs a = {};
    a.rows = rows, a.vocab = vocab, a.cols = cols;
    a.ids = ids, a.id_bytes = id_bytes, a.scale = (float)scale;
    a.dy = dy, a.lddy = rows > 1 ? lddy : 0;
    a.dweight = dweight, a.ld_dweight = vocab > 1 ? ld_dweight : 0, a.accumulate = accumulate;
    hipStream_t s = (hipStream_t)stream;
    MSAMP_LAUNCH(MSAMP_KERNEL_EMBEDDING_SORT, s, launch_embedding_sort(a, workspace, s));
    MSAMP_LAUNCH(MSAMP_KERNEL_EMBEDDING_BACKWARD, s, launch_embedding_backward(dtype, a, workspace, s));
    return MSAMP_OK;
  });
}

int64_t msamp_recurrence_forward_workspace(const msamp_recurrence* args) {
  return workspace_of([&](int64_t* bytes) -> msamp_status {
    MSAMP_TRY(check_recurrence(args, false));
    *bytes = recurrence_workspace(*args, false);
    return MSAMP_OK;
  });
}

int64_t msamp_recurrence_backward_workspace(const msamp_recurrence* args) {
  return workspace_of([&](int64_t* bytes) -> msamp_status {
    MSAMP_TRY(check_recurrence(args, true));
    *bytes = recurrence_workspace(*args, true);
    return MSAMP_OK;
  });
}

msamp_status msamp_recurrence_forward(const msamp_recurrence* args, void* workspace, int64_t workspace_bytes,
                                      void* stream) {
  return guarded([&]() -> msamp_status {
    clear_error();
    return run_recurrence(args, false, workspace, workspace_bytes, (hipStream_t)stream);
  });
}

msamp_status msamp_recurrence_backward(const msamp_recurrence* args, void* workspace, int64_t workspace_bytes,
                                       void* stream) {
  return guarded([&]() -> msamp_status {
    clear_error();
    return run_recurrence(args, true, workspace, workspace_bytes, (hipStream_t)stream);
  });
}

int64_t msamp_distill_forward_workspace(const msamp_vocab_loss* args) {
  return workspace_of([&](int64_t* bytes) -> msamp_status {
    MSAMP_TRY(check_loss(args, false, false));
    *bytes = loss_workspace(false, *args);
    return MSAMP_OK;
  });
}

int64_t msamp_policy_forward_workspace(const msamp_vocab_loss* args) {
  return workspace_of([&](int64_t* bytes) -> msamp_status {
    MSAMP_TRY(check_loss(args, true, false));
    *bytes = loss_workspace(true, *args);
    return MSAMP_OK;
  });
}

msamp_status msamp_distill_forward(const msamp_vocab_loss* args, void* workspace, int64_t workspace_bytes,
                                   void* stream) {
  return guarded([&]() -> msamp_status {
    clear_error();
    return run_loss_forward(args, false, workspace, workspace_bytes, (hipStream_t)stream);
  });
}

msamp_status msamp_policy_forward(const msamp_vocab_loss* args, void* workspace, int64_t workspace_bytes,
                                  void* stream) {
  return guarded([&]() -> msamp_status {
    clear_error();
    return run_loss_forward(args, true, workspace, workspace_bytes, (hipStream_t)stream);
  });
}

msamp_status msamp_distill_backward(const msamp_vocab_loss* args, void* stream) {
  return guarded([&]() -> msamp_status {
    clear_error();
    return run_loss_backward(args, false, (hipStream_t)stream);
  });
}

msamp_status msamp_policy_backward(const msamp_vocab_loss* args, void* stream) {
  return guarded([&]() -> msamp_status {
    clear_error();
    return run_loss_backward(args, true, (hipStream_t)stream);
  });
}

}  // extern "C"
