// host.hpp -- what the files of the C ABI share on the host: the per-thread
// error text, the exception barrier of every entry point, and the optional
// event timing around each kernel launch. Defined in abi.hip. Internal.
#pragma once

#include <hip/hip_runtime.h>

#include <exception>
#include <new>
#include <string>
#include <type_traits>

#include "msamp.h"

namespace msamp {

// Sets the calling thread's error text and returns 'st'.
msamp_status fail(msamp_status st, const std::string& msg);
msamp_status fail_hip(hipError_t e, const char* what);
void clear_error();

#define MSAMP_TRY(expr)                 \
  do {                                  \
    msamp_status st__ = (expr);         \
    if (st__ != MSAMP_OK) return st__;  \
  } while (0)

// Runs 'launch' (which enqueues one kernel and returns its launch status),
// bracketed by events when profiling is on.
hipError_t timed_call(msamp_kernel_kind kind, hipStream_t s, hipError_t (*launch)(void*), void* ctx);

template <typename F>
hipError_t timed(msamp_kernel_kind kind, hipStream_t s, F&& launch) {
  return timed_call(
      kind, s, [](void* f) -> hipError_t { return (*static_cast<std::remove_reference_t<F>*>(f))(); }, &launch);
}

#define MSAMP_LAUNCH(kind, stream, call)                                   \
  do {                                                                     \
    hipError_t e__ = timed((kind), (stream), [&]() { return (call); });   \
    if (e__ != hipSuccess) return fail_hip(e__, msamp_kernel_name(kind));  \
  } while (0)

// No C++ exception crosses the C interface.
template <typename F>
msamp_status guarded(F&& f) {
  try {
    return f();
  } catch (const std::bad_alloc&) {
    return fail(MSAMP_E_NO_MEMORY, "host allocation failed");
  } catch (const std::exception& ex) {
    return fail(MSAMP_E_INVALID_ARG, std::string("internal error: ") + ex.what());
  } catch (...) {
    return fail(MSAMP_E_INVALID_ARG, "internal error");
  }
}

}  // namespace msamp
