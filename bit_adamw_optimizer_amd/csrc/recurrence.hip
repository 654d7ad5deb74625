// recurrence.hip -- the gated linear recurrence, forward and backward, on
// gfx950. The definition is in msamp.h.
//
// Two channels to a lane: h_t = a_t h_{t-1} + (1 - a_t) x_t has no products
// between channels, so all of it is bound by memory, or, where there are few
// channels, by the chain over time.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "checkpoint.hpp"
#include "model.hpp"

namespace msamp {
namespace {

constexpr int kChunk = MSAMP_RECURRENCE_CHUNK;

// Two consecutive channels as they lie in memory; n (1 or 2) of them are the
// tensor's.
template <typename T>
struct Pair;
template <>
struct Pair<float> {
  typedef u32x2 raw;
  static __device__ __forceinline__ raw load(const float* p, int n) {
    if (n >= 2) return *(const GLOBAL u32x2_any*)p;
    return raw{*(const GLOBAL uint32_t*)p, 0u};
  }
  static __device__ __forceinline__ float2 values(raw r) {
    return make_float2(__uint_as_float(r.x), __uint_as_float(r.y));
  }
  static __device__ __forceinline__ void store(float* p, int n, float2 v) {
    if (n >= 2) *(GLOBAL u32x2_any*)p = u32x2{__float_as_uint(v.x), __float_as_uint(v.y)};
    else *(GLOBAL float*)p = v.x;
  }
};
typedef uint32_t u32_any __attribute__((aligned(1)));
template <typename T>
struct Pair {
  typedef uint32_t raw;
  static __device__ __forceinline__ raw load(const T* p, int n) {
    if (n >= 2) return *(const GLOBAL u32_any*)p;
    return (raw) * (const GLOBAL uint16_t*)p;
  }
  static __device__ __forceinline__ float2 values(raw r) {
    return make_float2(to_f32(__builtin_bit_cast(T, (uint16_t)(r & 0xFFFFu))),
                       to_f32(__builtin_bit_cast(T, (uint16_t)(r >> 16))));
  }
  static __device__ __forceinline__ void store(T* p, int n, float2 v) {
    const uint32_t lo = __builtin_bit_cast(uint16_t, from_f32<T>(v.x));
    if (n >= 2) *(GLOBAL u32_any*)p = lo | (uint32_t)__builtin_bit_cast(uint16_t, from_f32<T>(v.y)) << 16;
    else *(GLOBAL uint16_t*)p = (uint16_t)lo;
  }
};

// a = 1 / (1 + e^-g) and keep = 1 - a = 1 / (1 + e^g) from one exponential,
// e^-|g|, so that the smaller of the two keeps its digits.
__device__ __forceinline__ void gate1(float g, float* a, float* keep) {
  const float e = __builtin_amdgcn_exp2f(-__builtin_fabsf(g) * 1.44269504088896341f);
  const float big = __builtin_amdgcn_rcpf(1.0f + e), small = e * big;
  *a = g >= 0.0f ? big : small;
  *keep = g >= 0.0f ? small : big;
}
__device__ __forceinline__ void gate2(float2 g, float2* a, float2* keep) {
  gate1(g.x, &a->x, &keep->x);
  gate1(g.y, &a->y, &keep->y);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  return make_float2(__builtin_fmaf(a.x, b.x, c.x), __builtin_fmaf(a.y, b.y, c.y));
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return make_float2(a.x * b.x, a.y * b.y); }

__device__ __forceinline__ int64_t length_of(const msamp_recurrence& a, int64_t b) {
  if (a.lengths == nullptr) return a.time;
  const int64_t n = load_int(a.lengths, a.length_bytes, b);
  return n < 0 ? 0 : n < a.time ? n : a.time;
}

// ------------------------------------------------------ one lane, all steps ---

constexpr int kBlock = 256;

// Each lane goes through all steps of its two channels.
template <typename T>
__global__ __launch_bounds__(kBlock) void k_forward_lane(msamp_recurrence a, int64_t pairs) {
  const int64_t i = (int64_t)blockIdx.x * kBlock + threadIdx.x;
  if (i >= a.batch * pairs) return;
  const int64_t b = i / pairs, c = (i - b * pairs) * 2;
  const int n = a.channels - c < 2 ? 1 : 2;
  const int64_t len = length_of(a, b);
  float2 h = a.h0 == nullptr ? make_float2(0.0f, 0.0f)
                             : Pair<float>::values(Pair<float>::load(a.h0 + b * a.ld_h0 + c, n));
  const T* x = (const T*)a.x + b * a.x_batch + c;
  const T* g = (const T*)a.gate + b * a.gate_batch + c;
  T* y = (T*)a.y + b * a.y_batch + c;
  float* states = a.states == nullptr ? nullptr : a.states + b * ((a.time + kChunk - 1) / kChunk) * a.channels + c;
  for (int64_t t = 0; t < len; ++t) {
    if (states != nullptr && t % kChunk == 0) Pair<float>::store(states + t / kChunk * a.channels, n, h);
    float2 av, keep;
    gate2(Pair<T>::values(Pair<T>::load(g + t * a.gate_time, n)), &av, &keep);
    h = fma2(av, h, mul2(keep, Pair<T>::values(Pair<T>::load(x + t * a.x_time, n))));
    Pair<T>::store(y + t * a.y_time, n, h);
  }
  if (a.h_last != nullptr) Pair<float>::store(a.h_last + b * a.ld_h_last + c, n, h);
}

// The same backward in time: h before each step of a chunk again from the
// chunk's state, then the gradients. 'm' is a_{t+1} l_{t+1}.
template <typename T>
__global__ __launch_bounds__(kBlock) void k_backward_lane(msamp_recurrence a, int64_t pairs) {
  const int64_t i = (int64_t)blockIdx.x * kBlock + threadIdx.x;
  if (i >= a.batch * pairs) return;
  const int64_t b = i / pairs, c = (i - b * pairs) * 2;
  const int n = a.channels - c < 2 ? 1 : 2;
  const int64_t len = length_of(a, b);
  float2 m = a.dh_last == nullptr ? make_float2(0.0f, 0.0f)
                                  : Pair<float>::values(Pair<float>::load(a.dh_last + b * a.ld_dh_last + c, n));
  const T* x = (const T*)a.x + b * a.x_batch + c;
  const T* g = (const T*)a.gate + b * a.gate_batch + c;
  const T* dy = (const T*)a.dy + b * a.dy_batch + c;
  T* dx = (T*)a.dx + b * a.dx_batch + c;
  T* dg = (T*)a.dgate + b * a.dgate_batch + c;
  const int64_t chunks = (a.time + kChunk - 1) / kChunk;
  for (int64_t k = (len + kChunk - 1) / kChunk - 1; k >= 0; --k) {
    const int64_t t0 = k * kChunk;
    const int steps = (int)(len - t0 < kChunk ? len - t0 : kChunk);
    float2 h = Pair<float>::values(Pair<float>::load(a.states + (b * chunks + k) * a.channels + c, n));
    float2 av[kChunk], keep[kChunk], slope[kChunk];
#pragma unroll
    for (int r = 0; r < kChunk; ++r) {
      if (r < steps) {
        const float2 xv = Pair<T>::values(Pair<T>::load(x + (t0 + r) * a.x_time, n));
        gate2(Pair<T>::values(Pair<T>::load(g + (t0 + r) * a.gate_time, n)), &av[r], &keep[r]);
        slope[r] = mul2(make_float2(h.x - xv.x, h.y - xv.y), mul2(av[r], keep[r]));
        h = fma2(av[r], h, mul2(keep[r], xv));
      }
    }
#pragma unroll
    for (int r = kChunk - 1; r >= 0; --r) {
      if (r < steps) {
        const float2 d = Pair<T>::values(Pair<T>::load(dy + (t0 + r) * a.dy_time, n));
        const float2 l = make_float2(d.x + m.x, d.y + m.y);
        Pair<T>::store(dx + (t0 + r) * a.dx_time, n, mul2(keep[r], l));
        Pair<T>::store(dg + (t0 + r) * a.dgate_time, n, mul2(slope[r], l));
        m = mul2(av[r], l);
      }
    }
  }
  if (a.dh0 != nullptr) Pair<float>::store(a.dh0 + b * a.ld_dh0 + c, n, m);
}

template <typename T>
hipError_t forward(const msamp_recurrence& a, void*, hipStream_t s) {
  const int64_t pairs = (a.channels + 1) / 2;
  k_forward_lane<T><<<(unsigned)((a.batch * pairs + kBlock - 1) / kBlock), kBlock, 0, s>>>(a, pairs);
  return hipGetLastError();
}

template <typename T>
hipError_t backward(const msamp_recurrence& a, void*, hipStream_t s) {
  const int64_t pairs = (a.channels + 1) / 2;
  k_backward_lane<T><<<(unsigned)((a.batch * pairs + kBlock - 1) / kBlock), kBlock, 0, s>>>(a, pairs);
  return hipGetLastError();
}

}  // namespace

int64_t recurrence_workspace(const msamp_recurrence&, bool) { return 0; }

hipError_t launch_recurrence_forward(const msamp_recurrence& a, void* ws, hipStream_t s) {
  return a.dtype == MSAMP_F32 ? forward<float>(a, ws, s)
                              : a.dtype == MSAMP_F16 ? forward<f16>(a, ws, s) : forward<bf16>(a, ws, s);
}

hipError_t launch_recurrence_backward(const msamp_recurrence& a, void* ws, hipStream_t s) {
  return a.dtype == MSAMP_F32 ? backward<float>(a, ws, s)
                              : a.dtype == MSAMP_F16 ? backward<f16>(a, ws, s) : backward<bf16>(a, ws, s);
}

}  // namespace msamp
