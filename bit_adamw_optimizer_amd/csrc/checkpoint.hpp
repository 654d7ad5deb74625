// checkpoint.hpp -- device side of the 8-bit activation checkpoint (groups of
// 32 elements of a row, one power-of-two scale each; defined in msamp.h), and
// the 8-element loads and stores that its kernels and the norms share.
//
// Eight consecutive elements belong to one lane, so a group is four
// neighbouring lanes and its largest magnitude takes two exchanges.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "codec.hpp"
#include "device.hpp"
#include "train.hpp"

namespace msamp {

typedef __bf16 bf16;
typedef _Float16 f16;

// 16-byte, 8-byte accesses at any address that is aligned for the element:
// the hardware takes such addresses, so odd row lengths need no other path.
typedef u32x4 u32x4_any __attribute__((aligned(1)));
typedef u32x2 u32x2_any __attribute__((aligned(1)));

constexpr int kGroup = MSAMP_CHECKPOINT_GROUP;
constexpr float kF32Max = 3.402823466e+38f;
constexpr float kBf16Max = 3.3895313892515355e+38f;

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(f16 v) { return (float)v; }
__device__ __forceinline__ float to_f32(bf16 v) { return (float)v; }

// One rounding to nearest even (as_f32: no fusing of an earlier rounding).
template <typename T>
__device__ __forceinline__ T from_f32(float v) {
  if constexpr (sizeof(T) == 4)
    return v;
  else
    return (T)as_f32(v);
}

// n (<= 8) consecutive elements from p; zeros behind them.
template <typename T>
__device__ __forceinline__ void load8(const T* p, int n, float* f) {
  if (n >= 8) {
    if constexpr (sizeof(T) == 4) {
      u32x4 a = *(const GLOBAL u32x4_any*)p, b = *((const GLOBAL u32x4_any*)p + 1);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        f[k] = __uint_as_float(a[k]);
        f[k + 4] = __uint_as_float(b[k]);
      }
    } else {
      u32x4 a = *(const GLOBAL u32x4_any*)p;
      typedef T t8 __attribute__((ext_vector_type(8)));
      t8 v = __builtin_bit_cast(t8, a);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = to_f32(v[k]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = k < n ? to_f32(((const GLOBAL T*)p)[k]) : 0.0f;
  }
}

// STREAM: past the caches.
template <typename T, bool STREAM = false>
__device__ __forceinline__ void store8(T* p, int n, const float* f) {
  auto put = [](u32x4 v, GLOBAL u32x4_any* q) {
    if constexpr (STREAM) __builtin_nontemporal_store(v, q);
    else *q = v;
  };
  if (n >= 8) {
    if constexpr (sizeof(T) == 4) {
      u32x4 a, b;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        a[k] = __float_as_uint(f[k]);
        b[k] = __float_as_uint(f[k + 4]);
      }
      put(a, (GLOBAL u32x4_any*)p);
      put(b, (GLOBAL u32x4_any*)p + 1);
    } else {
      typedef T t8 __attribute__((ext_vector_type(8)));
      t8 v;
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = from_f32<T>(f[k]);
      put(__builtin_bit_cast(u32x4, v), (GLOBAL u32x4_any*)p);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) ((GLOBAL T*)p)[k] = from_f32<T>(f[k]);
  }
}

// 2^e for e in [-126, 127].
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// The smallest e with amax <= fp8_max * 2^e (fp8_max = 1.75 * 2^emax), at
// least -126; 0 for amax 0, Inf or NaN. 'bits': amax as binary32 bits.
template <int FMT>
__device__ __forceinline__ int group_exponent(uint32_t bits) {
  constexpr int emax = FMT == kE4M3 ? 8 : 15;
  if (bits == 0u || bits >= 0x7F800000u) return 0;
  int e = (int)(bits >> 23) - 127 - emax + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return e < -126 ? -126 : e;
}

// Codes of a lane's eight elements (f, zeros behind the row's end) and their
// group's exponent. The four lanes of a group run this together.
template <int FMT>
__device__ __forceinline__ u32x2 encode_group8(const float* f, int* e) {
  uint32_t m = 0u;
#pragma unroll
  for (int k = 0; k < 8; ++k) m = umax(m, abs_bits(f[k]));
  m = umax(m, (uint32_t)__shfl_xor((int)m, 1, 64));
  m = umax(m, (uint32_t)__shfl_xor((int)m, 2, 64));
  *e = group_exponent<FMT>(m);
  const float s = pow2i(-*e);
  float g[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) g[k] = f[k] * s;
  u32x2 q;
  if (m <= 0x7F800000u) {  // no NaN in the group
    q = enc8<FMT>(g);
  } else {
    q.x = enc4_nan<FMT>(g);
    q.y = enc4_nan<FMT>(g + 4);
  }
  return q;
}

__device__ __forceinline__ void store_codes8(uint8_t* p, int n, u32x2 q) {
  if (n >= 8) {
    *(GLOBAL u32x2_any*)p = q;
  } else {
    for (int k = 0; k < n; ++k) ((GLOBAL uint8_t*)p)[k] = (uint8_t)((k < 4 ? q.x : q.y) >> (8 * (k & 3)));
  }
}

// Saves a lane's eight elements (column col of its row, n <= 8 of them real)
// into a checkpoint's row: all four lanes of a group call it together.
__device__ __forceinline__ void save_group8(int fmt, uint8_t* codes, uint8_t* scales, int64_t col, int n,
                                            const float* f) {
  int e;
  u32x2 q = fmt == kE4M3 ? encode_group8<kE4M3>(f, &e) : encode_group8<kE5M2>(f, &e);
  if (n <= 0) return;
  store_codes8(codes + col, n, q);
  if (col % kGroup == 0) ((GLOBAL uint8_t*)scales)[col / kGroup] = (uint8_t)(e + 127);
}

// Finite range of an output type: a finite value beyond it becomes the
// largest finite one (a code may round up to the next power of two).
__device__ __forceinline__ float clamp_finite(float v, float lim) {
  const float c = __builtin_amdgcn_fmed3f(v, -lim, lim);
  return __builtin_isnan(v) ? v : c;
}

// The values of eight codes with their group's scale byte.
__device__ __forceinline__ void decode_group8(int fmt, u32x2 q, uint32_t b, float* f) {
  if (fmt == kE4M3) dec8<kE4M3>(q, f); else dec8<kE5M2>(q, f);
  const float s = __uint_as_float(b << 23);
#pragma unroll
  for (int k = 0; k < 8; ++k) f[k] *= s;
  if (b >= 127u + 112u) {  // 57344 * 2^112 and above may leave binary32
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = clamp_finite(f[k], kF32Max);
  }
}

// n (<= 8) values of a checkpoint's row from column col; zeros behind them.
__device__ __forceinline__ void load_ckpt8(int fmt, const uint8_t* codes, const uint8_t* scales, int64_t col, int n,
                                           float* f) {
  u32x2 q = {0u, 0u};
  uint32_t b = 127u;
  if (n >= 8) {
    q = *(const GLOBAL u32x2_any*)(codes + col);
  } else {
    for (int k = 0; k < n; ++k) {
      const uint32_t c = (uint32_t)((const GLOBAL uint8_t*)codes)[col + k] << (8 * (k & 3));
      if (k < 4) q.x |= c; else q.y |= c;
    }
  }
  if (n > 0) b = ((const GLOBAL uint8_t*)scales)[col / kGroup];
  decode_group8(fmt, q, b, f);
}

}  // namespace msamp
