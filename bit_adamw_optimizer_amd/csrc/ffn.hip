// ffn.hip -- the gated feed-forward block on gfx950: gate and up projections,
// activation and product in one kernel, and its backward pass, which forms
// gate and up again from the block's input. The definitions are in msamp.h.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "checkpoint.hpp"
#include "ffn.hpp"

namespace msamp {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef f16 f16x8 __attribute__((ext_vector_type(8)));
typedef bf16 bf16x8 __attribute__((ext_vector_type(8)));

template <typename T>
struct Frag;
template <>
struct Frag<f16> {
  typedef f16x8 type;
  static __device__ __forceinline__ f32x16 mma(f16x8 a, f16x8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
  }
};
template <>
struct Frag<bf16> {
  typedef bf16x8 type;
  static __device__ __forceinline__ f32x16 mma(bf16x8 a, bf16x8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
};

// ------------------------------------------------------------ activation ---

// act(g) and act'(g).
__device__ __forceinline__ void act_and_grad(int act, float g, float* a, float* d) {
  if (act == MSAMP_ACT_SILU) {
    const float s = 1.0f / (1.0f + __expf(-g));
    *a = g * s;
    *d = s * (1.0f + g * (1.0f - s));
  } else if (act == MSAMP_ACT_GELU) {
    const float phi = 0.5f * (1.0f + erff(g * 0.70710678118654752f));
    *a = g * phi;
    *d = phi + g * 0.39894228040143268f * __expf(-0.5f * g * g);
  } else {
    // (1 + tanh(z)) / 2 = 1 / (1 + e^(-2z))
    const float z2 = 1.5957691216057308f * (g + 0.044715f * g * g * g);
    const float s = 1.0f / (1.0f + __expf(-z2));
    *a = g * s;
    *d = s + g * s * (1.0f - s) * 1.5957691216057308f * (1.0f + 0.134145f * g * g);
  }
}

// -------------------------------------------------------- matrix product ---

// C[m, n] = sum_k A[m, k] B[n, k] with any strides; 64 x 64 tiles.
enum Mode { kForward, kRecompute, kDx, kDw };

struct Product {
  int64_t M, N, K;
  const void *a0, *a1;  // a1: the second sum's left operand (kDx)
  int64_t am, ak;
  const void *b0, *b1;  // b1: up (kForward, kRecompute), the second sum's right operand (kDx)
  int64_t bn0, bk0, bn1, bk1;
  int act;
  void* out;  // h, dx or a weight gradient
  int64_t ldo;
  bool out_f32;
  int accumulate;
  const void* dh;
  int64_t lddh;
  void *dg, *du;
  int64_t ldd;
};

constexpr int kTileM = 64, kTileN = 64, kTileK = 32, kPad = 8;

template <typename T>
__device__ __forceinline__ void stage(T (*lds)[kTileK + kPad], const T* src, int64_t rows, int64_t K, int64_t sr,
                                      int64_t sk, int64_t r0, int64_t k0) {
  for (int i = threadIdx.x; i < 64 * kTileK; i += 256) {
    // consecutive threads along the consecutive elements
    const int r = sk == 1 ? i / kTileK : i % 64, k = sk == 1 ? i % kTileK : i / 64;
    T v = (T)0.0f;
    if (r0 + r < rows && k0 + k < K) v = src[(r0 + r) * sr + (k0 + k) * sk];
    lds[r][k] = v;
  }
}

template <typename T, int MODE>
__global__ __launch_bounds__(256) void k_product(Product p) {
  typedef typename Frag<T>::type frag;
  constexpr bool kTwo = MODE == kForward || MODE == kRecompute;
  __shared__ __attribute__((aligned(16))) T As[kTileM][kTileK + kPad];
  __shared__ __attribute__((aligned(16))) T Bs[kTwo ? 2 : 1][kTileN][kTileK + kPad];
  const int64_t m0 = (int64_t)blockIdx.y * kTileM, n0 = (int64_t)blockIdx.x * kTileN;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32;
  f32x16 acc0 = {}, acc1 = {};
  for (int pass = 0; pass < (MODE == kDx ? 2 : 1); ++pass) {
    const T* A = (const T*)(pass == 0 ? p.a0 : p.a1);
    const T* B = (const T*)(pass == 0 ? p.b0 : p.b1);
    const int64_t bn = pass == 0 ? p.bn0 : p.bn1, bk = pass == 0 ? p.bk0 : p.bk1;
    for (int64_t k0 = 0; k0 < p.K; k0 += kTileK) {
      __syncthreads();
      stage(As, A, p.M, p.K, p.am, p.ak, m0, k0);
      stage(Bs[0], B, p.N, p.K, bn, bk, n0, k0);
      if constexpr (kTwo) stage(Bs[1], (const T*)p.b1, p.N, p.K, p.bn1, p.bk1, n0, k0);
      __syncthreads();
#pragma unroll
      for (int kk = 0; kk < kTileK; kk += 16) {
        const frag a = *(const frag*)&As[wm + (lane & 31)][kk + (lane >> 5) * 8];
        const frag b = *(const frag*)&Bs[0][wn + (lane & 31)][kk + (lane >> 5) * 8];
        acc0 = Frag<T>::mma(a, b, acc0);
        if constexpr (kTwo) {
          const frag c = *(const frag*)&Bs[1][wn + (lane & 31)][kk + (lane >> 5) * 8];
          acc1 = Frag<T>::mma(a, c, acc1);
        }
      }
    }
  }
  const int64_t n = n0 + wn + (lane & 31);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int64_t m = m0 + wm + (i / 4) * 8 + (lane >> 5) * 4 + (i & 3);
    if (m >= p.M || n >= p.N) continue;
    if constexpr (kTwo) {
      float a, d;
      act_and_grad(p.act, acc0[i], &a, &d);
      if (p.out != nullptr) ((T*)p.out)[m * p.ldo + n] = from_f32<T>(a * acc1[i]);
      if constexpr (MODE == kRecompute) {
        const float dh = to_f32(((const T*)p.dh)[m * p.lddh + n]);
        ((T*)p.dg)[m * p.ldd + n] = from_f32<T>(dh * acc1[i] * d);
        ((T*)p.du)[m * p.ldd + n] = from_f32<T>(dh * a);
      }
    } else if (p.out_f32) {
      float* o = (float*)p.out + m * p.ldo + n;
      *o = p.accumulate ? *o + acc0[i] : acc0[i];
    } else {
      ((T*)p.out)[m * p.ldo + n] = from_f32<T>(acc0[i]);
    }
  }
}

template <int MODE>
hipError_t launch_product(int dtype, const Product& p, hipStream_t s) {
  const dim3 g((unsigned)((p.N + kTileN - 1) / kTileN), (unsigned)((p.M + kTileM - 1) / kTileM));
  if (dtype == MSAMP_F16) k_product<f16, MODE><<<g, dim3(256), 0, s>>>(p);
  else k_product<bf16, MODE><<<g, dim3(256), 0, s>>>(p);
  return hipGetLastError();
}

int64_t round256(int64_t n) { return (n + 255) / 256 * 256; }

}  // namespace

int64_t ffn_forward_workspace(const msamp_gated_ffn&) { return 0; }

int64_t ffn_backward_workspace(const msamp_gated_ffn& a) {
  return 2 * round256(a.tokens * a.ffn * 2) + (a.x_ckpt != nullptr ? round256(a.tokens * a.hidden * 2) : 0);
}

msamp_status ffn_forward(const msamp_gated_ffn& a, void*, hipStream_t s) {
  if (a.tokens == 0 || a.ffn == 0) return MSAMP_OK;
  Product p = {};
  p.M = a.tokens, p.N = a.ffn, p.K = a.hidden;
  p.a0 = a.x, p.am = a.ldx, p.ak = 1;
  p.b0 = a.w_gate, p.bn0 = a.ld_gate, p.bk0 = 1;
  p.b1 = a.w_up, p.bn1 = a.ld_up, p.bk1 = 1;
  p.act = a.act;
  p.out = a.h, p.ldo = a.ldh;
  MSAMP_LAUNCH(MSAMP_KERNEL_FFN_FORWARD, s, launch_product<kForward>(a.dtype, p, s));
  return MSAMP_OK;
}

msamp_status ffn_backward(const msamp_gated_ffn& a, void* ws, hipStream_t s) {
  char* w = (char*)ws;
  void* dg = w;
  w += round256(a.tokens * a.ffn * 2);
  void* du = w;
  w += round256(a.tokens * a.ffn * 2);
  const void* x = a.x;
  int64_t ldx = a.ldx;
  if (a.x_ckpt != nullptr && a.tokens > 0 && a.hidden > 0) {
    const CkptRef ck = {a.x_ckpt->codes, a.x_ckpt->ld, a.x_ckpt->scales, a.x_ckpt->ld_scales, (int)a.x_ckpt->fmt};
    MSAMP_LAUNCH(MSAMP_KERNEL_FFN_LAYOUT, s,
                 launch_checkpoint_load(a.dtype, a.tokens, a.hidden, ck, w, a.hidden, s));
    x = w;
    ldx = a.hidden;
  }
  Product p = {};
  if (a.tokens > 0 && a.ffn > 0) {
    p.M = a.tokens, p.N = a.ffn, p.K = a.hidden;
    p.a0 = x, p.am = ldx, p.ak = 1;
    p.b0 = a.w_gate, p.bn0 = a.ld_gate, p.bk0 = 1;
    p.b1 = a.w_up, p.bn1 = a.ld_up, p.bk1 = 1;
    p.act = a.act;
    p.out = a.h, p.ldo = a.ldh;
    p.dh = a.dh, p.lddh = a.lddh;
    p.dg = dg, p.du = du, p.ldd = a.ffn;
    MSAMP_LAUNCH(MSAMP_KERNEL_FFN_RECOMPUTE, s, launch_product<kRecompute>(a.dtype, p, s));
  }
  if (a.hidden == 0) return MSAMP_OK;
  if (a.tokens > 0) {
    p = {};
    p.M = a.tokens, p.N = a.hidden, p.K = a.ffn;
    p.a0 = dg, p.a1 = du, p.am = a.ffn, p.ak = 1;
    p.b0 = a.w_gate, p.bn0 = 1, p.bk0 = a.ld_gate;
    p.b1 = a.w_up, p.bn1 = 1, p.bk1 = a.ld_up;
    p.out = a.dx, p.ldo = a.lddx;
    MSAMP_LAUNCH(MSAMP_KERNEL_FFN_DX, s, launch_product<kDx>(a.dtype, p, s));
  }
  for (int i = 0; i < 2 && a.ffn > 0; ++i) {
    p = {};
    p.M = a.ffn, p.N = a.hidden, p.K = a.tokens;
    p.a0 = i == 0 ? dg : du, p.am = 1, p.ak = a.ffn;
    p.b0 = x, p.bn0 = 1, p.bk0 = ldx;
    p.out = i == 0 ? a.dw_gate : a.dw_up, p.ldo = i == 0 ? a.ld_dw_gate : a.ld_dw_up;
    p.out_f32 = a.dw_dtype == MSAMP_F32;
    p.accumulate = a.dw_accumulate;
    MSAMP_LAUNCH(MSAMP_KERNEL_FFN_DW, s, launch_product<kDw>(a.dtype, p, s));
  }
  return MSAMP_OK;
}

}  // namespace msamp
