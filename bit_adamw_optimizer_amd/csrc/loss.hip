// loss.hip -- losses over a vocabulary and their gradients on gfx950:
// distillation from a teacher's top logits, and the clipped policy loss with a
// KL term. The definitions are in msamp.h.
//
// Both are a softmax over each row's logits and a correction at a few classes:
//   dlogits = c (q - sum over the entries of p at their classes)
// so they share everything but the few numbers of a row: its entries (up to
// 1,024 with the teacher's p, or the action with p = 1) and c.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cmath>

#include "checkpoint.hpp"
#include "lanes.hpp"
#include "model.hpp"

namespace msamp {
namespace {

constexpr int kBlock = 512, kWaves = kBlock / 64;
constexpr int kTop = MSAMP_DISTILL_MAX_TOP;
constexpr float kLog2e = 1.44269504088896341f;

struct LossArgs {
  msamp_vocab_loss a;
  float inv_tau;                     // 1 / tau
  double inv_tau64;
  double log_low, log_high;          // logarithms of the clip's bounds
  float low, high, kl;
};

__device__ __forceinline__ float lane_max(float v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v = __builtin_fmaxf(v, __shfl_xor(v, off, 64));
  return v;
}

// Largest value and sum over the workgroup, given to every thread.
__device__ __forceinline__ float block_largest(float v) {
  __shared__ float part[kWaves];
  v = lane_max(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  v = part[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) v = __builtin_fmaxf(v, part[w]);
  return v;
}
__device__ __forceinline__ float block_sum(float v) {
  __shared__ float part[kWaves];
  v = wave_sum(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  v = part[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) v += part[w];
  return v;
}

// The entries of a row: classes and their p, in LDS.
struct Entries {
  int32_t id[kTop];
  float p[kTop];
};

__device__ __forceinline__ float teacher_at(const msamp_vocab_loss& a, int64_t row, int j) {
  const int64_t i = row * a.ld_teacher + j;
  if (a.teacher_dtype == MSAMP_F32) return ((const GLOBAL float*)a.teacher)[i];
  if (a.teacher_dtype == MSAMP_F16) return to_f32(((const GLOBAL f16*)a.teacher)[i]);
  return to_f32(((const GLOBAL bf16*)a.teacher)[i]);
}

// Fills e with the row's entries (class -1: none). Returns whether the row has
// any; *log_p is what the logarithm of an entry's p is less than its
// (teacher - largest) / tau, which stays in e.p until p is formed.
template <bool POLICY>
__device__ __forceinline__ bool load_entries(const LossArgs& l, int64_t row, Entries& e, float* teacher_max,
                                             float* teacher_sum) {
  const msamp_vocab_loss& a = l.a;
  if constexpr (POLICY) {
    const int64_t id = load_int(a.ids, a.id_bytes, row);
    const bool live = id >= 0 && id < a.vocab;
    if (threadIdx.x == 0) {
      e.id[0] = live ? (int32_t)id : -1;
      e.p[0] = 1.0f;
    }
    __syncthreads();
    return live;
  } else {
    float most = -INFINITY;
    bool nan = false;
    for (int j = threadIdx.x; j < a.top; j += kBlock) {
      const int64_t id = load_int(a.ids, a.id_bytes, row * a.ld_ids + j);
      float t = teacher_at(a, row, j);
      if (id < 0 || id >= a.vocab) t = -INFINITY;
      e.id[j] = t == -INFINITY ? -1 : (int32_t)id;
      e.p[j] = t;
      nan |= t != t;
      most = __builtin_fmaxf(most, t);
    }
    if (nan) most = INFINITY;  // INFINITY - INFINITY: the row's results are NaN
    most = block_largest(most);
    float sum = 0.0f;
    for (int j = threadIdx.x; j < a.top; j += kBlock) {
      const float t = e.id[j] < 0 ? -INFINITY : (e.p[j] - most) * l.inv_tau;
      e.p[j] = t;
      sum += e.id[j] < 0 ? 0.0f : __expf(t);
    }
    sum = block_sum(sum);
    *teacher_max = most;
    *teacher_sum = sum;
    return most != -INFINITY;
  }
}

template <typename T, bool POLICY, bool BACKWARD>
__global__ __launch_bounds__(kBlock) void k_loss(LossArgs l) {
  __shared__ Entries e;
  const msamp_vocab_loss& a = l.a;
  const int top = POLICY ? 1 : (int)a.top;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* z = (const T*)a.logits + row * a.ld_logits;
    T* dz = (T*)a.dlogits + row * a.ld_dlogits;
    float teacher_max = 0.0f, teacher_sum = 1.0f;
    __syncthreads();
    bool live = load_entries<POLICY>(l, row, e, &teacher_max, &teacher_sum);
    float largest = 0.0f, sum = 0.0f;
    if (live) {
      if constexpr (BACKWARD) {
        largest = a.stats[2 * row];
        sum = a.stats[2 * row + 1];
      } else {
        float most = -INFINITY;
        for (int64_t v = threadIdx.x * 8; v < a.vocab; v += kBlock * 8) {
          const int n = (int)(a.vocab - v < 8 ? a.vocab - v : 8);
          float f[8];
          load8(z + v, n, f);
#pragma unroll
          for (int k = 0; k < 8; ++k) most = k < n ? __builtin_fmaxf(most, f[k]) : most;
        }
        largest = block_largest(most);
        // sums of at most 64 pieces are joined, so that no running sum has many terms
        for (int64_t v0 = threadIdx.x * 8; v0 < a.vocab; v0 += 64 * kBlock * 8) {
          float part = 0.0f;
          for (int64_t v = v0; v < a.vocab && v < v0 + 64 * kBlock * 8; v += kBlock * 8) {
            const int n = (int)(a.vocab - v < 8 ? a.vocab - v : 8);
            float f[8];
            load8(z + v, n, f);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              f[k] = k < n ? __builtin_amdgcn_exp2f((f[k] - largest) * (l.inv_tau * kLog2e)) : 0.0f;
            part += ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
          }
          sum += part;
        }
        sum = block_sum(sum);
      }
      if (largest == -INFINITY) live = false, sum = 0.0f;
    }
    if (!BACKWARD && a.stats != nullptr && threadIdx.x == 0) {
      a.stats[2 * row] = largest;
      a.stats[2 * row + 1] = sum;
    }
    // the loss and the factor of the gradient
    float c = 0.0f;
    if (live) {
      const float dloss = a.dlogits == nullptr ? 0.0f : a.dloss == nullptr ? 1.0f : a.dloss[row];
      if constexpr (POLICY) {
        const double lp = (double)(to_f32(z[e.id[0]]) - largest) * l.inv_tau64 - log((double)sum);
        const double d = lp - (double)a.old_logp[row];
        const float adv = a.advantages[row], r = expf((float)d);
        const bool over = adv > 0.0f && d > l.log_high, under = adv < 0.0f && d < l.log_low;
        const float away = l.kl != 0.0f ? (float)((double)a.ref_logp[row] - lp) : 0.0f;
        const float more = expm1f(away);
        if (!BACKWARD && threadIdx.x == 0) {
          const float first = adv == 0.0f ? 0.0f : (over ? l.high : under ? l.low : r) * adv;
          a.loss[row] = l.kl * (more - away) - first;
          if (a.logp != nullptr) a.logp[row] = (float)lp;
        }
        const float g = -l.kl * more - (over || under || adv == 0.0f ? 0.0f : r * adv);
        c = -dloss * g * l.inv_tau;
      } else {
        const float log_sum = logf(sum), log_teacher = logf(teacher_sum), inv = 1.0f / teacher_sum;
        float part = 0.0f;
        for (int j = threadIdx.x; j < top; j += kBlock) {
          if (e.id[j] < 0) continue;
          const float t = e.p[j], p = __expf(t) * inv;
          if (!BACKWARD && p != 0.0f) {
            const float q = (to_f32(z[e.id[j]]) - largest) * l.inv_tau;
            part += p * ((t - log_teacher) - (q - log_sum));
          }
          e.p[j] = p;
        }
        if (!BACKWARD) {
          const float tau = (float)a.temperature;
          part = block_sum(part);
          if (threadIdx.x == 0) a.loss[row] = tau * tau * part;
        }
        c = dloss * (float)a.temperature;
      }
    } else if (!BACKWARD && threadIdx.x == 0) {
      a.loss[row] = 0.0f;
      if (POLICY && a.logp != nullptr) a.logp[row] = 0.0f;
    }
    if (a.dlogits == nullptr) continue;
    if (!live) {
      const float zero[8] = {};
      for (int64_t v = threadIdx.x * 8; v < a.vocab; v += kBlock * 8)
        store8<T, true>(dz + v, (int)(a.vocab - v < 8 ? a.vocab - v : 8), zero);
      continue;
    }
    const float inv = 1.0f / sum, scale = l.inv_tau * kLog2e;
    __syncthreads();  // every p is in LDS
    float at[(kTop + kBlock - 1) / kBlock];
    for (int j = threadIdx.x, i = 0; j < top; j += kBlock, ++i) {
      at[i] = 0.0f;
      if (e.id[j] < 0) continue;
      float p = 0.0f;  // of every entry of this class, in their order: the same sum from each of them
      for (int k = 0; k < top; ++k)
        if (e.id[k] == e.id[j]) p += e.p[k];
      at[i] = (__builtin_amdgcn_exp2f((to_f32(z[e.id[j]]) - largest) * scale) * inv - p) * c;
    }
    __syncthreads();  // the classes' logits are read before dlogits, which may be logits, is written
    for (int64_t v = threadIdx.x * 8; v < a.vocab; v += kBlock * 8) {
      const int n = (int)(a.vocab - v < 8 ? a.vocab - v : 8);
      float f[8];
      load8(z + v, n, f);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = __builtin_amdgcn_exp2f((f[k] - largest) * scale) * inv * c;
      store8(dz + v, n, f);
    }
    __syncthreads();  // the entries' values go over the others'
    for (int j = threadIdx.x, i = 0; j < top; j += kBlock, ++i)
      if (e.id[j] >= 0) dz[e.id[j]] = from_f32<T>(at[i]);
  }
}

LossArgs loss_args(const msamp_vocab_loss& a) {
  LossArgs l;
  l.a = a;
  l.inv_tau = (float)(1.0 / a.temperature);
  l.inv_tau64 = 1.0 / a.temperature;
  l.log_low = std::log(1.0 - a.clip_low);
  l.log_high = std::log1p(a.clip_high);
  l.low = (float)(1.0 - a.clip_low);
  l.high = (float)(1.0 + a.clip_high);
  l.kl = (float)a.kl;
  return l;
}

template <bool POLICY, bool BACKWARD>
hipError_t run(const msamp_vocab_loss& a, hipStream_t s) {
  const LossArgs l = loss_args(a);
  const unsigned grid = (unsigned)(a.rows < (1 << 20) ? a.rows : 1 << 20);
  if (a.dtype == MSAMP_F32) k_loss<float, POLICY, BACKWARD><<<grid, kBlock, 0, s>>>(l);
  else if (a.dtype == MSAMP_F16) k_loss<f16, POLICY, BACKWARD><<<grid, kBlock, 0, s>>>(l);
  else k_loss<bf16, POLICY, BACKWARD><<<grid, kBlock, 0, s>>>(l);
  return hipGetLastError();
}

}  // namespace

int64_t loss_workspace(const msamp_vocab_loss&) { return 0; }

hipError_t launch_loss_forward(bool policy, const msamp_vocab_loss& a, void*, hipStream_t s) {
  return policy ? run<true, false>(a, s) : run<false, false>(a, s);
}

hipError_t launch_loss_backward(bool policy, const msamp_vocab_loss& a, hipStream_t s) {
  return policy ? run<true, true>(a, s) : run<false, true>(a, s);
}

}  // namespace msamp
