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

constexpr double kLog2e = 1.44269504088896341;

struct LossArgs {
  msamp_vocab_loss a;
  int64_t row0;              // of the launch's first workgroup
  float inv_tau, scale;      // 1 / tau, log2(e) / tau, rounded once each
  double inv_tau64;
  double log_low, log_high;  // logarithms of the clip's bounds
  double low, high, kl;
};

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v = __builtin_fmaxf(v, __shfl_xor(v, off, 64));
  return v;
}

// A piece of a row: the 16 bytes of 8 logits, or of 4 in binary32, as they lie
// in memory.
template <typename T>
constexpr int kPer = 16 / (int)sizeof(T);

template <typename T>
__device__ __forceinline__ void values(u32x4 r, float* f) {
  struct V {
    T v[kPer<T>];
  };
  const V v = __builtin_bit_cast(V, r);
#pragma unroll
  for (int k = 0; k < kPer<T>; ++k) f[k] = to_f32(v.v[k]);
}
template <typename T>
__device__ __forceinline__ u32x4 rounded(const float* f) {
  struct V {
    T v[kPer<T>];
  } v;
#pragma unroll
  for (int k = 0; k < kPer<T>; ++k) v.v[k] = from_f32<T>(f[k]);
  return __builtin_bit_cast(u32x4, v);
}

// The pieces of a row start at its first logit on 16 bytes. They are read and
// written through a buffer that ends behind the last whole one, so that a piece
// has one offset and none is beyond the row. The few logits before and behind
// the pieces are a thread's each.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_buffer(const void* p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00020000);
}
constexpr int kPastCaches = 2;             // nt
constexpr uint32_t kOutside = 0x80000000u;  // beyond every buffer: read as 0, not written

// Nothing to the hardware; to the compiler another value, so that it unpacks a
// row's logits again in each pass instead of keeping them in twice the
// registers.
__device__ __forceinline__ void again(u32x4& r) { asm volatile("" : "+v"(r)); }

// A row's softmax while it is formed: the largest logit and the sum of
// exp2((z - largest) scale). Logits of -Inf alone leave the largest at -Inf
// and the sum at 0; a NaN makes the sum NaN.
// Both are binary32, as the stats that the backward pass takes are: terms are
// added as trees of 8 over pieces, lanes and waves, and an exponent is off by
// 2^-23 of itself, that is least where a term has weight. log(sum) is off by
// 3e-8 at the median (rows of 512 binary32 logits), half a step of the stored
// sum.
struct Soft {
  float largest, sum;
};
__device__ __forceinline__ Soft join(Soft a, Soft b, float scale) {
  const float m = __builtin_fmaxf(a.largest, b.largest), base = m == -INFINITY ? 0.0f : m;
  return {m, a.sum * __builtin_amdgcn_exp2f((a.largest - base) * scale) +
                 b.sum * __builtin_amdgcn_exp2f((b.largest - base) * scale)};
}
template <int N>
__device__ __forceinline__ float sum_exp(const float* f, float base, float scale) {
  float e[N];
#pragma unroll
  for (int k = 0; k < N; ++k) e[k] = __builtin_amdgcn_exp2f((f[k] - base) * scale);
#pragma unroll
  for (int n = N / 2; n > 0; n /= 2)
#pragma unroll
    for (int k = 0; k < n; ++k) e[k] += e[k + n];
  return e[0];
}

__device__ __forceinline__ float teacher_at(const msamp_vocab_loss& a, int64_t row, int j) {
  const int64_t i = row * a.ld_teacher + j;
  if (a.teacher_dtype == MSAMP_F32) return ((const GLOBAL float*)a.teacher)[i];
  if (a.teacher_dtype == MSAMP_F16) return to_f32(((const GLOBAL f16*)a.teacher)[i]);
  return to_f32(((const GLOBAL bf16*)a.teacher)[i]);
}

// The pieces of a row, or of a part of it, that a workgroup holds.
template <typename T, int BLOCK, int NCH>
struct Held {
  u32x4 raw[NCH];
  float single;      // this thread's logit outside the pieces; -Inf: none
  int whole;         // pieces
  int64_t start;     // of the pieces
  int64_t lo, hi;    // of the part, with the logits outside the pieces
  int64_t single_v;  // where this thread's is; -1: none

  __device__ __forceinline__ uint32_t at(int i) const {
    const int p = i * BLOCK + (int)threadIdx.x;
    return p < whole ? (uint32_t)p * 16 : kOutside;
  }
  __device__ __forceinline__ void cut(const T* z, int part, int64_t vocab) {
    constexpr int N = kPer<T>, kMost = BLOCK * NCH;
    int64_t head = (-(int64_t)(uintptr_t)z & 15) / (int)sizeof(T);
    if (head > vocab) head = vocab;
    start = head + (int64_t)part * (kMost * N);
    const int64_t left = vocab > start ? (vocab - start) / N : 0;
    whole = left < kMost ? (int)left : kMost;
    const int64_t end = start + (int64_t)whole * N;
    const bool last = whole < kMost;
    lo = part == 0 ? 0 : start;
    hi = last ? vocab : end;
    const int i = threadIdx.x;
    single_v = part == 0 && i < head ? i : last && i >= 16 && end + i - 16 < vocab ? end + i - 16 : -1;
  }
  template <int CACHES>
  __device__ __forceinline__ void load(const T* z) {
    const auto b = row_buffer(z + start, (int64_t)whole * 16);
#pragma unroll
    for (int i = 0; i < NCH; ++i)
      raw[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(b, at(i), 0, CACHES));
    single = single_v >= 0 ? to_f32(((const GLOBAL T*)z)[single_v]) : -INFINITY;
  }
  // What was read beyond the whole pieces is -Inf from here on.
  __device__ __forceinline__ void mask() {
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      if ((i + 1) * BLOCK <= whole) continue;  // the whole workgroup
      constexpr uint32_t none = sizeof(T) == 4 ? 0xFF800000u : __is_same(T, f16) ? 0xFC00FC00u : 0xFF80FF80u;
      if (i * BLOCK + (int)threadIdx.x >= whole) raw[i] = u32x4{none, none, none, none};
    }
  }
};

// Largest logit of a thread's pieces over its wave. 16-bit logits that are not
// negative order as their bits do, two to an instruction, so only where a wave
// has none of those are the values compared.
template <typename T, int N>
__device__ __forceinline__ float largest_of(u32x4 (&raw)[N], float single) {
  if constexpr (sizeof(T) == 2) {
    typedef short s2 __attribute__((ext_vector_type(2)));
    s2 m = {INT16_MIN, INT16_MIN};
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t two = raw[i][k];
        m = __builtin_elementwise_max(m, __builtin_bit_cast(s2, two));
      }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1)
      m = __builtin_elementwise_max(m, __builtin_bit_cast(s2, __shfl_xor(__builtin_bit_cast(int, m), off, 64)));
    const short most = m.x > m.y ? m.x : m.y;
    if (most >= 0) return wave_max(__builtin_fmaxf(single, to_f32(__builtin_bit_cast(T, most))));
  }
  float m = single;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float f[kPer<T>];
    again(raw[i]);
    values<T>(raw[i], f);
#pragma unroll
    for (int k = 0; k < kPer<T>; ++k) m = __builtin_fmaxf(m, f[k]);
  }
  return wave_max(m);
}

template <typename T, int BLOCK, int NCH>
__device__ __forceinline__ Soft wave_softmax(Held<T, BLOCK, NCH>& held, float scale) {
  held.mask();
  const float largest = largest_of<T, NCH>(held.raw, held.single), base = largest == -INFINITY ? 0.0f : largest;
  float sum = __builtin_amdgcn_exp2f((held.single - base) * scale);
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    float f[kPer<T>];
    again(held.raw[i]);
    values<T>(held.raw[i], f);
    sum += sum_exp<kPer<T>>(f, base, scale);
  }
  return {largest, wave_sum(sum)};
}

enum { kPolicy = 0, kFewClasses = 1, kManyClasses = 2 };  // up to 64 classes: one to a lane of the first wave
enum { kOwnSums = 0, kGivenSums = 1, kPartSums = 2 };

// Where rows are cut into parts: what the first launch leaves to the second.
struct Parts {
  int count;
  Soft* soft;  // [rows][count]
  float* z;    // [rows][top]: the logits at the entries' classes, which the second launch may overwrite
};

// Whether the row takes part, and (kPolicy, kFewClasses) this lane's class in
// *id, -1 if it has none. Every wave looks for itself, so that no logit of a
// row that is left out is read.
template <int KIND>
__device__ __forceinline__ bool row_is_live(const msamp_vocab_loss& a, int64_t row, int lane, int64_t* id, float* t) {
  *id = -1;
  *t = -INFINITY;
  if constexpr (KIND == kPolicy) {
    const int64_t act = load_int(a.ids, a.id_bytes, row);
    const bool live = act >= 0 && act < a.vocab;
    if (live) *id = act;
    return live;
  } else if constexpr (KIND == kFewClasses) {
    if (lane < a.top) {
      *id = load_int(a.ids, a.id_bytes, row * a.ld_ids + lane);
      *t = teacher_at(a, row, lane);
    }
    if (*id < 0 || *id >= a.vocab || *t == -INFINITY) *id = -1, *t = -INFINITY;
    return __ballot(*id >= 0) != 0;
  } else {
    bool any = false;
    for (int j = lane; j < a.top; j += 64) {
      const int64_t i = load_int(a.ids, a.id_bytes, row * a.ld_ids + j);
      any |= i >= 0 && i < a.vocab && teacher_at(a, row, j) != -INFINITY;
    }
    return __ballot(any) != 0;
  }
}

// A row's entries in LDS (kManyClasses): classes (-1: none), the teacher's
// exponentials, and what the gradient is there.
struct Entries {
  int32_t* id;
  float* e;
  float* at;
};

// One workgroup of BLOCK threads to a row, or to a part of one, of which each
// thread holds NCH pieces in registers from the sums to the gradient, so that
// the row is read once. NCH 0: rows of any length.
//
// Bound by memory: 8,192 x 32,000 bfloat16 logits with their gradient, 1.05 GB,
// take 185 us (5.7 TB/s), 4,096 x 50,257 147 us, the gradient alone of 500 x
// 131,072 binary32 97 us (5.4 TB/s); three passes over the row in memory took
// 366 us for the first. The arithmetic, two exponentials and about ten other
// operations a logit, is 60% of the vector units' time at that rate, so several
// rows have to be in different stages on a compute unit: that takes few
// registers (70 for 32,000 16-bit logits, three workgroups a compute unit), for
// which there is no loop over rows (its constants would stay in registers: 112)
// and the logits are unpacked again in each pass (145). Rows that start
// anywhere are cut at their first 16 bytes (4,096 x 50,257: 178 us from the
// row's start). Logits and gradient bypass the caches (without that on the
// loads 200 us). The first wave alone has the entries; what it needs of memory
// is under way before the row is.
template <typename T, int KIND, int FROM, int BLOCK, int NCH>
__global__ __launch_bounds__(BLOCK) void k_loss(LossArgs l, Parts parts) {
  constexpr int kWaves = BLOCK / 64;
  constexpr int64_t kStep = BLOCK * kPer<T>;
  extern __shared__ char lds[];
  __shared__ Soft soft[kWaves];
  __shared__ float part_of_loss[kWaves];
  __shared__ float factor, teacher[2];
  const msamp_vocab_loss& a = l.a;
  const int top = KIND == kPolicy ? 1 : (int)a.top;
  const Entries e = {(int32_t*)lds, (float*)lds + top, (float*)lds + 2 * top};
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const float scale = l.scale;
  const bool first = FROM != kGivenSums && blockIdx.y == 0;  // writes the loss
  const int64_t row = l.row0 + blockIdx.x;
  const T* z = (const T*)a.logits + row * a.ld_logits;
  T* dz = (T*)a.dlogits + row * a.ld_dlogits;
  Held<T, BLOCK, (NCH > 0 ? NCH : 1)> held;
  held.cut(z, NCH > 0 ? blockIdx.y : 0, a.vocab);
  if (NCH == 0) held.lo = 0, held.hi = a.vocab;
  int64_t id;
  float t;
  bool live = row_is_live<KIND>(a, row, lane, &id, &t);
  Soft s = {0.0f, 0.0f};
  float zc = 0.0f, old = 0.0f, adv = 0.0f, ref = 0.0f, dloss = 1.0f;
  if (live) {
    if (wave == 0) {
      if (KIND != kManyClasses && id >= 0)
        zc = FROM == kPartSums ? parts.z[row * top + (KIND == kPolicy ? 0 : lane)] : to_f32(((const GLOBAL T*)z)[id]);
      if (KIND == kPolicy) {
        old = a.old_logp[row];
        adv = a.advantages[row];
        if (l.kl != 0.0) ref = a.ref_logp[row];
      }
    }
    if (a.dlogits != nullptr && a.dloss != nullptr) dloss = a.dloss[row];
    if constexpr (FROM == kGivenSums) s = {a.stats[2 * row], a.stats[2 * row + 1]};
    if constexpr (NCH > 0) {
      if (FROM == kOwnSums || a.dlogits != nullptr) held.template load<kPastCaches>(z);
    }
  }
  // the teacher's softmax: its exponentials, and their sum over the entries of one's own class
  float teacher_log = 0.0f, teacher_inv = 0.0f, own = 0.0f, mine = 0.0f;
  if (KIND == kFewClasses && live && wave == 0) {
    const float most = wave_max(t != t ? INFINITY : t);  // NaN as Inf: Inf - Inf makes the row's results NaN
    t = (t - most) * l.inv_tau;
    own = id >= 0 ? __expf(t) : 0.0f;
    const float sum = wave_sum(own);
    teacher_log = logf(sum);
    teacher_inv = 1.0f / sum;
    for (int k = 0; k < top; ++k) {  // in the entries' order: the same sum for each entry of a class
      const int other = __builtin_amdgcn_readlane((int)id, k);
      const float p = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(own), k));
      mine += (int)id == other ? p : 0.0f;
    }
  }
  if (KIND == kManyClasses && live && wave == 0) {
    float most = -INFINITY, sum = 0.0f;
    for (int j = lane; j < top; j += 64) {
      const int64_t i = load_int(a.ids, a.id_bytes, row * a.ld_ids + j);
      float u = teacher_at(a, row, j);
      if (i < 0 || i >= a.vocab) u = -INFINITY;
      e.id[j] = u == -INFINITY ? -1 : (int32_t)i;
      e.at[j] = u;
      most = __builtin_fmaxf(most, u != u ? INFINITY : u);
    }
    most = wave_max(most);
    for (int j = lane; j < top; j += 64) {
      const float u = (e.at[j] - most) * l.inv_tau, x = e.id[j] < 0 ? 0.0f : __expf(u);
      e.at[j] = u;
      e.e[j] = x;
      sum += x;
    }
    sum = wave_sum(sum);
    if (lane == 0) teacher[0] = logf(sum), teacher[1] = 1.0f / sum;
  }
  if constexpr (FROM == kOwnSums) {
    if (live) {
      if constexpr (NCH > 0) {
        s = wave_softmax<T, BLOCK, NCH>(held, scale);
      }
      if (kWaves > 1) {
        if (lane == 0) soft[wave] = s;
        __syncthreads();
        s = soft[0];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) s.largest = __builtin_fmaxf(s.largest, soft[w].largest);
        const float base = s.largest == -INFINITY ? 0.0f : s.largest;
        s.sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
          s.sum += soft[w].sum * __builtin_amdgcn_exp2f((soft[w].largest - base) * scale);
      }
    }
  }
  if constexpr (FROM == kPartSums) {
    if (live) {
      s = parts.soft[row * parts.count];
      for (int k = 1; k < parts.count; ++k) s = join(s, parts.soft[row * parts.count + k], scale);
    }
  }
  if (KIND == kManyClasses && (FROM != kOwnSums || kWaves == 1)) __syncthreads();  // the entries are in LDS
  if (first && a.stats != nullptr && threadIdx.x == 0) {
    a.stats[2 * row] = s.largest;
    a.stats[2 * row + 1] = s.sum;
  }
  if (live && s.largest == -INFINITY && s.sum == 0.0f) live = false;
  if (!live) {
    if (first && threadIdx.x == 0) {
      a.loss[row] = 0.0f;
      if (KIND == kPolicy && a.logp != nullptr) a.logp[row] = 0.0f;
    }
    if (a.dlogits != nullptr) {
      const float zero[8] = {};
      for (int64_t v = held.lo + threadIdx.x * 8; v < held.hi; v += BLOCK * 8)
        store8<T, true>(dz + v, (int)(held.hi - v < 8 ? held.hi - v : 8), zero);
    }
    return;
  }
  // the loss, the gradient at the entries' classes ('at'), and its factor elsewhere
  const float inv = 1.0f / s.sum;
  float c = 0.0f, at = 0.0f;
  if constexpr (KIND == kPolicy) {
    if (wave == 0) {
      // binary64 from the row's binary32 sum on: one lane's work, while near the reference policy e^d - d - 1 is d^2 / 2
      // and would keep no digits of binary32
      const double lp = ((double)zc - (double)s.largest) * l.inv_tau64 - log((double)s.sum);
      const double d = lp - (double)old, r = exp(d);
      const bool over = adv > 0.0f && d > l.log_high, under = adv < 0.0f && d < l.log_low;
      const double away = l.kl != 0.0 ? (double)ref - lp : 0.0, more = expm1(away);
      if (first && lane == 0) {
        const double won = adv == 0.0f ? 0.0 : (over ? l.high : under ? l.low : r) * (double)adv;
        const double apart = away == INFINITY ? away : more - away;  // the reference allows what the mask does not
        a.loss[row] = (float)(l.kl * apart - won);
        if (a.logp != nullptr) a.logp[row] = (float)lp;
      }
      const double g = -l.kl * more - (over || under || adv == 0.0f ? 0.0 : r * (double)adv);
      c = (float)(-(double)dloss * g * l.inv_tau64);
      if (kWaves > 1 && lane == 0) factor = c;
      at = (__builtin_amdgcn_exp2f((zc - s.largest) * scale) * inv - 1.0f) * c;
      if (kWaves > 1 && lane == 0) part_of_loss[0] = at;
    }
    if (a.dlogits != nullptr && kWaves > 1) {
      __syncthreads();
      c = factor;
      at = part_of_loss[0];
    }
  } else {
    const float tau = (float)a.temperature, log_sum = logf(s.sum);
    c = dloss * tau;
    if constexpr (KIND == kFewClasses) {
      if (wave == 0) {
        const float zv = zc - s.largest, p = own * teacher_inv;
        float loss = p != 0.0f ? p * ((t - teacher_log) - (zv * l.inv_tau - log_sum)) : 0.0f;
        loss = wave_sum(loss);
        if (first && lane == 0) a.loss[row] = tau * (tau * loss);
        at = (__builtin_amdgcn_exp2f(zv * scale) * inv - mine * teacher_inv) * c;
      }
      // these logits are read before the gradient, which may go over them, is written (the barrier of the sums does
      // where they are formed here, and parts have them from the first launch)
      if (FROM == kGivenSums && kWaves > 1) __syncthreads();
    } else {
      const float log_teacher = teacher[0], inv_teacher = teacher[1];
      float loss = 0.0f;
      for (int j = threadIdx.x; j < top; j += BLOCK) {
        const int32_t i = e.id[j];
        if (i < 0) continue;
        const float zv = (FROM == kPartSums ? parts.z[row * top + j] : to_f32(((const GLOBAL T*)z)[i])) - s.largest;
        const float p = e.e[j] * inv_teacher;
        if (p != 0.0f) loss += p * ((e.at[j] - log_teacher) - (zv * l.inv_tau - log_sum));
        float sum = 0.0f;
        for (int k = 0; k < top; ++k) sum += e.id[k] == i ? e.e[k] : 0.0f;
        e.at[j] = (__builtin_amdgcn_exp2f(zv * scale) * inv - sum * inv_teacher) * c;
      }
      loss = wave_sum(loss);
      if (lane == 0) part_of_loss[wave] = loss;
      __syncthreads();  // and the classes' logits are read before the gradient is written
      if (first && threadIdx.x == 0) {
        loss = part_of_loss[0];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) loss += part_of_loss[w];
        a.loss[row] = tau * (tau * loss);
      }
    }
  }
  if (a.dlogits != nullptr) {
    const float k = c * inv;
    constexpr int N = kPer<T>;
    auto gradient = [&](int64_t v, u32x4 r) {
      float f[N];
      values<T>(r, f);
#pragma unroll
      for (int j = 0; j < N; ++j) f[j] = __builtin_amdgcn_exp2f((f[j] - s.largest) * scale) * k;
      if (KIND == kPolicy && id >= v && id < v + N) {  // the action is in this piece
#pragma unroll
        for (int j = 0; j < N; ++j) f[j] = id == v + j ? at : f[j];
      }
      return rounded<T>(f);
    };
    auto single = [&](int64_t v, float zv) {
      const float g = __builtin_amdgcn_exp2f((zv - s.largest) * scale) * k;
      dz[v] = from_f32<T>(KIND == kPolicy && v == id ? at : g);
    };
    if constexpr (NCH > 0) {
      const auto db = row_buffer(dz + held.start, (int64_t)held.whole * 16);
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
        again(held.raw[i]);
        __builtin_amdgcn_raw_buffer_store_b128(gradient(held.start + i * kStep + threadIdx.x * N, held.raw[i]), db, held.at(i), 0,
                                               kPastCaches);
      }
      if (held.single_v >= 0) single(held.single_v, held.single);
    } else {
      const int64_t whole = a.vocab / N * N;
      for (int64_t v = threadIdx.x * N; v < whole; v += kStep)
        *(GLOBAL u32x4_any*)(dz + v) = gradient(v, *(const GLOBAL u32x4_any*)(z + v));
      if (whole + threadIdx.x < a.vocab) single(whole + threadIdx.x, to_f32(((const GLOBAL T*)z)[whole + threadIdx.x]));
    }
    if (KIND != kPolicy) {
      __syncthreads();  // the classes' values go over the others'
      if (KIND == kFewClasses) {
        if (wave == 0 && id >= held.lo && id < held.hi) dz[id] = from_f32<T>(at);
      } else {
        for (int j = threadIdx.x; j < top; j += BLOCK)
          if (e.id[j] >= held.lo && e.id[j] < held.hi) dz[e.id[j]] = from_f32<T>(e.at[j]);
      }
    }
  }
}

// The sums of a row's parts, and the logits at its entries' classes.
template <typename T, int KIND, int BLOCK, int NCH>
__global__ __launch_bounds__(BLOCK) void k_parts(LossArgs l, Parts parts) {
  constexpr int kWaves = BLOCK / 64;
  __shared__ Soft soft[kWaves];
  const msamp_vocab_loss& a = l.a;
  const int top = KIND == kPolicy ? 1 : (int)a.top;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const float scale = l.scale;
  const int64_t row = l.row0 + blockIdx.x;
  const T* z = (const T*)a.logits + row * a.ld_logits;
  Held<T, BLOCK, NCH> held;
  held.cut(z, blockIdx.y, a.vocab);
  int64_t id;
  float t;
  if (!row_is_live<KIND>(a, row, lane, &id, &t)) return;  // the whole workgroup
  held.template load<0>(z);  // read again by the second launch
  if (blockIdx.y == 0) {
    for (int j = threadIdx.x; j < top; j += BLOCK) {
      const int64_t i = load_int(a.ids, a.id_bytes, KIND == kPolicy ? row : row * a.ld_ids + j);
      if (i >= 0 && i < a.vocab) parts.z[row * top + j] = to_f32(((const GLOBAL T*)z)[i]);
    }
  }
  Soft s = wave_softmax<T, BLOCK, NCH>(held, scale);
  if (lane == 0) soft[wave] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kWaves; ++w) s = join(s, soft[w], scale);
    parts.soft[row * parts.count + blockIdx.y] = s;
  }
}

LossArgs loss_args(const msamp_vocab_loss& a) {
  LossArgs l;
  l.a = a;
  l.row0 = 0;
  l.inv_tau = (float)(1.0 / a.temperature);
  l.scale = (float)(kLog2e / a.temperature);
  l.inv_tau64 = 1.0 / a.temperature;
  l.log_low = std::log(1.0 - a.clip_low);
  l.log_high = std::log1p(a.clip_high);
  l.low = 1.0 - a.clip_low;
  l.high = 1.0 + a.clip_high;
  l.kl = (float)a.kl != 0.0f ? a.kl : 0.0;  // as the check of ref_logp takes it
  return l;
}

// One workgroup to a row (a loop over rows would keep its constants in
// registers), at most 2^20 rows a launch.
template <typename F>
hipError_t each_rows(const LossArgs& l, F&& f) {
  LossArgs part = l;
  for (part.row0 = 0; part.row0 < l.a.rows; part.row0 += 1 << 20) {
    const int64_t left = l.a.rows - part.row0;
    f(part, (unsigned)(left < (1 << 20) ? left : 1 << 20));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename T, int KIND, int FROM, int BLOCK, int NCH>
hipError_t launch(const LossArgs& l, const Parts& parts, int count, hipStream_t s) {
  const size_t lds = KIND == kManyClasses ? 12 * (size_t)l.a.top : 0;
  return each_rows(l, [&](const LossArgs& p, unsigned rows) {
    k_loss<T, KIND, FROM, BLOCK, NCH><<<dim3(rows, (unsigned)count), BLOCK, lds, s>>>(p, parts);
  });
}

// Rows that one workgroup does not hold in registers are cut into parts of
// 32,768 16-bit or 16,384 binary32 logits. Loss and gradient in one call read
// such rows twice: 4,096 x 128,256 bfloat16, 2.1 GB, take 208 + 390 us, 2,048 x
// 50,257 binary32, 823 MB, 75 + 136.
constexpr int kPartBlock = 512, kPartPieces = 8;
int64_t bytes_of(const msamp_vocab_loss& a) { return a.vocab * (a.dtype == MSAMP_F32 ? 4 : 2); }
int64_t parts_of(const msamp_vocab_loss& a) {
  return (bytes_of(a) + kPartBlock * kPartPieces * 16 - 1) / (kPartBlock * kPartPieces * 16);
}
bool in_parts(const msamp_vocab_loss& a) { return bytes_of(a) > 512 * 16 * 16; }

// The smallest workgroup that holds a row in registers. Rows fit where their
// pieces do: those logits behind the last whole piece have a register of their
// own. Each size against the next one, distillation of 2^27 bfloat16 logits with
// their gradient, us: 512 a row 213 and 248, 1,024 132 and 177, 2,048 113 and
// 187 (256 threads of one piece), 4,096 111 and 151, 8,192 91 and 139, 16,384 89
// and 121, 32,768 97 and 106; 13 pieces and 16 at 34,000 108 and 121, at 45,000
// 103 and 107, at 50,257 105 and 108.
template <typename T, int KIND, int FROM>
hipError_t whole(const LossArgs& l, hipStream_t s) {
  const int64_t pieces = (bytes_of(l.a) + 15) / 16;
  const Parts none = {1, nullptr, nullptr};
  if (pieces <= 64) return launch<T, KIND, FROM, 64, 1>(l, none, 1, s);
  if (pieces <= 128) return launch<T, KIND, FROM, 64, 2>(l, none, 1, s);
  if (pieces <= 256) return launch<T, KIND, FROM, 64, 4>(l, none, 1, s);
  if (pieces <= 512) return launch<T, KIND, FROM, 256, 2>(l, none, 1, s);
  if (pieces <= 1024) return launch<T, KIND, FROM, 256, 4>(l, none, 1, s);
  if (pieces <= 2048) return launch<T, KIND, FROM, 512, 4>(l, none, 1, s);
  if (pieces <= 4096) return launch<T, KIND, FROM, 512, 8>(l, none, 1, s);
  if (pieces <= 6656) return launch<T, KIND, FROM, 512, 13>(l, none, 1, s);
  return launch<T, KIND, FROM, 512, 16>(l, none, 1, s);
}

template <typename T, int KIND>
hipError_t forward(const LossArgs& l, void* ws, hipStream_t s) {
  if (!in_parts(l.a)) return whole<T, KIND, kOwnSums>(l, s);
  const int count = (int)parts_of(l.a);
  const Parts parts = {count, (Soft*)ws, (float*)ws + 2 * l.a.rows * count};
  const hipError_t e = each_rows(l, [&](const LossArgs& p, unsigned rows) {
    k_parts<T, KIND, kPartBlock, kPartPieces><<<dim3(rows, (unsigned)count), kPartBlock, 0, s>>>(p, parts);
  });
  if (e != hipSuccess) return e;
  return launch<T, KIND, kPartSums, kPartBlock, kPartPieces>(l, parts, l.a.dlogits != nullptr ? count : 1, s);
}

// Parts read the logits at every class, so in place a long row stays with one
// workgroup, which reads them before it writes: 500 x 131,072 binary32 take 106
// us (96 in parts, the gradient apart), 4,096 x 128,256 bfloat16 418 (393).
template <typename T, int KIND>
hipError_t backward(const LossArgs& l, hipStream_t s) {
  if (!in_parts(l.a)) return whole<T, KIND, kGivenSums>(l, s);
  const Parts none = {1, nullptr, nullptr};
  if (l.a.dlogits == l.a.logits) return launch<T, KIND, kGivenSums, kPartBlock, 0>(l, none, 1, s);
  return launch<T, KIND, kGivenSums, kPartBlock, kPartPieces>(l, none, (int)parts_of(l.a), s);
}

template <typename T>
hipError_t run(const LossArgs& l, bool policy, bool back, void* ws, hipStream_t s) {
  if (policy) return back ? backward<T, kPolicy>(l, s) : forward<T, kPolicy>(l, ws, s);
  if (l.a.top <= 64) return back ? backward<T, kFewClasses>(l, s) : forward<T, kFewClasses>(l, ws, s);
  return back ? backward<T, kManyClasses>(l, s) : forward<T, kManyClasses>(l, ws, s);
}

hipError_t run(const msamp_vocab_loss& a, bool policy, bool back, void* ws, hipStream_t s) {
  const LossArgs l = loss_args(a);
  return a.dtype == MSAMP_F32 ? run<float>(l, policy, back, ws, s)
                              : a.dtype == MSAMP_F16 ? run<f16>(l, policy, back, ws, s) : run<bf16>(l, policy, back, ws, s);
}

}  // namespace

int64_t loss_workspace(bool policy, const msamp_vocab_loss& a) {
  return in_parts(a) ? a.rows * (8 * parts_of(a) + 4 * (policy ? 1 : a.top)) : 0;
}

hipError_t launch_loss_forward(bool policy, const msamp_vocab_loss& a, void* ws, hipStream_t s) {
  return run(a, policy, false, ws, s);
}

hipError_t launch_loss_backward(bool policy, const msamp_vocab_loss& a, hipStream_t s) {
  return run(a, policy, true, nullptr, s);
}

}  // namespace msamp
