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
constexpr int kPastCaches = 2, kThroughCaches = 0;  // nt, or not

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
  static __device__ __forceinline__ raw load(__amdgpu_buffer_rsrc_t b, uint32_t at) {
    return __builtin_bit_cast(raw, __builtin_amdgcn_raw_buffer_load_b64(b, at, 0, 0));
  }
  static __device__ __forceinline__ raw load_one(__amdgpu_buffer_rsrc_t b, uint32_t at) {
    return raw{__builtin_amdgcn_raw_buffer_load_b32(b, at, 0, 0), 0u};
  }
  static __device__ __forceinline__ raw second(raw r) { return raw{r.y, 0u}; }
  template <int CACHES>
  static __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t b, uint32_t at, float2 v) {
    __builtin_amdgcn_raw_buffer_store_b64(u32x2{__float_as_uint(v.x), __float_as_uint(v.y)}, b, at, 0, CACHES);
  }
  static __device__ __forceinline__ void store_one(__amdgpu_buffer_rsrc_t b, uint32_t at, float2 v) {
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v.x), b, at, 0, 0);
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
  static __device__ __forceinline__ raw packed(float2 v) {
    typedef float f2 __attribute__((ext_vector_type(2)));
    typedef T t2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(raw, __builtin_convertvector((f2{v.x, v.y}), t2));
  }
  static __device__ __forceinline__ void store(T* p, int n, float2 v) {
    if (n >= 2) *(GLOBAL u32_any*)p = packed(v);
    else *(GLOBAL T*)p = from_f32<T>(v.x);
  }
  static __device__ __forceinline__ raw load(__amdgpu_buffer_rsrc_t b, uint32_t at) {
    return __builtin_amdgcn_raw_buffer_load_b32(b, at, 0, 0);
  }
  static __device__ __forceinline__ raw load_one(__amdgpu_buffer_rsrc_t b, uint32_t at) {
    return (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(b, at, 0, 0);
  }
  static __device__ __forceinline__ raw second(raw r) { return r >> 16; }
  template <int CACHES>
  static __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t b, uint32_t at, float2 v) {
    __builtin_amdgcn_raw_buffer_store_b32(packed(v), b, at, 0, CACHES);
  }
  static __device__ __forceinline__ void store_one(__amdgpu_buffer_rsrc_t b, uint32_t at, float2 v) {
    __builtin_amdgcn_raw_buffer_store_b16((uint16_t)(packed(v) & 0xFFFFu), b, at, 0, 0);
  }
};

// a = 1 / (1 + e^-g) and keep = 1 - a = 1 / (1 + e^g) from one exponential,
// e^-|g|, so that the smaller of the two keeps its digits. 2^p takes a p rounded
// to binary32, which alone would be off by |g| 2^-24 of itself: what the
// rounding left out of -|g| is put back as a factor 1 + rest. The larger one is
// 1 less the smaller, half a step off, since gradients take products of it over
// all of a channel's memory: with 1 / (1 + e) from v_rcp and without the rest dh0
// of 9,000 bfloat16 steps was off by 1.5e-6 (now 1.8e-7).
__device__ __forceinline__ void gate1(float g, float* a, float* keep) {
  const float x = -__builtin_fabsf(g), p = x * 1.44269504088896341f;
  const float rest = __builtin_fmaxf(__builtin_fmaf(p, -0.693147180559945309f, x), -1.0f);  // -1 where it is Inf - Inf
  const float e0 = __builtin_amdgcn_exp2f(p), e = __builtin_fmaf(e0, rest, e0);
  const float small = e * __builtin_amdgcn_rcpf(1.0f + e), big = 1.0f - small;
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

// ------------------------------------------- tiles: waves side by side in time ---

// A workgroup takes a block of 2 * LANES channels through its span of the
// sequence, 32 * WAVES steps at a time: each wave has a chunk of 32 steps,
// each of its 64 / LANES groups of lanes R consecutive steps of it in
// registers. A run of steps maps the state before it to the state behind it
// by h -> A h + S, so the groups form (A, S) of their steps, join them over
// the wave's lanes and (through LDS, one barrier) over the waves, and only
// then go through their steps with the state they start from. The next tile's
// loads are under way meanwhile.
//
// Bound by memory: 4 x 4,096 steps of 4,096 bfloat16 channels take 91 us
// forward (411 MB, 4.5 TB/s; 72 where the last call left part in the cache) and
// 159 us backward (679 MB, 4.3 TB/s; 135; x, gate and dy are read once, h comes
// from the saved states); a lane that goes through all steps alone takes 2,627 and 5,664 us. A tile's loads have to be under way
// for the whole of the tile before it: nothing in the loop may wait for memory
// (a state loaded before the loop is waited for there, no value goes through
// scratch, the odd channel's block has a loop of its own), and the two channels
// of a 16-bit step share a register until they are used. 16 waves, or 32
// channels to a workgroup and twice the workgroups, were slower (99 us forward).
//
// Where batch and channels alone give too few workgroups, sequences are cut
// into spans: a first launch forms each span's (A, S), and each workgroup of
// the second joins those before its own. 1 x 16,384 x 2,048: 25 + 35 us forward
// and 25 + 56 backward; 256 workgroups, twice as many take 28 + 38 and 25 + 60.
struct Spans {
  int64_t blocks;  // of channels
  int32_t steps;   // of a span, a multiple of the tile's
  int32_t count;
  int32_t run;     // neighbouring blocks on a die
  bool whole;      // every step starts on 128 bytes
  float4* joined;  // [batch][count][pairs]: (A, S) of each span
  float2* first;   // [batch][pairs]: the state before all spans, which the last state may go over
  int64_t pairs;
};

template <typename T>
constexpr int lanes_of() {
  return sizeof(T) == 2 ? 32 : 16;  // 128 bytes of a step
}

struct Affine {  // v -> a v + s
  float2 a, s;
};
__device__ __forceinline__ float2 apply(const Affine& f, float2 v) { return fma2(f.a, v, f.s); }
// f after g
__device__ __forceinline__ Affine after(const Affine& f, const Affine& g) { return {mul2(f.a, g.a), fma2(f.a, g.s, f.s)}; }

__device__ __forceinline__ float2 shuffle2(float2 v, int lane) {
  return make_float2(__shfl(v.x, lane, 64), __shfl(v.y, lane, 64));
}
__device__ __forceinline__ Affine shuffle(const Affine& f, int lane) {
  return {shuffle2(f.a, lane), shuffle2(f.s, lane)};
}

__device__ __forceinline__ float2 pick(bool c, float2 a, float2 b) { return make_float2(c ? a.x : b.x, c ? a.y : b.y); }

// What the groups before (FORWARD: earlier, otherwise later in time) this
// lane's map a state to, in *before; the whole wave's map in the last group
// (FORWARD: the highest) of *all.
template <int LANES, bool FORWARD>
__device__ __forceinline__ void join_groups(int lane, const Affine& mine, Affine* before, Affine* all) {
  Affine sum = mine;
#pragma unroll
  for (int off = LANES; off < 64; off <<= 1) {
    const int from = FORWARD ? lane - off : lane + off;
    const Affine f = shuffle(sum, from & 63), both = after(sum, f);
    const bool in = from >= 0 && from < 64;
    sum.a = pick(in, both.a, sum.a);
    sum.s = pick(in, both.s, sum.s);
  }
  const int from = FORWARD ? lane - LANES : lane + LANES;
  const Affine f = shuffle(sum, from & 63);
  const bool in = from >= 0 && from < 64;
  before->a = pick(in, f.a, make_float2(1.0f, 1.0f));
  before->s = pick(in, f.s, make_float2(0.0f, 0.0f));
  *all = sum;
}

// Place of a workgroup: block of channels, sequence, span.
struct Place {
  int lane, wave, group, n;
  bool odd, none;     // the block has an odd number of channels; there is no block
  bool ends, single;  // this lane has the last of an odd number, behind others; there is one channel
  int64_t b, c, span, len, t0, t1;  // steps [t0, t1) of the span
};
// A tensor's part of one tile, through a buffer whose bounds end behind its
// last step and channel: what lies outside is read as 0 and not written. The
// lane's own offset goes through an empty asm once a tile, so that the compiler
// forms each step's offset with one addition instead of holding all of them in
// registers over the whole loop.
constexpr uint32_t kOutside = 0x80000000u;  // beyond every buffer, also with a tile's steps added
struct Steps {
  int64_t stride;  // elements
  uint32_t lane;   // this lane's byte in a tile
};
__device__ __forceinline__ Steps steps_of(int64_t stride, int64_t step, int64_t c, int n, int size) {
  return {stride, n > 0 ? (uint32_t)((step * stride + c) * size) : kOutside};
}
template <typename T>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const T* p, const Steps& s, int64_t t, int64_t steps,
                                                            int64_t channels) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)(p + t * s.stride), 0,
                                           (int)(((steps - 1) * s.stride + channels) * (int64_t)sizeof(T)), 0x00020000);
}
__device__ __forceinline__ uint32_t once(uint32_t v) {
  asm volatile("" : "+v"(v));
  return v;
}
// Nothing to the hardware; to the compiler another value, which it unpacks
// again where it is used instead of keeping it in twice the registers.
__device__ __forceinline__ uint32_t again(uint32_t v) { return once(v); }
__device__ __forceinline__ u32x2 again(u32x2 v) { return v; }  // nothing is unpacked

// Formed here and not where it is used next, behind what it is formed from.
__device__ __forceinline__ void formed(float2& v) { asm volatile("" : "+v"(v.x), "+v"(v.y)); }

// ODD: the block holds the last of an odd number of channels. Its lane reads
// the pair that ends with it, so that a step is one load for all lanes, and
// writes it alone; a single channel has no pair.
template <typename T, int R, bool ODD>
__device__ __forceinline__ void load_steps(__amdgpu_buffer_rsrc_t b, const Steps& s, const Place& p,
                                           typename Pair<T>::raw* v) {
  const uint32_t row = (uint32_t)(s.stride * (int64_t)sizeof(T));
  const uint32_t at = once(ODD && p.ends ? s.lane - (uint32_t)sizeof(T) : s.lane);
  if (ODD && p.single) {
#pragma unroll
    for (int r = 0; r < R; ++r) v[r] = Pair<T>::load_one(b, at + r * row);
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r) v[r] = Pair<T>::load(b, at + r * row);
  }
}
template <typename T, bool ODD>
__device__ __forceinline__ float2 own(const Place& p, typename Pair<T>::raw v) {
  return Pair<T>::values(ODD && p.ends ? Pair<T>::second(v) : v);
}
template <typename T, int R, bool ODD>
__device__ __forceinline__ void store_steps(__amdgpu_buffer_rsrc_t b, const Steps& s, const Place& p, bool whole,
                                            const float2* v) {
  const uint32_t row = (uint32_t)(s.stride * (int64_t)sizeof(T));
  const uint32_t at = once(ODD && p.n < 2 ? kOutside : s.lane);
  if (whole) {
#pragma unroll
    for (int r = 0; r < R; ++r) Pair<T>::template store<kPastCaches>(b, at + r * row, v[r]);
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r) Pair<T>::template store<kThroughCaches>(b, at + r * row, v[r]);
  }
  if (ODD && p.n == 1) {
    const uint32_t one = once(s.lane);
#pragma unroll
    for (int r = 0; r < R; ++r) Pair<T>::store_one(b, one + r * row, v[r]);
  }
}

template <int LANES>
__device__ __forceinline__ Place place_of(const msamp_recurrence& a, const Spans& sp) {
  Place p;
  p.lane = threadIdx.x & 63;
  p.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  p.group = p.lane / LANES;
  // workgroups go to the 8 dies in turn: neighbouring blocks to one of them, whose cache then has both halves of a
  // line that they share (rows that do not start on 128 bytes)
  const uint32_t run = (uint32_t)sp.run, i = blockIdx.x / (8 * run) * (8 * run) + blockIdx.x % 8 * run + blockIdx.x / 8 % run;
  const uint32_t per = (uint32_t)(sp.blocks * sp.count);
  p.b = i / per;
  p.none = p.b >= a.batch;
  if (p.none) return p;
  const uint32_t rest = i - (uint32_t)p.b * per;
  p.span = rest / (uint32_t)sp.blocks;
  const int64_t block = rest - (uint32_t)p.span * (uint32_t)sp.blocks;
  p.c = (block * LANES + p.lane % LANES) * 2;
  const int64_t left = a.channels - p.c;
  p.n = left <= 0 ? 0 : left == 1 ? 1 : 2;
  p.odd = (a.channels & 1) && block == sp.blocks - 1;
  p.ends = p.n == 1 && p.c > 0;
  p.single = a.channels == 1;
  p.len = __builtin_amdgcn_readfirstlane((int)length_of(a, p.b));
  p.t0 = p.span * sp.steps;
  p.t1 = p.t0 + sp.steps < p.len ? p.t0 + sp.steps : p.len;
  return p;
}

template <typename T, int WAVES>
struct Tile {
  static constexpr int kLanes = lanes_of<T>(), kGroups = 64 / kLanes, kSteps = kChunk / kGroups;
  static constexpr int kTile = kChunk * WAVES, kThreads = 64 * WAVES;
};

// Maps of the steps' (a, b) in time's order.
template <int R>
__device__ __forceinline__ Affine run_of(const float2* av, const float2* bv) {
  Affine f = {av[0], bv[0]};
#pragma unroll
  for (int r = 1; r < R; ++r) f = {mul2(f.a, av[r]), fma2(av[r], f.s, bv[r])};
  return f;
}

// PASS 0: y, states and h_last. PASS 1: the spans' maps alone.
template <typename T, int WAVES, int PASS, bool ODD>
__device__ __forceinline__ void forward_tiles(const msamp_recurrence& a, const Spans& sp, const Place& p,
                                         float4 (&wave_map)[2][WAVES][lanes_of<T>()]) {
  typedef Tile<T, WAVES> K;
  constexpr int R = K::kSteps;
  const T* x = (const T*)a.x + p.b * a.x_batch;
  const T* g = (const T*)a.gate + p.b * a.gate_batch;
  T* y = PASS == 0 ? (T*)a.y + p.b * a.y_batch : nullptr;
  const int mine = p.wave * kChunk + p.group * R;  // this group's steps in a tile
  const Steps sx = steps_of(a.x_time, mine, p.c, p.n, sizeof(T)), sg = steps_of(a.gate_time, mine, p.c, p.n, sizeof(T));
  const Steps sy = steps_of(a.y_time, mine, p.c, p.n, sizeof(T));
  Affine total = {make_float2(1.0f, 1.0f), make_float2(0.0f, 0.0f)};
  float2 h = make_float2(0.0f, 0.0f);
  if (PASS == 0 && p.n > 0) {
    if (a.h0 != nullptr) {
      if (sp.count > 1) h = sp.first[p.b * sp.pairs + p.c / 2];
      else h = Pair<float>::values(Pair<float>::load(a.h0 + p.b * a.ld_h0 + p.c, p.n));
    }
    for (int64_t s = 0; s < p.span; ++s) {
      const float4 f = sp.joined[(p.b * sp.count + s) * sp.pairs + p.c / 2];
      h = fma2(make_float2(f.x, f.y), h, make_float2(f.z, f.w));
    }
  }
  formed(h);  // waited for here: in the loop that would wait for the next tile's loads too
  typename Pair<T>::raw xr[R], gr[R];
  auto steps_at = [&](int64_t t) { return t + K::kTile < p.t1 ? (int64_t)K::kTile : p.t1 - t; };
  auto load = [&](int64_t t) {
    load_steps<T, R, ODD>(buffer_of(g, sg, t, steps_at(t), a.channels), sg, p, gr);
    load_steps<T, R, ODD>(buffer_of(x, sx, t, steps_at(t), a.channels), sx, p, xr);
  };
  if (p.t0 < p.t1) load(p.t0);
  int turn = 0;
  for (int64_t t = p.t0; t < p.t1; t += K::kTile, turn ^= 1) {
    const int64_t at = t + mine;
    typename Pair<T>::raw xc[R], gc[R];
#pragma unroll
    for (int r = 0; r < R; ++r) xc[r] = xr[r], gc[r] = gr[r];
    if (t + K::kTile < p.t1) load(t + K::kTile);
    float2 av[R], bv[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float2 keep;
      gate2(own<T, ODD>(p, gc[r]), &av[r], &keep);
      bv[r] = mul2(keep, own<T, ODD>(p, xc[r]));
    }
    if (t + K::kTile > p.t1) {  // steps behind the end keep the state
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (at + r >= p.t1) av[r] = make_float2(1.0f, 1.0f), bv[r] = make_float2(0.0f, 0.0f);
    }
    Affine before, all;
    join_groups<K::kLanes, true>(p.lane, run_of<R>(av, bv), &before, &all);
    if (WAVES > 1) {
      if (p.group == K::kGroups - 1)
        wave_map[turn][p.wave][p.lane % K::kLanes] = make_float4(all.a.x, all.a.y, all.s.x, all.s.y);
      __syncthreads();
    } else {
      all = shuffle(all, 64 - K::kLanes + p.lane % K::kLanes);
    }
    float2 start = h;
    if (PASS == 1) start = total.s;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      if (WAVES > 1) {
        const float4 f = wave_map[turn][w][p.lane % K::kLanes];
        all = {make_float2(f.x, f.y), make_float2(f.z, f.w)};
      }
      if (PASS == 1) {
        total = after(all, total);
      } else {
        if (w == p.wave) start = h;
        h = apply(all, h);
      }
    }
    if (PASS == 1) continue;
    if (a.states != nullptr && p.group == 0 && p.n > 0 && t + p.wave * kChunk < p.t1)
      Pair<float>::store(a.states + (p.b * ((a.time + kChunk - 1) / kChunk) + t / kChunk + p.wave) * a.channels + p.c, p.n,
                         start);
    float2 v = apply(before, start);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      v = fma2(av[r], v, bv[r]);
      bv[r] = v;
    }
    store_steps<T, R, ODD>(buffer_of(y, sy, t, steps_at(t), a.channels), sy, p, sp.whole, bv);
  }
  if (p.n == 0 || threadIdx.x >= K::kLanes) return;
  if (PASS == 1) {
    sp.joined[(p.b * sp.count + p.span) * sp.pairs + p.c / 2] = make_float4(total.a.x, total.a.y, total.s.x, total.s.y);
    if (p.span == 0 && a.h0 != nullptr)
      sp.first[p.b * sp.pairs + p.c / 2] = Pair<float>::values(Pair<float>::load(a.h0 + p.b * a.ld_h0 + p.c, p.n));
  } else if (a.h_last != nullptr && (p.len == 0 ? p.span == 0 : p.t0 < p.len && p.len <= p.t0 + sp.steps)) {
    Pair<float>::store(a.h_last + p.b * a.ld_h_last + p.c, p.n, h);
  }
}

template <typename T, int WAVES, int PASS>
__global__ __launch_bounds__(64 * WAVES) void k_forward_tile(msamp_recurrence a, Spans sp) {
  __shared__ float4 wave_map[2][WAVES][lanes_of<T>()];
  const Place p = place_of<lanes_of<T>()>(a, sp);
  if (p.none) return;
  if (p.odd) forward_tiles<T, WAVES, PASS, true>(a, sp, p, wave_map);
  else forward_tiles<T, WAVES, PASS, false>(a, sp, p, wave_map);
}

// Backward in time, m_t = a_t l_t = a_t (dy_t + m_{t+1}); h again from the
// state before each wave's chunk. PASS 1: the spans' maps of m alone.
template <typename T, int WAVES, int PASS, bool ODD>
__device__ __forceinline__ void backward_tiles(const msamp_recurrence& a, const Spans& sp, const Place& p,
                                         float4 (&wave_map)[2][WAVES][lanes_of<T>()]) {
  typedef Tile<T, WAVES> K;
  constexpr int R = K::kSteps;
  const T* x = (const T*)a.x + p.b * a.x_batch;
  const T* g = (const T*)a.gate + p.b * a.gate_batch;
  const T* dy = (const T*)a.dy + p.b * a.dy_batch;
  T* dx = (T*)a.dx + p.b * a.dx_batch;
  T* dg = (T*)a.dgate + p.b * a.dgate_batch;
  const float* states = a.states + p.b * ((a.time + kChunk - 1) / kChunk) * a.channels + p.c;
  const int mine = p.wave * kChunk + p.group * R;
  const Steps sx = steps_of(a.x_time, mine, p.c, p.n, sizeof(T)), sg = steps_of(a.gate_time, mine, p.c, p.n, sizeof(T));
  const Steps sd = steps_of(a.dy_time, mine, p.c, p.n, sizeof(T)), ox = steps_of(a.dx_time, mine, p.c, p.n, sizeof(T));
  const Steps og = steps_of(a.dgate_time, mine, p.c, p.n, sizeof(T));
  Affine total = {make_float2(1.0f, 1.0f), make_float2(0.0f, 0.0f)};
  float2 m = make_float2(0.0f, 0.0f);
  if (PASS == 0 && p.n > 0) {
    if (a.dh_last != nullptr) {
      if (sp.count > 1) m = sp.first[p.b * sp.pairs + p.c / 2];
      else m = Pair<float>::values(Pair<float>::load(a.dh_last + p.b * a.ld_dh_last + p.c, p.n));
    }
    const int64_t last = (p.len + sp.steps - 1) / sp.steps - 1;  // the span with the last step
    for (int64_t s = last; s > p.span; --s) {
      const float4 f = sp.joined[(p.b * sp.count + s) * sp.pairs + p.c / 2];
      m = fma2(make_float2(f.x, f.y), m, make_float2(f.z, f.w));
    }
  }
  formed(m);
  typename Pair<T>::raw xr[R], gr[R], dr[R];
  float2 state = make_float2(0.0f, 0.0f);
  auto steps_at = [&](int64_t t) { return t + K::kTile < p.t1 ? (int64_t)K::kTile : p.t1 - t; };
  auto load_state = [&](int64_t t) {
    if (p.n > 0 && t + p.wave * kChunk < p.t1)
      state = Pair<float>::values(Pair<float>::load(states + (t / kChunk + p.wave) * a.channels, p.n));
  };
  const int64_t tiles = p.t0 < p.t1 ? (p.t1 - p.t0 + K::kTile - 1) / K::kTile : 0;
  if (tiles > 0) {
    const int64_t t = p.t0 + (tiles - 1) * K::kTile;
    load_steps<T, R, ODD>(buffer_of(g, sg, t, steps_at(t), a.channels), sg, p, gr);
    if (PASS == 0) {
      load_steps<T, R, ODD>(buffer_of(x, sx, t, steps_at(t), a.channels), sx, p, xr);
      load_state(t);
    }
    load_steps<T, R, ODD>(buffer_of(dy, sd, t, steps_at(t), a.channels), sd, p, dr);
  }
  int turn = 0;
  for (int64_t i = tiles - 1; i >= 0; --i, turn ^= 1) {
    const int64_t t = p.t0 + i * K::kTile, at = t + mine;
    const bool cut = t + K::kTile > p.t1, more = i > 0;  // steps behind the end leave m and h as they are
    float2 av[R], keep[R], slope[R];
    typename Pair<T>::raw gc[R];
#pragma unroll
    for (int r = 0; r < R; ++r) gc[r] = gr[r];
    if (more) load_steps<T, R, ODD>(buffer_of(g, sg, t - K::kTile, K::kTile, a.channels), sg, p, gr);
#pragma unroll
    for (int r = 0; r < R; ++r) gate2(own<T, ODD>(p, gc[r]), &av[r], &keep[r]);
    if (cut) {
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (at + r >= p.t1) av[r] = make_float2(1.0f, 1.0f), keep[r] = make_float2(0.0f, 0.0f);
    }
    if (PASS == 0) {
      // h before each step, and dgate's factor (h - x) a (1 - a)
      Affine f = {av[0], mul2(keep[0], own<T, ODD>(p, xr[0]))}, before, all;
#pragma unroll
      for (int r = 1; r < R; ++r) f = {mul2(f.a, av[r]), fma2(av[r], f.s, mul2(keep[r], own<T, ODD>(p, xr[r])))};
      join_groups<K::kLanes, true>(p.lane, f, &before, &all);
      float2 h = apply(before, state);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float2 xv = own<T, ODD>(p, again(xr[r]));
        slope[r] = mul2(make_float2(h.x - xv.x, h.y - xv.y), mul2(av[r], keep[r]));
        formed(slope[r]);
        h = fma2(av[r], h, mul2(keep[r], xv));
      }
      if (more) {
        load_steps<T, R, ODD>(buffer_of(x, sx, t - K::kTile, K::kTile, a.channels), sx, p, xr);
        load_state(t - K::kTile);
      }
    }
    if (cut) {  // a dy that repeats its steps is within its bounds behind the end too
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (at + r >= p.t1) dr[r] = typename Pair<T>::raw{};
    }
    Affine f = {av[R - 1], mul2(av[R - 1], own<T, ODD>(p, again(dr[R - 1])))}, before, all;
#pragma unroll
    for (int r = R - 2; r >= 0; --r) {
      const float2 d = own<T, ODD>(p, again(dr[r]));
      f = {mul2(f.a, av[r]), mul2(av[r], make_float2(d.x + f.s.x, d.y + f.s.y))};
    }
    join_groups<K::kLanes, false>(p.lane, f, &before, &all);
    if (WAVES > 1) {
      if (p.group == 0) wave_map[turn][p.wave][p.lane] = make_float4(all.a.x, all.a.y, all.s.x, all.s.y);
      __syncthreads();
    } else {
      all = shuffle(all, p.lane % K::kLanes);
    }
    float2 start = m;
#pragma unroll
    for (int w = WAVES - 1; w >= 0; --w) {
      if (WAVES > 1) {
        const float4 q = wave_map[turn][w][p.lane % K::kLanes];
        all = {make_float2(q.x, q.y), make_float2(q.z, q.w)};
      }
      if (PASS == 1) {
        total = after(all, total);
      } else {
        if (w == p.wave) start = m;
        m = apply(all, m);
      }
    }
    if (PASS == 0) {
      float2 v = apply(before, start);
#pragma unroll
      for (int r = R - 1; r >= 0; --r) {
        const float2 d = own<T, ODD>(p, again(dr[r])), l = make_float2(d.x + v.x, d.y + v.y);
        keep[r] = mul2(keep[r], l);
        slope[r] = mul2(slope[r], l);
        v = mul2(av[r], l);
      }
    }
    if (more) load_steps<T, R, ODD>(buffer_of(dy, sd, t - K::kTile, K::kTile, a.channels), sd, p, dr);
    if (PASS == 0) {
      store_steps<T, R, ODD>(buffer_of(dx, ox, t, steps_at(t), a.channels), ox, p, sp.whole, keep);
      store_steps<T, R, ODD>(buffer_of(dg, og, t, steps_at(t), a.channels), og, p, sp.whole, slope);
    }
  }
  if (p.n == 0 || threadIdx.x >= K::kLanes) return;
  if (PASS == 1) {
    sp.joined[(p.b * sp.count + p.span) * sp.pairs + p.c / 2] = make_float4(total.a.x, total.a.y, total.s.x, total.s.y);
    if (p.span == 0 && a.dh_last != nullptr)
      sp.first[p.b * sp.pairs + p.c / 2] =
          Pair<float>::values(Pair<float>::load(a.dh_last + p.b * a.ld_dh_last + p.c, p.n));
  } else if (a.dh0 != nullptr && p.span == 0)
    Pair<float>::store(a.dh0 + p.b * a.ld_dh0 + p.c, p.n, m);
}

template <typename T, int WAVES, int PASS>
__global__ __launch_bounds__(64 * WAVES) void k_backward_tile(msamp_recurrence a, Spans sp) {
  __shared__ float4 wave_map[2][WAVES][lanes_of<T>()];
  const Place p = place_of<lanes_of<T>()>(a, sp);
  if (p.none) return;
  if (p.odd) backward_tiles<T, WAVES, PASS, true>(a, sp, p, wave_map);
  else backward_tiles<T, WAVES, PASS, false>(a, sp, p, wave_map);
}

// Steps up to which a lane goes through them alone (channels 4,096, bfloat16). Forward, 64 sequences of 8 steps: 5.6 us,
// the tiles with 9 8.5; 256 sequences 10 and 27. Backward, 64 of 4 steps 11, of 8 16 as the tiles with 9; 256 of 8 steps
// 70 and 48.
constexpr int64_t kFewForward = 16, kFewBackward = 4;
constexpr int64_t kEnoughGroups = 192;  // workgroups from which sequences are left whole
constexpr int64_t kSpanGroups = 256;    // of sequences that are cut
constexpr int64_t kMostSpans = 64;

// The waves side by side that a sequence fills, up to 8. Measured (4,096 bfloat16 channels, us forward): 64 x 32 steps 11
// with 1 wave, 19 with 2; 64 x 64 21 with 2, 20 with 1, 34 with 4; 32 x 128 21 with 4, 46 with 8; 4 x 256 7.9 with 8, 8.4
// with 4, 17 with 1; 16 x 256 26 with 8, 21 with 4.
// A launch has less than 2^32 threads: 2^22 sequences of up to 64 binary32 channels, two workgroups each, take 4 waves.
int waves_of(const msamp_recurrence& a) {
  const int64_t channels = a.dtype == MSAMP_F32 ? 32 : 64;  // of a workgroup
  if (a.time <= kChunk) return 1;
  if (a.time <= 2 * kChunk) return 2;
  return a.time <= 4 * kChunk || a.batch * ((a.channels + channels - 1) / channels) > (1 << 22) ? 4 : 8;
}

bool whole_lines(const msamp_recurrence& a, bool backward) {
  const int64_t size = a.dtype == MSAMP_F32 ? 4 : 2;
  auto whole = [&](const void* p, int64_t batch, int64_t time) {
    return (((uintptr_t)p | (uintptr_t)(batch * size) | (uintptr_t)(time * size)) & 127) == 0;
  };
  if (!whole(a.x, a.x_batch, a.x_time) || !whole(a.gate, a.gate_batch, a.gate_time)) return false;
  if (!backward) return whole(a.y, a.y_batch, a.y_time);
  return whole(a.dy, a.dy_batch, a.dy_time) && whole(a.dx, a.dx_batch, a.dx_time) &&
         whole(a.dgate, a.dgate_batch, a.dgate_time);
}

Spans spans_of(const msamp_recurrence& a, void* ws, bool backward) {
  Spans s;
  const int64_t lanes = a.dtype == MSAMP_F32 ? lanes_of<float>() : lanes_of<f16>();
  s.pairs = (a.channels + 1) / 2;
  s.blocks = (s.pairs + lanes - 1) / lanes;
  const int64_t tile = kChunk * waves_of(a), tiles = (a.time + tile - 1) / tile;
  const int64_t groups = s.blocks * a.batch;
  int64_t count = groups >= kEnoughGroups ? 1 : (kSpanGroups + groups - 1) / groups;
  if (count > kMostSpans) count = kMostSpans;
  if (count > tiles) count = tiles;
  const int64_t each = (tiles + count - 1) / count;
  s.count = (int32_t)((tiles + each - 1) / each);
  s.steps = (int32_t)(each * tile);
  // (Times here are of gates two operations shorter, 1 to 2% less.)
  // Lines that neighbours share (steps that do not start on 128 bytes): all of a die's workgroups side by side. 2 x
  // 16,411 x 1,000: 40 us forward and 73 backward, in turn 55 and 103. Whole lines: in turn (4 x 4,096 x
  // 4,096: 88 us and 156; four to a die 92 and 164). Outputs go past the caches where lines are whole (there 88 and
  // 156, through them 90 and 159) and through them where the cache can join a line's parts (2 x 16,411 x 999
  // backward: 138 us past them, 127 through).
  const int64_t all = s.blocks * s.count * a.batch;
  s.whole = whole_lines(a, backward);
  s.run = s.whole ? 1 : (int32_t)((all + 7) / 8);
  s.joined = (float4*)ws;
  s.first = (float2*)(s.joined + a.batch * s.count * s.pairs);
  return s;
}

template <typename T, int WAVES, bool BACKWARD>
hipError_t tiles(const msamp_recurrence& a, const Spans& sp, hipStream_t s) {
  const int64_t turn = 8 * sp.run;
  const unsigned grid = (unsigned)((sp.blocks * sp.count * a.batch + turn - 1) / turn * turn);
  if (sp.count > 1) {
    if (BACKWARD) k_backward_tile<T, WAVES, 1><<<grid, 64 * WAVES, 0, s>>>(a, sp);
    else k_forward_tile<T, WAVES, 1><<<grid, 64 * WAVES, 0, s>>>(a, sp);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (BACKWARD) k_backward_tile<T, WAVES, 0><<<grid, 64 * WAVES, 0, s>>>(a, sp);
  else k_forward_tile<T, WAVES, 0><<<grid, 64 * WAVES, 0, s>>>(a, sp);
  return hipGetLastError();
}

// A lane goes through all steps of few, where a tile's steps do not lie within
// the 2^31 bytes of a buffer, and where steps share elements: the bounds of
// such a buffer end inside a pair of a step behind it, which is read as a whole.
bool lane_alone(const msamp_recurrence& a, bool backward) {
  if (a.time <= (backward ? kFewBackward : kFewForward)) return true;
  const int64_t most = ((int64_t)1 << 31) / (a.dtype == MSAMP_F32 ? 4 : 2) - a.channels;
  const int64_t tile = kChunk * waves_of(a);
  auto alone = [&](int64_t stride) { return stride >= most / tile || (stride > 0 && stride < a.channels); };
  if (alone(a.x_time) || alone(a.gate_time)) return true;
  return backward ? alone(a.dy_time) || alone(a.dx_time) || alone(a.dgate_time) : alone(a.y_time);
}

template <typename T, bool BACKWARD>
hipError_t run(const msamp_recurrence& a, void* ws, hipStream_t s) {
  if (lane_alone(a, BACKWARD)) {
    const int64_t pairs = (a.channels + 1) / 2;
    const unsigned grid = (unsigned)((a.batch * pairs + kBlock - 1) / kBlock);
    if (BACKWARD) k_backward_lane<T><<<grid, kBlock, 0, s>>>(a, pairs);
    else k_forward_lane<T><<<grid, kBlock, 0, s>>>(a, pairs);
    return hipGetLastError();
  }
  const Spans sp = spans_of(a, ws, BACKWARD);
  switch (waves_of(a)) {
    case 1: return tiles<T, 1, BACKWARD>(a, sp, s);
    case 2: return tiles<T, 2, BACKWARD>(a, sp, s);
    case 4: return tiles<T, 4, BACKWARD>(a, sp, s);
    default: return tiles<T, 8, BACKWARD>(a, sp, s);
  }
}

}  // namespace

int64_t recurrence_workspace(const msamp_recurrence& a, bool backward) {
  if (a.batch == 0 || a.channels == 0 || lane_alone(a, backward)) return 0;
  const Spans s = spans_of(a, nullptr, backward);
  return s.count > 1 ? a.batch * s.pairs * (s.count * (int64_t)sizeof(float4) + (int64_t)sizeof(float2)) : 0;
}

hipError_t launch_recurrence_forward(const msamp_recurrence& a, void* ws, hipStream_t s) {
  return a.dtype == MSAMP_F32 ? run<float, false>(a, ws, s)
                              : a.dtype == MSAMP_F16 ? run<f16, false>(a, ws, s) : run<bf16, false>(a, ws, s);
}

hipError_t launch_recurrence_backward(const msamp_recurrence& a, void* ws, hipStream_t s) {
  return a.dtype == MSAMP_F32 ? run<float, true>(a, ws, s)
                              : a.dtype == MSAMP_F16 ? run<f16, true>(a, ws, s) : run<bf16, true>(a, ws, s);
}

}  // namespace msamp
