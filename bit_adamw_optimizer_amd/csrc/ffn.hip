// ffn.hip -- the gated feed-forward block on gfx950: gate and up projections,
// activation and product in one kernel, and its backward pass, which forms
// gate and up again from the block's input. The definitions are in msamp.h.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cmath>
#include <iterator>
#include <type_traits>

#include "checkpoint.hpp"
#include "ffn.hpp"

namespace msamp {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef f16 f16x8 __attribute__((ext_vector_type(8)));
typedef bf16 bf16x8 __attribute__((ext_vector_type(8)));

typedef short s16x4 __attribute__((ext_vector_type(4)));

#define LDS __attribute__((address_space(3)))

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

// act(g) and act'(g). The exponential (of the argument times log2 e, which makes
// the result off by about |argument| units in the last place of binary32) and
// the reciprocal (one unit) are the hardware's.
template <int ACT>
__device__ __forceinline__ void act_and_grad(float g, float* a, float* d) {
  if constexpr (ACT == MSAMP_ACT_SILU) {
    const float s = __builtin_amdgcn_rcpf(1.0f + __expf(-g));
    *a = g * s;
    *d = s * __builtin_fmaf(g, 1.0f - s, 1.0f);
  } else if constexpr (ACT == MSAMP_ACT_GELU) {
    // erfc keeps the digits of the left tail, which 1 + erf cancels (none left from -5.5 on)
    const float phi = 0.5f * erfcf(g * -0.70710678118654752f);
    *a = g * phi;
    *d = phi + g * 0.39894228040143268f * __expf(-0.5f * g * g);
  } else {
    // (1 + tanh(z)) / 2 = 1 / (1 + e^(-2z))
    const float g2 = g * g;
    const float z2 = 1.5957691216057308f * __builtin_fmaf(0.044715f * g2, g, g);
    const float s = __builtin_amdgcn_rcpf(1.0f + __expf(-z2));
    *a = g * s;
    // far out, s (1 - s) is 0 and outweighs the slope of z, which may overflow
    const float t = s * (1.0f - s);
    *d = s + (t == 0.0f ? 0.0f : g * t * 1.5957691216057308f * __builtin_fmaf(0.134145f, g2, 1.0f));
  }
}

// f(std::integral_constant of the activation).
template <typename F>
__device__ __forceinline__ void with_act(int act, F&& f) {
  if (act == MSAMP_ACT_SILU) f(std::integral_constant<int, MSAMP_ACT_SILU>());
  else if (act == MSAMP_ACT_GELU) f(std::integral_constant<int, MSAMP_ACT_GELU>());
  else f(std::integral_constant<int, MSAMP_ACT_GELU_TANH>());
}

// -------------------------------------------------------- matrix product ---
//
// out[r, c] = sum_k R(r, k) C(c, k), summed in binary32 by 32x32x16 MFMA.
//
// A workgroup of 8 waves (2 along r, 4 along c) forms a tile of 64 * FR rows
// and 256 columns, 64 k a step. Both operand tiles of the next step travel to
// LDS by buffer loads that write it directly while the current one is
// multiplied (two LDS stages). C is the instruction's left operand and R its
// right one, so that a lane ends with four consecutive columns of one row.
//
// An operand is stored with k along its rows (kAlong: x, the weights and
// [dg | du] as they are read by the products over hidden and inner units) or
// with k across them (kAcross: the same memory in the products over tokens
// and, for the weights, inner units). Either goes to LDS as it lies in memory,
// in pieces of 16 bytes whose order within a row is permuted so that the reads
// of a fragment spread over all banks:
//   kAlong   LDS row = 64 k of one r or c, 8 pieces; piece p of row i at p ^ (i / 2 & 7),
//            so that 16 rows at one k cover the 256 bytes of all banks
//   kAcross  LDS row = all r or c of one k; piece p of row k at p ^ ((k & 3) << 2);
//            read by the transposing LDS load, four k of 16 columns at a time
// Nothing is copied or transposed beforehand unless rows are not 16-byte
// aligned.
//
// Reads past an operand's last row or k return zero (buffer bounds, and a
// comparison in the last step along k), so ragged sizes need no other path.
//
// Bound by the matrix units at the clock that the power limit leaves (about 1.7
// GHz): at 4096 tokens, hidden 4096, 11008 inner units, bf16, the forward
// projections take 645 us (1145 TFLOP/s; instructions in the matrix units 62%
// of the time), those of the backward pass 684 us (55%), both gradients 1273 us
// (1160 TFLOP/s, 61%); LDS bank conflicts 1% to 3% of the LDS cycles. In a row
// of launches under the profiler the forward projections slow down to 803 us
// when the power limit acts and end at 710; passes with other work between them
// took 608 to 645 us. With
// zeros for operands the same code runs 15% faster. One workgroup of 8 waves a
// compute unit holds 128 KB of LDS; 128 x 128 tiles on 4 waves, 32 k in four
// stages, two such workgroups, and two groups of waves half a step apart were
// slower or equal.

enum Mode { kForward, kRecompute, kDx, kDw };
// Modes whose tile is a pair, gate and up of the same 128 inner units.
constexpr bool is_pair(int mode) { return mode == kForward || mode == kRecompute; }

struct Product {
  int64_t R, C, K;  // output rows and columns (inner units for kForward, kRecompute), sum length of a pass
  const void *r0, *r1;  // r1: left operand of the second pass (kDx), the up half (kDw)
  int64_t ldr;
  const void *c0, *c1;  // c1: up weights
  int64_t ldc0, ldc1;
  uint32_t tiles_r, tiles_c;
  // The sum over k in 'splits' parts of 'part' steps each: their sums go to
  // 'partial', one unit after another, and are joined by a second launch.
  uint32_t splits;
  int64_t part;
  float* partial;
  int act;
  void *out0, *out1;  // h or dx; dw_gate and dw_up
  int64_t ldo0, ldo1;
  bool out_f32;
  int accumulate;
  const void* dh;
  int64_t lddh;
  void* dgu;  // [R, 2 * half] of dg | du (kRecompute)
  int64_t half;
};

constexpr int kThreads = 512;
constexpr int kStepK = 64;
constexpr int kTileC = 256;

// Operands hold whole pieces of 8 elements: rows that do not end on one are
// padded with zeros (lay_out, kRecompute's dg | du).
__device__ __forceinline__ int64_t round8(int64_t n) { return (n + 7) & ~(int64_t)7; }

// Descriptor of a buffer of 'bytes' bytes (raw, bounds-checked).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* p, int64_t bytes) {
  const int64_t b = bytes < 0 ? 0 : (bytes > 0x7FFFFFFF ? 0x7FFFFFFF : bytes);
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)b, 0x00020000);
}

__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t r, LDS char* lds, int voffset, int soffset) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (LDS void*)lds, 16, voffset, soffset, 0, 0);
}

constexpr int kOutside = 0x7FFFFFF0;  // beyond every buffer

// One operand tile of ROWS = 64 * FR rows (r or c), k along: its loads to LDS.
template <int FR>
struct Along {
  int voff[FR];
  int piece;  // first k of this lane's piece
  __device__ __forceinline__ void init(int wave, int lane, int64_t ld) {
    piece = ((lane & 7) ^ (((wave & 1) << 2) | (lane >> 4))) * 8;
#pragma unroll
    for (int j = 0; j < FR; ++j) voff[j] = (int)((64 * j + 8 * wave + (lane >> 3)) * ld * 2) + piece * 2;
  }
  // k0: first k of the step; left: k that remain from there (0: none, all
  // zeros). The scalar offset stays within the buffer, whose bounds are
  // compared with it subtracted.
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, LDS char* lds, int wave, int j, int64_t k0,
                                       int64_t left) const {
    const int v = piece < left ? voff[j] : kOutside;
    load_to_lds(r, lds + (64 * j + 8 * wave) * 128, v, left > 0 ? (int)(k0 * 2) : 0);
  }
};

// One operand tile of 64 * FR columns, k across.
template <int FR>
struct Across {
  static constexpr int kPieces = 8 * FR;         // of an LDS row
  static constexpr int kRows = 64 / kPieces;     // k rows of one load
  static constexpr int kSpread = FR == 1 ? 1 : 3;
  int voff[FR];
  __device__ __forceinline__ void init(int wave, int lane, int64_t ld) {
#pragma unroll
    for (int j = 0; j < FR; ++j) {
      const int k = (wave + 8 * j) * kRows + lane / kPieces;
      voff[j] = (int)(k * ld * 2) + ((lane % kPieces) ^ ((k & kSpread) << 2)) * 16;
    }
  }
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, LDS char* lds, int wave, int j) const {
    load_to_lds(r, lds + (wave + 8 * j) * 1024, voff[j], 0);
  }
};

template <typename T>
__device__ __forceinline__ typename Frag<T>::type along_frag(const LDS char* lds, int block, int kk, int lane) {
  const int off = (lane & 31) * 128 + (((kk * 2 + (lane >> 5)) ^ ((lane >> 1) & 7)) * 16);
  return *(const LDS typename Frag<T>::type*)(lds + block * 32 * 128 + off);
}

template <typename T, int FR>
__device__ __forceinline__ typename Frag<T>::type across_frag(const LDS char* lds, int block, int kk, int lane) {
  const int s = lane & 15, q = (s >> 2) & Across<FR>::kSpread;
  const int off = ((lane >> 5) * 8 + (s >> 2)) * (FR * 128) + ((block ^ q) * 64) + ((lane >> 4) & 1) * 32 + (s & 3) * 8;
  const LDS char* p = lds + kk * 16 * (FR * 128) + off;
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS s16x4*)p);
  const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS s16x4*)(p + 4 * (FR * 128)));
  return __builtin_bit_cast(typename Frag<T>::type, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// Where a workgroup's tile lies: unit 'id' of 'n'. Workgroups go to the 8 XCDs
// in turn; each XCD gets a contiguous run of units, in blocks of 8 tiles along
// r, so that the 32 tiles it works on at a time share 8 row tiles and 4 column
// tiles in its L2.
struct Place {
  uint32_t tr, tc, part, z, unit;
};
__device__ __forceinline__ Place place_of(const Product& p, uint32_t id, uint32_t n) {
  Place q;
  const uint32_t tiles = p.tiles_r * p.tiles_c;
  const uint32_t xcd = id & 7, i = id >> 3, full = n >> 3, rest = n & 7;
  q.unit = xcd * full + (xcd < rest ? xcd : rest) + i;
  const uint32_t zs = q.unit / tiles, t = q.unit - zs * tiles;
  q.z = zs / p.splits;
  q.part = zs - q.z * p.splits;
  const uint32_t per = 8 * p.tiles_c;
  const uint32_t g = t / per, in = t - g * per;
  const uint32_t rows = p.tiles_r - g * 8 < 8 ? p.tiles_r - g * 8 : 8;
  q.tc = in / rows;
  q.tr = g * 8 + (in - q.tc * rows);
  return q;
}

// The accumulators of a wave: FR blocks of 32 rows by 2 blocks of 32 columns
// (kForward, kRecompute: gate and up of the same 32 inner units).
template <int FR>
struct Acc {
  f32x16 v[FR][2];
};

// The loads of step 'next' into the stage wr; zeros from step 'end' on. Those
// of operands with k along (the projections) have no branch, so that they are
// spread between matrix instructions. The bounds of one with k across (both
// gradients) compile to a uniform branch, at which scheduling ends.
template <typename T, int MODE, int FR>
__device__ __forceinline__ void load_step(const Product& p, LDS char* wr, const Along<FR>& ra, const Across<FR>& rx,
                                          const Along<4>& ca, const Across<4>& cx, const Across<4>& cy, int64_t row0,
                                          int64_t col0, int z, int wave, int64_t next, int64_t steps1, int64_t end) {
  const bool second = MODE == kDx && next >= steps1;
  const int64_t k0 = (second ? next - steps1 : next) * kStepK;
  const int64_t left = next < end ? p.K - k0 : 0;
  const int64_t ks = left < kStepK ? left : kStepK;
  if constexpr (MODE == kDw) {
    const T* r = (const T*)(z == 0 ? p.r0 : p.r1) + k0 * p.ldr + row0;
    const auto b = buffer_of(r, ks <= 0 ? 0 : ((ks - 1) * p.ldr + round8(p.R) - row0) * 2);
#pragma unroll
    for (int j = 0; j < FR; ++j) rx.load(b, wr, wave, j);
  } else {
    const T* r = (const T*)(second ? p.r1 : p.r0) + row0 * p.ldr;
    const int64_t rows = p.R - row0 < 64 * FR ? p.R - row0 : 64 * FR;
    const auto b = buffer_of(r, ((rows - 1) * p.ldr + round8(p.K)) * 2);
#pragma unroll
    for (int j = 0; j < FR; ++j) ra.load(b, wr, wave, j, k0, left);
  }
  LDS char* wc = wr + FR * 64 * 128;
  if constexpr (is_pair(MODE)) {
    const int64_t rows = p.C - col0 < 128 ? p.C - col0 : 128;
    const auto bg = buffer_of((const T*)p.c0 + col0 * p.ldc0, ((rows - 1) * p.ldc0 + round8(p.K)) * 2);
    const auto bu = buffer_of((const T*)p.c1 + col0 * p.ldc1, ((rows - 1) * p.ldc1 + round8(p.K)) * 2);
    // LDS rows 0..127 gate, 128..255 up; ca holds the gate's offsets, then the up's
#pragma unroll
    for (int j = 0; j < 4; ++j) ca.load(j < 2 ? bg : bu, wc, wave, j, k0, left);
  } else {
    const int64_t ld = second ? p.ldc1 : p.ldc0;
    const T* c = (const T*)(second ? p.c1 : p.c0) + k0 * ld + col0;
    const auto b = buffer_of(c, ks <= 0 ? 0 : ((ks - 1) * ld + round8(p.C) - col0) * 2);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      load_to_lds(b, wc + (wave + 8 * j) * 1024, MODE == kDx && second ? cy.voff[j] : cx.voff[j], 0);
  }
}

// The operands of 16 k from a stage: blocks of 32 rows and of 32 columns.
template <typename T, int FR>
struct Frags {
  typename Frag<T>::type r[FR], c[2];
};

template <typename T, int MODE, int FR>
__device__ __forceinline__ void read_frags(const LDS char* rd, int wave, int lane, int kk, Frags<T, FR>& f) {
  const LDS char* rc = rd + FR * 64 * 128;
  const int rb = (wave >> 2) * FR, cb = wave & 3;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    if constexpr (is_pair(MODE)) f.c[c] = along_frag<T>(rc, cb + 4 * c, kk, lane);
    else f.c[c] = across_frag<T, 4>(rc, cb * 2 + c, kk, lane);
  }
#pragma unroll
  for (int r = 0; r < FR; ++r) {
    if constexpr (MODE == kDw) f.r[r] = across_frag<T, FR>(rd, rb + r, kk, lane);
    else f.r[r] = along_frag<T>(rd, rb + r, kk, lane);
  }
}

template <typename T, int FR>
__device__ __forceinline__ void multiply(const Frags<T, FR>& f, Acc<FR>& acc) {
#pragma unroll
  for (int r = 0; r < FR; ++r)
#pragma unroll
    for (int c = 0; c < 2; ++c) acc.v[r][c] = Frag<T>::mma(f.c[c], f.r[r], acc.v[r][c]);
}

// Spreads a section's LDS reads and loads evenly between its 2 FR matrix
// instructions.
template <int READS, int LOADS, int FR>
__device__ __forceinline__ void interleave() {
  constexpr int kMfma = 0x8, kVmem = 0x10, kDsRead = 0x100, n = 2 * FR;
#pragma unroll
  for (int g = 0; g < n; ++g) {
    __builtin_amdgcn_sched_group_barrier(kMfma, 1, 0);
    if constexpr (READS >= n) __builtin_amdgcn_sched_group_barrier(kDsRead, (READS + n - 1) / n, 0);
    else if (g < READS) __builtin_amdgcn_sched_group_barrier(kDsRead, 1, 0);
    if constexpr (LOADS >= n) __builtin_amdgcn_sched_group_barrier(kVmem, (LOADS + n - 1) / n, 0);
    else if (g < LOADS) __builtin_amdgcn_sched_group_barrier(kVmem, 1, 0);
  }
}

// One step of 64 k: four sections of 16 k, each reading the operands of the
// next section while it multiplies its own. Before the last section all reads
// of this stage have arrived; the barrier there lets the waves write over it
// (the loads of step i + 2, into 'again', the same stage) and, as every wave
// has waited for its own loads of step i + 1, read the other stage 'nx'. So the
// loads have a whole step to arrive. In the projections a wave goes on behind
// the barrier with matrix instructions between its reads and loads; in the
// gradients the branch in load_step keeps 8 to 12 LDS reads, the loads and their
// descriptors before the section's first one.
template <typename T, int MODE, int FR>
__device__ __forceinline__ void step(const Product& p, const LDS char* __restrict__ rd,
                                     const LDS char* __restrict__ nx, LDS char* __restrict__ again,
                                     const Along<FR>& ra, const Across<FR>& rx, const Along<4>& ca,
                                     const Across<4>& cx, const Across<4>& cy, int64_t row0, int64_t col0, int z,
                                     int wave, int lane, int64_t i, int64_t steps1, int64_t end, Frags<T, FR>& f,
                                     Acc<FR>& acc) {
  constexpr int kReads = (is_pair(MODE) ? 2 : 4) + (MODE == kDw ? 2 * FR : FR);
#pragma unroll
  for (int kk = 0; kk < 3; ++kk) {
    Frags<T, FR> next;
    read_frags<T, MODE, FR>(rd, wave, lane, kk + 1, next);
    multiply<T, FR>(f, acc);
    interleave<kReads, 0, FR>();
    f = next;
  }
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
  Frags<T, FR> next;
  read_frags<T, MODE, FR>(nx, wave, lane, 0, next);
  load_step<T, MODE, FR>(p, again, ra, rx, ca, cx, cy, row0, col0, z, wave, i + 2, steps1, end);
  multiply<T, FR>(f, acc);
  interleave<kReads, FR + 4, FR>();
  f = next;
}

// 16-bit tile in LDS on its way out (or dh on its way in): rows of COLS
// columns, pieces of 16 bytes, piece p of row i at p ^ (i & (pieces - 1)).
template <int COLS>
__device__ __forceinline__ int tile_piece(int row, int piece) {
  return row * (COLS * 2) + ((piece ^ (row & (COLS / 8 - 1))) * 16);
}

template <typename T, int COLS, int ROWS>
__device__ __forceinline__ void store_tile(const LDS char* lds, T* out, int64_t ld, int64_t rows, int64_t cols) {
  for (int i = threadIdx.x; i < ROWS * (COLS / 8); i += kThreads) {
    const int row = i / (COLS / 8), piece = i % (COLS / 8);
    if (row < rows && piece * 8 < cols) {
      const u32x4 v = *(const LDS u32x4*)(lds + tile_piece<COLS>(row, piece));
      T* o = out + row * ld + piece * 8;
      if (cols - piece * 8 >= 8) {
        *(GLOBAL u32x4_any*)o = v;
      } else {
        typedef T t8 __attribute__((ext_vector_type(8)));
        const t8 e = __builtin_bit_cast(t8, v);
        for (int k = 0; k < cols - piece * 8; ++k) ((GLOBAL T*)o)[k] = e[k];
      }
    }
  }
}

template <typename T>
__device__ __forceinline__ uint64_t pack4(const float* f) {
  typedef T t4 __attribute__((ext_vector_type(4)));
  t4 v;
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = from_f32<T>(f[k]);
  return __builtin_bit_cast(uint64_t, v);
}

// dh of a tile as it lies in memory, 16 bytes a thread and piece: loaded
// before the sums, so that it is there when they are.
template <typename T, int FR>
struct Incoming {
  u32x4 v[64 * FR * 16 / kThreads];
  __device__ __forceinline__ void load(const Product& p, int64_t row0, int64_t col0) {
#pragma unroll
    for (int k = 0; k < 64 * FR * 16 / kThreads; ++k) {
      const int i = threadIdx.x + k * kThreads, row = i / 16, piece = i % 16;
      const int64_t n = p.C - col0 - piece * 8;
      v[k] = u32x4{0u, 0u, 0u, 0u};
      if (row0 + row < p.R && n > 0) {
        const GLOBAL T* q = (const GLOBAL T*)p.dh + (row0 + row) * p.lddh + col0 + piece * 8;
        if (n >= 8) {
          v[k] = *(const GLOBAL u32x4_any*)q;
        } else {
          typedef T t8 __attribute__((ext_vector_type(8)));
          t8 e = __builtin_bit_cast(t8, v[k]);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j < n) e[j] = q[j];
          v[k] = __builtin_bit_cast(u32x4, e);
        }
      }
    }
  }
  __device__ __forceinline__ void to_lds(LDS char* lds) const {
#pragma unroll
    for (int k = 0; k < 64 * FR * 16 / kThreads; ++k) {
      const int i = threadIdx.x + k * kThreads;
      *(LDS u32x4*)(lds + tile_piece<128>(i / 16, i % 16)) = v[k];
    }
  }
};

// The tile's sums to where they go.
template <typename T, int MODE, int FR>
__device__ __forceinline__ void finish(const Product& p, LDS char* lds, int64_t row0, int64_t col0, int z, int wave,
                                       int lane, const Acc<FR>& acc, const Incoming<T, FR>& dh) {
  constexpr int kRows = 64 * FR;
  const int64_t rows = p.R - row0;
  const int lrow = (wave >> 2) * (32 * FR) + (lane & 31);  // + 32 r
  __syncthreads();  // the stages have been read
  if constexpr (is_pair(MODE)) {
    const int lcol = (wave & 3) * 32;  // + 8 q + 4 (lane / 32) + e
    LDS char* second = lds + kRows * 256;
    const int64_t cols = p.C - col0;
    auto place = [&](int r, int q) { return tile_piece<128>(lrow + 32 * r, (lcol >> 3) + q) + (lane >> 5) * 8; };
    uint64_t du[MODE == kRecompute ? FR : 1][4];
    if constexpr (MODE == kRecompute) {
      dh.to_lds(lds);
      __syncthreads();
    }
    with_act(p.act, [&](auto act) {
#pragma unroll
      for (int r = 0; r < FR; ++r)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float a[4], d[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) act_and_grad<decltype(act)::value>(acc.v[r][0][q * 4 + e], &a[e], &d[e]);
          const int at = place(r, q);
          if constexpr (MODE == kRecompute) {  // dg takes dh's place; dg and du are rounded to T, as MFMA operands
            typedef T t4 __attribute__((ext_vector_type(4)));
            const t4 in = *(const LDS t4*)(lds + at);
            float g[4], u[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              g[e] = to_f32(in[e]) * acc.v[r][1][q * 4 + e] * d[e];
              u[e] = to_f32(in[e]) * a[e];
            }
            *(LDS uint64_t*)(lds + at) = pack4<T>(g);
            du[r][q] = pack4<T>(u);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) a[e] *= acc.v[r][1][q * 4 + e];
          *(LDS uint64_t*)((MODE == kForward ? lds : second) + at) = pack4<T>(a);
        }
    });
    __syncthreads();
    T* out = (T*)p.out0 + row0 * p.ldo0 + col0;
    if constexpr (MODE == kForward) {
      store_tile<T, 128, kRows>(lds, out, p.ldo0, rows, cols);
    } else {
      // columns behind the last inner unit are zero: they are operands of the next products
      T* o = (T*)p.dgu + row0 * (2 * p.half) + col0;
      store_tile<T, 128, kRows>(lds, o, 2 * p.half, rows, p.half - col0);
      if (p.out0 != nullptr) store_tile<T, 128, kRows>(second, out, p.ldo0, rows, cols);
      __syncthreads();
#pragma unroll
      for (int r = 0; r < FR; ++r)
#pragma unroll
        for (int q = 0; q < 4; ++q) *(LDS uint64_t*)(lds + place(r, q)) = du[r][q];
      __syncthreads();
      store_tile<T, 128, kRows>(lds, o + p.half, 2 * p.half, rows, p.half - col0);
    }
  } else {
    void* base = MODE == kDw && z == 1 ? p.out1 : p.out0;
    const int64_t ld = MODE == kDw && z == 1 ? p.ldo1 : p.ldo0;
    const int64_t cols = p.C - col0;
    const int lcol = (wave & 3) * 64 + (lane >> 5) * 4;  // + 32 c + 8 q + e
    if (MODE == kDw && p.out_f32) {
#pragma unroll
      for (int r = 0; r < FR; ++r) {
        const int row = lrow + 32 * r;
        float* o = (float*)base + (row0 + row) * ld + col0;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int col = lcol + 32 * c + 8 * q;
            typedef f32x4 f32x4_any __attribute__((aligned(4)));
            if (row < rows && col + 4 <= cols) {
              f32x4 v;
#pragma unroll
              for (int e = 0; e < 4; ++e) v[e] = acc.v[r][c][q * 4 + e];
              if (p.accumulate) v += *(const GLOBAL f32x4_any*)(o + col);
              *(GLOBAL f32x4_any*)(o + col) = v;
            } else if (row < rows) {
              for (int e = 0; e < 4; ++e)
                if (col + e < cols) {
                  const float v = acc.v[r][c][q * 4 + e];
                  o[col + e] = p.accumulate ? o[col + e] + v : v;
                }
            }
          }
      }
      return;
    }
#pragma unroll
    for (int r = 0; r < FR; ++r)
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = acc.v[r][c][q * 4 + e];
          const int at = tile_piece<256>(lrow + 32 * r, ((lcol + 32 * c) >> 3) + q) + (lane >> 5) * 8;
          *(LDS uint64_t*)(lds + at) = pack4<T>(v);
        }
    __syncthreads();
    store_tile<T, 256, kRows>(lds, (T*)base + row0 * ld + col0, ld, rows, cols);
  }
}

// Bytes of LDS of a workgroup: two stages; they also hold the outgoing tiles.
template <int FR>
constexpr int stage_bytes() {
  return FR * 64 * 128 + kTileC * 128;
}

// Unit 'id' of the 'n' of a product.
template <typename T, int MODE, int FR>
__device__ __forceinline__ void run_unit(const Product& p, LDS char* lds, uint32_t id, uint32_t n) {
  constexpr bool kPair = is_pair(MODE);
  constexpr int kStage = stage_bytes<FR>();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const Place at = place_of(p, id, n);
  const int z = MODE == kDw ? (int)at.z : 0;
  const int64_t row0 = (int64_t)at.tr * (64 * FR), col0 = (int64_t)at.tc * (kPair ? 128 : 256);
  Along<FR> ra;
  Across<FR> rx;
  Along<4> ca;
  Across<4> cx, cy;  // cy: the second pass's
  if constexpr (MODE == kDw) rx.init(wave, lane, p.ldr);
  else ra.init(wave, lane, p.ldr);
  if constexpr (kPair) {
    ca.init(wave, lane, p.ldc0);
    Along<4> up;
    up.init(wave, lane, p.ldc1);
    ca.voff[2] = up.voff[0];
    ca.voff[3] = up.voff[1];
  } else {
    cx.init(wave, lane, p.ldc0);
    if constexpr (MODE == kDx) cy.init(wave, lane, p.ldc1);
  }
  Incoming<T, FR> dh;
  if constexpr (MODE == kRecompute) {
    if (p.splits == 1) dh.load(p, row0, col0);
  }
  Acc<FR> acc;
#pragma unroll
  for (int r = 0; r < FR; ++r) acc.v[r][0] = acc.v[r][1] = f32x16{};
  const int64_t steps1 = (p.K + kStepK - 1) / kStepK;
  const int64_t steps = MODE == kDx ? 2 * steps1 : steps1;
  const int64_t begin = (int64_t)at.part * p.part;
  const int64_t end = steps < begin + p.part ? steps : begin + p.part;
  load_step<T, MODE, FR>(p, lds, ra, rx, ca, cx, cy, row0, col0, z, wave, begin, steps1, end);
  __syncthreads();
  load_step<T, MODE, FR>(p, lds + kStage, ra, rx, ca, cx, cy, row0, col0, z, wave, begin + 1, steps1, end);
  Frags<T, FR> f;
  read_frags<T, MODE, FR>(lds, wave, lane, 0, f);
  for (int64_t i = begin; i < end; ++i) {
    const int cur = (int)((i - begin) & 1) * kStage;
    step<T, MODE, FR>(p, lds + cur, lds + (kStage - cur), lds + cur, ra, rx, ca, cx, cy, row0, col0, z, wave, lane, i,
                      steps1, end, f, acc);
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the last loads to LDS, of zeros, are still under way
  if (p.splits > 1) {
    f32x4* o = (f32x4*)p.partial + (int64_t)at.unit * (64 * FR * kTileC / 4) + wave * (FR * 2 * 4 * 64) + lane;
    const int lrow = (wave >> 2) * (32 * FR) + (lane & 31);
#pragma unroll
    for (int r = 0; r < FR; ++r)
      if (row0 + lrow + 32 * r < p.R) {
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            f32x4 v;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = acc.v[r][c][q * 4 + e];
            o[((r * 2 + c) * 4 + q) * 64] = v;
          }
      }
    return;
  }
  finish<T, MODE, FR>(p, lds, row0, col0, z, wave, lane, acc, dh);
}

// Joins the parts of a split sum, in their order, and finishes the tile: unit
// 'id' of the 'n' tiles.
template <typename T, int MODE, int FR>
__device__ __forceinline__ void join_unit(const Product& p, LDS char* lds, uint32_t id, uint32_t n) {
  constexpr bool kPair = is_pair(MODE);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  Product one = p;
  one.splits = 1;
  const Place at = place_of(one, id, n);
  const int z = MODE == kDw ? (int)at.z : 0;
  const int64_t row0 = (int64_t)at.tr * (64 * FR), col0 = (int64_t)at.tc * (kPair ? 128 : 256);
  const uint32_t tiles = p.tiles_r * p.tiles_c;
  const int64_t tile = at.unit - at.z * tiles;
  Incoming<T, FR> dh;
  if constexpr (MODE == kRecompute) dh.load(p, row0, col0);
  Acc<FR> acc;
#pragma unroll
  for (int r = 0; r < FR; ++r) acc.v[r][0] = acc.v[r][1] = f32x16{};
  const int lrow = (wave >> 2) * (32 * FR) + (lane & 31);
  constexpr int kAhead = FR == 4 ? 2 : 4;  // parts whose loads are under way at a time
  const int64_t size = 64 * FR * kTileC / 4;  // of a unit, in f32x4
  const f32x4* from = (const f32x4*)p.partial + ((int64_t)at.z * p.splits * tiles + tile) * size +
                      wave * (FR * 2 * 4 * 64) + lane;
#pragma unroll
  for (int r = 0; r < FR; ++r)
    if (row0 + lrow + 32 * r < p.R)
      for (uint32_t part = 0; part < p.splits; part += kAhead) {
        f32x4 v[kAhead][8];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
#pragma unroll
          for (int q = 0; q < 8; ++q)
            if (part + k < p.splits) v[k][q] = from[(int64_t)(part + k) * tiles * size + (r * 8 + q) * 64];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
          if (part + k < p.splits) {
#pragma unroll
            for (int q = 0; q < 8; ++q)
#pragma unroll
              for (int e = 0; e < 4; ++e) acc.v[r][q >> 2][(q & 3) * 4 + e] += v[k][q][e];
          }
      }
  finish<T, MODE, FR>(p, lds, row0, col0, z, wave, lane, acc, dh);
}

// Gate and up projections (kForward, kRecompute): tiles of both for the same
// units, so that the activation and the product need no pass of their own.
template <typename T, int MODE, int FR>
__global__ __launch_bounds__(kThreads) void k_projections(Product p) {
  __shared__ __attribute__((aligned(16))) char smem[2 * stage_bytes<FR>()];
  run_unit<T, MODE, FR>(p, (LDS char*)smem, blockIdx.x, gridDim.x);
}

template <typename T, int MODE, int FR>
__global__ __launch_bounds__(kThreads) void k_projections_join(Product p) {
  __shared__ __attribute__((aligned(16))) char smem[64 * FR * 512];
  join_unit<T, MODE, FR>(p, (LDS char*)smem, blockIdx.x, gridDim.x);
}

// dx and the weights' gradients in one launch: nx units of dx first (their sums
// are the longer ones), then those of the weights, which fill the compute units
// that dx leaves.
template <typename T, int FR>
__global__ __launch_bounds__(kThreads) void k_gradients(Product x, Product w, uint32_t nx) {
  __shared__ __attribute__((aligned(16))) char smem[2 * stage_bytes<FR>()];
  if (blockIdx.x < nx) run_unit<T, kDx, FR>(x, (LDS char*)smem, blockIdx.x, nx);
  else run_unit<T, kDw, FR>(w, (LDS char*)smem, blockIdx.x - nx, gridDim.x - nx);
}

// The same for the tiles whose sums were split (none of dx: nx = 0; none of the
// weights: all of the grid is nx).
template <typename T, int FR>
__global__ __launch_bounds__(kThreads) void k_gradients_join(Product x, Product w, uint32_t nx) {
  __shared__ __attribute__((aligned(16))) char smem[64 * FR * 512];
  if (blockIdx.x < nx) join_unit<T, kDx, FR>(x, (LDS char*)smem, blockIdx.x, nx);
  else join_unit<T, kDw, FR>(w, (LDS char*)smem, blockIdx.x - nx, gridDim.x - nx);
}

constexpr int kUnits = 256;  // workgroups that run at a time, one a compute unit
constexpr int64_t kMaxUnits = UINT32_MAX / kThreads;  // of a launch

// How a product is cut: its tiles, and parts of the sum over k.
struct Cut {
  uint32_t tiles_r, tiles_c, splits;
  int64_t part;
  int64_t bytes;  // of partial sums
};

int64_t steps_of(int mode, int64_t K) { return (K + kStepK - 1) / kStepK * (mode == kDx ? 2 : 1); }

// Units (workgroups) of a cut, and tiles.
int64_t tiles_of(int mode, const Cut& c) { return (int64_t)c.tiles_r * c.tiles_c * (mode == kDw ? 2 : 1); }

// The cut with tiles of 64 * fr rows and the sums in 'splits' parts of whole
// steps (false: there is none, or it fills the device more than four times, or
// has more units than a launch).
bool cut_of(int mode, int fr, int64_t splits, int64_t R, int64_t C, int64_t K, Cut* c) {
  const int64_t steps = steps_of(mode, K), tc = is_pair(mode) ? 128 : 256;
  const int64_t part = (steps + splits - 1) / splits;
  if ((steps + part - 1) / part != splits || (splits > 1 && part < 2)) return false;
  *c = {(uint32_t)((R + 64 * fr - 1) / (64 * fr)), (uint32_t)((C + tc - 1) / tc), (uint32_t)splits, part, 0};
  if (splits == 1) return tiles_of(mode, *c) <= kMaxUnits;
  if (tiles_of(mode, *c) > 4 * kUnits / splits) return false;
  c->bytes = tiles_of(mode, *c) * splits * (64 * fr * kTileC * 4);
  return true;
}

// Times in us, fitted to measurements of every cut of 14 problems (tokens 64 to
// 8192, hidden 128 to 8192, 128 to 13824 inner units; on these the cut they
// choose is within 2% of the best one on average, 18% at most).
double unit_us(int fr, const Cut& c) {
  return c.part * (fr == 4 ? 1.8 : (fr == 2 ? 1.05 : 0.8)) + (fr == 4 ? 13.0 : (fr == 2 ? 7.5 : 2.0));
}
// Joining parts: each takes a workgroup so long at least, and all pass twice
// through memory at 8 TB/s.
double join_us(int fr, const Cut& c) {
  if (c.splits == 1) return 0.0;
  const double each = c.splits * (fr == 4 ? 2.0 : (fr == 2 ? 0.6 : 0.25)), all = c.bytes * 2 / 8e6;
  return 3.5 + (each > all ? each : all);
}

// Numbers of parts that are looked at (a plan is made on the host at each
// call, in about a microsecond).
constexpr int kSplits[] = {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64};

struct Candidate {
  Cut cut;
  double units, unit, join;
};

// The cuts with tiles of 64 * fr rows.
int candidates(int mode, int fr, int64_t R, int64_t C, int64_t K, Candidate* out) {
  int n = 0;
  for (int splits : kSplits) {
    Candidate& c = out[n];
    if (!cut_of(mode, fr, splits, R, C, K, &c.cut)) continue;
    c.units = (double)tiles_of(mode, c.cut) * splits;
    c.unit = unit_us(fr, c.cut);
    c.join = join_us(fr, c.cut);
    ++n;
  }
  return n;
}

// The cut of a projection with the least estimated time, and its fr (0: none).
int choose_projection(int mode, int64_t R, int64_t C, int64_t K, Cut* best) {
  double least = 1e30;
  int fr_best = 0;
  Candidate c[std::size(kSplits)];
  for (int fr = 4; fr >= 1; fr /= 2) {
    const int n = candidates(mode, fr, R, C, K, c);
    for (int i = 0; i < n; ++i) {
      const double t = std::ceil(c[i].units / kUnits) * c[i].unit + c[i].join;
      if (t < least) {
        least = t;
        *best = c[i].cut;
        fr_best = fr;
      }
    }
  }
  return fr_best;
}

// The cuts of both gradients, which run side by side with the same fr: the
// time of the longer unit (a quarter more with others after it on the device),
// or of all of them, half a unit of dW, which come last, and 0.15 of the longer
// (fitted to 18 problems: within 5% of the best cut on average, 27% at most).
// 0: none fits a launch.
int choose_gradients(int64_t T, int64_t K, int64_t F, Cut* x, Cut* w) {
  double least = 1e30;
  int fr_best = 0;
  Candidate cx[std::size(kSplits)], cw[std::size(kSplits)];
  for (int fr = 4; fr >= 1; fr /= 2) {
    const int nx = candidates(kDx, fr, T, K, F, cx), nw = candidates(kDw, fr, F, K, T, cw);
    for (int i = 0; i < nx; ++i)
      for (int j = 0; j < nw; ++j) {
        if (cx[i].units + cw[j].units > kMaxUnits) continue;
        double t = cx[i].unit > cw[j].unit ? cx[i].unit : cw[j].unit;
        if (cx[i].units + cw[j].units > kUnits) {
          const double all =
              (cx[i].units * cx[i].unit + cw[j].units * cw[j].unit) / kUnits + 0.5 * cw[j].unit + 0.15 * t;
          t = all > 1.25 * t ? all : 1.25 * t;
        }
        t += cx[i].join > cw[j].join ? cx[i].join : cw[j].join;
        if (t < least) {
          least = t;
          *x = cx[i].cut;
          *w = cw[j].cut;
          fr_best = fr;
        }
      }
  }
  return fr_best;
}

void apply(const Cut& c, float* partial, Product* p) {
  p->tiles_r = c.tiles_r, p->tiles_c = c.tiles_c, p->splits = c.splits, p->part = c.part, p->partial = partial;
}

template <typename T, int MODE, int FR>
hipError_t launch_projections(const Product& p, bool join, hipStream_t s) {
  const uint32_t tiles = p.tiles_r * p.tiles_c;
  if (join) k_projections_join<T, MODE, FR><<<dim3(tiles), dim3(kThreads), 0, s>>>(p);
  else k_projections<T, MODE, FR><<<dim3(tiles * p.splits), dim3(kThreads), 0, s>>>(p);
  return hipGetLastError();
}

template <int MODE>
hipError_t launch_projections(int dtype, int fr, const Product& p, bool join, hipStream_t s) {
  if (dtype == MSAMP_F16)
    return fr == 4 ? launch_projections<f16, MODE, 4>(p, join, s)
                   : (fr == 2 ? launch_projections<f16, MODE, 2>(p, join, s) : launch_projections<f16, MODE, 1>(p, join, s));
  return fr == 4 ? launch_projections<bf16, MODE, 4>(p, join, s)
                 : (fr == 2 ? launch_projections<bf16, MODE, 2>(p, join, s) : launch_projections<bf16, MODE, 1>(p, join, s));
}

template <typename T, int FR>
hipError_t launch_gradients(const Product& x, const Product& w, bool join, hipStream_t s) {
  uint32_t nx = x.tiles_r * x.tiles_c, nw = 2 * w.tiles_r * w.tiles_c;
  if (join) {
    nx = x.splits > 1 ? nx : 0;
    nw = w.splits > 1 ? nw : 0;
    k_gradients_join<T, FR><<<dim3(nx + nw), dim3(kThreads), 0, s>>>(x, w, nx);
  } else {
    nx *= x.splits;
    k_gradients<T, FR><<<dim3(nx + nw * w.splits), dim3(kThreads), 0, s>>>(x, w, nx);
  }
  return hipGetLastError();
}

template <typename T>
hipError_t launch_gradients(int fr, const Product& x, const Product& w, bool join, hipStream_t s) {
  return fr == 4 ? launch_gradients<T, 4>(x, w, join, s)
                 : (fr == 2 ? launch_gradients<T, 2>(x, w, join, s) : launch_gradients<T, 1>(x, w, join, s));
}

hipError_t launch_gradients(int dtype, int fr, const Product& x, const Product& w, bool join, hipStream_t s) {
  return dtype == MSAMP_F16 ? launch_gradients<f16>(fr, x, w, join, s) : launch_gradients<bf16>(fr, x, w, join, s);
}

// Hands out pieces of the workspace (or only counts them).
struct Arena {
  char* base;
  int64_t used = 0;
  void* take(int64_t bytes) {
    if (bytes == 0) return nullptr;
    void* p = base == nullptr ? nullptr : base + used;
    used += (bytes + 255) / 256 * 256;
    return p;
  }
};

msamp_status too_many_tiles() { return fail(MSAMP_E_INVALID_ARG, "the product has too many tiles"); }

// Plans the tiled projections (taking their partial sums' workspace) and runs
// them.
template <int MODE>
msamp_status tiled_projections(msamp_kernel_kind kind, int dtype, Product p, Arena& ws, bool run, hipStream_t s) {
  Cut c;
  const int fr = choose_projection(MODE, p.R, p.C, p.K, &c);
  if (fr == 0) return too_many_tiles();
  apply(c, (float*)ws.take(c.bytes), &p);
  if (!run) return MSAMP_OK;
  MSAMP_LAUNCH(kind, s, launch_projections<MODE>(dtype, fr, p, false, s));
  if (c.splits > 1) MSAMP_LAUNCH(MSAMP_KERNEL_FFN_REDUCE, s, launch_projections<MODE>(dtype, fr, p, true, s));
  return MSAMP_OK;
}

// The same for both gradients.
msamp_status gradients(int dtype, Product x, Product w, Arena& ws, bool run, hipStream_t s) {
  Cut cx, cw;
  const int fr = choose_gradients(x.R, x.C, x.K, &cx, &cw);
  if (fr == 0) return too_many_tiles();
  apply(cx, (float*)ws.take(cx.bytes), &x);
  apply(cw, (float*)ws.take(cw.bytes), &w);
  if (!run) return MSAMP_OK;
  MSAMP_LAUNCH(MSAMP_KERNEL_FFN_GRADIENTS, s, launch_gradients(dtype, fr, x, w, false, s));
  if (cx.splits > 1 || cw.splits > 1)
    MSAMP_LAUNCH(MSAMP_KERNEL_FFN_REDUCE, s, launch_gradients(dtype, fr, x, w, true, s));
  return MSAMP_OK;
}

// -------------------------------------------------------------- few rows ---
//
// Up to 64 tokens the gate and up projections are bound by reading the
// weights, each once. A workgroup forms 16 inner units for all tokens; its 8
// waves share the sum over k and read their parts of the 32 weight rows
// straight into the operands of 16x16x32 MFMA, 128 bytes of every row at a
// time (k is taken in the order of the bytes a lane holds, the same for x), so
// no LDS and no barrier stand between the loads. The waves' sums are joined
// through LDS. At 1 token, 4096 and 11008 (180 MB of weights): 34.7 us, 5.2
// TB/s. With one token the rate of the memory bounds it: 4, 8 or 16 waves and
// 2, 4 or 8 chunks of loads under way all take 34.2 to 37.4 us there and 50.2
// to 52.1 us at 8192 and 8192; 8 waves with 2 chunks are within 2% of the best
// at every size tried.

template <typename T>
struct Frag16;
template <>
struct Frag16<f16> {
  static __device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                  0);
  }
};
template <>
struct Frag16<bf16> {
  static __device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
  }
};

constexpr int kFewRows = 64, kFewWaves = 8, kFewThreads = 64 * kFewWaves;

// n (<= 8) consecutive elements at any address; zeros behind them.
template <typename T>
__device__ __forceinline__ u32x4 load_piece(const T* p, int64_t n) {
  if (n >= 8) return *(const GLOBAL u32x4_any*)p;
  typedef T t8 __attribute__((ext_vector_type(8)));
  t8 v = {};
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (k < n) v[k] = ((const GLOBAL T*)p)[k];
  return __builtin_bit_cast(u32x4, v);
}

// ALIGNED: 16-byte aligned rows of whole pieces, read through buffers whose
// bounds give the zeros behind the last row and k. Otherwise the rows behind
// the last one repeat it (their sums go nowhere), and the chunk that k ends in
// is read on its own.
template <typename T, int MODE, int NT, bool ALIGNED>
__global__ __launch_bounds__(kFewThreads) void k_few_rows(Product p) {
  constexpr int kUnroll = 2;  // chunks of 64 k whose loads are under way at a time (see above)
  __shared__ f32x4 sums[kFewWaves][NT][2][64];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int64_t col0 = (int64_t)blockIdx.x * 16;
  // rows of this block's weights that exist (none: columns that pad dg | du)
  const int64_t left = p.C - col0, cols = left < 0 ? 0 : (left < 16 ? left : 16);
  const int piece = (lane >> 4) * 16;  // this lane's 16 k of a chunk of 64
  constexpr int kOuts = (NT * 256 + kFewThreads - 1) / kFewThreads;  // values of h a thread ends with
  T dh[MODE == kRecompute ? kOuts : 1];
  if constexpr (MODE == kRecompute) {  // here early, as the sums
#pragma unroll
    for (int k = 0; k < kOuts; ++k) {
      const int i = threadIdx.x + k * kFewThreads;
      const int64_t row = 16 * (i / 256) + ((i / 16) & 15), col = col0 + (i & 15);
      dh[k] = i < NT * 256 && row < p.R && col < p.C ? ((const GLOBAL T*)p.dh)[row * p.lddh + col] : (T)0.0f;
    }
  }
  f32x4 acc[NT][2] = {};
  const int chunks = (int)(ALIGNED ? (p.K + 63) / 64 : p.K / 64);
  auto multiply = [&](const u32x4(&g)[2], const u32x4(&u)[2], const u32x4(&x)[NT][2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        acc[t][0] = Frag16<T>::mma(g[h], x[t][h], acc[t][0]);
        acc[t][1] = Frag16<T>::mma(u[h], x[t][h], acc[t][1]);
      }
  };
  if constexpr (ALIGNED) {
    const auto bg = buffer_of((const T*)p.c0 + col0 * p.ldc0, cols == 0 ? 0 : ((cols - 1) * p.ldc0 + round8(p.K)) * 2);
    const auto bu = buffer_of((const T*)p.c1 + col0 * p.ldc1, cols == 0 ? 0 : ((cols - 1) * p.ldc1 + round8(p.K)) * 2);
    const auto bx = buffer_of(p.r0, ((p.R - 1) * p.ldr + round8(p.K)) * 2);
    const int og = (int)((lane & 15) * p.ldc0 * 2) + piece * 2, ou = (int)((lane & 15) * p.ldc1 * 2) + piece * 2;
    int ox[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) ox[t] = (int)(((lane & 15) + 16 * t) * p.ldr * 2) + piece * 2;
    for (int i = wave * kUnroll; i < chunks; i += kFewWaves * kUnroll) {
      u32x4 g[kUnroll][2], u[kUnroll][2], x[kUnroll][NT][2];
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        const int k0 = (i + j) * 64;
        const int64_t rest = p.K - k0 - piece;  // k of this lane that exist
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const bool in = rest > 8 * h;
          g[j][h] = __builtin_amdgcn_raw_buffer_load_b128(bg, in ? og + k0 * 2 + 16 * h : kOutside, 0, 0);
          u[j][h] = __builtin_amdgcn_raw_buffer_load_b128(bu, in ? ou + k0 * 2 + 16 * h : kOutside, 0, 0);
#pragma unroll
          for (int t = 0; t < NT; ++t)
            x[j][t][h] = __builtin_amdgcn_raw_buffer_load_b128(bx, in ? ox[t] + k0 * 2 + 16 * h : kOutside, 0, 0);
        }
      }
      __builtin_amdgcn_sched_barrier(0);  // all of these loads are under way before the first is waited for
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) multiply(g[j], u[j], x[j]);
    }
  } else {
    const int64_t row = col0 + (lane & 15) < p.C ? col0 + (lane & 15) : p.C - 1;
    const T* pg = (const T*)p.c0 + row * p.ldc0 + piece;
    const T* pu = (const T*)p.c1 + row * p.ldc1 + piece;
    const T* px[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int64_t token = (lane & 15) + 16 * t;
      px[t] = (const T*)p.r0 + (token < p.R ? token : p.R - 1) * p.ldr + piece;
    }
    for (int i = wave * kUnroll; i < chunks; i += kFewWaves * kUnroll) {
      u32x4 g[kUnroll][2], u[kUnroll][2], x[kUnroll][NT][2];
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        // in the place of a chunk behind the last whole one the first is read, and not used
        const bool in = i + j < chunks;
        const int64_t k0 = in ? (int64_t)(i + j) * 64 : 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          g[j][h] = *(const GLOBAL u32x4_any*)(pg + k0 + 8 * h);
          u[j][h] = *(const GLOBAL u32x4_any*)(pu + k0 + 8 * h);
#pragma unroll
          for (int t = 0; t < NT; ++t) x[j][t][h] = *(const GLOBAL u32x4_any*)(px[t] + k0 + 8 * h);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < kUnroll; ++j)
        if (i + j < chunks) multiply(g[j], u[j], x[j]);
    }
    if (p.K % 64 != 0 && wave == chunks % kFewWaves) {
      u32x4 g[2], u[2], x[NT][2];
      const int64_t k0 = (int64_t)chunks * 64;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t n = p.K - k0 - piece - 8 * h;
        g[h] = load_piece(pg + k0 + 8 * h, n);
        u[h] = load_piece(pu + k0 + 8 * h, n);
#pragma unroll
        for (int t = 0; t < NT; ++t) x[t][h] = load_piece(px[t] + k0 + 8 * h, n);
      }
      multiply(g, u, x);
    }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    sums[wave][t][0][lane] = acc[t][0];
    sums[wave][t][1][lane] = acc[t][1];
  }
  __syncthreads();
  // element e of sums[..][lane]: inner unit 4 * (lane / 16) + e, token lane % 16
#pragma unroll
  for (int k = 0; k < kOuts; ++k) {
    const int i = threadIdx.x + k * kFewThreads;
    if (i >= NT * 256) break;
    const int t = i / 256, token = (i / 16) & 15, unit = i & 15;
    const int64_t row = 16 * t + token, col = col0 + unit;
    if (row >= p.R) continue;
    const int from = (unit >> 2) * 16 + token;
    float g = 0.0f, u = 0.0f;
#pragma unroll
    for (int w = 0; w < kFewWaves; ++w) {
      g += sums[w][t][0][from][unit & 3];
      u += sums[w][t][1][from][unit & 3];
    }
    float a, d;
    with_act(p.act, [&](auto act) { act_and_grad<decltype(act)::value>(g, &a, &d); });
    if (col < p.C && p.out0 != nullptr) ((GLOBAL T*)p.out0)[row * p.ldo0 + col] = from_f32<T>(a * u);
    if constexpr (MODE == kRecompute) {
      GLOBAL T* o = (GLOBAL T*)p.dgu + row * (2 * p.half) + col;
      o[0] = from_f32<T>(to_f32(dh[k]) * u * d);
      o[p.half] = from_f32<T>(to_f32(dh[k]) * a);
    }
  }
}

// Whether the matrix kernels can read an operand where it lies: 16-byte
// aligned rows of whole 16-byte pieces, and a tile of 256 rows within the 2^31
// bytes of a buffer.
bool direct(const void* p, int64_t ld, int64_t cols) {
  return ((uintptr_t)p & 15u) == 0 && ld % 8 == 0 && cols % 8 == 0 && ld >= cols && ld < (1 << 22);
}

template <typename T, int MODE, bool ALIGNED>
hipError_t launch_few_rows(const Product& p, hipStream_t s) {
  const int64_t cols = MODE == kRecompute ? p.half : p.C;
  const dim3 g((unsigned)((cols + 15) / 16)), b(kFewThreads);
  if (p.R <= 16) k_few_rows<T, MODE, 1, ALIGNED><<<g, b, 0, s>>>(p);
  else if (p.R <= 32) k_few_rows<T, MODE, 2, ALIGNED><<<g, b, 0, s>>>(p);
  else k_few_rows<T, MODE, 4, ALIGNED><<<g, b, 0, s>>>(p);
  return hipGetLastError();
}

template <int MODE>
hipError_t launch_few(int dtype, const Product& p, hipStream_t s) {
  if constexpr (MODE == kForward) {  // the backward pass lays its operands out anyway
    if (!direct(p.r0, p.ldr, p.K) || !direct(p.c0, p.ldc0, p.K) || !direct(p.c1, p.ldc1, p.K))
      return dtype == MSAMP_F16 ? launch_few_rows<f16, MODE, false>(p, s) : launch_few_rows<bf16, MODE, false>(p, s);
  }
  return dtype == MSAMP_F16 ? launch_few_rows<f16, MODE, true>(p, s) : launch_few_rows<bf16, MODE, true>(p, s);
}

// Whether the kernel for few tokens takes the gate and up projections. Every
// workgroup of it reads all of x, from L2: with more than about 8e8 products
// (100 MB of it) that costs more than the partial sums of the tiled kernel
// save. Measured at hidden 4096, 11008 inner units: 16 tokens 40.1 us against
// 50.3 us by tiles, 24 tokens 49.5 against 50.5, 64 tokens 79.5 against 57.8;
// at 768 and 2048, 64 tokens 8.3 against 11.2. Its waves take their parts of k
// one after another, with several blocks of tokens 128 k at a time: beyond a
// hidden size of 1024 that takes longer than a split sum (56 tokens at 3136
// and 1920: 18.5 us).
bool few_rows(int64_t R, int64_t C, int64_t K) {
  return R <= kFewRows && C <= (1 << 22) && (double)R * (double)C * (double)K <= 8e8 && (R <= 16 || K <= 1024);
}

// The gate and up projections by the kernel that suits the number of tokens.
template <int MODE>
msamp_status projections(msamp_kernel_kind kind, int dtype, const Product& p, Arena& ws, bool run, hipStream_t s) {
  if (!few_rows(p.R, p.C, p.K)) return tiled_projections<MODE>(kind, dtype, p, ws, run, s);
  if (run) MSAMP_LAUNCH(kind, s, launch_few<MODE>(dtype, p, s));
  return MSAMP_OK;
}

// ---------------------------------------------------------------- layout ---

// out [rows, ld] <- src [rows, cols] or a checkpoint's values (rounded to T, the
// operand type of the matrix instructions), zeros behind the last column; up to
// three matrices in one launch. Bound by memory: 4096 x 4096 from a checkpoint,
// 51 MB, take 13 us; the products read the result 43 times, so decoding there
// would cost more.
struct Layout {
  int64_t rows, cols;
  const void* src;  // null: ck
  int64_t lds;
  CkptRef ck;
  void* out;
  int64_t ld;
};
struct Layouts {
  Layout job[3];
  int n;
};

template <typename T>
__global__ __launch_bounds__(256) void k_layout(Layouts all) {
  const Layout a = all.job[blockIdx.y];
  const int64_t per = a.ld / 8, total = a.rows * per;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t row = (uint64_t)total <= UINT32_MAX ? (int64_t)((uint32_t)i / (uint32_t)per) : i / per;
    const int64_t col = (i - row * per) * 8, left = a.cols - col;
    const int n = left < 0 ? 0 : (left < 8 ? (int)left : 8);
    float f[8];
    if (a.src != nullptr) {
      load8((const T*)a.src + row * a.lds + col, n, f);
    } else {
      load_ckpt8(a.ck.fmt, a.ck.codes + row * a.ck.ld, a.ck.scales + row * a.ck.ld_scales, col, n, f);
      const float lim = __is_same(T, f16) ? kF16Max : kBf16Max;
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = clamp_finite(f[k], lim);
    }
    store8((T*)a.out + row * a.ld + col, 8, f);
  }
}

hipError_t launch_layout(int dtype, const Layouts& all, hipStream_t s) {
  int64_t blocks = 1;
  for (int i = 0; i < all.n; ++i) {
    const int64_t b = (all.job[i].rows * (all.job[i].ld / 8) + 255) / 256;
    blocks = b > blocks ? b : blocks;
  }
  const dim3 g((unsigned)(blocks < 65536 ? blocks : 65536), (unsigned)all.n);
  if (dtype == MSAMP_F16) k_layout<f16><<<g, dim3(256), 0, s>>>(all);
  else k_layout<bf16><<<g, dim3(256), 0, s>>>(all);
  return hipGetLastError();
}

// ------------------------------------------------------------------ plan ---

int64_t round64(int64_t n) { return (n + 63) / 64 * 64; }

struct Operand {
  const void* p;
  int64_t ld;
};

// An operand [rows, cols]: where it lies, or its place in the workspace with
// the job that lays it out there.
msamp_status lay_out(int64_t rows, int64_t cols, const void* p, int64_t ld, const msamp_checkpoint* ck, Arena& ws,
                     Layouts& jobs, Operand* out) {
  *out = {p, ld};
  if (ck == nullptr && direct(p, ld, cols)) return MSAMP_OK;
  const int64_t lp = round64(cols);
  if (lp >= (1 << 22)) return fail(MSAMP_E_INVALID_ARG, "hidden exceeds 2^22 - 64");
  Layout& j = jobs.job[jobs.n++];
  j = {rows, cols, ck == nullptr ? p : nullptr, ld, CkptRef{}, ws.take(rows * lp * 2), lp};
  if (ck != nullptr) j.ck = {ck->codes, ck->ld, ck->scales, ck->ld_scales, (int)ck->fmt};
  *out = {j.out, lp};
  return MSAMP_OK;
}

msamp_status run_layouts(int dtype, const Layouts& jobs, hipStream_t s) {
  if (jobs.n > 0) MSAMP_LAUNCH(MSAMP_KERNEL_FFN_LAYOUT, s, launch_layout(dtype, jobs, s));
  return MSAMP_OK;
}

// Output of zeros: the sums of nothing.
template <typename T>
__global__ void k_fill_zero(int64_t rows, int64_t cols, T* out, int64_t ld) {
  const int64_t total = rows * cols;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256)
    out[i / cols * ld + i % cols] = (T)0.0f;
}

msamp_status fill_zero(int dtype, int64_t rows, int64_t cols, void* out, int64_t ld, hipStream_t s) {
  if (rows == 0 || cols == 0) return MSAMP_OK;
  const int64_t blocks = (rows * cols + 255) / 256;
  const dim3 g((unsigned)(blocks < 65536 ? blocks : 65536));
  auto launch = [&]() {
    if (dtype == MSAMP_F32) k_fill_zero<float><<<g, dim3(256), 0, s>>>(rows, cols, (float*)out, ld);
    else k_fill_zero<uint16_t><<<g, dim3(256), 0, s>>>(rows, cols, (uint16_t*)out, ld);
    return hipGetLastError();
  };
  MSAMP_LAUNCH(MSAMP_KERNEL_FFN_LAYOUT, s, launch());
  return MSAMP_OK;
}

// Counts the workspace (run = false) or makes the call.
msamp_status forward(const msamp_gated_ffn& a, Arena& ws, bool run, hipStream_t s) {
  if (a.tokens == 0 || a.ffn == 0) return MSAMP_OK;
  if (a.hidden == 0) return run ? fill_zero(a.dtype, a.tokens, a.ffn, a.h, a.ldh, s) : MSAMP_OK;
  Operand x = {a.x, a.ldx}, g = {a.w_gate, a.ld_gate}, u = {a.w_up, a.ld_up};
  if (!few_rows(a.tokens, a.ffn, a.hidden)) {
    Layouts jobs = {};
    MSAMP_TRY(lay_out(a.tokens, a.hidden, a.x, a.ldx, nullptr, ws, jobs, &x));
    MSAMP_TRY(lay_out(a.ffn, a.hidden, a.w_gate, a.ld_gate, nullptr, ws, jobs, &g));
    MSAMP_TRY(lay_out(a.ffn, a.hidden, a.w_up, a.ld_up, nullptr, ws, jobs, &u));
    if (run) MSAMP_TRY(run_layouts(a.dtype, jobs, s));
  }
  Product p = {};
  p.R = a.tokens, p.C = a.ffn, p.K = a.hidden;
  p.r0 = x.p, p.ldr = x.ld;
  p.c0 = g.p, p.ldc0 = g.ld, p.c1 = u.p, p.ldc1 = u.ld;
  p.act = a.act;
  p.out0 = a.h, p.ldo0 = a.ldh;
  return projections<kForward>(MSAMP_KERNEL_FFN_FORWARD, a.dtype, p, ws, run, s);
}

msamp_status backward(const msamp_gated_ffn& a, Arena& ws, bool run, hipStream_t s) {
  const int64_t T = a.tokens, K = a.hidden, F = a.ffn;
  if (T == 0 || F == 0 || K == 0) {  // sums of nothing
    if (!run) return MSAMP_OK;
    if (a.h != nullptr) MSAMP_TRY(fill_zero(a.dtype, T, F, a.h, a.ldh, s));
    MSAMP_TRY(fill_zero(a.dtype, T, K, a.dx, a.lddx, s));
    if (a.dw_accumulate) return MSAMP_OK;
    MSAMP_TRY(fill_zero(a.dw_dtype, F, K, a.dw_gate, a.ld_dw_gate, s));
    return fill_zero(a.dw_dtype, F, K, a.dw_up, a.ld_dw_up, s);
  }
  Operand x, g, u;
  Layouts jobs = {};
  MSAMP_TRY(lay_out(T, K, a.x, a.ldx, a.x_ckpt, ws, jobs, &x));
  MSAMP_TRY(lay_out(F, K, a.w_gate, a.ld_gate, nullptr, ws, jobs, &g));
  MSAMP_TRY(lay_out(F, K, a.w_up, a.ld_up, nullptr, ws, jobs, &u));
  if (run) MSAMP_TRY(run_layouts(a.dtype, jobs, s));
  const int64_t half = round64(F);
  if (2 * half >= (1 << 22)) return fail(MSAMP_E_INVALID_ARG, "ffn exceeds 2^21 - 64");
  char* dgu = (char*)ws.take(T * 2 * half * 2);  // null while only counting
  Product p = {};
  p.R = T, p.C = F, p.K = K;
  p.r0 = x.p, p.ldr = x.ld;
  p.c0 = g.p, p.ldc0 = g.ld, p.c1 = u.p, p.ldc1 = u.ld;
  p.act = a.act;
  p.out0 = a.h, p.ldo0 = a.ldh;
  p.dh = a.dh, p.lddh = a.lddh;
  p.dgu = dgu, p.half = half;
  // the partial sums of both launches take turns in the same memory
  const int64_t mark = ws.used;
  MSAMP_TRY(projections<kRecompute>(MSAMP_KERNEL_FFN_RECOMPUTE, a.dtype, p, ws, run, s));
  const int64_t most = ws.used;
  ws.used = mark;

  Product dx = {};
  dx.R = T, dx.C = K, dx.K = F;
  dx.r0 = dgu, dx.r1 = run ? dgu + half * 2 : nullptr, dx.ldr = 2 * half;
  dx.c0 = g.p, dx.ldc0 = g.ld, dx.c1 = u.p, dx.ldc1 = u.ld;
  dx.out0 = a.dx, dx.ldo0 = a.lddx;

  Product dw = {};
  dw.R = F, dw.C = K, dw.K = T;
  dw.r0 = dx.r0, dw.r1 = dx.r1, dw.ldr = dx.ldr;
  dw.c0 = x.p, dw.ldc0 = x.ld;
  dw.out0 = a.dw_gate, dw.ldo0 = a.ld_dw_gate, dw.out1 = a.dw_up, dw.ldo1 = a.ld_dw_up;
  dw.out_f32 = a.dw_dtype == MSAMP_F32, dw.accumulate = a.dw_accumulate;
  MSAMP_TRY(gradients(a.dtype, dx, dw, ws, run, s));
  ws.used = ws.used > most ? ws.used : most;
  return MSAMP_OK;
}

}  // namespace

msamp_status ffn_forward_workspace(const msamp_gated_ffn& a, int64_t* bytes) {
  Arena ws = {nullptr};
  MSAMP_TRY(forward(a, ws, false, nullptr));
  *bytes = ws.used;
  return MSAMP_OK;
}

msamp_status ffn_backward_workspace(const msamp_gated_ffn& a, int64_t* bytes) {
  Arena ws = {nullptr};
  MSAMP_TRY(backward(a, ws, false, nullptr));
  *bytes = ws.used;
  return MSAMP_OK;
}

msamp_status ffn_plan(const msamp_gated_ffn& a, bool backward, int32_t* plan) {
  const int64_t T = a.tokens, K = a.hidden, F = a.ffn;
  for (int i = 0; i < 6; ++i) plan[i] = 0;
  if (T == 0 || K == 0 || F == 0) return MSAMP_OK;
  Cut x, w;
  if (!few_rows(T, F, K)) {
    plan[0] = 64 * choose_projection(backward ? kRecompute : kForward, T, F, K, &x);
    if (plan[0] == 0) return too_many_tiles();
    plan[1] = (int32_t)x.splits;
  }
  if (!backward) return MSAMP_OK;
  plan[2] = plan[4] = 64 * choose_gradients(T, K, F, &x, &w);
  if (plan[2] == 0) return too_many_tiles();
  plan[3] = (int32_t)x.splits, plan[5] = (int32_t)w.splits;
  return MSAMP_OK;
}

msamp_status ffn_forward(const msamp_gated_ffn& a, void* ws, hipStream_t s) {
  Arena arena = {(char*)ws};
  return forward(a, arena, true, s);
}

msamp_status ffn_backward(const msamp_gated_ffn& a, void* ws, hipStream_t s) {
  Arena arena = {(char*)ws};
  return backward(a, arena, true, s);
}

}  // namespace msamp
