// norm.hip -- 8-bit activation checkpoints (save, load) and layer norm / RMS
// norm (forward, backward) on gfx950. The definitions are in msamp.h.
//
// All of these are bound by memory: one pass over the data, the row of a norm
// held in registers between its statistics and its output.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "checkpoint.hpp"

namespace msamp {
namespace {

// ----------------------------------------------------------- checkpoints ---

constexpr int kCkBlock = 256;

// Work units of 8 elements, whole groups per row (units behind the row's last
// element take part in their group's exchange and store nothing). At most
// 2^30 a launch, so that their row is a 32-bit division.
struct Units {
  uint32_t total;
  uint32_t per_row;
};

// Bound by memory: 16,384 rows of 4,096 bfloat16 columns, 203 MB each way, take
// 36.2 us to save (5.6 TB/s) and 31.0 us to load (6.6 TB/s, some of the codes
// being in cache still). The load's output is stored past the caches (save and
// load there: 68 us against 76; stored that way, the save's codes would come
// back from memory, 75 us). One unit a thread: more of them, loaded ahead, were
// slower (both, before those stores: 76 us with one, 81 with two, 87 with four).
template <typename T>
__global__ __launch_bounds__(kCkBlock) void k_checkpoint_save(Units u, int64_t cols, const T* x, int64_t ldx,
                                                              CkptRef ck) {
  const uint32_t i = blockIdx.x * kCkBlock + threadIdx.x;
  // a group's four lanes are inside or outside together (total is a multiple of 4)
  if (i >= u.total) return;
  const uint32_t r = i / u.per_row;
  const int64_t row = r;
  const int64_t col = (int64_t)(i - r * u.per_row) * 8;
  const int n = (int)(cols - col < 8 ? cols - col : 8);
  float f[8];
  load8(x + row * ldx + col, n, f);
  save_group8(ck.fmt, ck.codes + row * ck.ld, ck.scales + row * ck.ld_scales, col, n, f);
}

template <typename T>
__global__ __launch_bounds__(kCkBlock) void k_checkpoint_load(Units u, int64_t cols, CkptRef ck, T* out,
                                                              int64_t ldout) {
  const uint32_t i = blockIdx.x * kCkBlock + threadIdx.x;
  if (i >= u.total) return;
  const uint32_t r = i / u.per_row;
  const int64_t row = r;
  const int64_t col = (int64_t)(i - r * u.per_row) * 8;
  const int n = (int)(cols - col < 8 ? cols - col : 8);
  if (n <= 0) return;
  float f[8];
  load_ckpt8(ck.fmt, ck.codes + row * ck.ld, ck.scales + row * ck.ld_scales, col, n, f);
  if constexpr (sizeof(T) == 2) {
    const float lim = __is_same(T, f16) ? kF16Max : kBf16Max;
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = clamp_finite(f[k], lim);
  }
  store8<T, true>(out + row * ldout + col, n, f);
}

// ----------------------------------------------------------------- norms ---

// Sum over the 64 lanes, given to all of them: four shifts within the rows of
// 16 lanes, two carries between them (the total ends in lane 63), no LDS.
template <int CTRL, int ROWS>
__device__ __forceinline__ float add_dpp(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROWS, 0xf, true));
}
__device__ __forceinline__ float wave_sum(float v) {
  v = add_dpp<0x111, 0xf>(v);  // row_shr:1
  v = add_dpp<0x112, 0xf>(v);
  v = add_dpp<0x114, 0xf>(v);
  v = add_dpp<0x118, 0xf>(v);
  v = add_dpp<0x142, 0xa>(v);  // row_bcast:15 into rows 1 and 3
  v = add_dpp<0x143, 0xc>(v);  // row_bcast:31 into rows 2 and 3
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// Sum over each 16 or 32 neighbouring lanes, given to all of them.
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
  if constexpr (LANES == 64) return wave_sum(v);
  v = add_dpp<0xB1, 0xf>(v);   // quad_perm: 1 0 3 2
  v = add_dpp<0x4E, 0xf>(v);   // quad_perm: 2 3 0 1
  v = add_dpp<0x141, 0xf>(v);  // row_half_mirror: the other four of eight
  v = add_dpp<0x140, 0xf>(v);  // row_mirror: the other eight
  if constexpr (LANES == 32) v += __shfl_xor(v, 16, 64);
  return v;
}

// Sums of a and b over the lanes of a row: LANES neighbours of a wave, or (64)
// WAVES whole waves, GROUPS rows side by side in the workgroup. 'turn'
// alternates between two sets of partials, so that one barrier a sum is enough.
template <int LANES, int WAVES, int GROUPS>
__device__ __forceinline__ void row_sum2(float& a, float& b, int turn) {
  a = lanes_sum<LANES>(a);
  b = lanes_sum<LANES>(b);
  if constexpr (WAVES > 1) {
    __shared__ float part[2][GROUPS][2][WAVES];
    const int wave = threadIdx.x >> 6, group = wave / WAVES;
    if ((threadIdx.x & 63) == 0) {
      part[turn][group][0][wave % WAVES] = a;
      part[turn][group][1][wave % WAVES] = b;
    }
    __syncthreads();
    a = part[turn][group][0][0];
    b = part[turn][group][1][0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) {
      a += part[turn][group][0][w];
      b += part[turn][group][1][w];
    }
  }
}

// Threads of a workgroup: a row per wave (four rows), or a row per workgroup.
template <int WAVES>
constexpr int norm_block() {
  return WAVES == 1 ? 256 : WAVES * 64;
}

template <typename T>
__device__ __forceinline__ void load_weight8(const void* w, bool f32, int64_t col, int n, float fill, float* f) {
  if (w == nullptr) {
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = fill;
  } else if (sizeof(T) == 2 && !f32) {
    load8((const T*)w + col, n, f);
  } else {
    load8((const float*)w + col, n, f);
  }
}

template <typename T>
__device__ __forceinline__ void load_x8(const NormArgs& a, int64_t row, int64_t col, int n, float* f) {
  if (a.x != nullptr)
    load8((const T*)a.x + row * a.ldx + col, n, f);
  else
    load_ckpt8(a.ck.fmt, a.ck.codes + row * a.ck.ld, a.ck.scales + row * a.ck.ld_scales, col, n, f);
}

// One row per LANES lanes of a wave or per WAVES waves; a lane holds NCH pieces
// of 8 columns in registers, so that the row is read once: mean, then the
// squares around it, then the output. Bound by memory: 16,384 x 4,096 bfloat16
// with its checkpoint saved, 338 MB, take 62 us (5.5 TB/s). A wave alone holds
// up to 2,048 columns, as its sums need no barrier; four share up to 8,192.
template <typename T, int LANES, int WAVES, int NCH>
__global__ __launch_bounds__(norm_block<WAVES>()) void k_norm_forward(NormArgs a) {
  constexpr int kLanes = WAVES * LANES;
  const int lane = threadIdx.x % kLanes;
  const int64_t row = (int64_t)blockIdx.x * (norm_block<WAVES>() / kLanes) + threadIdx.x / kLanes;
  if (row >= a.rows) return;  // all lanes of a row; with WAVES > 1 no row is beyond
  float v[NCH][8];
  int n[NCH];
  float sum = 0.0f, sq = 0.0f;
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int64_t col = ((int64_t)c * kLanes + lane) * 8;
    n[c] = (int)(a.cols - col < 8 ? a.cols - col : 8);
    if (n[c] < 0) n[c] = 0;
    load_x8<T>(a, row, col, n[c], v[c]);
  }
  if (a.save.codes != nullptr) {
#pragma unroll
    for (int c = 0; c < NCH; ++c)
      save_group8(a.save.fmt, a.save.codes + row * a.save.ld, a.save.scales + row * a.save.ld_scales,
                  ((int64_t)c * kLanes + lane) * 8, n[c], v[c]);
  }
  const float inv = 1.0f / (float)a.cols;
  float mu = 0.0f;
  if (a.mean != nullptr) {
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int k = 0; k < 8; ++k) sum += v[c][k];
    row_sum2<LANES, WAVES, 1>(sum, sq, 0);
    mu = sum * inv;
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int k = 0; k < 8; ++k) v[c][k] = k < n[c] ? v[c][k] - mu : 0.0f;
    sum = 0.0f;
  }
#pragma unroll
  for (int c = 0; c < NCH; ++c)
#pragma unroll
    for (int k = 0; k < 8; ++k) sq = __builtin_fmaf(v[c][k], v[c][k], sq);
  row_sum2<LANES, WAVES, 1>(sq, sum, 1);
  const float rstd = 1.0f / __builtin_sqrtf(__builtin_fmaf(sq, inv, a.eps));
  if (lane == 0) {
    if (a.mean != nullptr) a.mean[row] = mu;
    a.rstd[row] = rstd;
  }
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int64_t col = ((int64_t)c * kLanes + lane) * 8;
    if (n[c] > 0) {
      float w[8], b[8], y[8];
      load_weight8<T>(a.weight, a.weight_f32, col, n[c], 1.0f, w);
      load_weight8<T>(a.bias, a.weight_f32, col, n[c], 0.0f, b);
#pragma unroll
      for (int k = 0; k < 8; ++k) y[k] = __builtin_fmaf(v[c][k] * rstd, w[k], b[k]);
      store8((T*)a.y + row * a.ldy + col, n[c], y);
    }
  }
}

// A lane's pieces of a row as they lie in memory: of a matrix of T, or of a
// checkpoint's codes with their scales. Pieces behind the last column hold
// anything (the row's first piece, loaded without a branch, or zeros).
template <typename T, bool CK, int NCH>
struct RawRow {
  typedef T t8 __attribute__((ext_vector_type(8)));
  t8 v[CK ? 1 : NCH];
  u32x2 q[CK ? NCH : 1];
  uint8_t s[CK ? NCH : 1];
};

template <typename T, int NCH, int LANES, bool TAIL>
__device__ __forceinline__ void load_raw(const T* row, int cols, int lane, RawRow<T, false, NCH>& r) {
  typedef T t8 __attribute__((ext_vector_type(8)));
  typedef t8 t8_any __attribute__((aligned(sizeof(T))));
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int col = (c * LANES + lane) * 8;
    if constexpr (!TAIL) {
      r.v[c] = *(const GLOBAL t8_any*)(row + (col < cols ? col : 0));
    } else if (col + 8 <= cols) {
      r.v[c] = *(const GLOBAL t8_any*)(row + col);
    } else {
      r.v[c] = t8{};
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (col + k < cols) r.v[c][k] = ((const GLOBAL T*)row)[col + k];
    }
  }
}

template <typename T, int NCH, int LANES, bool TAIL>
__device__ __forceinline__ void load_raw(const CkptRef& ck, int64_t row, int cols, int lane,
                                         RawRow<T, true, NCH>& r) {
  const uint8_t* codes = ck.codes + row * ck.ld;
  const uint8_t* scales = ck.scales + row * ck.ld_scales;
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int col = (c * LANES + lane) * 8, at = col < cols ? col : 0;
    r.s[c] = ((const GLOBAL uint8_t*)scales)[at / kGroup];
    if constexpr (!TAIL) {
      r.q[c] = *(const GLOBAL u32x2_any*)(codes + at);
    } else if (col + 8 <= cols) {
      r.q[c] = *(const GLOBAL u32x2_any*)(codes + col);
    } else {
      r.q[c] = u32x2{0u, 0u};
      for (int k = 0; k < 8 && col + k < cols; ++k) {
        const uint32_t b = (uint32_t)((const GLOBAL uint8_t*)codes)[col + k] << (8 * (k & 3));
        if (k < 4) r.q[c].x |= b; else r.q[c].y |= b;
      }
    }
  }
}

template <typename T, int NCH>
__device__ __forceinline__ void unpack(const RawRow<T, false, NCH>& r, int, int c, float* f) {
#pragma unroll
  for (int k = 0; k < 8; ++k) f[k] = to_f32(r.v[c][k]);
}
template <typename T, int NCH>
__device__ __forceinline__ void unpack(const RawRow<T, true, NCH>& r, int fmt, int c, float* f) {
  decode_group8(fmt, r.q[c], r.s[c], f);
}

// Each workgroup walks over rows: GROUPS sets of WAVES waves, each with a row,
// or with 64 / LANES rows of LANES lanes. A lane holds the same NCH pieces of 8
// columns throughout and sums their share of dweight and dbias in registers.
// The next row is on its way while one is worked on; two rows where several
// waves share one of a 16-bit checkpoint, whose rows are the shortest in bytes
// (from a checkpoint, 16,384 x 2,560: 54 us with two, 58 with one; 65,536 x 512:
// 39.7 and 38.2; from a matrix, 8,192 x 768: 15.9 and 14.9). They lie in a ring
// of buffers that the unrolled loop names one after another, and are loaded
// without branches (behind the last row the last again): where buffers are
// copied, the compiler waits for every load under way.
// TAIL: the columns end inside a piece. Lanes behind the last column work on
// dy = 0, which adds nothing to a row's sums (dy * xh is 0 or, in a row whose
// statistics are not finite anyway, NaN).
// Bound by memory where rows are many: 16,384 x 4,096 bfloat16 from a checkpoint,
// 338 MB, take 61 us (5.5 TB/s); 8,192 x 768 fp16, 38 MB, take 12.6 us, where the
// start and the end of four turns weigh as much.
template <typename T, bool CK, bool TAIL, int LANES, int WAVES, int NCH, int GROUPS>
__global__ __launch_bounds__(WAVES* GROUPS * 64) void k_norm_backward(NormArgs a) {
  constexpr int kLanes = WAVES * LANES, kRows = WAVES * GROUPS * 64 / kLanes;
  const int lane = (int)threadIdx.x % kLanes;
  const int64_t stride = (int64_t)gridDim.x * kRows;
  const int cols = (int)a.cols;
  const float inv = 1.0f / (float)cols;
  const bool centered = a.mean != nullptr, bias = a.dbias != nullptr;
  // With several pieces a lane, registers are short: the weights are then read
  // for every row (from cache), and no row is loaded ahead. A thread of 1,024
  // has 128 registers, and what it holds of four pieces (beyond 16,384 columns)
  // does not fit: 106 to 179 registers go through scratch (264 to 512 bytes a
  // lane), of two pieces up to 16. 4,096 rows, bfloat16: 16,384 columns take 96
  // us (4.2 TB/s), 32,768 columns 501 us (1.6 TB/s); binary32 159 and 634 us.
  constexpr bool kKeep = NCH == 1;
  constexpr int kAhead = !kKeep ? 0 : (CK && sizeof(T) == 2 && WAVES >= 4 ? 2 : 1);
  float w[NCH][8], sw[NCH][8], sb[NCH][8];
  auto load_weights = [&](int c) {
    const int col = (c * kLanes + lane) * 8;
    const int n = cols - col < 8 ? (cols > col ? cols - col : 0) : 8;
    load_weight8<T>(a.weight, a.weight_f32, col, n, 1.0f, w[c]);
  };
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    if constexpr (kKeep) load_weights(c);
#pragma unroll
    for (int k = 0; k < 8; ++k) sw[c][k] = sb[c][k] = 0.0f;
  }
  struct Row {
    RawRow<T, CK, NCH> x;
    RawRow<T, false, NCH> g;
    float mu, rstd;
  };
  Row ring[kAhead + 1];
  const float* mean = centered ? a.mean : a.rstd;  // read in any case, used if centered
  auto fetch = [&](int64_t row, Row& r) {
    row = row < a.rows ? row : a.rows - 1;
    if constexpr (CK) load_raw<T, NCH, kLanes, TAIL>(a.ck, row, cols, lane, r.x);
    else load_raw<T, NCH, kLanes, TAIL>((const T*)a.x + row * a.ldx, cols, lane, r.x);
    load_raw<T, NCH, kLanes, TAIL>((const T*)a.dy + row * a.lddy, cols, lane, r.g);
    r.mu = mean[row];
    r.rstd = a.rstd[row];
  };
  int turn = 0;
  auto work = [&](int64_t row, const Row& in) {
    const bool live = row < a.rows;
    const float mu = in.mu, rstd = in.rstd;
    float xh[NCH][8], g[NCH][8];
    float c1 = 0.0f, c2 = 0.0f;
    if (live) {
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        unpack<T, NCH>(in.x, a.ck.fmt, c, xh[c]);
        unpack<T, NCH>(in.g, 0, c, g[c]);
        if ((c * kLanes + lane) * 8 >= cols) {
#pragma unroll
          for (int k = 0; k < 8; ++k) g[c][k] = 0.0f;
        }
        if constexpr (!kKeep) load_weights(c);
        if (centered) {
#pragma unroll
          for (int k = 0; k < 8; ++k) xh[c][k] -= mu;
        }
        if (bias) {
#pragma unroll
          for (int k = 0; k < 8; ++k) sb[c][k] += g[c][k];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          xh[c][k] *= rstd;
          sw[c][k] = __builtin_fmaf(g[c][k], xh[c][k], sw[c][k]);
          g[c][k] *= w[c][k];
          c2 = __builtin_fmaf(g[c][k], xh[c][k], c2);
        }
        if (centered) {
#pragma unroll
          for (int k = 0; k < 8; ++k) c1 += g[c][k];
        }
      }
    }
    row_sum2<LANES, WAVES, GROUPS>(c1, c2, turn);
    turn ^= 1;
    if (live) {
      c1 *= inv * rstd;
      c2 *= inv * rstd;
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        const int col = (c * kLanes + lane) * 8;
        if (col < cols) {
          float o[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) o[k] = __builtin_fmaf(-xh[c][k], c2, __builtin_fmaf(g[c][k], rstd, -c1));
          store8((T*)a.dx + row * a.lddx + col, TAIL && cols - col < 8 ? cols - col : 8, o);
        }
      }
    }
  };
  int64_t row = (int64_t)blockIdx.x * kRows + (int)threadIdx.x / kLanes;
#pragma unroll
  for (int b = 0; b < kAhead; ++b) fetch(row + b * stride, ring[b]);
  // all rows of a workgroup make the same number of turns: the sums have a barrier
  for (int64_t base = (int64_t)blockIdx.x * kRows; base < a.rows;) {
#pragma unroll
    for (int b = 0; b <= kAhead; ++b) {
      fetch(row + kAhead * stride, ring[(b + kAhead) % (kAhead + 1)]);
      work(row, ring[b]);
      base += stride, row += stride;
      if (base >= a.rows) break;
    }
  }
  if (a.dweight == nullptr && a.dbias == nullptr) return;
  const int group = (int)threadIdx.x / (WAVES * 64);
  if constexpr (LANES < 64) {  // a wave's rows
#pragma unroll
    for (int off = LANES; off < 64; off *= 2)
#pragma unroll
      for (int c = 0; c < NCH; ++c)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          sw[c][k] += __shfl_xor(sw[c][k], off, 64);
          sb[c][k] += __shfl_xor(sb[c][k], off, 64);
        }
  }
  // one workgroup alone has the whole sums; several leave theirs for k_norm_reduce
  const bool alone = a.partial == nullptr;
  float* pw = alone ? a.dweight : a.partial + (int64_t)blockIdx.x * a.cols;
  float* pb = alone ? a.dbias : pw + a.nparts * a.cols;
  const bool add = alone && a.accumulate;
  if constexpr (GROUPS > 1) {  // the groups' sums of the same columns meet in LDS, and are added in order
    __shared__ __attribute__((aligned(16))) float acc[GROUPS][NCH * kLanes * 8];
    auto join = [&](const float(&sums)[NCH][8], float* out) {
      __syncthreads();  // acc has been read
      if (LANES == 64 || (int)(threadIdx.x & 63) < LANES) {
#pragma unroll
        for (int c = 0; c < NCH; ++c)
#pragma unroll
          for (int k = 0; k < 8; ++k) acc[group][(c * kLanes + lane) * 8 + k] = sums[c][k];
      }
      __syncthreads();
      for (int col = threadIdx.x; col < cols; col += WAVES * GROUPS * 64) {
        float t = acc[0][col];
#pragma unroll
        for (int g = 1; g < GROUPS; ++g) t += acc[g][col];
        out[col] = add ? out[col] + t : t;
      }
    };
    if (a.dweight != nullptr) join(sw, pw);
    if (bias) join(sb, pb);
  } else {
    auto store = [&](float(&sums)[NCH][8], float* out) {
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        const int col = (c * kLanes + lane) * 8;
        const int n = TAIL && cols - col < 8 ? cols - col : 8;
        if (col < cols) {
          if (add) {
            float old[8];
            load8(out + col, n, old);
#pragma unroll
            for (int k = 0; k < 8; ++k) sums[c][k] += old[k];
          }
          store8(out + col, n, sums[c]);
        }
      }
    };
    if (a.dweight != nullptr) store(sw, pw);
    if (bias) store(sb, pb);
  }
}

// 32 columns per workgroup, 32 threads a column, each over every 32nd part, in
// this order always. Latency bounds it: 3.9 us for 512 parts of 768 columns,
// 4.8 us for 256 of 4,096.
__global__ __launch_bounds__(1024) void k_norm_reduce(NormArgs a) {
  float* out = blockIdx.y == 0 ? a.dweight : a.dbias;
  if (out == nullptr) return;
  const float* p = a.partial + (int64_t)blockIdx.y * a.nparts * a.cols;
  const int64_t col = (int64_t)blockIdx.x * 32 + (threadIdx.x & 31);
  const int part = threadIdx.x >> 5;
  __shared__ float acc[32][33];
  float s = 0.0f;
  if (col < a.cols) {
#pragma unroll 8
    for (int64_t i = part; i < a.nparts; i += 32) s += p[i * a.cols + col];
  }
  acc[part][threadIdx.x & 31] = s;
  __syncthreads();
  if (part == 0 && col < a.cols) {
    s = 0.0f;
    for (int k = 0; k < 32; ++k) s += acc[k][threadIdx.x];
    out[col] = a.accumulate ? out[col] + s : s;
  }
}

template <typename T, int LANES, int WAVES, int NCH>
void norm_fwd(const NormArgs& a, hipStream_t s) {
  constexpr int kRows = norm_block<WAVES>() / (WAVES * LANES);
  k_norm_forward<T, LANES, WAVES, NCH>
      <<<dim3((unsigned)((a.rows + kRows - 1) / kRows)), dim3(norm_block<WAVES>()), 0, s>>>(a);
}
template <typename T, bool CK, int LANES, int WAVES, int NCH, int GROUPS>
void norm_bwd_of(const NormArgs& a, hipStream_t s) {
  const dim3 g((unsigned)a.nparts), b(WAVES * GROUPS * 64);
  if (a.cols % 8 == 0) k_norm_backward<T, CK, false, LANES, WAVES, NCH, GROUPS><<<g, b, 0, s>>>(a);
  else k_norm_backward<T, CK, true, LANES, WAVES, NCH, GROUPS><<<g, b, 0, s>>>(a);
}
template <typename T, int LANES, int WAVES, int NCH, int GROUPS>
void norm_bwd(const NormArgs& a, hipStream_t s) {
  if (a.x != nullptr) norm_bwd_of<T, false, LANES, WAVES, NCH, GROUPS>(a, s);
  else norm_bwd_of<T, true, LANES, WAVES, NCH, GROUPS>(a, s);
}

template <typename T>
void norm_fwd_any(const NormArgs& a, hipStream_t s) {
  if (a.cols <= 128) norm_fwd<T, 16, 1, 1>(a, s);
  else if (a.cols <= 256) norm_fwd<T, 32, 1, 1>(a, s);
  else if (a.cols <= 512) norm_fwd<T, 64, 1, 1>(a, s);
  else if (a.cols <= 1024) norm_fwd<T, 64, 1, 2>(a, s);
  else if (a.cols <= 2048) norm_fwd<T, 64, 1, 4>(a, s);
  else if (a.cols <= 4096) norm_fwd<T, 64, 4, 2>(a, s);
  else if (a.cols <= 8192) norm_fwd<T, 64, 4, 4>(a, s);
  else if (a.cols <= 16384) norm_fwd<T, 64, 16, 2>(a, s);
  else norm_fwd<T, 64, 16, 4>(a, s);
}
// Waves of a row, pieces of a lane and rows side by side of the backward pass:
// one piece of 8 columns a lane wherever a workgroup can be wide enough (with
// two, the sums of the weight gradients take the registers of half the waves:
// 8,192 rows of 768 columns took 22 us against 15). At most 256 workgroups of
// wide rows (one per compute unit, whose partial sums are 3% of the traffic),
// 512 of narrow ones (32,000 rows of 1,024 columns from a checkpoint: 38 us
// against 43 with 256, 8,192 x 768: equal; the rule goes by the columns alone and
// loses where few rows of binary32 meet it: 2,000 x 1,000, 15 against 12).
int norm_rows(int64_t cols) {
  if (cols <= 512) return cols <= 128 ? 32 : (cols <= 256 ? 16 : 8);
  return cols <= 2048 ? 4 : (cols <= 4096 ? 2 : 1);
}

template <typename T>
void norm_bwd_any(const NormArgs& a, hipStream_t s) {
  if (a.cols <= 128) norm_bwd<T, 16, 1, 1, 8>(a, s);
  else if (a.cols <= 256) norm_bwd<T, 32, 1, 1, 8>(a, s);
  else if (a.cols <= 512) norm_bwd<T, 64, 1, 1, 8>(a, s);
  else if (a.cols <= 1024) norm_bwd<T, 64, 2, 1, 4>(a, s);
  else if (a.cols <= 2048) norm_bwd<T, 64, 4, 1, 4>(a, s);
  else if (a.cols <= 4096) norm_bwd<T, 64, 8, 1, 2>(a, s);
  else if (a.cols <= 8192) norm_bwd<T, 64, 16, 1, 1>(a, s);
  else if (a.cols <= 16384) norm_bwd<T, 64, 16, 2, 1>(a, s);
  else norm_bwd<T, 64, 16, 4, 1>(a, s);
}

constexpr int64_t kSlabUnits = (int64_t)1 << 30;

Units units_of(int64_t rows, int64_t cols) {
  const int64_t per_row = (cols + kGroup - 1) / kGroup * (kGroup / 8);
  return {(uint32_t)(rows * per_row), (uint32_t)per_row};
}
int64_t slab_rows(int64_t cols) {
  const int64_t per_row = (cols + kGroup - 1) / kGroup * (kGroup / 8);
  return per_row >= kSlabUnits ? 1 : kSlabUnits / per_row;
}

template <typename T>
hipError_t checkpoint_save(int64_t rows, int64_t cols, const T* x, int64_t ldx, CkptRef ck, hipStream_t s) {
  const int64_t slab = slab_rows(cols);
  for (;; rows -= slab) {
    const Units u = units_of(rows < slab ? rows : slab, cols);
    k_checkpoint_save<T><<<dim3((u.total + kCkBlock - 1) / kCkBlock), dim3(kCkBlock), 0, s>>>(u, cols, x, ldx, ck);
    if (rows <= slab) return hipGetLastError();
    x += slab * ldx;
    ck.codes += slab * ck.ld;
    ck.scales += slab * ck.ld_scales;
  }
}

template <typename T>
hipError_t checkpoint_load(int64_t rows, int64_t cols, CkptRef ck, T* out, int64_t ldout, hipStream_t s) {
  const int64_t slab = slab_rows(cols);
  for (;; rows -= slab) {
    const Units u = units_of(rows < slab ? rows : slab, cols);
    k_checkpoint_load<T><<<dim3((u.total + kCkBlock - 1) / kCkBlock), dim3(kCkBlock), 0, s>>>(u, cols, ck, out,
                                                                                             ldout);
    if (rows <= slab) return hipGetLastError();
    out += slab * ldout;
    ck.codes += slab * ck.ld;
    ck.scales += slab * ck.ld_scales;
  }
}

}  // namespace

hipError_t launch_checkpoint_save(int dtype, int64_t rows, int64_t cols, const void* x, int64_t ldx,
                                  const CkptRef& ck, hipStream_t s) {
  if (dtype == MSAMP_F32) return checkpoint_save(rows, cols, (const float*)x, ldx, ck, s);
  if (dtype == MSAMP_F16) return checkpoint_save(rows, cols, (const f16*)x, ldx, ck, s);
  return checkpoint_save(rows, cols, (const bf16*)x, ldx, ck, s);
}

hipError_t launch_checkpoint_load(int dtype, int64_t rows, int64_t cols, const CkptRef& ck, void* out, int64_t ldout,
                                  hipStream_t s) {
  if (dtype == MSAMP_F32) return checkpoint_load(rows, cols, ck, (float*)out, ldout, s);
  if (dtype == MSAMP_F16) return checkpoint_load(rows, cols, ck, (f16*)out, ldout, s);
  return checkpoint_load(rows, cols, ck, (bf16*)out, ldout, s);
}

hipError_t launch_norm_forward(int dtype, const NormArgs& all, hipStream_t s) {
  // at most 2^21 rows a launch: with up to 1024 threads a row, they stay below 2^32
  constexpr int64_t kSlab = (int64_t)1 << 21;
  const int64_t es = dtype == MSAMP_F32 ? 4 : 2;
  NormArgs a = all;
  for (int64_t done = 0; done < all.rows; done += kSlab) {
    a.rows = all.rows - done < kSlab ? all.rows - done : kSlab;
    if (dtype == MSAMP_F32) norm_fwd_any<float>(a, s);
    else if (dtype == MSAMP_F16) norm_fwd_any<f16>(a, s);
    else norm_fwd_any<bf16>(a, s);
    if (a.rows < kSlab) break;
    if (a.x != nullptr) a.x = (const char*)a.x + kSlab * a.ldx * es;
    a.ck.codes += kSlab * a.ck.ld;
    a.ck.scales += kSlab * a.ck.ld_scales;
    if (a.save.codes != nullptr) {
      a.save.codes += kSlab * a.save.ld;
      a.save.scales += kSlab * a.save.ld_scales;
    }
    a.y = (char*)a.y + kSlab * a.ldy * es;
    if (a.mean != nullptr) a.mean += kSlab;
    a.rstd += kSlab;
  }
  return hipGetLastError();
}

// One workgroup alone, which needs no second launch, walks over the rows of two,
// or over those of four where rows are narrow and end on a piece (8 x 768: 4.8 us
// alone against 6.6, 16 x 768: 6.2 against 6.6, 32 x 768: 8.9 against 6.6; 30 x 500:
// 8.9 against 7.5; 4 x 4,096: 6.4 against 7.9, 8 x 4,096: 8.5 against 7.9).
int64_t norm_backward_parts(int64_t rows, int64_t cols) {
  const int64_t g = norm_rows(cols), blocks = (rows + g - 1) / g;
  const int64_t alone = cols <= 1024 && cols % 8 == 0 ? 4 : 2, most = cols <= 1024 ? 512 : 256;
  if (blocks <= alone) return blocks > 0;
  return blocks < most ? blocks : most;
}

hipError_t launch_norm_backward(int dtype, const NormArgs& a, hipStream_t s) {
  if (dtype == MSAMP_F32) norm_bwd_any<float>(a, s);
  else if (dtype == MSAMP_F16) norm_bwd_any<f16>(a, s);
  else norm_bwd_any<bf16>(a, s);
  return hipGetLastError();
}

hipError_t launch_norm_reduce(const NormArgs& a, hipStream_t s) {
  k_norm_reduce<<<dim3((unsigned)((a.cols + 31) / 32), 2), dim3(1024), 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace msamp
