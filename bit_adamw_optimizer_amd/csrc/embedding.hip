// embedding.hip -- embedding lookup with scaling and its gradient by sorted
// tokens on gfx950. The definitions are in msamp.h.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "checkpoint.hpp"
#include "model.hpp"

namespace msamp {
namespace {

constexpr int kBlock = 256;
constexpr int64_t kMaxGroups = 1 << 20;  // workgroups of a launch

// --------------------------------------------------------------- lookup ---

// LANES neighbours take a row, 8 columns each at a time, 256 / LANES rows a
// workgroup. Bound by memory: the rows named are read, y is written past the
// caches; 16,384 rows of 4,096 bfloat16 columns with the frequencies of a text
// take 31.6 us (5.7 TB/s), 16 rows of 768 2.6 us.
template <typename T, int LANES>
__global__ __launch_bounds__(kBlock) void k_embedding_forward(EmbeddingArgs a) {
  constexpr int kRows = kBlock / LANES;
  const int lane = threadIdx.x % LANES;
  for (int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / LANES; row < a.rows;
       row += (int64_t)gridDim.x * kRows) {
    const int64_t id = load_int(a.ids, a.id_bytes, row);
    const bool live = id >= 0 && id < a.vocab;
    const T* w = (const T*)a.weight + (live ? id : 0) * a.ldw;
    T* y = (T*)a.y + row * a.ldy;
    for (int64_t col = lane * 8; col < a.cols; col += LANES * 8) {
      const int n = (int)(a.cols - col < 8 ? a.cols - col : 8);
      float f[8];
      if (live) {
        load8(w + col, n, f);
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] *= a.scale;
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = 0.0f;
      }
      store8<T, true>(y + col, n, f);
    }
  }
}

// The fewest lanes that hold a row, up to 64 with 8 columns each; measured, us, against the neighbouring sizes
// (2^26 bfloat16 elements, ids spread evenly): 64 columns 12 with 8 lanes, 23 with 32; 256 columns 40 with 32, 50 with
// 64; 512 columns 40 with 64, 54 with 256; 1,024 columns 43 with 256, 40 with 64; 4,096 columns 40 and 42.
template <typename T>
hipError_t forward(const EmbeddingArgs& a, hipStream_t s) {
  auto run = [&](auto lanes) -> hipError_t {
    constexpr int L = decltype(lanes)::value;
    const int64_t groups = (a.rows + kBlock / L - 1) / (kBlock / L);
    k_embedding_forward<T, L><<<(unsigned)(groups < kMaxGroups ? groups : kMaxGroups), kBlock, 0, s>>>(a);
    return hipGetLastError();
  };
  const int64_t units = (a.cols + 7) / 8;
  if (units <= 8) return run(std::integral_constant<int, 8>());
  if (units <= 32) return run(std::integral_constant<int, 32>());
  if (units <= 64) return run(std::integral_constant<int, 64>());
  return run(std::integral_constant<int, 256>());
}

// ----------------------------------------------------------------- sort ---

// Ids are cut into ranges of 'span', one to a workgroup, so that no workgroup
// waits for another: each goes through all rows, its 16 waves through 16 runs
// of consecutive rows, first counting the rows of each of its ids (and the rows
// of all smaller ids, where its output starts), then placing the rows' numbers
// by id, in their order. Two ids' counters never meet, and a wave places its
// rows by itself, so neither pass has an order that could change. Every
// workgroup reads all ids, from cache: 13 us for 16,384 rows, 9 us for 5,003,
// most of it latency (ids in two passes over memory, one load after another:
// 20 us). The work grows with rows times workgroups, and beyond 16,384 rows ids
// are read twice: 43 us for 65,536 rows, of 32,000 ids as of 131,072.
constexpr int kSortBlock = 1024, kSortWaves = kSortBlock / 64;
constexpr int kMostIds = 512;   // ids of a workgroup: 16 counters each in LDS
constexpr int kAhead = 16;      // loads of 64 ids under way

struct Sorted {
  int32_t* order;  // [rows] row numbers, by id and then by number
  int32_t* key;    // [rows] their ids
  int32_t* first;  // [vocab + 1] where each id's rows start
  float* partial;  // [2 * pieces][cols]
};

int64_t sort_span(int64_t vocab) {
  const int64_t span = (vocab + 255) / 256;  // a workgroup for each compute unit
  return span < kMostIds ? span : kMostIds;
}

// kAhead times 64 ids from row r on, one of 64 neighbours to a lane; -1 from
// row 'end' on and for those that name nothing. Through a buffer, whose bounds
// need no branch around each load, so that all of them are under way at once.
__device__ __forceinline__ void load_ids(const EmbeddingArgs& a, int64_t r, int64_t end, int lane, int32_t* id) {
  const int rows = (int)(end - r < 64 * kAhead ? end - r : 64 * kAhead);
  const auto b = __builtin_amdgcn_make_buffer_rsrc((char*)const_cast<void*>(a.ids) + r * a.id_bytes, 0,
                                                   rows * a.id_bytes, 0x00020000);
  if (a.id_bytes == 8) {
    u32x2 v[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      v[k] = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(b, (k * 64 + lane) * 8, 0, 0));
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      id[k] = k * 64 + lane < rows && v[k].y == 0 && v[k].x < (uint64_t)a.vocab ? (int32_t)v[k].x : -1;
  } else {
    uint32_t v[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) v[k] = __builtin_amdgcn_raw_buffer_load_b32(b, (k * 64 + lane) * 4, 0, 0);
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      id[k] = k * 64 + lane < rows && v[k] < (uint64_t)a.vocab ? (int32_t)v[k] : -1;
  }
}

__global__ __launch_bounds__(kSortBlock) void k_sort(EmbeddingArgs a, int span, Sorted out) {
  __shared__ int32_t count[kSortWaves][kMostIds];
  __shared__ int32_t before[kSortWaves];
  __shared__ int32_t sums[kMostIds / 64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t lo = (int32_t)blockIdx.x * span;
  const int32_t ids = a.vocab - lo < span ? (int32_t)a.vocab - lo : span;
  const int64_t run = ((a.rows + kSortWaves - 1) / kSortWaves + 63) / 64 * 64;
  const int64_t r0 = wave * run, r1 = r0 + run < a.rows ? r0 + run : a.rows;
  const bool once = run <= 64 * kAhead;  // the ids stay in registers
  int32_t id[kAhead];
  if (once && r0 < r1) load_ids(a, r0, r1, lane, id);
  for (int w = 0; w < kSortWaves; ++w)
    if (threadIdx.x < span) count[w][threadIdx.x] = 0;
  __syncthreads();
  int32_t smaller = 0;
  for (int64_t r = r0; r < r1; r += 64 * kAhead) {
    if (!once) load_ids(a, r, r1, lane, id);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      smaller += id[k] >= 0 && id[k] < lo;
      const int32_t i = id[k] - lo;
      if (i >= 0 && i < ids) atomicAdd(&count[wave][i], 1);
    }
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) smaller += __shfl_xor(smaller, off, 64);
  if (lane == 0) before[wave] = smaller;
  __syncthreads();
  // counters into starting places: of the waves within an id, of the ids within the range
  const int32_t i = threadIdx.x;
  int32_t n[kSortWaves], sum = 0;
  if (wave < kMostIds / 64) {
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) n[w] = i < ids ? count[w][i] : 0;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) sum += n[w];
    const int32_t own = sum;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int32_t up = __shfl_up(sum, off, 64);
      if (lane >= off) sum += up;
    }
    if (lane == 63) sums[wave] = sum;
    sum -= own;
  }
  __syncthreads();
  if (wave < kMostIds / 64) {
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) sum += before[w];
#pragma unroll
    for (int w = 0; w < kMostIds / 64; ++w) sum += w < wave ? sums[w] : 0;
    if (i < ids) out.first[lo + i] = sum;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      if (i < ids) count[w][i] = sum;
      sum += n[w];
    }
    if (i == ids - 1 && lo + ids == a.vocab) out.first[a.vocab] = sum;
  }
  __syncthreads();
  for (int64_t r = r0; r < r1; r += 64 * kAhead) {
    if (!once) load_ids(a, r, r1, lane, id);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int32_t local = id[k] - lo;
      const bool mine = local >= 0 && local < ids;
      // the lanes of each id in turn, few where most rows are of other ranges
      uint64_t left = __ballot(mine);
      if (left == 0) continue;  // the whole wave
      uint64_t same = 0;
      int leader = lane;
      while (left != 0) {
        const int one = __ffsll((unsigned long long)left) - 1;
        const uint64_t these = __ballot(mine && local == __builtin_amdgcn_readlane(local, one));
        if ((these >> lane) & 1) same = these, leader = one;
        left &= ~these;
      }
      // the first lane of each id takes places for all of them
      int32_t at = 0;
      if (mine && lane == leader) at = atomicAdd(&count[wave][local], (int32_t)__popcll(same));
      at = __shfl(at, leader, 64);
      if (mine) {
        at += __popcll(same & ((1ull << lane) - 1));
        out.order[at] = (int32_t)(r + k * 64 + lane);
        out.key[at] = lo + local;
      }
    }
  }
}

// -------------------------------------------------------------- gradient ---

// Rows of one id beyond which its sum is cut into pieces of so many sorted
// rows each: what one workgroup may have to add up alone. Longer for many
// rows, so that the join has no more than about 1,024 pieces to add.
__host__ __device__ inline int64_t piece_rows(int64_t rows) {
  int64_t n = 16;
  while (n * 1024 < rows) n *= 2;
  return n;
}

// Four consecutive elements as they lie in memory, n (<= 4) of them from p.
template <typename T>
struct Raw4 {
  uint32_t w[sizeof(T)];
};
template <typename T>
__device__ __forceinline__ Raw4<T> raw4(const T* p, int n) {
  if (n >= 4) {
    if constexpr (sizeof(T) == 4) return __builtin_bit_cast(Raw4<T>, (u32x4) * (const GLOBAL u32x4_any*)p);
    else return __builtin_bit_cast(Raw4<T>, (u32x2) * (const GLOBAL u32x2_any*)p);
  }
  struct V {
    T v[4];
  } v;
#pragma unroll
  for (int k = 0; k < 4; ++k) v.v[k] = k < n ? ((const GLOBAL T*)p)[k] : (T)0.0f;
  return __builtin_bit_cast(Raw4<T>, v);
}
template <typename T>
__device__ __forceinline__ void values4(const Raw4<T>& r, float* f) {
  struct V {
    T v[4];
  };
  const V v = __builtin_bit_cast(V, r);
#pragma unroll
  for (int k = 0; k < 4; ++k) f[k] = to_f32(v.v[k]);
}
template <typename T>
__device__ __forceinline__ void load4(const T* p, int n, float* f) {
  values4(raw4(p, n), f);
}

__device__ __forceinline__ void store4(float* p, int n, const float* f) {
  if (n >= 4) {
    u32x4 v;
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = __float_as_uint(f[k]);
    *(GLOBAL u32x4_any*)p = v;
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < n) ((GLOBAL float*)p)[k] = f[k];
  }
}

// Adds dy's columns col[c] of sorted rows [p0, p1), in their order, U rows'
// loads under way at a time. WAVE: p0 and p1 are the whole wave's, whose lanes
// load 64 rows' numbers at once and read them from each other: all 64 have to
// come here, those without columns (n <= 0, nothing is loaded for them) too.
template <typename T, int CH, int U, bool WAVE>
__device__ __forceinline__ void sum_rows(const EmbeddingArgs& a, const int32_t* order, int64_t p0, int64_t p1,
                                         int64_t col, int step, const int* n, float (*f)[4]) {
  const int lane = threadIdx.x & 63;
  for (int64_t p = p0; p < p1; p += WAVE ? 64 : U) {
    int32_t mine = 0;
    if (WAVE && p + lane < p1) mine = ((const GLOBAL int32_t*)order)[p + lane];
    const int rows = (int)(p1 - p < (WAVE ? 64 : U) ? p1 - p : (WAVE ? 64 : U));
    auto at = [&](int i) {
      const int32_t r = WAVE ? __builtin_amdgcn_readlane(mine, i) : ((const GLOBAL int32_t*)order)[p + i];
      return (const T*)a.dy + (int64_t)r * a.lddy + col;
    };
    auto add = [&](const Raw4<T>& v, float* sum) {
      float x[4];
      values4(v, x);
#pragma unroll
      for (int k = 0; k < 4; ++k) sum[k] += x[k];
    };
    int u0 = 0;
    for (; u0 + 1 < rows; u0 += U) {  // behind the last row: the last row again, not added
      Raw4<T> v[U][CH];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const T* row = at(u0 + u < rows ? u0 + u : rows - 1);
#pragma unroll
        for (int c = 0; c < CH; ++c) v[u][c] = raw4(row + c * step, n[c]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (u0 + u < rows) {
#pragma unroll
          for (int c = 0; c < CH; ++c) add(v[u][c], f[c]);
        }
    }
    if (u0 < rows) {
      const T* row = at(u0);
#pragma unroll
      for (int c = 0; c < CH; ++c) add(raw4(row + c * step, n[c]), f[c]);
    }
  }
}

// Parts of the ids with more than 'piece' rows: sorted rows [p * piece, (p + 1)
// * piece) hold the end of at most one of them (slot 2p) and the start of at
// most one (2p + 1).
template <typename T>
__global__ __launch_bounds__(kBlock) void k_pieces(EmbeddingArgs a, Sorted s, int64_t piece) {
  const int64_t col = ((int64_t)blockIdx.y * kBlock + threadIdx.x) * 4;
  const int n = (int)(a.cols - col < 4 ? a.cols - col : 4);
  const int64_t p = blockIdx.x, p0 = p * piece;
  int64_t p1 = p0 + piece < a.rows ? p0 + piece : a.rows;
  const int64_t total = s.first[a.vocab];
  const int32_t head = s.key[p0];
  int32_t tail = s.key[p1 - 1];  // of the rows sorted; what lies behind them is not used
  if (p0 >= total) return;
  if (p1 > total) {
    p1 = total;
    tail = s.key[p1 - 1];
  }
  const int64_t head0 = s.first[head], head1 = s.first[head + 1], tail0 = s.first[tail], tail1 = s.first[tail + 1];
  if (head1 - head0 > piece) {
    float f[1][4] = {};
    sum_rows<T, 1, 16, true>(a, s.order, p0, head1 < p1 ? head1 : p1, col, 0, &n, f);
    store4(s.partial + 2 * p * a.cols + col, n, f[0]);
  }
  if (tail != head && tail1 - tail0 > piece) {
    float f[1][4] = {};
    sum_rows<T, 1, 16, true>(a, s.order, tail0, p1, col, 0, &n, f);
    store4(s.partial + (2 * p + 1) * a.cols + col, n, f[0]);
  }
}

// LANES neighbours take a row of dweight, CH times 4 columns each at a time. An
// id of no row is most of the work: zeros to write. 32,000 x 4,096 from 16,384
// rows, 524 MB of it, take 126 us (of no rows 89 us, 5.9 TB/s); with the dy of a
// row loaded column by column, or unpacked where it is loaded (138 registers),
// 250 us. BY_ROW: a workgroup's rows
// are found from sorted rows that are the first of their id, so that ids of no
// row (which accumulating leaves alone) are not looked at.
template <typename T, int LANES, int CH, bool BY_ROW>
__global__ __launch_bounds__(kBlock) void k_embedding_backward(EmbeddingArgs a, Sorted s, int64_t piece, int64_t group0) {
  constexpr int kRows = kBlock / LANES, kStep = LANES * 4;
  constexpr bool kWave = LANES >= 64;
  const int lane = threadIdx.x % LANES;
  int64_t v = (group0 + blockIdx.x) * kRows + threadIdx.x / LANES;
  if (BY_ROW) {
    if (v >= a.rows) return;
    const int64_t total = s.first[a.vocab];
    const int32_t id = s.key[v], before = v > 0 ? s.key[v - 1] : -1;
    if (v >= total || id == before) return;
    v = id;
  } else if (v >= a.vocab) {
    return;
  }
  int32_t q0 = s.first[v], q1 = s.first[v + 1];
  if (kWave) q0 = __builtin_amdgcn_readfirstlane(q0), q1 = __builtin_amdgcn_readfirstlane(q1);
  const int64_t p0 = q0, p1 = q1;
  float* out = a.dweight + v * a.ld_dweight;
  // a wave stays together while it has columns, its lanes behind the last one too (sum_rows)
  const int in_wave = kWave ? lane & 63 : lane;
  for (int64_t first = lane - in_wave; first * 4 < a.cols; first += CH * LANES) {
    const int64_t col = (first + in_wave) * 4;
    int n[CH];
    float f[CH][4] = {};
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int64_t left = a.cols - (col + c * kStep);
      n[c] = left < 0 ? 0 : left < 4 ? (int)left : 4;
    }
    if (p1 - p0 <= piece) {
      sum_rows<T, CH, (CH == 1 ? 8 : 4) * 2 / (int)sizeof(T), kWave>(a, s.order, p0, p1, col, kStep, n, f);
    } else {
      const int64_t k0 = p0 / piece, k1 = (p1 + piece - 1) / piece;
#pragma unroll(CH == 1 ? 16 : 4)
      for (int64_t q = k0; q < k1; ++q) {
        const float* part = s.partial + (2 * q + (q * piece < p0 ? 1 : 0)) * a.cols + col;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          float t[4];
          load4(part + c * kStep, n[c], t);
#pragma unroll
          for (int k = 0; k < 4; ++k) f[c][k] += t[k];
        }
      }
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (BY_ROW) {
        float t[4];
        load4(out + col + c * kStep, n[c], t);
#pragma unroll
        for (int k = 0; k < 4; ++k) f[c][k] = __builtin_fmaf(f[c][k], a.scale, t[k]);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) f[c][k] *= a.scale;
      }
      store4(out + col + c * kStep, n[c], f[c]);
    }
  }
}

int64_t round16(int64_t bytes) { return (bytes + 15) / 16 * 16; }

int64_t pieces_of(int64_t rows) {
  const int64_t piece = piece_rows(rows);
  return rows > piece ? (rows + piece - 1) / piece : 0;
}

Sorted sorted(const EmbeddingArgs& a, void* ws) {
  Sorted s;
  s.order = (int32_t*)ws;
  s.key = (int32_t*)((char*)ws + round16(4 * a.rows));
  s.first = (int32_t*)((char*)s.key + round16(4 * a.rows));
  s.partial = (float*)((char*)s.first + round16(4 * (a.vocab + 1)));
  return s;
}

template <typename T>
hipError_t backward(const EmbeddingArgs& a, void* ws, hipStream_t s) {
  const Sorted st = sorted(a, ws);
  const int64_t piece = piece_rows(a.rows), pieces = pieces_of(a.rows);
  if (pieces > 0) {
    const dim3 grid((unsigned)pieces, (unsigned)((a.cols + 4 * kBlock - 1) / (4 * kBlock)));
    k_pieces<T><<<grid, kBlock, 0, s>>>(a, st, piece);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  auto run = [&](auto lanes, auto chunks) -> hipError_t {
    constexpr int L = decltype(lanes)::value, CH = decltype(chunks)::value, R = kBlock / L;
    const int64_t groups = ((a.accumulate ? a.rows : a.vocab) + R - 1) / R;
    for (int64_t g = 0; g < groups; g += kMaxGroups) {
      const unsigned n = (unsigned)(groups - g < kMaxGroups ? groups - g : kMaxGroups);
      if (a.accumulate) k_embedding_backward<T, L, CH, true><<<n, kBlock, 0, s>>>(a, st, piece, g);
      else k_embedding_backward<T, L, CH, false><<<n, kBlock, 0, s>>>(a, st, piece, g);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  };
  // lanes and columns a lane that hold a row, up to 4,096 columns at a time; us against the neighbouring sizes (the
  // forward rows' gradient into 2^27 elements): 32 columns 202 with 8 lanes, 301 with 32; 128 columns 288 with 32, 279
  // with 64; 256 columns 319, with 64 x 2 303; 512 columns 243 with 64 x 2, 332 x 1, 337 x 4; 1,024 columns 182 with 64
  // x 4, 166 x 2, 267 with 128 x 4; 2,048 columns 160 with 128 x 4, 156 with 64, 227 with 256; 4,096 columns 143 with
  // 256 x 4, 145 with 128
  const int64_t units = (a.cols + 3) / 4;
  using std::integral_constant;
  if (units <= 8) return run(integral_constant<int, 8>(), integral_constant<int, 1>());
  if (units <= 32) return run(integral_constant<int, 32>(), integral_constant<int, 1>());
  if (units <= 64) return run(integral_constant<int, 64>(), integral_constant<int, 1>());
  if (units <= 128) return run(integral_constant<int, 64>(), integral_constant<int, 2>());
  if (units <= 256) return run(integral_constant<int, 64>(), integral_constant<int, 4>());
  if (units <= 512) return run(integral_constant<int, 128>(), integral_constant<int, 4>());
  return run(integral_constant<int, 256>(), integral_constant<int, 4>());
}

}  // namespace

hipError_t launch_embedding_forward(int dtype, const EmbeddingArgs& a, hipStream_t s) {
  return dtype == MSAMP_F32 ? forward<float>(a, s) : dtype == MSAMP_F16 ? forward<f16>(a, s) : forward<bf16>(a, s);
}

int64_t embedding_workspace(int64_t rows, int64_t vocab, int64_t cols) {
  return 2 * round16(4 * rows) + round16(4 * (vocab + 1)) + 2 * pieces_of(rows) * cols * 4;
}

hipError_t launch_embedding_sort(const EmbeddingArgs& a, void* ws, hipStream_t s) {
  const int span = (int)sort_span(a.vocab);
  k_sort<<<(unsigned)((a.vocab + span - 1) / span), kSortBlock, 0, s>>>(a, span, sorted(a, ws));
  return hipGetLastError();
}

hipError_t launch_embedding_backward(int dtype, const EmbeddingArgs& a, void* ws, hipStream_t s) {
  return dtype == MSAMP_F32 ? backward<float>(a, ws, s)
                            : dtype == MSAMP_F16 ? backward<f16>(a, ws, s) : backward<bf16>(a, ws, s);
}

}  // namespace msamp
