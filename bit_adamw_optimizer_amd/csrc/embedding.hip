// embedding.hip -- embedding lookup with scaling and its gradient by sorted
// tokens on gfx950. The definitions are in msamp.h.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "checkpoint.hpp"
#include "model.hpp"

namespace msamp {
namespace {

constexpr int kBlock = 256;
constexpr int64_t kMaxGroups = 1 << 20;  // workgroups of a launch; they walk over the rest

// --------------------------------------------------------------- lookup ---

// LANES neighbours take a row, 8 columns each at a time, 256 / LANES rows a
// workgroup. Bound by memory: the rows named are read, y is written past the
// caches.
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
// rows by itself, so neither pass has an order that could change.
constexpr int kSortBlock = 1024, kSortWaves = kSortBlock / 64;
constexpr int kMostIds = 512;   // ids of a workgroup: 16 counters each in LDS
constexpr int kAhead = 4;       // loads of 64 ids under way

struct Sorted {
  int32_t* order;  // [rows] row numbers, by id and then by number
  int32_t* first;  // [vocab + 1] where each id's rows start
  float* partial;  // [2 * pieces][cols]
};

int64_t sort_span(int64_t vocab) {
  const int64_t span = (vocab + 255) / 256;  // a workgroup for each compute unit
  return span < 16 ? 16 : span < kMostIds ? span : kMostIds;
}

template <typename F>
__device__ __forceinline__ void each_id(const void* ids, int bytes, int64_t lo, int64_t hi, int lane, F&& f) {
  for (int64_t r = lo; r < hi; r += 64 * kAhead) {
    int64_t id[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int64_t row = r + k * 64 + lane;
      id[k] = row < hi ? load_int(ids, bytes, row) : -1;
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) f(r + k * 64 + lane, id[k]);
  }
}

__global__ __launch_bounds__(kSortBlock) void k_sort(EmbeddingArgs a, int span, Sorted out) {
  __shared__ int32_t count[kSortWaves][kMostIds];
  __shared__ int32_t start[kMostIds];
  __shared__ int32_t before[kSortWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t lo = (int64_t)blockIdx.x * span;
  const int64_t ids = a.vocab - lo < span ? a.vocab - lo : span;
  for (int i = threadIdx.x; i < kSortWaves * kMostIds; i += kSortBlock) (&count[0][0])[i] = 0;
  __syncthreads();
  const int64_t run = ((a.rows + kSortWaves - 1) / kSortWaves + 63) / 64 * 64;
  const int64_t r0 = wave * run, r1 = r0 + run < a.rows ? r0 + run : a.rows;
  int32_t smaller = 0;
  each_id(a.ids, a.id_bytes, r0, r1, lane, [&](int64_t, int64_t id) {
    smaller += id >= 0 && id < lo;
    if (id >= lo && id < lo + ids) atomicAdd(&count[wave][id - lo], 1);
  });
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) smaller += __shfl_xor(smaller, off, 64);
  if (lane == 0) before[wave] = smaller;
  __syncthreads();
  // counters into starting places: first within the range (one wave), then each wave's within its id
  if (wave == 0) {
    int32_t base = 0;
    for (int w = 0; w < kSortWaves; ++w) base += before[w];
    for (int i0 = 0; i0 < ids; i0 += 64) {
      const int i = i0 + lane;
      int32_t n = 0;
      if (i < ids)
        for (int w = 0; w < kSortWaves; ++w) n += count[w][i];
      int32_t sum = n;
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const int32_t up = __shfl_up(sum, off, 64);
        if (lane >= off) sum += up;
      }
      if (i < ids) {
        start[i] = base + sum - n;
        out.first[lo + i] = base + sum - n;
      }
      base += __shfl(sum, 63, 64);
    }
    if (lane == 0 && lo + ids == a.vocab) out.first[a.vocab] = base;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < ids; i += kSortBlock) {
    int32_t at = start[i];
    for (int w = 0; w < kSortWaves; ++w) {
      const int32_t n = count[w][i];
      count[w][i] = at;
      at += n;
    }
  }
  __syncthreads();
  int bits = 0;
  while ((1 << bits) < span) ++bits;
  each_id(a.ids, a.id_bytes, r0, r1, lane, [&](int64_t row, int64_t id) {
    const bool mine = id >= lo && id < lo + ids;
    uint64_t same = __ballot(mine);
    if (same == 0) return;  // the whole wave
    const int local = mine ? (int)(id - lo) : 0;
    for (int b = 0; b < bits; ++b) {
      const uint64_t set = __ballot(mine && ((local >> b) & 1));
      same &= (local >> b) & 1 ? set : ~set;
    }
    // the first lane of each id takes places for all of them
    const int leader = mine ? __ffsll((unsigned long long)same) - 1 : lane;
    int32_t at = 0;
    if (mine && lane == leader) at = atomicAdd(&count[wave][local], (int32_t)__popcll(same));
    at = __shfl(at, leader, 64);
    if (mine) out.order[at + __popcll(same & ((1ull << lane) - 1))] = (int32_t)row;
  });
}

// -------------------------------------------------------------- gradient ---

// Rows of one id beyond which its sum is cut into pieces of so many sorted
// rows each: what one workgroup may have to add up alone. Longer for many
// rows, so that the join has no more than about 1,024 pieces to add.
__host__ __device__ inline int64_t piece_rows(int64_t rows) {
  int64_t n = 64;
  while (n * 1024 < rows) n *= 2;
  return n;
}

// Sum over sorted rows [p0, p1) of dy's columns [col, col + 4).
template <typename T>
__device__ __forceinline__ void load4(const T* p, int n, float* f) {
  if (n >= 4) {
    if constexpr (sizeof(T) == 4) {
      const u32x4 v = *(const GLOBAL u32x4_any*)p;
#pragma unroll
      for (int k = 0; k < 4; ++k) f[k] = __uint_as_float(v[k]);
    } else {
      typedef T t4 __attribute__((ext_vector_type(4)));
      const t4 v = __builtin_bit_cast(t4, (u32x2) * (const GLOBAL u32x2_any*)p);
#pragma unroll
      for (int k = 0; k < 4; ++k) f[k] = to_f32(v[k]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = k < n ? to_f32(((const GLOBAL T*)p)[k]) : 0.0f;
  }
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

template <typename T>
__device__ __forceinline__ void sum_rows(const EmbeddingArgs& a, const int32_t* order, int64_t p0, int64_t p1,
                                         int64_t col, int n, float* f) {
  constexpr int U = 4;
  int64_t p = p0;
  for (; p + U <= p1; p += U) {
    int32_t r[U];
    float v[U][4];
#pragma unroll
    for (int u = 0; u < U; ++u) r[u] = ((const GLOBAL int32_t*)order)[p + u];
#pragma unroll
    for (int u = 0; u < U; ++u) load4((const T*)a.dy + r[u] * a.lddy + col, n, v[u]);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < 4; ++k) f[k] += v[u][k];
  }
  for (; p < p1; ++p) {
    float v[4];
    load4((const T*)a.dy + ((const GLOBAL int32_t*)order)[p] * a.lddy + col, n, v);
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] += v[k];
  }
}

// Parts of the ids with more than 'piece' rows: sorted rows [p * piece, (p + 1)
// * piece) hold the end of at most one of them (slot 2p) and the start of at
// most one (2p + 1).
template <typename T>
__global__ __launch_bounds__(kBlock) void k_pieces(EmbeddingArgs a, Sorted s, int64_t piece, int64_t pieces) {
  const int64_t col = ((int64_t)blockIdx.y * kBlock + threadIdx.x) * 4;
  const int n = (int)(a.cols - col < 4 ? a.cols - col : 4);
  const int64_t total = s.first[a.vocab];
  for (int64_t p = blockIdx.x; p < pieces; p += gridDim.x) {
    const int64_t p0 = p * piece, p1 = p0 + piece < total ? p0 + piece : total;
    if (p0 >= p1) return;
    const int64_t head = load_int(a.ids, a.id_bytes, s.order[p0]);
    const int64_t tail = load_int(a.ids, a.id_bytes, s.order[p1 - 1]);
    const int64_t head0 = s.first[head], head1 = s.first[head + 1], tail0 = s.first[tail], tail1 = s.first[tail + 1];
    if (n <= 0) continue;
    if (head1 - head0 > piece) {
      float f[4] = {};
      sum_rows<T>(a, s.order, p0, head1 < p1 ? head1 : p1, col, n, f);
      store4(s.partial + 2 * p * a.cols + col, n, f);
    }
    if (tail != head && tail1 - tail0 > piece) {
      float f[4] = {};
      sum_rows<T>(a, s.order, tail0, p1, col, n, f);
      store4(s.partial + (2 * p + 1) * a.cols + col, n, f);
    }
  }
}

// LANES neighbours take a row of dweight, 4 columns each at a time; an id of
// no row is most of the work: zeros to write, or nothing when accumulating.
template <typename T, int LANES>
__global__ __launch_bounds__(kBlock) void k_embedding_backward(EmbeddingArgs a, Sorted s, int64_t piece) {
  constexpr int kRows = kBlock / LANES;
  const int lane = threadIdx.x % LANES;
  for (int64_t v = (int64_t)blockIdx.x * kRows + threadIdx.x / LANES; v < a.vocab; v += (int64_t)gridDim.x * kRows) {
    const int64_t p0 = s.first[v], p1 = s.first[v + 1];
    if (p0 == p1 && a.accumulate) continue;
    float* out = a.dweight + v * a.ld_dweight;
    for (int64_t col = lane * 4; col < a.cols; col += LANES * 4) {
      const int n = (int)(a.cols - col < 4 ? a.cols - col : 4);
      float f[4] = {};
      if (p1 - p0 <= piece) {
        sum_rows<T>(a, s.order, p0, p1, col, n, f);
      } else {
        const int64_t q0 = p0 / piece, q1 = (p1 + piece - 1) / piece;
        for (int64_t q = q0; q < q1; ++q) {
          float t[4];
          load4(s.partial + (2 * q + (q * piece < p0 ? 1 : 0)) * a.cols + col, n, t);
#pragma unroll
          for (int k = 0; k < 4; ++k) f[k] += t[k];
        }
      }
      if (a.accumulate) {
        float t[4];
        load4(out + col, n, t);
#pragma unroll
        for (int k = 0; k < 4; ++k) f[k] = __builtin_fmaf(f[k], a.scale, t[k]);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) f[k] *= a.scale;
      }
      store4(out + col, n, f);
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
  s.first = (int32_t*)((char*)ws + round16(4 * a.rows));
  s.partial = (float*)((char*)s.first + round16(4 * (a.vocab + 1)));
  return s;
}

template <typename T>
hipError_t backward(const EmbeddingArgs& a, void* ws, hipStream_t s) {
  const Sorted st = sorted(a, ws);
  const int64_t piece = piece_rows(a.rows), pieces = pieces_of(a.rows);
  if (pieces > 0) {
    const dim3 grid((unsigned)(pieces < 65536 ? pieces : 65536), (unsigned)((a.cols + 4 * kBlock - 1) / (4 * kBlock)));
    k_pieces<T><<<grid, kBlock, 0, s>>>(a, st, piece, pieces);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  auto run = [&](auto lanes) -> hipError_t {
    constexpr int L = decltype(lanes)::value;
    const int64_t groups = (a.vocab + kBlock / L - 1) / (kBlock / L);
    k_embedding_backward<T, L><<<(unsigned)(groups < kMaxGroups ? groups : kMaxGroups), kBlock, 0, s>>>(a, st, piece);
    return hipGetLastError();
  };
  const int64_t units = (a.cols + 3) / 4;
  if (units <= 8) return run(std::integral_constant<int, 8>());
  if (units <= 32) return run(std::integral_constant<int, 32>());
  if (units <= 64) return run(std::integral_constant<int, 64>());
  return run(std::integral_constant<int, 256>());
}

}  // namespace

hipError_t launch_embedding_forward(int dtype, const EmbeddingArgs& a, hipStream_t s) {
  return dtype == MSAMP_F32 ? forward<float>(a, s) : dtype == MSAMP_F16 ? forward<f16>(a, s) : forward<bf16>(a, s);
}

int64_t embedding_workspace(int64_t rows, int64_t vocab, int64_t cols) {
  return round16(4 * rows) + round16(4 * (vocab + 1)) + 2 * pieces_of(rows) * cols * 4;
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
