// lanes.hpp -- sums over the lanes of a wave, without LDS. Internal.
#pragma once

#include <hip/hip_runtime.h>

namespace msamp {

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

}  // namespace msamp
