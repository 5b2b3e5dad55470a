// Sums, running sums and maxima over the 64 lanes of a wave by DPP moves.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w4 {

template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {   // 0 where no lane is named
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
}
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ uint64_t dpp_u64(uint64_t v) {
  return ((uint64_t)dpp_u32<CTRL, ROWS>((uint32_t)(v >> 32)) << 32) | dpp_u32<CTRL, ROWS>((uint32_t)v);
}
__device__ __forceinline__ uint64_t lane_u64(uint64_t v, int lane) {
  return ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), lane) << 32) |
         (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, lane);
}
template <typename V>   // of 8 bytes
__device__ __forceinline__ V lane_value(V v, int lane) {
  return __builtin_bit_cast(V, lane_u64(__builtin_bit_cast(uint64_t, v), lane));
}

// Inclusive sums of v (8 bytes) over the lanes: within rows of 16, then from the
// last lanes of the rows before.
template <typename V>
__device__ __forceinline__ V wave_scan(V v) {
#define W4_ADD(...) v += __builtin_bit_cast(V, dpp_u64<__VA_ARGS__>(__builtin_bit_cast(uint64_t, v)))
  W4_ADD(0x111);        // row_shr 1
  W4_ADD(0x112);        // row_shr 2
  W4_ADD(0x114);        // row_shr 4
  W4_ADD(0x118);        // row_shr 8
  W4_ADD(0x142, 0xA);   // row_bcast 15 into rows 1 and 3
  W4_ADD(0x143, 0xC);   // row_bcast 31 into rows 2 and 3
#undef W4_ADD
  return v;
}
template <typename V>
__device__ __forceinline__ V wave_sum(V v) { return lane_value(wave_scan(v), 63); }

__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = max(v, dpp_u32<0xB1>(v));
  return max(v, dpp_u32<0x4E>(v));
}
// of quads' maxima
__device__ __forceinline__ uint32_t wave_max_of_quads(uint32_t v) {
  v = max(v, dpp_u32<0x141>(v));
  v = max(v, dpp_u32<0x140>(v));
  return max(max((uint32_t)__builtin_amdgcn_readlane((int)v, 0), (uint32_t)__builtin_amdgcn_readlane((int)v, 16)),
             max((uint32_t)__builtin_amdgcn_readlane((int)v, 32), (uint32_t)__builtin_amdgcn_readlane((int)v, 48)));
}

}  // namespace w4
