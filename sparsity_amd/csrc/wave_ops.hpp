// Values of other lanes of a wave without a way through LDS.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace bl {

// v of the lane that a DPP control names, `id` where there is none or the row mask leaves the lane out.
template <int CTRL, int ROWS, class T>
__device__ __forceinline__ T lane_move(T v, T id) {
  if constexpr (sizeof(T) == 8) {
    const uint2 x = __builtin_bit_cast(uint2, v), y = __builtin_bit_cast(uint2, id);
    const uint2 z = {(uint32_t)__builtin_amdgcn_update_dpp((int)y.x, (int)x.x, CTRL, ROWS, 0xF, false),
                     (uint32_t)__builtin_amdgcn_update_dpp((int)y.y, (int)x.y, CTRL, ROWS, 0xF, false)};
    return __builtin_bit_cast(T, z);
  } else {
    return __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, id), __builtin_bit_cast(int, v),
                                                             CTRL, ROWS, 0xF, false));
  }
}
// op over the lanes up to each one (id: what changes nothing), in registers: within rows of 16 lanes, then over
// them.  The order is fixed.
template <class T, class Op>
__device__ __forceinline__ T wave_scan(T v, T id, Op op) {
  v = op(lane_move<0x111, 0xF>(v, id), v);   // 1, 2, 4, 8 lanes up the row
  v = op(lane_move<0x112, 0xF>(v, id), v);
  v = op(lane_move<0x114, 0xF>(v, id), v);
  v = op(lane_move<0x118, 0xF>(v, id), v);
  v = op(lane_move<0x142, 0xA>(v, id), v);   // last lane of a row to the next one
  v = op(lane_move<0x143, 0xC>(v, id), v);   // of the lower half to the upper
  return v;
}
template <class T>
__device__ __forceinline__ T lane_value(T v, int lane) {
  if constexpr (sizeof(T) == 8) {
    const uint2 x = __builtin_bit_cast(uint2, v);
    const uint2 z = {(uint32_t)__builtin_amdgcn_readlane((int)x.x, lane), (uint32_t)__builtin_amdgcn_readlane((int)x.y, lane)};
    return __builtin_bit_cast(T, z);
  } else {
    return __builtin_bit_cast(T, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
  }
}
template <class T, class Op>
__device__ __forceinline__ T wave_all(T v, T id, Op op) {
  return lane_value(wave_scan(v, id, op), 63);
}

}  // namespace bl
