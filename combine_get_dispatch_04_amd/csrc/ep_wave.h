// ep_wave.h -- device helpers that the router's and the adapters' kernels share.
#pragma once

#include "ep_common.h"

namespace ep {

// Two fp32 values to bf16, nearest even, for any input: a NaN stays one (the
// integer form in ep_common.h, for finite values, could carry its payload away).
__device__ __forceinline__ uint32_t pack_bf16_any(float lo, float hi)
{
    typedef __bf16 b16x2 __attribute__((ext_vector_type(2)));
    const b16x2 v = {(__bf16)lo, (__bf16)hi};
    return __builtin_bit_cast(uint32_t, v);
}

constexpr float kNegInf = -__builtin_huge_valf();

// Row shifts inside 16 lanes, then the row broadcasts, as in
// wave_inclusive_scan: lane 63 ends up with all 64 lanes' value.  The order
// of the additions is fixed, so sums are the same for every run.
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_f(float old, float v)
{
    return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(
        (int)__float_as_uint(old), (int)__float_as_uint(v), CTRL, ROWS, 0xF, false));
}
__device__ __forceinline__ float last_lane(float v)
{
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}
__device__ __forceinline__ float lane_value(float v, int lane)
{
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), lane));
}
__device__ __forceinline__ float wave_sum_f(float v)
{
    v += dpp_f<0x111, 0xF>(0.0f, v);
    v += dpp_f<0x112, 0xF>(0.0f, v);
    v += dpp_f<0x114, 0xF>(0.0f, v);
    v += dpp_f<0x118, 0xF>(0.0f, v);
    v += dpp_f<0x142, 0xA>(0.0f, v);
    v += dpp_f<0x143, 0xC>(0.0f, v);
    return last_lane(v);
}
__device__ __forceinline__ float wave_max_f(float v)
{
    v = fmaxf(v, dpp_f<0x111, 0xF>(kNegInf, v));
    v = fmaxf(v, dpp_f<0x112, 0xF>(kNegInf, v));
    v = fmaxf(v, dpp_f<0x114, 0xF>(kNegInf, v));
    v = fmaxf(v, dpp_f<0x118, 0xF>(kNegInf, v));
    v = fmaxf(v, dpp_f<0x142, 0xA>(kNegInf, v));
    v = fmaxf(v, dpp_f<0x143, 0xC>(kNegInf, v));
    return last_lane(v);
}

}  // namespace ep
