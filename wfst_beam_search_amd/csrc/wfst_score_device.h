// Device helpers of the operators around the search. Not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>

#include "wfst_score.h"

namespace wfst {

namespace {

constexpr int kWaveSize = 64;
constexpr unsigned kMaxRowGrid = 1u << 18;      // workgroups of a launch over rows

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef float float4_t __attribute__((ext_vector_type(4)));

// N consecutive elements at any element alignment, as one load or store.
template <typename T, int N> struct __attribute__((packed, aligned(sizeof(T)))) Pack { T v[N]; };

__device__ __forceinline__ bool row_active(const RowSet &s, int64_t r)
{
    if (!s.lengths) return true;
    const int64_t b = r / s.T;
    return (int32_t)(r - b * s.T) < s.lengths[b];
}

// Reductions over a wavefront by data-parallel moves (all 64 lanes active): four
// steps inside rows of 16 lanes, two across rows, the result read from lane 63.
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_f(float id, float v)
{
    return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(id), __float_as_int(v), CTRL, ROWS, 0xf, false));
}

__device__ __forceinline__ float wave_max_f(float v)
{
    const float id = -INFINITY;
    v = fmaxf(v, dpp_f<0x111, 0xf>(id, v));
    v = fmaxf(v, dpp_f<0x112, 0xf>(id, v));
    v = fmaxf(v, dpp_f<0x114, 0xf>(id, v));
    v = fmaxf(v, dpp_f<0x118, 0xf>(id, v));
    v = fmaxf(v, dpp_f<0x142, 0xa>(id, v));
    v = fmaxf(v, dpp_f<0x143, 0xc>(id, v));
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

__device__ __forceinline__ float wave_sum_f(float v)
{
    v += dpp_f<0x111, 0xf>(0.0f, v);
    v += dpp_f<0x112, 0xf>(0.0f, v);
    v += dpp_f<0x114, 0xf>(0.0f, v);
    v += dpp_f<0x118, 0xf>(0.0f, v);
    v += dpp_f<0x142, 0xa>(0.0f, v);
    v += dpp_f<0x143, 0xc>(0.0f, v);
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

}  // namespace

}  // namespace wfst
