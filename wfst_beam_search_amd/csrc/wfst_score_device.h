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

// The same for a call of fewer than 2^32 rows (a division of 64 bits takes some 100
// instructions).
__device__ __forceinline__ bool row_active32(const RowSet &s, uint32_t r)
{
    if (!s.lengths) return true;
    const uint32_t b = r / (uint32_t)s.T;
    return (int32_t)(r - b * (uint32_t)s.T) < s.lengths[b];
}

// The adapter slot of row r of a call, -1: none.
__device__ __forceinline__ int row_adapter(const AdaptCall &ad, int64_t r)
{
    const int s = ad.ids[(uint32_t)r / (uint32_t)ad.per_id];
    return s >= 0 && s < ad.a.slots && ad.a.ranks[s] > 0 ? s : -1;
}

// N consecutive elements at any element alignment, as one load or store.
template <typename T, int N> struct __attribute__((packed, aligned(sizeof(T)))) Pack { T v[N]; };

__device__ __forceinline__ bool row_active(const RowSet &s, int64_t r)
{
    if (!s.lengths) return true;
    const int64_t b = r / s.T;
    return (int32_t)(r - b * s.T) < s.lengths[b];
}

// x[k .. k+7] of a row of K features (0 past them, and for a row that is not there).
template <typename XT>
__device__ __forceinline__ void load_x(const XT *row, bool there, int k, int K, float (&v)[8])
{
    if (there && k + 8 <= K) {
        const Pack<XT, 8> p = *(const Pack<XT, 8> *)(row + k);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = (float)p.v[j];
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = there && k + j < K ? (float)row[k + j] : 0.0f;
    }
}

// Reductions over a wavefront by data-parallel moves (all 64 lanes active): four
// steps inside rows of 16 lanes, two across rows, the result read from lane 63.
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_f(float id, float v)
{
    return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(id), __float_as_int(v), CTRL, ROWS, 0xf, false));
}

template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_i(int v)
{
    return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xf, false);
}

__device__ __forceinline__ int wave_sum_i(int v)
{
    v += dpp_i<0x111, 0xf>(v);
    v += dpp_i<0x112, 0xf>(v);
    v += dpp_i<0x114, 0xf>(v);
    v += dpp_i<0x118, 0xf>(v);
    v += dpp_i<0x142, 0xa>(v);
    v += dpp_i<0x143, 0xc>(v);
    return __builtin_amdgcn_readlane(v, 63);
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
