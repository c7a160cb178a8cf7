// gfx950 (CDNA4) kernels of the low-rank adapters beside the output layer: a slot laid out for the
// kernels, and the product of hidden states with the adapters' down matrices. What the up
// matrices give is added by the layer's kernels before they round (wfst_layer.hip).
#include "wfst_score_device.h"

namespace wfst {

namespace {

template <typename AT>
__global__ __launch_bounds__(256) void k_adapter_load(Adapters a, int32_t slot, AdapterSource src)
{
    const size_t t0 = (size_t)blockIdx.x * blockDim.x + threadIdx.x, step = (size_t)gridDim.x * blockDim.x;
    if (t0 == 0) {
        a.ranks[slot] = src.rank;
        a.scales[slot] = src.scale;
    }
    const int nb = (src.rank + 15) / 16;
    AT *down = (AT *)a.down + (size_t)slot * a.rb * 16 * a.kp;
    for (size_t i = t0; i < (size_t)src.rank * a.kp; i += step) {
        const size_t j = i / a.kp, k = i % a.kp;
        down[i] = k < (size_t)a.K ? ((const AT *)src.down)[j * src.down_stride + k] : (AT)0.0f;
    }
    AT *up = (AT *)a.up + (size_t)slot * a.nt * a.rb * 256;
    for (size_t i = t0; i < (size_t)a.nt * nb * 256; i += step) {
        const size_t tile = i / 256 / nb, jb = i / 256 % nb, lane = i / 4 % 64;
        const size_t n = tile * kTileN + lane % 16, j = jb * 16 + lane / 16 * 4 + i % 4;
        up[(tile * a.rb + jb) * 256 + i % 256] =
            n < (size_t)a.N && j < (size_t)src.rank ? ((const AT *)src.up)[n * src.up_stride + j] : (AT)0.0f;
    }
}

__global__ void k_adapters_clear(Adapters a)
{
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i < a.slots) {
        a.ranks[i] = 0;
        a.scales[i] = 0.0f;
    }
}

// One wavefront for each row and rank.
template <typename XT, typename AT>
__global__ __launch_bounds__(256) void k_adapt_shrink(LayerCall c, int32_t K)
{
    const AdaptCall &ad = c.ad;
    const int lane = threadIdx.x & 63, R = ad.a.rb * 16;
    const int64_t n = (int64_t)c.M * R, step = (int64_t)gridDim.x * 4;
    for (int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); i < n; i += step) {
        const int64_t m = i / R;
        const int j = (int)(i - m * R);
        if (!row_active(c.rows, m)) continue;
        const int slot = row_adapter(ad, m);
        if (slot < 0) continue;
        float sum = 0.0f;
        if (j < ad.a.ranks[slot]) {
            const AT *w = (const AT *)ad.a.down + ((size_t)slot * R + j) * ad.a.kp;
            const XT *x = (const XT *)c.x + m * c.x_stride;
            for (int k = lane * 8; k < K; k += kWaveSize * 8) {
                float v[8];
                load_x<XT>(x, true, k, K, v);
                const Pack<AT, 8> p = *(const Pack<AT, 8> *)(w + k);
#pragma unroll
                for (int e = 0; e < 8; ++e) sum = fmaf(v[e], (float)p.v[e], sum);
            }
            sum = wave_sum_f(sum) * ad.a.scales[slot];
        }
        if (lane == 0) ad.h[i] = sum;
    }
}

template <typename XT>
hipError_t shrink(const LayerCall &c, int32_t K, hipStream_t s)
{
    const int64_t n = ((int64_t)c.M * c.ad.a.rb * 16 + 3) / 4;
    const dim3 g((unsigned)std::min<int64_t>(n, kMaxRowGrid)), b(256);
    if (c.ad.a.dtype == kF32) hipLaunchKernelGGL((k_adapt_shrink<XT, float>), g, b, 0, s, c, K);
    else if (c.ad.a.dtype == kF16) hipLaunchKernelGGL((k_adapt_shrink<XT, _Float16>), g, b, 0, s, c, K);
    else hipLaunchKernelGGL((k_adapt_shrink<XT, __bf16>), g, b, 0, s, c, K);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_adapters_clear(const Adapters &a, hipStream_t s)
{
    hipLaunchKernelGGL(k_adapters_clear, dim3((a.slots + 255) / 256), dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_adapter_load(const Adapters &a, int32_t slot, const AdapterSource &src, hipStream_t s)
{
    const size_t items = std::max<size_t>((size_t)src.rank * a.kp, (size_t)a.nt * ((src.rank + 15) / 16) * 256);
    const dim3 g((unsigned)std::max<size_t>(1, std::min<size_t>((items + 255) / 256, 4096))), b(256);
    if (a.dtype == kF32) hipLaunchKernelGGL(k_adapter_load<float>, g, b, 0, s, a, slot, src);
    else if (a.dtype == kF16) hipLaunchKernelGGL(k_adapter_load<_Float16>, g, b, 0, s, a, slot, src);
    else hipLaunchKernelGGL(k_adapter_load<__bf16>, g, b, 0, s, a, slot, src);
    return hipGetLastError();
}

hipError_t launch_adapt_shrink(const LayerCall &c, int32_t K, hipStream_t s)
{
    if (c.x_dtype == kF32) return shrink<float>(c, K, s);
    if (c.x_dtype == kF16) return shrink<_Float16>(c, K, s);
    return shrink<__bf16>(c, K, s);
}

}  // namespace wfst
