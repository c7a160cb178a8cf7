// gfx950 (CDNA4) kernels that lay a low-rank adapter out in its slot. The products run beside the
// output layer's (wfst_adapters_device.h, wfst_layer_kernels.h).
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

}  // namespace wfst
