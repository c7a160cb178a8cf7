// The output layer with 4-bit weights: its arrays laid out, its workspace, and the choice of its
// kernels (wfst_layer_kernels.h).
#include "wfst_layer_kernels.h"

namespace wfst {

namespace {

// The caller's weights, scales and zeros into the layer's tiles; features past
// K hold q = 0 (their x is 0), features past N and groups past K scale 0.
template <typename ST>
__global__ __launch_bounds__(256) void k_layer_pack(Layer l, LayerSource src, uint4 *w, ST *scales, uint8_t *zeros,
                                                     float *bias)
{
    const size_t nthreads = (size_t)gridDim.x * blockDim.x;
    const size_t t0 = (size_t)blockIdx.x * blockDim.x + threadIdx.x;
    const size_t rowb = ((size_t)l.K + 1) / 2;
    for (size_t i = t0; i < (size_t)l.nt * l.kb * kWaveSize; i += nthreads) {
        const int lane = (int)(i & 63);
        const size_t tile = i >> 6;
        const int kb = (int)(tile % l.kb);
        const size_t n = (tile / l.kb) * kTileN + (lane & 15);
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int k0 = kb * kTileK + j * 32 + (lane >> 4) * 8;
            uint32_t v = 0;
            if (n < (size_t)l.N && k0 + 8 <= l.K) {
                // four bytes at once: their low halves to bits 0 .. 15, their high halves to 16 .. 31
                struct __attribute__((packed, aligned(1))) Word { uint32_t w; };
                uint32_t b = ((const Word *)(src.w + n * rowb + k0 / 2))->w;
                uint32_t lo = b & 0x0F0F0F0Fu, hi = (b >> 4) & 0x0F0F0F0Fu;
                lo = (lo | lo >> 4) & 0x00FF00FFu;
                hi = (hi | hi >> 4) & 0x00FF00FFu;
                v = ((lo | lo >> 8) & 0xFFFFu) | (hi | hi >> 8) << 16;
            } else {
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    const int k = k0 + 2 * p;
                    uint32_t byte = 0;
                    if (n < (size_t)l.N && k < l.K) byte = src.w[n * rowb + k / 2];
                    if (k + 1 >= l.K) byte &= 15u;
                    v |= (byte & 15u) << (4 * p) | (byte >> 4) << (16 + 4 * p);
                }
            }
            o[j] = v;
        }
        w[i] = make_uint4(o[0], o[1], o[2], o[3]);
    }
    const size_t ngroups = (l.K + (size_t)l.group - 1) / l.group;
    for (size_t i = t0; i < (size_t)l.nt * l.kb * kTileN * l.gpt; i += nthreads) {
        const int sub = (int)(i % l.gpt);
        const size_t tile = i / l.gpt / kTileN;
        const size_t n = tile / l.kb * kTileN + i / l.gpt % kTileN;
        const size_t k = tile % l.kb * kTileK + sub * (kTileK / l.gpt);
        const size_t g = k / l.group;
        const bool in = n < (size_t)l.N && g < ngroups;
        scales[i] = in ? ((const ST *)src.scales)[n * ngroups + g] : (ST)0.0f;
        if (zeros) zeros[i] = in ? (src.zeros[n * ngroups + g] & 15u) : 8;
    }
    if (bias)
        for (size_t i = t0; i < (size_t)l.N; i += nthreads) bias[i] = src.bias[i];
}

}  // namespace

hipError_t launch_layer_pack(const Layer &l, const LayerSource &src, uint4 *w, void *scales, uint8_t *zeros,
                             float *bias, hipStream_t s)
{
    const size_t items = (size_t)l.nt * l.kb * kWaveSize;
    const dim3 g((unsigned)std::min<size_t>((items + 255) / 256, 8192)), b(256);
    if (l.scale_dtype == kF32)
        hipLaunchKernelGGL(k_layer_pack<float>, g, b, 0, s, l, src, w, (float *)scales, zeros, bias);
    else if (l.scale_dtype == kF16)
        hipLaunchKernelGGL(k_layer_pack<_Float16>, g, b, 0, s, l, src, w, (_Float16 *)scales, zeros, bias);
    else
        hipLaunchKernelGGL(k_layer_pack<__bf16>, g, b, 0, s, l, src, w, (__bf16 *)scales, zeros, bias);
    return hipGetLastError();
}

AdaptBytes adapt_bytes(const Adapters &a, int32_t rows)
{
    // (groups of 16 to 64 rows, up to 4 lists each)
    const size_t r64 = ((size_t)rows + 63) / 64 * 64, r16 = ((size_t)rows + 15) / 16;
    return {r16 * a.rb * h_block_bytes(a.dtype), 4 * r64 * a.rb * sizeof(uint4), 4 * r16 * sizeof(int32_t)};
}

size_t layer_workspace(const Layer &l, int32_t rows, int32_t x_dtype)
{
    if (!many_tiles(l, rows, x_dtype)) return 0;
    const size_t blocks = (size_t)((rows + kRowsM - 1) / kRowsM) * l.kb;
    return operand_bytes(l, rows, x_dtype) + (x_dtype == kF16 ? 0 : blocks * kRowsM * 4);
}

hipError_t launch_layer(const Layer &l, const LayerCall &c, hipStream_t s)
{
    if (c.x_dtype == kF32) return launch_layer_f32(l, c, s);
    if (c.x_dtype == kF16) return launch_layer_f16(l, c, s);
    return launch_layer_bf16(l, c, s);
}

}  // namespace wfst
