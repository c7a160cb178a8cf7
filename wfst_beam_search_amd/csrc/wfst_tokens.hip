// gfx950 (CDNA4) kernels of the scores of given tokens: log-probability and rank of each, the
// distribution's entropy, the best alternatives.
#include "wfst_score_device.h"

namespace wfst {

namespace {

// m = max x, d = (x - m) / T, S = sum exp d, lz = log S:
// log-probability d - lz, entropy lz - (sum exp(d) d) / S.
constexpr int kThreads = 256;

struct Totals { float m, ones, sum, wsum; bool nan; };

__device__ __forceinline__ uint64_t order_key(float x, int32_t v)
{
    const uint32_t u = __float_as_uint(x + 0.0f);                     // (one zero)
    return (uint64_t)(u & 0x80000000u ? ~u : u | 0x80000000u) << 32 | (uint32_t)~v;
}

__device__ __forceinline__ float key_score(uint64_t k)
{
    const uint32_t u = (uint32_t)(k >> 32);
    return __uint_as_float(u & 0x80000000u ? u & 0x7FFFFFFFu : ~u);
}

template <typename F>
__device__ __forceinline__ float block_reduce(float v, float *red, F join)
{
    __syncthreads();
    for (int d = 32; d >= 1; d >>= 1) v = join(v, __shfl_xor(v, d, 64));
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    return join(join(red[0], red[1]), join(red[2], red[3]));
}

template <typename XT>
__global__ __launch_bounds__(kThreads) void k_token_scores(TokenCall c)
{
    __shared__ float red[4];
    __shared__ uint64_t kred[4];
    const int tid = threadIdx.x;
    const auto add = [](float a, float b) { return a + b; };
    const auto max2 = [](float a, float b) { return fmaxf(a, b); };
    for (int64_t r = blockIdx.x; r < c.rows; r += gridDim.x) {
        if (!row_active(c.set, r)) continue;
        const XT *x = (const XT *)c.x + r * c.x_stride;
        float t = c.temperatures ? c.temperatures[r] : c.temperature;
        t = t > 0.0f ? fminf(t, 3.402823466e38f) : 0.0f;
        float m = -INFINITY, bad = 0.0f;
        for (int v = tid; v < c.V; v += kThreads) {
            const float z = (float)x[v];
            bad = z != z || z == INFINITY ? 1.0f : bad;
            m = fmaxf(m, z);
        }
        m = block_reduce(m, red, max2);
        bad = block_reduce(bad, red, max2);
        // where z - m could pass binary32's range, half of it times 2 / T
        const float half = m > 0x1p100f ? 0.5f : 1.0f, inv = 1.0f / (fmaxf(t, 0x1p-125f) * half);
        float ones = 0.0f, sum = 0.0f, wsum = 0.0f;
        if (bad == 0.0f && m > -INFINITY && t > 0.0f)
            for (int v = tid; v < c.V; v += kThreads) {
                const float z = (float)x[v], d = fmaf(z, half, -m * half) * inv;
                if (z == m) { ones += 1.0f; continue; }
                const float e = expf(d);
                sum += e;
                if (e > 0.0f) wsum += e * d;
            }
        ones = block_reduce(ones, red, add);
        sum = block_reduce(sum, red, add);
        wsum = block_reduce(wsum, red, add);
        const float lz = bad != 0.0f ? NAN : m == -INFINITY || t == 0.0f ? 0.0f : log1pf((ones - 1.0f) + sum);
        const auto log_prob = [&](float z, int rank) {
            if (lz != lz) return NAN;
            if (!(z > -INFINITY)) return -INFINITY;
            return t == 0.0f ? (rank == 0 ? 0.0f : -INFINITY) : fmaf(z, half, -m * half) / t / half - lz;
        };
        if (tid == 0 && c.entropies) c.entropies[r] = lz == 0.0f ? lz : lz - wsum / (ones + sum);
        for (int i = 0; i < c.C; ++i) {
            const int tok = c.tokens[r * c.C + i];
            if (tok < 0 || tok >= c.V) {
                if (tid == 0) { c.log_probs[r * c.C + i] = -INFINITY; c.ranks[r * c.C + i] = -1; }
                continue;
            }
            float zt = (float)x[tok];
            if (zt != zt) zt = -INFINITY;
            float before = 0.0f;
            for (int v = tid; v < c.V; v += kThreads) {
                float z = (float)x[v];
                if (z != z) z = -INFINITY;
                if (z > zt || (z == zt && v < tok)) before += 1.0f;
            }
            before = block_reduce(before, red, add);
            if (tid == 0) { c.log_probs[r * c.C + i] = log_prob(zt, (int)before); c.ranks[r * c.C + i] = (int)before; }
        }
        uint64_t last = ~0ull;
        for (int i = 0; i < c.top_n; ++i) {
            uint64_t best = 0;
            for (int v = tid; v < c.V; v += kThreads) {
                const float z = (float)x[v];
                const uint64_t k = z > -INFINITY ? order_key(z, v) : 0;
                if (k < last && k > best) best = k;
            }
            for (int d = 32; d >= 1; d >>= 1) {
                const uint64_t o = __shfl_xor((unsigned long long)best, d, 64);
                best = o > best ? o : best;
            }
            __syncthreads();
            if ((tid & 63) == 0) kred[tid >> 6] = best;
            __syncthreads();
            for (int w = 0; w < 4; ++w) best = kred[w] > best ? kred[w] : best;
            last = best;
            if (tid == 0) {
                c.top_tokens[r * c.top_n + i] = best ? (int32_t)~(uint32_t)best : -1;
                c.top_log_probs[r * c.top_n + i] = best ? log_prob(key_score(best), i) : -INFINITY;
            }
        }
        __syncthreads();
    }
}

}  // namespace

size_t token_workspace(int64_t, int32_t, int32_t, int32_t, int32_t) { return 0; }

hipError_t launch_token_scores(const TokenCall &c, hipStream_t s)
{
    const dim3 g((unsigned)std::min<int64_t>(c.rows, kMaxRowGrid)), b(kThreads);
    if (c.x_dtype == kF32) hipLaunchKernelGGL(k_token_scores<float>, g, b, 0, s, c);
    else if (c.x_dtype == kF16) hipLaunchKernelGGL(k_token_scores<_Float16>, g, b, 0, s, c);
    else hipLaunchKernelGGL(k_token_scores<__bf16>, g, b, 0, s, c);
    return hipGetLastError();
}

}  // namespace wfst
