// gfx950 (CDNA4) kernels of the operators around the search: the output layer
// with 4-bit weights (hidden states to logits), the log-softmax (logits to the
// log-posteriors the search reads) and the draw of tokens from scores.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "wfst_score.h"

namespace wfst {

namespace {

constexpr int kWaveSize = 64;

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef float float4_t __attribute__((ext_vector_type(4)));

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

template <typename T>
__device__ __forceinline__ T wave_sum_t(T v)
{
#pragma unroll
    for (int d = kWaveSize / 2; d >= 1; d >>= 1) v += __shfl_xor(v, d, kWaveSize);
    return v;
}

// ---------------------------------------------------------------- output layer
//
// y[m, n] = bias[n] + sum_g s[n, g] * sum_{k in g} (q[n, k] - z[n, g]) x[m, k]
//
// Each wavefront owns 16 output features and up to 16 rows of x and runs
// v_mfma_f32_16x16x32_f16 with x as the left operand and the weights as the
// right one, so the lane that unpacks feature n's weights also receives n's
// sums and needs n's scale and zero alone. A weight is unpacked exactly: a mask
// puts two 4-bit values into the mantissas of two halves 1024 + q (or 1024 +
// 16 q), and one packed subtraction (or multiply-add by 1/16) of the zero point
// leaves q - z, an integer in [-15, 15]. Sums inside a group are the matrix
// unit's binary32 sums of exact products; a group's sum is multiplied by its
// scale in binary32 and added to the row's sum.
//
// x enters the matrix unit as binary16. bfloat16 and binary32 rows are scaled
// by a power of two per 128 features so that the block's largest finite value
// lies in [2^14, 2^15): a bfloat16 value then fits binary16 exactly or, 2^29
// below the block's largest, loses less than 2^-39 of that; a binary32 value is
// cut into a sum of two binary16 values (off by at most 2^-24 of itself, or
// 2^-39 of the block's largest).

constexpr int kLayerWaves = 4;
constexpr int kLayerThreads = kLayerWaves * kWaveSize;
constexpr int kRowsM = 16;
constexpr int kChunk = 512;                    // features of x staged at a time
constexpr int kXStride = kChunk + 8;           // halves; 16 bytes of padding keep the 16 rows on distinct banks

template <typename T> __device__ __forceinline__ float load_scale(const void *p, size_t i)
{
    return (float)((const T *)p)[i];
}

// The power of two that brings |x| <= mx into [2^14, 2^15), as its exponent.
__device__ __forceinline__ int block_exponent(float mx)
{
    if (!(mx > 0.0f)) return 0;
    int e;
    (void)frexpf(mx, &e);                      // mx = f * 2^e, f in [0.5, 1)
    e -= 15;
    return e < -120 ? -120 : e;                // 2^e and its inverse stay normal
}

template <typename XT, typename OT, typename ST>
__global__ __launch_bounds__(kLayerThreads) void k_layer(Layer l, LayerCall c)
{
    constexpr int kParts = sizeof(XT) == 4 ? 2 : 1;
    constexpr bool kScaled = !__is_same(XT, _Float16);
    __shared__ __align__(16) _Float16 xs[kParts][kRowsM * kXStride];
    __shared__ __align__(16) float xf[kChunk / kTileK][kRowsM];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int nt = blockIdx.x * kLayerWaves + wave;
    const int m0 = blockIdx.y * kRowsM;
    const int col = lane & 15, quad = lane >> 4;
    const bool live = nt < l.nt;
    float4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};

    for (int k0 = 0; k0 < l.K; k0 += kChunk) {
        __syncthreads();
        // stage x[m0 .. m0+15][k0 .. k0+511]: 16 consecutive threads take one row's 128 features
        for (int i = tid; i < kRowsM * (kChunk / 8); i += kLayerThreads) {
            const int r = i / (kChunk / 8), seg = i - r * (kChunk / 8);
            const int k = k0 + seg * 8, m = m0 + r;
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = (m < c.M && k + j < l.K) ? (float)((const XT *)c.x)[(int64_t)m * c.x_stride + k + j] : 0.0f;
            int e = 0;
            if (kScaled) {
                float mx = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float a = fabsf(v[j]);
                    mx = fmaxf(mx, a < INFINITY ? a : 0.0f);
                }
#pragma unroll
                for (int d = 8; d >= 1; d >>= 1) mx = fmaxf(mx, __shfl_xor(mx, d, 16));
                e = block_exponent(mx);
                if ((seg & 15) == 0) xf[seg >> 4][r] = ldexpf(1.0f, e);
            }
            half8_t hi, lo;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float s = kScaled ? ldexpf(v[j], -e) : v[j];
                hi[j] = (_Float16)s;
                const float d = s - (float)hi[j];
                lo[j] = (_Float16)(fabsf(s) < INFINITY ? d : 0.0f);   // (an infinity or NaN is in hi alone)
            }
            *(half8_t *)&xs[0][r * kXStride + seg * 8] = hi;
            if (kParts == 2) *(half8_t *)&xs[kParts - 1][r * kXStride + seg * 8] = lo;
        }
        __syncthreads();
        if (!live) continue;
        const int kb0 = k0 / kTileK, kbn = min(kChunk / kTileK, l.kb - kb0);
        for (int b = 0; b < kbn; ++b) {
            const uint4 w4 = l.w[((size_t)nt * l.kb + kb0 + b) * kWaveSize + lane];
            const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
            float4_t f = {1.0f, 1.0f, 1.0f, 1.0f};
            if (kScaled) f = *(const float4_t *)&xf[b][quad * 4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int k = (kb0 + b) * kTileK + j * 32;
                if (k >= l.K) break;
                const int g = k / l.group;
                const size_t gi = ((size_t)nt * l.ngroups + g) * kTileN + col;
                const float s = load_scale<ST>(l.scales, gi);
                const int z = l.zeros ? l.zeros[gi] : 8;
                const half2_t z0 = {(_Float16)(float)(-1024 - z), (_Float16)(float)(-1024 - z)};
                const half2_t z1 = {(_Float16)(float)(-64 - z), (_Float16)(float)(-64 - z)};
                const half2_t r16 = {(_Float16)0.0625f, (_Float16)0.0625f};
                union { uint32_t u[4]; half2_t h[4]; half8_t v; } q;
                const uint32_t w8 = w[j] >> 8;
                q.u[0] = (w[j] & 0x000F000Fu) | 0x64006400u;
                q.u[1] = (w[j] & 0x00F000F0u) | 0x64006400u;
                q.u[2] = (w8 & 0x000F000Fu) | 0x64006400u;
                q.u[3] = (w8 & 0x00F000F0u) | 0x64006400u;
                q.h[0] += z0;
                q.h[2] += z0;
                q.h[1] = __builtin_elementwise_fma(q.h[1], r16, z1);
                q.h[3] = __builtin_elementwise_fma(q.h[3], r16, z1);
                float4_t part = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int p = 0; p < kParts; ++p) {
                    const half8_t a = *(const half8_t *)&xs[p][col * kXStride + b * kTileK + j * 32 + quad * 8];
                    part = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, q.v, part, 0, 0, 0);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[i] = fmaf(part[i], kScaled ? s * f[i] : s, acc[i]);
            }
        }
    }
    const int n = nt * kTileN + col;
    if (!live || n >= l.N) return;
    const float bias = l.bias ? l.bias[n] : 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int m = m0 + quad * 4 + i;
        if (m < c.M && row_active(c.rows, m)) ((OT *)c.out)[(int64_t)m * c.out_stride + n] = (OT)(acc[i] + bias);
    }
}

// The caller's weights, scales and zeros into the layer's tiles; features past
// K hold q = 0 (their x is 0) and features past N scale 0.
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
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const int k = k0 + 2 * p;
                uint32_t byte = 0;
                if (n < (size_t)l.N && k < l.K) byte = src.w[n * rowb + k / 2];
                if (k + 1 >= l.K) byte &= 15u;
                v |= (byte & 15u) << (4 * p) | (byte >> 4) << (16 + 4 * p);
            }
            o[j] = v;
        }
        w[i] = make_uint4(o[0], o[1], o[2], o[3]);
    }
    for (size_t i = t0; i < (size_t)l.nt * l.ngroups * kTileN; i += nthreads) {
        const size_t g = (i / kTileN) % l.ngroups;
        const size_t n = i / kTileN / l.ngroups * kTileN + i % kTileN;
        const bool in = n < (size_t)l.N;
        scales[i] = in ? ((const ST *)src.scales)[n * l.ngroups + g] : (ST)0.0f;
        if (zeros) zeros[i] = in ? (src.zeros[n * l.ngroups + g] & 15u) : 8;
    }
    if (bias)
        for (size_t i = t0; i < (size_t)l.N; i += nthreads) bias[i] = src.bias[i];
}

template <typename XT, typename OT>
hipError_t layer_st(const Layer &l, const LayerCall &c, hipStream_t s)
{
    const dim3 g((l.nt + kLayerWaves - 1) / kLayerWaves, (c.M + kRowsM - 1) / kRowsM), b(kLayerThreads);
    if (l.scale_dtype == kF32) hipLaunchKernelGGL((k_layer<XT, OT, float>), g, b, 0, s, l, c);
    else if (l.scale_dtype == kF16) hipLaunchKernelGGL((k_layer<XT, OT, _Float16>), g, b, 0, s, l, c);
    else hipLaunchKernelGGL((k_layer<XT, OT, __bf16>), g, b, 0, s, l, c);
    return hipGetLastError();
}

template <typename XT>
hipError_t layer_ot(const Layer &l, const LayerCall &c, hipStream_t s)
{
    if (c.out_dtype == kF32) return layer_st<XT, float>(l, c, s);
    if (c.out_dtype == kF16) return layer_st<XT, _Float16>(l, c, s);
    return layer_st<XT, __bf16>(l, c, s);
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

hipError_t launch_layer(const Layer &l, const LayerCall &c, hipStream_t s)
{
    if (c.x_dtype == kF32) return layer_ot<float>(l, c, s);
    if (c.x_dtype == kF16) return layer_ot<_Float16>(l, c, s);
    return layer_ot<__bf16>(l, c, s);
}

// ---------------------------------------------------------------- log-softmax
//
// z = scale * x + bias, out = (z - max z) - log sum exp(z - max z), sums and
// statistics in binary32. The sum leaves the row's largest entries (each
// exactly 1) out and counts them, so that the logarithm of a row with one
// dominant label is log1p of a small number and keeps its digits. A row of
// -inf alone stays -inf; a row with +inf or NaN becomes NaN.

namespace {

constexpr unsigned kMaxRowGrid = 1u << 18;

// VEC consecutive elements at any element alignment, as one load or store.
template <typename T, int VEC> struct __attribute__((packed, aligned(sizeof(T)))) Pack { T v[VEC]; };

// Elements moved at once: 16 bytes of the wider of the two types.
template <typename A, typename B> constexpr int pack_len() { return 16 / (sizeof(A) > sizeof(B) ? sizeof(A) : sizeof(B)); }

// z of the VEC elements from v on (-inf past V).
template <typename XT, int VEC>
__device__ __forceinline__ void norm_load(const XT *x, const NormCall &c, int v, float (&z)[VEC])
{
    if (v + VEC <= c.V) {
        const Pack<XT, VEC> p = *(const Pack<XT, VEC> *)(x + v);
#pragma unroll
        for (int j = 0; j < VEC; ++j) z[j] = (float)p.v[j] * c.scale;
        if (c.bias) {
            const Pack<float, VEC> b = *(const Pack<float, VEC> *)(c.bias + v);
#pragma unroll
            for (int j = 0; j < VEC; ++j) z[j] += b.v[j];
        }
    } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            z[j] = -INFINITY;
            if (v + j < c.V) {
                z[j] = (float)x[v + j] * c.scale;
                if (c.bias) z[j] += c.bias[v + j];
            }
        }
    }
}

template <typename OT, int VEC>
__device__ __forceinline__ void norm_store(OT *o, int V, int v, const float (&y)[VEC])
{
    if (v + VEC <= V) {
        Pack<OT, VEC> p;
#pragma unroll
        for (int j = 0; j < VEC; ++j) p.v[j] = (OT)y[j];
        *(Pack<OT, VEC> *)(o + v) = p;
    } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j)
            if (v + j < V) o[v + j] = (OT)y[j];
    }
}

__device__ __forceinline__ float exp_diff(float d) { return __builtin_amdgcn_exp2f(d * 1.44269504088896341f); }

// Statistics of a set of z: the largest, how many equal it, and the sum of
// exp(z - largest) over the others. A NaN or +inf among the z makes the sum NaN
// (by itself, through z - largest), or the largest +inf where all else is -inf.
struct NormStat { float m, ones, sum; };

__device__ __forceinline__ NormStat norm_join(const NormStat &a, const NormStat &b)
{
    NormStat r;
    r.m = fmaxf(a.m, b.m);
    r.ones = (a.m == r.m ? a.ones : 0.0f) + (b.m == r.m ? b.ones : 0.0f);
    r.sum = 0.0f;
    if (r.m == INFINITY) {
        r.sum = NAN;
    } else if (r.m > -INFINITY) {
        r.sum += a.m == r.m ? a.sum : (a.sum + a.ones) * exp_diff(a.m - r.m);
        r.sum += b.m == r.m ? b.sum : (b.sum + b.ones) * exp_diff(b.m - r.m);
    }
    return r;
}

// out = (z - m) - lz of a row. A row of -inf alone is left as it is.
struct NormRow { float m, lz; };

__device__ __forceinline__ NormRow norm_row(const NormStat &s)
{
    NormRow r = {s.m, log1pf((s.ones - 1.0f) + s.sum)};
    if (s.m == -INFINITY) r = {0.0f, 0.0f};
    if (s.m == INFINITY) r = {0.0f, NAN};
    return r;
}

// Statistics of a row that WAVES wavefronts hold, NV packs a thread; red holds
// 3 * WAVES floats.
template <int VEC, int WAVES, int NV>
__device__ __forceinline__ NormStat norm_stats(const float (&z)[NV][VEC], float *red)
{
    const int wave = threadIdx.x >> 6;
    const bool first = (threadIdx.x & 63) == 0;
    NormStat s = {-INFINITY, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) s.m = fmaxf(s.m, z[i][j]);
    s.m = wave_max_f(s.m);
    if (WAVES > 1) {
        if (first) red[wave] = s.m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < WAVES; ++w) s.m = fmaxf(s.m, red[w]);
    }
    if (s.m > -INFINITY) {                            // (the same for all threads of the row)
        uint32_t ones = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float d = z[i][j] - s.m, e = exp_diff(d);
                const bool top = d == 0.0f;
                ones += __popcll(__ballot(top));      // (counted on the scalar unit)
                s.sum += top ? 0.0f : e;
            }
        s.ones = (float)ones;
    } else {
        bool nan = false;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) nan |= z[i][j] != z[i][j];
        s.sum = nan ? 1.0f : 0.0f;
    }
    s.sum = wave_sum_f(s.sum);
    if (WAVES > 1) {
        if (first) { red[WAVES + wave] = s.sum; red[2 * WAVES + wave] = s.ones; }
        __syncthreads();
        s.sum = s.ones = 0.0f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) { s.sum += red[WAVES + w]; s.ones += red[2 * WAVES + w]; }
    }
    if (s.m == -INFINITY && s.sum > 0.0f) s.m = INFINITY;
    return s;
}

// A row in the registers of WAVES wavefronts: read once, written once. A workgroup
// of one-wavefront rows holds four of them and no barrier.
template <typename XT, typename OT, int WAVES, int NV>
__global__ __launch_bounds__(WAVES == 1 ? 256 : WAVES * kWaveSize) void k_norm_row(NormCall c)
{
    constexpr int VEC = pack_len<XT, OT>();
    constexpr int kSpan = WAVES * kWaveSize * VEC;
    constexpr int kRows = WAVES == 1 ? 4 : 1;
    __shared__ float red[3 * WAVES];
    const int v0 = (WAVES == 1 ? (threadIdx.x & 63) : threadIdx.x) * VEC;
    const int64_t step = (int64_t)gridDim.x * kRows;
    for (int64_t r = (int64_t)blockIdx.x * kRows + (WAVES == 1 ? threadIdx.x >> 6 : 0); r < c.rows; r += step) {
        if (!row_active(c.set, r)) continue;
        const XT *x = (const XT *)c.x + r * c.x_stride;
        float z[NV][VEC];
#pragma unroll
        for (int i = 0; i < NV; ++i) norm_load<XT, VEC>(x, c, v0 + i * kSpan, z[i]);
        const NormRow n = norm_row(norm_stats<VEC, WAVES, NV>(z, red));
        OT *o = (OT *)c.out + r * c.out_stride;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float y[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) y[j] = (z[i][j] - n.m) - n.lz;
            if (v0 + i * kSpan < c.V) norm_store<OT, VEC>(o, c.V, v0 + i * kSpan, y);
        }
        if (WAVES > 1) __syncthreads();
    }
}

// Long or few rows, cut into pieces of 256 * VEC * kPieceNV elements: the first
// launch writes each piece's statistics, the second joins a row's and writes.
constexpr int kPieceWaves = 4;
constexpr int kPieceNV = 4;

template <typename XT, typename OT, bool WRITE>
__global__ __launch_bounds__(kPieceWaves *kWaveSize) void k_norm_piece(NormCall c, int pieces)
{
    constexpr int VEC = pack_len<XT, OT>();
    constexpr int kSpan = kPieceWaves * kWaveSize * VEC;
    __shared__ float red[3 * kPieceWaves];
    const int tid = threadIdx.x;
    NormStat *stats = (NormStat *)c.workspace;
    for (int64_t w = blockIdx.x; w < c.rows * pieces; w += gridDim.x) {
        const int64_t r = w / pieces;
        const int p = (int)(w - r * pieces);
        if (!row_active(c.set, r)) continue;
        const XT *x = (const XT *)c.x + r * c.x_stride;
        const int v0 = p * kSpan * kPieceNV + tid * VEC;
        float z[kPieceNV][VEC];
#pragma unroll
        for (int i = 0; i < kPieceNV; ++i) norm_load<XT, VEC>(x, c, v0 + i * kSpan, z[i]);
        if (!WRITE) {
            const NormStat s = norm_stats<VEC, kPieceWaves, kPieceNV>(z, red);
            if (tid == 0) stats[w] = s;
            __syncthreads();
            continue;
        }
        NormStat s = {-INFINITY, 0.0f, 0.0f};
        for (int q = tid & 63; q < pieces; q += kWaveSize) s = norm_join(s, stats[r * pieces + q]);
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) {
            const NormStat o = {__shfl_xor(s.m, d, 64), __shfl_xor(s.ones, d, 64), __shfl_xor(s.sum, d, 64)};
            s = norm_join(s, o);
        }
        const NormRow n = norm_row(s);
        OT *o = (OT *)c.out + r * c.out_stride;
#pragma unroll
        for (int i = 0; i < kPieceNV; ++i) {
            const int v = v0 + i * kSpan;
            float y[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) y[j] = (z[i][j] - n.m) - n.lz;
            if (v < c.V) norm_store<OT, VEC>(o, c.V, v, y);
        }
    }
}

// A row on 4 or 16 wavefronts, with just the packs it needs (a pack past the row
// costs its branch and registers: 5000 labels on 8 packs a thread instead of 5
// took 114 us instead of 92).
template <typename XT, typename OT>
void norm_wide(const NormCall &c, hipStream_t s)
{
    constexpr int kPack4 = 4 * kWaveSize * pack_len<XT, OT>();
    const dim3 g((unsigned)std::min<int64_t>(c.rows, kMaxRowGrid));
    switch ((c.V + kPack4 - 1) / kPack4) {
    case 1: case 2: case 3: hipLaunchKernelGGL((k_norm_row<XT, OT, 4, 3>), g, dim3(256), 0, s, c); break;
    case 4: hipLaunchKernelGGL((k_norm_row<XT, OT, 4, 4>), g, dim3(256), 0, s, c); break;
    case 5: hipLaunchKernelGGL((k_norm_row<XT, OT, 4, 5>), g, dim3(256), 0, s, c); break;
    case 6: hipLaunchKernelGGL((k_norm_row<XT, OT, 4, 6>), g, dim3(256), 0, s, c); break;
    case 7: case 8: hipLaunchKernelGGL((k_norm_row<XT, OT, 4, 8>), g, dim3(256), 0, s, c); break;
    case 9: case 10: case 11: case 12: hipLaunchKernelGGL((k_norm_row<XT, OT, 16, 3>), g, dim3(1024), 0, s, c); break;
    case 13: case 14: case 15: case 16: hipLaunchKernelGGL((k_norm_row<XT, OT, 16, 4>), g, dim3(1024), 0, s, c); break;
    case 17: case 18: case 19: case 20: hipLaunchKernelGGL((k_norm_row<XT, OT, 16, 5>), g, dim3(1024), 0, s, c); break;
    default: hipLaunchKernelGGL((k_norm_row<XT, OT, 16, 8>), g, dim3(1024), 0, s, c); break;
    }
}

template <typename XT, typename OT>
hipError_t norm_launch(const NormCall &c, hipStream_t s)
{
    constexpr int VEC = pack_len<XT, OT>();
    constexpr int kLane = kWaveSize * VEC;      // elements of one pack a lane
    const auto grid = [&](int64_t n) { return dim3((unsigned)std::min<int64_t>(n, kMaxRowGrid)); };
    const int pieces = norm_pieces(c.rows, c.V, c.x_dtype, c.out_dtype);
    if (pieces > 0) {
        const dim3 g = grid(c.rows * pieces), b(kPieceWaves * kWaveSize);
        hipLaunchKernelGGL((k_norm_piece<XT, OT, false>), g, b, 0, s, c, pieces);
        hipLaunchKernelGGL((k_norm_piece<XT, OT, true>), g, b, 0, s, c, pieces);
    } else if (c.V <= 2 * kLane) {
        hipLaunchKernelGGL((k_norm_row<XT, OT, 1, 2>), grid((c.rows + 3) / 4), dim3(256), 0, s, c);
    } else if (c.V <= 4 * kLane) {
        hipLaunchKernelGGL((k_norm_row<XT, OT, 1, 4>), grid((c.rows + 3) / 4), dim3(256), 0, s, c);
    } else if (c.V <= 8 * kLane) {
        hipLaunchKernelGGL((k_norm_row<XT, OT, 1, 8>), grid((c.rows + 3) / 4), dim3(256), 0, s, c);
    } else {
        norm_wide<XT, OT>(c, s);
    }
    return hipGetLastError();
}

template <typename XT>
hipError_t norm_ot(const NormCall &c, hipStream_t s)
{
    if (c.out_dtype == kF32) return norm_launch<XT, float>(c, s);
    if (c.out_dtype == kF16) return norm_launch<XT, _Float16>(c, s);
    return norm_launch<XT, __bf16>(c, s);
}

}  // namespace

// Pieces a row is cut into, 0 for rows that stay whole: rows longer than 16
// wavefronts hold, and rows so few that whole ones would leave most of the 256
// CUs idle while each takes more than one piece.
int norm_pieces(int64_t rows, int32_t V, int32_t x_dtype, int32_t out_dtype)
{
    const int vec = 16 / (int)std::max(dtype_size(x_dtype), dtype_size(out_dtype));
    const int span = kPieceWaves * kWaveSize * vec * kPieceNV;
    const int whole = 16 * 8 * kWaveSize * vec;
    const int pieces = (V + span - 1) / span;
    return V > whole || (rows <= 128 && pieces > 1) ? pieces : 0;
}

size_t norm_workspace(int64_t rows, int32_t V, int32_t x_dtype, int32_t out_dtype)
{
    return (size_t)rows * (size_t)norm_pieces(rows, V, x_dtype, out_dtype) * sizeof(NormStat);
}

hipError_t launch_log_softmax(const NormCall &c, hipStream_t s)
{
    if (c.x_dtype == kF32) return norm_ot<float>(c, s);
    if (c.x_dtype == kF16) return norm_ot<_Float16>(c, s);
    return norm_ot<__bf16>(c, s);
}

// ---------------------------------------------------------------- draw
//
// mass_i = exp((x_i - max) / T). Kept: the top_k largest (among equal scores the
// lowest indices), of these the shortest run of the largest whose mass reaches
// top_p of theirs, of these the ones with mass >= min_p. The token is the first
// kept i, in index order, whose running mass exceeds u times the kept mass.
//
// Every rule cuts at a value: the kept set is {key > tau} and the first r
// entries with key == tau, key being the score's bits in an order that integers
// compare. tau is found by digit (8 bits of the key at a time) from histograms
// of counts (top_k) or masses (top_p); nothing is sorted. Masses are computed in
// binary64 and summed as integers of 2^-bits, so sums do not depend on the order
// in which threads add, and a draw falls on the side of a border that the exact
// sums give except within about 2^-45 of it.

namespace {

constexpr int kSampleThreads = 1024;
constexpr int kSampleWaves = kSampleThreads / kWaveSize;
constexpr uint32_t kKeyNegInf = 0x007FFFFFu;
constexpr uint32_t kKeyPosInf = 0xFF800000u;

// Integers that compare as the scores do; -0 as +0, NaN as -inf.
__device__ __forceinline__ uint32_t score_key(float x)
{
    if (x != x) return kKeyNegInf;
    const uint32_t b = __float_as_uint(x + 0.0f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ float key_score(uint32_t k)
{
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

struct MassOf {
    double m, t;       // the row's maximum, the temperature
    double unit;       // 2^bits
    bool inf;          // the maximum is +inf: only +inf has mass
    __device__ __forceinline__ double operator()(uint32_t key) const
    {
        if (inf) return key == kKeyPosInf ? 1.0 : 0.0;
        if (key <= kKeyNegInf) return 0.0;
        return exp(((double)key_score(key) - m) / t);
    }
    __device__ __forceinline__ uint64_t fixed(uint32_t key) const { return (uint64_t)rint((*this)(key) * unit); }
};

template <typename XT>
__global__ __launch_bounds__(kSampleThreads) void k_sample(SampleCall c, int bits)
{
    __shared__ unsigned long long hmass[256];
    __shared__ uint32_t hcnt[256];
    __shared__ unsigned long long wsum[kSampleWaves + 1];
    __shared__ uint32_t wcnt[kSampleWaves], wtie[kSampleWaves];
    __shared__ uint32_t sel[4];
    __shared__ unsigned long long selm[2];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int V = c.V;
    // each wavefront owns one contiguous piece of the row
    const int seg = ((V + kSampleThreads - 1) / kSampleThreads) * kWaveSize;
    const int v0 = min(V, wave * seg), v1 = min(V, v0 + seg);

    for (int64_t r = blockIdx.x; r < c.rows; r += gridDim.x) {
        if (!row_active(c.set, r)) continue;
        __syncthreads();
        const XT *x = (const XT *)c.x + r * c.x_stride;
        const float T = c.temperatures ? c.temperatures[r] : c.temperature;
        const int topk = c.top_ks ? c.top_ks[r] : c.top_k;
        const float topp = c.top_ps ? c.top_ps[r] : c.top_p;
        const float minp = c.min_ps ? c.min_ps[r] : c.min_p;
        const bool greedy = !(T > 0.0f);

        uint32_t kmax = 0, valid = 0;
        for (int v = v0 + lane; v < v1; v += kWaveSize) {
            const uint32_t k = score_key((float)x[v]);
            kmax = max(kmax, k);
            valid += k > kKeyNegInf;
        }
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) kmax = max(kmax, (uint32_t)__shfl_xor((int)kmax, d, 64));
        valid = wave_sum_t(valid);
        if (lane == 0) { wcnt[wave] = valid; wtie[wave] = kmax; }
        __syncthreads();
        kmax = 0;
        valid = 0;
        for (int w = 0; w < kSampleWaves; ++w) { kmax = max(kmax, wtie[w]); valid += wcnt[w]; }
        __syncthreads();
        if (valid == 0) {
            if (tid == 0) {
                c.token[r] = -1;
                if (c.log_prob) c.log_prob[r] = -INFINITY;
                if (c.kept) c.kept[r] = 0;
            }
            continue;
        }
        if (kmax == kKeyPosInf) {                  // +inf scores leave only each other
            uint32_t n = 0;
            for (int v = v0 + lane; v < v1; v += kWaveSize) n += score_key((float)x[v]) == kKeyPosInf;
            n = wave_sum_t(n);
            if (lane == 0) wcnt[wave] = n;
            __syncthreads();
            valid = 0;
            for (int w = 0; w < kSampleWaves; ++w) valid += wcnt[w];
            __syncthreads();
        }
        MassOf mass;
        mass.m = (double)key_score(kmax);
        mass.t = greedy ? 1.0 : (double)T;
        mass.unit = (double)(1ull << bits);
        mass.inf = kmax == kKeyPosInf;

        // tau = 0, ties = 0: nothing cut yet (every valid key lies above tau)
        uint32_t tau = mass.inf ? kKeyPosInf - 1u : kKeyNegInf, ties = 0;
        for (int rule = 0; rule < 2; ++rule) {
            uint64_t target;     // rule 0: entries to keep, rule 1: mass to reach
            if (rule == 0) {
                const uint32_t k = greedy ? 1u : (topk > 0 ? (uint32_t)topk : 0u);
                if (k == 0 || k >= valid) continue;
                target = k;
            } else {
                if (greedy || !(topp < 1.0f)) continue;
                // the mass kept so far
                uint64_t z = 0;
                for (int v = v0 + lane; v < v1; v += kWaveSize) {
                    const uint32_t k = score_key((float)x[v]);
                    if (k > tau) z += mass.fixed(k);
                }
                z = wave_sum_t((unsigned long long)z);
                if (lane == 0) wsum[wave] = z;
                __syncthreads();
                z = 0;
                for (int w = 0; w < kSampleWaves; ++w) z += wsum[w];
                if (ties) z += (uint64_t)ties * mass.fixed(tau);
                const double want = ceil((double)topp * (double)z);
                target = want >= 1.0 ? (uint64_t)want : 1ull;
                if (target > z) target = z;
                __syncthreads();
            }
            // digits of tau from the top; `above` is what lies over the digits found so far
            const uint32_t tau0 = tau, ties0 = ties;
            const uint64_t tiemass0 = ties0 ? mass.fixed(tau0) : 0;
            uint32_t prefix = 0;
            uint64_t above = 0;
            uint64_t unit_w = 0;
            uint32_t nlast = 0;
            for (int shift = 24; shift >= 0; shift -= 8) {
                for (int i = tid; i < 256; i += kSampleThreads) { hmass[i] = 0; hcnt[i] = 0; }
                __syncthreads();
                for (int v = v0 + lane; v < v1; v += kWaveSize) {
                    const uint32_t k = score_key((float)x[v]);
                    if (k > tau0 && (shift == 24 || (k >> (shift + 8)) == prefix)) {
                        const uint32_t d = (k >> shift) & 255u;
                        atomicAdd(&hcnt[d], 1u);
                        if (rule == 1) atomicAdd(&hmass[d], (unsigned long long)mass.fixed(k));
                    }
                }
                // the ties that an earlier rule kept
                if (tid == 0 && ties0 && (shift == 24 || (tau0 >> (shift + 8)) == prefix)) {
                    atomicAdd(&hcnt[(tau0 >> shift) & 255u], ties0);
                    if (rule == 1) atomicAdd(&hmass[(tau0 >> shift) & 255u], (unsigned long long)(ties0 * tiemass0));
                }
                __syncthreads();
                if (tid == 0) {
                    uint64_t acc = above;
                    int d = 255;
                    for (; d > 0; --d) {
                        const uint64_t w = rule == 0 ? hcnt[d] : hmass[d];
                        if (acc + w >= target) break;
                        acc += w;
                    }
                    sel[0] = (uint32_t)d;
                    sel[1] = hcnt[d];
                    selm[0] = acc;
                    selm[1] = rule == 0 ? hcnt[d] : hmass[d];
                }
                __syncthreads();
                prefix = prefix << 8 | sel[0];
                nlast = sel[1];
                above = selm[0];
                unit_w = selm[1];
                __syncthreads();
            }
            tau = prefix;
            // nlast equal entries of one mass each: the fewest that reach the target
            const uint64_t each = rule == 0 ? 1 : (nlast ? unit_w / nlast : 0);
            uint64_t need = each ? (target - above + each - 1) / each : nlast;
            if (need < 1) need = 1;
            ties = (uint32_t)(need < nlast ? need : nlast);
        }

        // kept mass, count and equal entries of each wavefront's piece
        const bool cut = !greedy && minp > 0.0f;
        const double lim = minp < 1.0f ? (double)minp : 1.0;
        uint64_t z = 0;
        uint32_t cnt = 0, tie = 0;
        for (int v = v0 + lane; v < v1; v += kWaveSize) {
            const uint32_t k = score_key((float)x[v]);
            if (k < tau || k <= kKeyNegInf) continue;
            if (k == tau) { ++tie; continue; }
            const double w = mass(k);
            if (cut && !(w >= lim)) continue;
            z += (uint64_t)rint(w * mass.unit);
            ++cnt;
        }
        z = wave_sum_t((unsigned long long)z);
        cnt = wave_sum_t(cnt);
        tie = wave_sum_t(tie);
        if (lane == 0) { wsum[wave] = z; wcnt[wave] = cnt; wtie[wave] = tie; }
        __syncthreads();
        if (tid == 0) {
            const double wt = mass(tau);
            const bool tie_ok = ties && !(cut && !(wt >= lim));
            const uint64_t ft = (uint64_t)rint(wt * mass.unit);
            uint32_t left = tie_ok ? ties : 0, total = 0;
            uint64_t acc = 0;
            for (int w = 0; w < kSampleWaves; ++w) {      // wsum: mass before the piece; wtie: ties it keeps
                const uint32_t t = min(left, wtie[w]);
                left -= t;
                const uint64_t mine = wsum[w] + t * ft;
                total += wcnt[w] + t;
                wtie[w] = t;
                wsum[w] = acc;
                acc += mine;
            }
            wsum[kSampleWaves] = acc;
            double want = (double)c.u[r];
            want = want > 0.0 ? floor(want * (double)acc) : 0.0;
            uint64_t t64 = want >= (double)acc ? acc - 1 : (uint64_t)want;
            if (t64 > acc - 1) t64 = acc - 1;
            selm[0] = t64;
            selm[1] = ft;
            sel[2] = total;
        }
        __syncthreads();
        const uint64_t want = selm[0], total = wsum[kSampleWaves], ft = selm[1];
        if (wsum[wave] <= want && want < wsum[wave + 1]) {   // exactly one wavefront: its piece holds the token
            uint64_t base = wsum[wave];
            uint32_t left = wtie[wave];
            for (int vb = v0; vb < v1; vb += kWaveSize) {
                const int v = vb + lane;
                const uint32_t k = v < v1 ? score_key((float)x[v]) : 0u;
                const bool is_tie = v < v1 && k == tau && k > kKeyNegInf;
                const unsigned long long tm = __ballot(is_tie);
                const uint32_t rank = __popcll(tm & ((1ull << lane) - 1ull));
                uint64_t w = 0;
                if (is_tie) w = rank < left ? ft : 0;
                else if (v < v1 && k > tau && k > kKeyNegInf) {
                    const double d = mass(k);
                    if (!(cut && !(d >= lim))) w = (uint64_t)rint(d * mass.unit);
                }
                uint64_t run = w;
#pragma unroll
                for (int d = 1; d < 64; d <<= 1) {
                    const unsigned long long o = __shfl_up((unsigned long long)run, d, 64);
                    if (lane >= d) run += o;
                }
                const unsigned long long hit = __ballot(base + run > want);
                if (hit) {
                    if (lane == __ffsll((unsigned long long)hit) - 1) {
                        c.token[r] = v;
                        if (c.log_prob) {
                            const double e = mass.inf || greedy ? 0.0 : ((double)key_score(k) - mass.m) / mass.t;
                            c.log_prob[r] = (float)(e - log((double)total / mass.unit));
                        }
                        if (c.kept) c.kept[r] = (int32_t)sel[2];
                    }
                    break;
                }
                base += __shfl((unsigned long long)run, 63, 64);
                const uint32_t nt = __popcll(tm);
                left -= min(left, nt);
            }
        }
    }
}

}  // namespace

hipError_t launch_sample(const SampleCall &c, hipStream_t s)
{
    // V masses of at most 2^bits each stay below 2^62
    int lg = 0;
    while ((1ll << lg) < (long long)c.V) ++lg;
    const int bits = std::min(52, 62 - lg);
    const dim3 g((unsigned)std::min<int64_t>(c.rows, kMaxRowGrid)), b(kSampleThreads);
    if (c.x_dtype == kF32) hipLaunchKernelGGL(k_sample<float>, g, b, 0, s, c, bits);
    else if (c.x_dtype == kF16) hipLaunchKernelGGL(k_sample<_Float16>, g, b, 0, s, c, bits);
    else hipLaunchKernelGGL(k_sample<__bf16>, g, b, 0, s, c, bits);
    return hipGetLastError();
}

}  // namespace wfst
