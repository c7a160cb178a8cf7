// gfx950 (CDNA4) kernels of the log-softmax: logits to the log-posteriors the search reads.
#include "wfst_score_device.h"

namespace wfst {

// z = scale * x + bias, out = (z - max z) - log sum exp(z - max z), sums and
// statistics in binary32. The sum leaves the row's largest entries (each
// exactly 1) out and counts them, so that the logarithm of a row with one
// dominant label is log1p of a small number and keeps its digits. A row of
// -inf alone stays -inf; a row with +inf or NaN becomes NaN.

namespace {

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

// Rows past those, cut into pieces of 256 * VEC * kPieceNV elements: the first
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
    const int pieces = norm_pieces(c.V, c.x_dtype, c.out_dtype);
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

// Pieces a row is cut into, 0 for rows that 16 wavefronts hold: whole rows are
// faster there however few they are (1, 64, 256 rows of 32768 binary32 labels, whole /
// in pieces: 9 / 14, 9 / 14, 15 / 21 us).
int norm_pieces(int32_t V, int32_t x_dtype, int32_t out_dtype)
{
    const int vec = 16 / (int)std::max(dtype_size(x_dtype), dtype_size(out_dtype));
    const int span = kPieceWaves * kWaveSize * vec * kPieceNV;
    const int whole = 16 * 8 * kWaveSize * vec;
    return V > whole ? (V + span - 1) / span : 0;
}

size_t norm_workspace(int64_t rows, int32_t V, int32_t x_dtype, int32_t out_dtype)
{
    return (size_t)rows * (size_t)norm_pieces(V, x_dtype, out_dtype) * sizeof(NormStat);
}

hipError_t launch_log_softmax(const NormCall &c, hipStream_t s)
{
    if (c.x_dtype == kF32) return norm_ot<float>(c, s);
    if (c.x_dtype == kF16) return norm_ot<_Float16>(c, s);
    return norm_ot<__bf16>(c, s);
}

}  // namespace wfst
