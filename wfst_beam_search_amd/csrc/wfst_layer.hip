// gfx950 (CDNA4) kernels of the output layer with 4-bit weights: hidden states to logits.
#include "wfst_score_device.h"

namespace wfst {

namespace {

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
// lies in [2^14, 2^15): a bfloat16 value then fits binary16 exactly or, 2^30
// below the block's largest, loses less than 2^-39 of that. A binary32 value is
// cut into hi + lo / 2^11, two binary16 values: off by at most 2^-23 of itself, or
// 2^-50 of the block's largest. Without the 2^11 lo would end at binary16's smallest
// number, 2^-39 of the block's largest: 16 bits of 0.01 beside 1e5. lo meets
// weights divided by 2^11 (exact), so the sum stays one, or (few rows, one scale a
// tile) has a sum of its own: one row x 131072 x 4096 of binary32, groups of 128, divided
// weights / own sum 75 / 68 us, groups of 64 79 / 78, groups of 32 88 / 99; for many
// rows the sums would pass the registers. Exact values would take a third part, half
// as many products again.

constexpr int kLayerWaves = 4;
constexpr int kLayerThreads = kLayerWaves * kWaveSize;
constexpr int kRowsM = 16;                     // rows of x one matrix instruction takes

// The exponent e for which |x| <= mx lies below 2^15 when scaled by 2^-e.
__device__ __forceinline__ int block_exponent(float mx)
{
    if (!(mx > 0.0f)) return 0;
    int e;
    (void)frexpf(mx, &e);                      // mx = f * 2^e, f in [0.5, 1)
    e -= 15;
    return e < -120 ? -120 : e;                // 2^e and its inverse stay normal
}

template <typename XT> constexpr int kParts = sizeof(XT) == 4 ? 2 : 1;
template <typename XT> constexpr bool kScaled = !__is_same(XT, _Float16);

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

__device__ __forceinline__ float finite_max(const float (&v)[8], float mx)
{
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float a = fabsf(v[j]);
        mx = fmaxf(mx, a < INFINITY ? a : 0.0f);
    }
    return mx;
}

// The binary16 operand (and for binary32 its remainder, times 2^11) of eight values, scaled by `inv`, a power of two.
template <typename XT>
__device__ __forceinline__ void to_half(const float (&v)[8], float inv, half8_t &hi, half8_t &lo)
{
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float s = kScaled<XT> ? v[j] * inv : v[j];
        hi[j] = (_Float16)s;
        if (kParts<XT> == 2) {
            const float d = s - (float)hi[j];
            lo[j] = (_Float16)(fabsf(s) < INFINITY ? d * 2048.0f : 0.0f);      // (an infinity or NaN is in hi alone)
        }
    }
}

// Scales and zero points of one lane's output feature in one tile.
template <int WS, int GPT> struct TileScale {
    uint32_t s[WS * GPT < 4 ? 1 : WS * GPT / 4];
    uint32_t z;
};

template <int WS, int GPT>
__device__ __forceinline__ TileScale<WS, GPT> load_tile_scale(const Layer &l, size_t i)
{
    TileScale<WS, GPT> t;
    if constexpr (WS * GPT == 2) {
        t.s[0] = ((const uint16_t *)l.scales)[i];
    } else {
        const uint32_t *p = (const uint32_t *)l.scales + i * (WS * GPT / 4);
#pragma unroll
        for (int j = 0; j < WS * GPT / 4; ++j) t.s[j] = p[j];
    }
    t.z = 0x08080808u;
    if (l.zeros) {
        if constexpr (GPT == 1) t.z = l.zeros[i];
        else if constexpr (GPT == 2) t.z = ((const uint16_t *)l.zeros)[i];
        else t.z = ((const uint32_t *)l.zeros)[i];
    }
    return t;
}

template <int WS, int GPT>
__device__ __forceinline__ float scale_of(const TileScale<WS, GPT> &t, int g, bool bf16)
{
    if constexpr (WS == 4) return __uint_as_float(t.s[g]);
    const uint32_t h = (t.s[g / 2] >> (16 * (g & 1))) & 0xFFFFu;
    union { uint16_t u; _Float16 h; } c;
    c.u = (uint16_t)h;
    return bf16 ? __uint_as_float(h << 16) : (float)c.h;
}

// The eight weights q - z of one word, exact in binary16.
struct ZeroPair { half2_t whole, sixteenth; };

__device__ __forceinline__ ZeroPair zero_pair(uint32_t z)
{
    const _Float16 h = (_Float16)(float)z;
    const _Float16 a = (_Float16)-1024.0f - h, b = (_Float16)-64.0f - h;
    return {{a, a}, {b, b}};
}

__device__ __forceinline__ half8_t unpack_word(uint32_t w, uint32_t magic, const ZeroPair &z)
{
    union { uint32_t u[4]; half2_t h[4]; half8_t v; } q;
    const half2_t r16 = {(_Float16)0.0625f, (_Float16)0.0625f};
    const uint32_t w8 = w >> 8;
    q.u[0] = (w & 0x000F000Fu) | magic;
    q.u[1] = (w & 0x00F000F0u) | magic;
    q.u[2] = (w8 & 0x000F000Fu) | magic;
    q.u[3] = (w8 & 0x00F000F0u) | magic;
    q.h[0] += z.whole;
    q.h[2] += z.whole;
    q.h[1] = __builtin_elementwise_fma(q.h[1], r16, z.sixteenth);
    q.h[3] = __builtin_elementwise_fma(q.h[3], r16, z.sixteenth);
    return q.v;
}

// 1024 in both halves, in a vector register that the compiler does not fold: a
// mask and this then combine in one instruction.
__device__ __forceinline__ uint32_t magic_1024()
{
    uint32_t m;
    asm("v_mov_b32 %0, 0x64006400" : "=v"(m));
    return m;
}

__device__ __forceinline__ void store_y(const LayerCall &c, int64_t m, int n, float y)
{
    const int64_t i = m * c.out_stride + n;
    if (c.out_dtype == kF32) ((float *)c.out)[i] = y;
    else if (c.out_dtype == kF16) ((_Float16 *)c.out)[i] = (_Float16)y;
    else ((__bf16 *)c.out)[i] = (__bf16)y;
}

// Up to 16 rows of x at a time (blockIdx.y: which 16), which the workgroup itself turns into
// binary16 in LDS, kc blocks of 128 features per slice at a time, laid out as the
// matrix instruction reads it: [32 features][8 features][row][8]. Only RP rows
// (the power of two that holds them) are kept; lanes of rows past them repeat
// the last one and their sums are dropped. KS = 1: a wavefront owns 16 output
// features and walks all of K. KS = 4: the four wavefronts of a workgroup own
// the same 16 features and a quarter of K each, joined in LDS at the end.
// Weights stream D tiles ahead of their use. SPL = 1 (at most 4 rows, whose staging
// takes one run of 8 features a thread) leaves registers for 4 wavefronts a SIMD (118
// of bfloat16): one row x 131072 x 4096 takes 59 us with 3 tiles ahead (62, 61, 71
// with 4, 2, 6), where the general staging's (174) leave 2 and it takes 74; 278 MB at
// 4.7 TB/s, 92 % of what a large copy moves on this card.
template <int KS, int SPL> constexpr int kTilesAhead = KS == 1 ? (SPL == 1 ? 3 : 4) : 2;

template <typename XT, int WS, int GPT, int KS, int SPL>
__global__ __launch_bounds__(kLayerThreads) void k_layer_few(Layer l, LayerCall c, int RP, int kc)
{
    constexpr int P = kParts<XT>;
    constexpr int D = kTilesAhead<KS, SPL>;
    constexpr bool kLow = P == 2 && GPT == 1;                           // second parts have a sum of their own
    extern __shared__ __align__(16) char smem[];
    half8_t *xs = (half8_t *)smem;                                      // [P][KS * kc * 16][RP]
    const int part = KS * kc * 16 * RP;
    float *xf = (float *)(xs + P * part);                               // [KS * kc][RP]
    float4_t *joint = (float4_t *)(smem);                               // (KS = 4, after the last use of xs)
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int m0 = blockIdx.y * kRowsM, M = min(kRowsM, c.M - m0);
    const int nt = min((int)(KS == 1 ? blockIdx.x * kLayerWaves + wave : blockIdx.x), l.nt - 1);
    const bool live = KS > 1 || blockIdx.x * kLayerWaves + wave < l.nt;
    const int col = lane & 15, quad = lane >> 4;
    const int slice = KS == 1 ? 0 : wave;
    const int b0 = (int)((int64_t)l.kb * slice / KS), nb = (int)((int64_t)l.kb * (slice + 1) / KS) - b0;
    const bool bf16s = l.scale_dtype == kBF16;
    const uint32_t magic = magic_1024();
    const XT *x = (const XT *)c.x + (int64_t)m0 * c.x_stride;
    const size_t tile0 = (size_t)nt * l.kb + b0;

    uint4 wq[D];
    TileScale<WS, GPT> sq[D];
#pragma unroll
    for (int i = 0; i < D; ++i) {
        const size_t t = tile0 + min(i, max(nb - 1, 0));
        wq[i] = l.w[min(t, (size_t)l.nt * l.kb - 1) * kWaveSize + lane];
        sq[i] = load_tile_scale<WS, GPT>(l, min(t, (size_t)l.nt * l.kb - 1) * kTileN + col);
    }

    // staging: 16 * RP threads (at most 64) take a block of 128 features, each up to four runs of 8
    const int per = min(64, 16 * RP), bpw = 64 / per;
    const int l2 = lane % per, sr = l2 % RP, s0 = l2 / RP, sstep = per / RP, spl = SPL == 1 ? 1 : 16 / sstep;
    const bool there = sr < M && row_active(c.rows, m0 + sr);
    const int longest = (l.kb + KS - 1) / KS;
    float4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
    const int arow = min(col, RP - 1), frow = min(quad * 4, RP - 1);

    for (int c0 = 0; c0 < longest; c0 += kc) {
        if (c0) __syncthreads();
        for (int u = wave * bpw + lane / per; u < KS * kc; u += kLayerWaves * bpw) {
            const int sl = u / kc, b = c0 + u % kc;
            const int sb0 = (int)((int64_t)l.kb * sl / KS), sbn = (int)((int64_t)l.kb * (sl + 1) / KS) - sb0;
            const bool in = b < sbn;
            float v[SPL][8];
            float mx = 0.0f;
#pragma unroll
            for (int i = 0; i < SPL; ++i) {
                if (i < spl) {
                    load_x<XT>(x + (int64_t)sr * c.x_stride, there && in, (sb0 + b) * kTileK + (s0 + i * sstep) * 8, l.K, v[i]);
                    if (kScaled<XT>) mx = finite_max(v[i], mx);
                }
            }
            float inv = 1.0f;
            if (kScaled<XT>) {
                for (int d = RP; d < per; d <<= 1) mx = fmaxf(mx, __shfl_xor(mx, d, 64));
                const int e = block_exponent(mx);
                inv = ldexpf(1.0f, -e);
                if (s0 == 0) xf[u * RP + sr] = ldexpf(1.0f, e);
            }
#pragma unroll
            for (int i = 0; i < SPL; ++i) {
                if (i < spl) {
                    half8_t hi, lo;
                    to_half<XT>(v[i], inv, hi, lo);
                    const int at = (u * 16 + s0 + i * sstep) * RP + sr;
                    xs[at] = hi;
                    if (P == 2) xs[part + at] = lo;
                }
            }
        }
        __syncthreads();
        const int end = min(nb, c0 + kc);
        for (int t = c0; t < end; t += D) {
#pragma unroll
            for (int i = 0; i < D; ++i) {
                if (t + i >= end) break;
                const uint4 w4 = wq[i];
                const TileScale<WS, GPT> ts = sq[i];
                const size_t nx = tile0 + min(t + i + D, nb - 1);
                wq[i] = l.w[nx * kWaveSize + lane];
                sq[i] = load_tile_scale<WS, GPT>(l, nx * kTileN + col);
                const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
                const int u = slice * kc + t + i - c0;
                float4_t sum = {0.0f, 0.0f, 0.0f, 0.0f}, low = sum, tile = sum;       // (low: of the second parts)
                ZeroPair z = zero_pair(ts.z & 255u);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (j && j % (4 / GPT) == 0) z = zero_pair((ts.z >> (8 * (j * GPT / 4))) & 255u);
                    const half8_t q = unpack_word(w[j], magic, z);
const int at = (u * 16 + j * 4 + quad) * RP + arow;
                    sum = __builtin_amdgcn_mfma_f32_16x16x32_f16(xs[at], q, sum, 0, 0, 0);
                    if constexpr (kLow) low = __builtin_amdgcn_mfma_f32_16x16x32_f16(xs[part + at], q, low, 0, 0, 0);
                    else if constexpr (P == 2)
                        sum = __builtin_amdgcn_mfma_f32_16x16x32_f16(xs[part + at], q * (_Float16)(1.0f / 2048.0f), sum, 0, 0, 0);
                    if ((j + 1) % (4 / GPT) == 0) {
                        const float s = scale_of<WS, GPT>(ts, j * GPT / 4, bf16s);
#pragma unroll
                        for (int q4 = 0; q4 < 4; ++q4) {
                            if (kLow) sum[q4] = fmaf(low[q4], 1.0f / 2048.0f, sum[q4]);
                            if (!kScaled<XT>) acc[q4] = fmaf(sum[q4], s, acc[q4]);
                            else if (j < 4 / GPT) tile[q4] = sum[q4] * s;
                            else tile[q4] = fmaf(sum[q4], s, tile[q4]);
                            sum[q4] = low[q4] = 0.0f;
                        }
                    }
                }
                // (the block's factor comes last: its product with a small scale alone may be subnormal)
                if (kScaled<XT>) {
#pragma unroll
                    for (int q4 = 0; q4 < 4; ++q4) acc[q4] = fmaf(tile[q4], xf[u * RP + min(frow + q4, RP - 1)], acc[q4]);
                }
            }
        }
    }
    if (KS > 1) {
        __syncthreads();
        if (wave) joint[(wave - 1) * kWaveSize + lane] = acc;
        __syncthreads();
        if (wave) return;
#pragma unroll
        for (int s = 0; s < KS - 1; ++s) acc += joint[s * kWaveSize + lane];
    }
    const int n = nt * kTileN + col;
    if (!live || n >= l.N) return;
    const float bias = l.bias ? l.bias[n] : 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int m = quad * 4 + i;
        if (m < M && row_active(c.rows, m0 + m)) store_y(c, m0 + m, n, acc[i] + bias);
    }
}

// Many rows: x is first turned into matrix operands, once, in the workspace:
// per 16 rows and 128 features, [P][32 features][lane][8 halves] and the 16
// scale factors. One wavefront makes one such block.
constexpr size_t kBlockHalves = 4 * 64 * 8;            // halves of one part of a block

template <typename XT>
__global__ __launch_bounds__(256) void k_layer_operands(Layer l, LayerCall c, half8_t *xa, float *xf)
{
    constexpr int P = kParts<XT>;
    const int lane = threadIdx.x & 63;
    const int row = lane & 15, quad = lane >> 4;
    const int64_t nblk = (int64_t)((c.M + kRowsM - 1) / kRowsM) * l.kb;
    const int64_t u = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (u >= nblk) return;
    const int64_t mt = u / l.kb;
    const int b = (int)(u - mt * l.kb);
    const int64_t m = mt * kRowsM + row;
    const bool there = m < c.M && row_active(c.rows, m);
    const XT *x = (const XT *)c.x + (there ? m : 0) * c.x_stride;
    float v[4][8], mx = 0.0f, inv = 1.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        load_x<XT>(x, there, b * kTileK + j * 32 + quad * 8, l.K, v[j]);
        if (kScaled<XT>) mx = finite_max(v[j], mx);
    }
    if (kScaled<XT>) {
        mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
        mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
        const int e = block_exponent(mx);
        inv = ldexpf(1.0f, -e);
        if (quad == 0) xf[u * kRowsM + row] = ldexpf(1.0f, e);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        half8_t hi, lo;
        to_half<XT>(v[j], inv, hi, lo);
        xa[(u * P * 4 + j) * 64 + lane] = hi;
        if (P == 2) xa[(u * P * 4 + 4 + j) * 64 + lane] = lo;
    }
}

// The product for many rows: a workgroup of 8 wavefronts makes 16 MT rows by 128
// output features. Each wavefront owns 32 features; the two halves of the
// workgroup take alternate blocks of 128 input features (joined in LDS at the
// end), so that each wavefront's matrix instructions share every operand of x
// read from LDS between two weight tiles. Operands of the next step are loaded
// into registers during a step and stored into the other LDS buffer after it, or
// (64 rows, one part, one scale a tile) loaded into that buffer directly, which
// frees the matrix instructions of the stores: 4096 x 131072 x 4096 binary16 8.3 -> 6.5
// ms (670 TFLOP/s), bfloat16 9.4 -> 8.6; with two parts, smaller groups or fewer rows
// the wait for the loads costs more (binary32 3 % of its 12.8 ms, groups of 32 3 %, 32
// rows 7 %).
template <typename XT, int WS, int GPT, int MT>
__global__ __launch_bounds__(512) void k_layer_many(Layer l, LayerCall c, const half8_t *xa, const float *xf)
{
    constexpr int P = kParts<XT>;
    constexpr int NT = 2;
    constexpr int kBlk = P * 4 * 64;                    // half8 of one block (16 rows, 128 features)
    constexpr int kStep = 2 * MT * kBlk;                // half8 of one step
    constexpr int kCopies = kStep / 512;
    constexpr bool kDirect = MT == 4 && P == 1 && GPT == 1;
    extern __shared__ __align__(16) char smem[];
    half8_t *buf = (half8_t *)smem;                     // [2][2 halves][MT][P][4][64]
    float *fac = (float *)(buf + 2 * kStep);            // [2][2][MT][16]
    float4_t *joint = (float4_t *)smem;                 // [4][MT * NT][64], after the last step
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int col = lane & 15, quad = lane >> 4;
    const int half = wave >> 2;
    const int nt0 = blockIdx.x * 8 + (wave & 3) * NT;
    const int mblk = blockIdx.y;
    const int mtiles = (c.M + kRowsM - 1) / kRowsM;
    const bool bf16s = l.scale_dtype == kBF16;
    const uint32_t magic = magic_1024();
    const int steps = (l.kb + 1) / 2;

    // block (half h, row tile mt) of a step: clamped to one that exists
    const auto block = [&](int step, int h, int mt) {
        const int64_t t = min(mblk * MT + mt, mtiles - 1);
        return t * l.kb + min(step * 2 + h, l.kb - 1);
    };
    half8_t reg[kDirect ? 1 : kCopies];
    float freg = 1.0f;
    const auto fetch = [&](int step, int slot) {
        if constexpr (kDirect) {
            typedef const __attribute__((address_space(1))) uint32_t *Global;
            typedef __attribute__((address_space(3))) uint32_t *Local;
#pragma unroll
            for (int i = 0; i < kCopies; ++i) {
                const int first = __builtin_amdgcn_readfirstlane(i * 512 + (tid & ~63));     // the wavefront's 64
                const int u = first / kBlk;
                const half8_t *src = xa + block(step, u / MT, u % MT) * kBlk + first % kBlk + lane;
                __builtin_amdgcn_global_load_lds((Global)src, (Local)(buf + slot * kStep + first), 16, 0, 0);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kCopies; ++i) {
                const int u = (i * 512 + tid) / kBlk;       // (the same for a wavefront)
                reg[i] = xa[block(step, u / MT, u % MT) * kBlk + (i * 512 + tid) % kBlk];
            }
        }
        if (kScaled<XT> && tid < 2 * MT * 16) freg = xf[block(step, tid / 16 / MT, tid / 16 % MT) * kRowsM + tid % 16];
    };
    const auto put = [&](int slot) {
        if constexpr (kDirect) {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");      // (this wavefront's part has arrived in LDS)
        } else {
#pragma unroll
            for (int i = 0; i < kCopies; ++i) buf[slot * kStep + i * 512 + tid] = reg[i];
        }
        if (kScaled<XT> && tid < 2 * MT * 16) fac[slot * 2 * MT * 16 + tid] = freg;
    };
    uint4 wq[NT];
    TileScale<WS, GPT> sq[NT];
    const auto weights = [&](int step) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const size_t t = (size_t)min(nt0 + n, l.nt - 1) * l.kb + min(step * 2 + half, l.kb - 1);
            wq[n] = l.w[t * kWaveSize + lane];
            sq[n] = load_tile_scale<WS, GPT>(l, t * kTileN + col);
        }
    };

    float4_t acc[MT][NT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[m][n] = (float4_t){0.0f, 0.0f, 0.0f, 0.0f};
    weights(0);
    fetch(0, 0);
    put(0);
    __syncthreads();
    for (int step = 0; step < steps; ++step) {
        const int slot = step & 1;
        uint4 w4[NT];
        TileScale<WS, GPT> ts[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) { w4[n] = wq[n]; ts[n] = sq[n]; }
        if (step + 1 < steps) {
            weights(step + 1);
            fetch(step + 1, slot ^ 1);
        }
        if (step * 2 + half < l.kb) {
            const half8_t *a0 = buf + slot * kStep + half * MT * kBlk + lane;
            float4_t tile[MT][NT], sum[MT][NT];
            ZeroPair z[NT];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool first = j % (4 / GPT) == 0, last = (j + 1) % (4 / GPT) == 0;
                half8_t q[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if (first) z[n] = zero_pair((ts[n].z >> (8 * (j * GPT / 4))) & 255u);
                    const uint32_t w = j == 0 ? w4[n].x : j == 1 ? w4[n].y : j == 2 ? w4[n].z : w4[n].w;
                    q[n] = unpack_word(w, magic, z[n]);
                }
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    if (p) {
#pragma unroll
                        for (int n = 0; n < NT; ++n) q[n] *= (_Float16)(1.0f / 2048.0f);       // (as the second part is held)
                    }
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        const half8_t a = a0[m * kBlk + (p * 4 + j) * 64];
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            if (first && p == 0) sum[m][n] = (float4_t){0.0f, 0.0f, 0.0f, 0.0f};
                            sum[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, q[n], sum[m][n], 0, 0, 0);
                        }
                    }
                }
                if (last) {
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const float s = scale_of<WS, GPT>(ts[n], j * GPT / 4, bf16s);
#pragma unroll
                        for (int m = 0; m < MT; ++m)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                if (!kScaled<XT>) acc[m][n][i] = fmaf(sum[m][n][i], s, acc[m][n][i]);
                                else if (j < 4 / GPT) tile[m][n][i] = sum[m][n][i] * s;
                                else tile[m][n][i] = fmaf(sum[m][n][i], s, tile[m][n][i]);
                            }
                    }
                }
            }
            if (kScaled<XT>) {
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const float4_t f = *(const float4_t *)(fac + ((slot * 2 + half) * MT + m) * 16 + quad * 4);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[m][n][i] = fmaf(tile[m][n][i], f[i], acc[m][n][i]);
                }
            }
        }
        if (step + 1 < steps) put(slot ^ 1);
        __syncthreads();
    }
    if (half) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n) joint[((wave & 3) * MT * NT + m * NT + n) * 64 + lane] = acc[m][n];
    }
    __syncthreads();
    if (half) return;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int f = (nt0 + n) * kTileN + col;
        if (nt0 + n >= l.nt || f >= l.N) continue;
        const float bias = l.bias ? l.bias[f] : 0.0f;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const float4_t y = acc[m][n] + joint[((wave & 3) * MT * NT + m * NT + n) * 64 + lane];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t r = ((int64_t)mblk * MT + m) * kRowsM + quad * 4 + i;
                if (r < c.M && row_active(c.rows, r)) store_y(c, r, f, y[i] + bias);
            }
        }
    }
}

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

template <typename XT, int WS, int GPT, int KS, int SPL>
hipError_t few_launch(const Layer &l, const LayerCall &c, int RP, hipStream_t s)
{
    constexpr int D = kTilesAhead<KS, SPL>;
    // blocks of 128 features staged at a time: all, or what 40 KiB hold
    const int longest = (l.kb + KS - 1) / KS;
    const size_t per = (size_t)KS * RP * (256 * kParts<XT> + 4);
    const int kc = std::min<int>(longest, std::max<int>(D, (int)(40960 / per) / D * D));
    const size_t lds = std::max<size_t>(per * kc, KS > 1 ? (KS - 1) * 64 * sizeof(float4_t) : 0);
    const dim3 g(KS > 1 ? l.nt : (l.nt + kLayerWaves - 1) / kLayerWaves, (c.M + kRowsM - 1) / kRowsM);
    hipLaunchKernelGGL((k_layer_few<XT, WS, GPT, KS, SPL>), g, dim3(kLayerThreads), lds, s, l, c, RP, kc);
    return hipGetLastError();
}

// Few tiles of features: K over the wavefronts of a workgroup, to have enough of
// them. One row of bfloat16, one / four wavefronts a tile, us, K = 512, 1024, 2050, 4096:
//  250 tiles 4.5 / 4.0, 5.7 / 4.5, 9.3 / 6.8, 13.4 / 7.9
// 1000 tiles 4.6 / 5.0, 5.9 / 5.9, 9.5 / 9.0, 15.3 / 12.5
// 1500 tiles 5.1 / 6.4, 6.8 / 7.6, 11.4 / 12.9, 18.5 / 18.0
// 2001 tiles 5.2 / 7.4, 6.9 / 8.9, 12.5 / 15.8, 19.2 / 21.1
// The border lies lower the smaller K is; one for all K gives up 1.3 us at 1500 x 512.
template <typename XT, int WS, int GPT>
hipError_t layer_few(const Layer &l, const LayerCall &c, hipStream_t s)
{
    int RP = 1;
    while (RP < std::min(c.M, kRowsM)) RP *= 2;
    if (l.nt < 1536) return RP <= 4 ? few_launch<XT, WS, GPT, 4, 1>(l, c, RP, s) : few_launch<XT, WS, GPT, 4, 4>(l, c, RP, s);
    return RP <= 4 ? few_launch<XT, WS, GPT, 1, 1>(l, c, RP, s) : few_launch<XT, WS, GPT, 1, 4>(l, c, RP, s);
}

// Row tiles of 16 a workgroup of k_layer_many takes (1, 2 or 4); 0: k_layer_few
// serves, because the workgroups would be too few to fill the card or the rows are
// few. Two launches cost some 6 us: below 16384 weight tiles they pay past 16 rows
// only (17000 x 1024, 16 rows: few 12 .. 23 us, many 14); above, from 3 rows of
// bfloat16 or binary32 on and from 5 of binary16, whose staging is a copy (32003 x
// 2050, few / many: 2 rows 18 / 18, 20 / 20, 13 / 18 us; 4 rows 22 / 19, 34 / 20, 15 / 19;
// 8 rows 42 / 19, 44 / 20, 28 / 19). By workgroups, bfloat16, few / many: 4 (64 x 500 x
// 512) 5 / 14, 40 (64 x 5000 x 1024) 14 / 18, 63 (64 x 8000 x 2048) 33 / 26, 64 (1024 x
// 500 x 512) 14 / 15, 80 (128 x 5000 x 1024) 25 / 19, 94 (64 x 12000 x 1024) 29 / 18, 160
// (256 x 5000 x 1024) 46 / 19: 128 keeps every size where few is faster, and between
// 60 and 128 some where many would be.
int many_tiles(const Layer &l, int32_t rows, int32_t x_dtype)
{
    const bool large = (int64_t)l.nt * l.kb >= 16384;
    if (rows < (!large ? kRowsM + 1 : x_dtype == kF16 ? 5 : 3)) return 0;
    const int mt = rows <= kRowsM ? 1 : rows <= 2 * kRowsM ? 2 : 4;
    const int64_t groups = (int64_t)((l.nt + 7) / 8) * ((rows + mt * kRowsM - 1) / (mt * kRowsM));
    return groups >= 128 ? mt : 0;
}

size_t operand_bytes(const Layer &l, int32_t rows, int32_t x_dtype)
{
    const size_t blocks = (size_t)((rows + kRowsM - 1) / kRowsM) * l.kb;
    return blocks * kBlockHalves * 2 * (x_dtype == kF32 ? 2 : 1);
}

template <typename XT, int WS, int GPT, int MT>
hipError_t layer_many(const Layer &l, const LayerCall &c, hipStream_t s)
{
    const int64_t blocks = (int64_t)((c.M + kRowsM - 1) / kRowsM) * l.kb;
    half8_t *xa = (half8_t *)c.workspace;
    float *xf = (float *)((char *)c.workspace + operand_bytes(l, c.M, c.x_dtype));
    hipLaunchKernelGGL(k_layer_operands<XT>, dim3((unsigned)((blocks + 3) / 4)), dim3(256), 0, s, l, c, xa, xf);
    const size_t lds = 2 * 2 * MT * (kParts<XT> * kBlockHalves * 2 + 64);
    const dim3 g((l.nt + 7) / 8, (c.M + MT * kRowsM - 1) / (MT * kRowsM));
    hipLaunchKernelGGL((k_layer_many<XT, WS, GPT, MT>), g, dim3(512), lds, s, l, c, (const half8_t *)xa, (const float *)xf);
    return hipGetLastError();
}

template <typename XT, int WS, int GPT>
hipError_t layer_rows(const Layer &l, const LayerCall &c, hipStream_t s)
{
    const int mt = many_tiles(l, c.M, c.x_dtype);
    if (mt == 4) return layer_many<XT, WS, GPT, 4>(l, c, s);
    if (mt == 2) return layer_many<XT, WS, GPT, 2>(l, c, s);
    if (mt == 1) return layer_many<XT, WS, GPT, 1>(l, c, s);
    return layer_few<XT, WS, GPT>(l, c, s);
}

template <typename XT>
hipError_t layer_xt(const Layer &l, const LayerCall &c, hipStream_t s)
{
    if (l.scale_dtype == kF32) {
        if (l.gpt == 1) return layer_rows<XT, 4, 1>(l, c, s);
        if (l.gpt == 2) return layer_rows<XT, 4, 2>(l, c, s);
        return layer_rows<XT, 4, 4>(l, c, s);
    }
    if (l.gpt == 1) return layer_rows<XT, 2, 1>(l, c, s);
    if (l.gpt == 2) return layer_rows<XT, 2, 2>(l, c, s);
    return layer_rows<XT, 2, 4>(l, c, s);
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

size_t layer_workspace(const Layer &l, int32_t rows, int32_t x_dtype)
{
    if (!many_tiles(l, rows, x_dtype)) return 0;
    const size_t blocks = (size_t)((rows + kRowsM - 1) / kRowsM) * l.kb;
    return operand_bytes(l, rows, x_dtype) + (x_dtype == kF16 ? 0 : blocks * kRowsM * 4);
}

hipError_t launch_layer(const Layer &l, const LayerCall &c, hipStream_t s)
{
    if (c.x_dtype == kF32) return layer_xt<float>(l, c, s);
    if (c.x_dtype == kF16) return layer_xt<_Float16>(l, c, s);
    return layer_xt<__bf16>(l, c, s);
}

}  // namespace wfst
