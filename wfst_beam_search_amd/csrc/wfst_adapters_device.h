// Device code of the low-rank adapters beside the output layer, for wfst_layer_kernels.h. Not part of the ABI.
#pragma once

#include "wfst_score_device.h"

namespace wfst {

namespace {

// y[m, n] += sum_j up[n, j] h[m, j], h[m, j] = scale * sum_k down[j, k] x[m, k]
//
// h is made once, by a launch before the layer's product (in the one that makes the
// layer's operands where there is such a launch), and meets up in the layer's epilogue,
// 16 rows, 16 features and 16 ranks to a block, so that the result is rounded once
// and never read back. h keeps its binary32 digits: with up in binary32 the matrix
// unit's binary32 products take it as it is; with up in bfloat16 as three bfloat16 parts
// of 8 bits; with up in binary16 as hi + lo / 2^11, two binary16 values scaled by a
// power of two per row and 16 ranks (off by at most 2^-23 of itself or 2^-50 of the
// largest of those 16). 16000 rows x 5000 x 1024 of binary16, one slot of rank 16, 32, 128, us
// for the whole call: 399, 415, 554, without a slot 357, the layer alone 318; 64 rows x 32003 x
// 2050 of binary32 over 64 slots of rank 16, 32: 72, 107 in binary32 (up is 131, 262 MB, of which
// repeated calls find a part in the last cache), 65, 79 in bfloat16; without a slot 48, the layer
// alone 45.

constexpr int kRowsTile = 16;

typedef short short4_t __attribute__((ext_vector_type(4)));
typedef _Float16 half4_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf8_t __attribute__((ext_vector_type(8)));

// A block of h, 16 rows by 16 ranks, as the matrix instruction reads it: [parts][64
// lanes][4], lane l holds row l % 16 and ranks 4 (l / 16) .. + 3; binary16: then one
// factor a row.
__host__ __device__ constexpr int h_block_bytes(int32_t dtype) { return dtype == kF32 ? 1024 : dtype == kF16 ? 1088 : 1536; }

// The exponent e for which |x| <= mx lies below 2^15 when scaled by 2^-e.
__device__ __forceinline__ int block_exponent(float mx)
{
    if (!(mx > 0.0f)) return 0;
    int e;
    (void)frexpf(mx, &e);                      // mx = f * 2^e, f in [0.5, 1)
    e -= 15;
    return e < -120 ? -120 : e;                // 2^e and its inverse stay normal
}

// Writes h of one row (of 16) and rank (of 16); mx: the largest finite |h| of the row's 16.
// An infinite up meets the first part alone, which therefore is 0 only where h is: below
// its type's smallest number it holds that one, and the next part the difference.
template <typename AT>
__device__ __forceinline__ void put_h(char *block, int row, int j, float v, float mx)
{
    const int at = ((j >> 2) * 16 + row) * 4 + (j & 3);
    if constexpr (sizeof(AT) == 4) {
        ((float *)block)[at] = v;
    } else if constexpr (__is_same(AT, _Float16)) {
        const int e = block_exponent(mx);
        const float s = v * ldexpf(1.0f, -e);
        _Float16 hi = (_Float16)s;
        if (hi == (_Float16)0.0f && v != 0.0f) hi = (_Float16)copysignf(0x1p-24f, v);      // (lo takes it back)
        ((_Float16 *)block)[at] = hi;
        ((_Float16 *)block)[256 + at] = (_Float16)(fabsf(s) < INFINITY ? (s - (float)hi) * 2048.0f : 0.0f);
        if (j == 0) ((float *)(block + 1024))[row] = ldexpf(1.0f, e);
    } else {
        // (cut, not rounded: the parts add up to v and none passes the largest number)
        const bool finite = fabsf(v) < INFINITY;
        float a = finite ? __uint_as_float(__float_as_uint(v) & 0xFFFF0000u) : v;
        if (a == 0.0f && v != 0.0f) a = copysignf(0x1p-133f, v);
        const float b = finite ? v - a : 0.0f, b1 = __uint_as_float(__float_as_uint(b) & 0xFFFF0000u);
        ((__bf16 *)block)[at] = (__bf16)a;
        ((__bf16 *)block)[256 + at] = (__bf16)b1;
        ((__bf16 *)block)[512 + at] = (__bf16)(b - b1);
    }
}

__device__ __forceinline__ float finite_abs(float v)
{
    const float a = fabsf(v);
    return a < INFINITY ? a : 0.0f;
}

constexpr int kRowWaves = 16;

// Row by row: a workgroup of 16 wavefronts for each row and 16 ranks, a wavefront for
// each rank, lanes along K.
template <typename XT, typename AT>
__device__ __forceinline__ void shrink_row(const LayerCall &c, int32_t K, int64_t item, float *red)
{
    const AdaptCall &ad = c.ad;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t m = item / ad.a.rb;
    const int jb = (int)(item - m * ad.a.rb);
    int slot = row_active32(c.rows, (uint32_t)m) ? ad.ids[(uint32_t)m / (uint32_t)ad.per_id] : -1;
    if (slot >= ad.a.slots) slot = -1;
    const int rank = slot >= 0 ? ad.a.ranks[slot] : 0, j = jb * 16 + wave;
    if (jb * 16 >= rank) return;
    float sum = 0.0f;
    if (j < rank) {
        const AT *w = (const AT *)ad.a.down + ((size_t)slot * ad.a.rb * 16 + j) * ad.a.kp;
        const XT *x = (const XT *)c.x + m * c.x_stride;
        float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        int k = lane * 8;
        for (; k + 3 * kWaveSize * 8 + 8 <= K; k += 4 * kWaveSize * 8) {
            Pack<XT, 8> v[4];
            Pack<AT, 8> p[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                v[q] = *(const Pack<XT, 8> *)(x + k + q * kWaveSize * 8);
                p[q] = *(const Pack<AT, 8> *)(w + k + q * kWaveSize * 8);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int e = 0; e < 8; ++e) part[q] = fmaf((float)v[q].v[e], (float)p[q].v[e], part[q]);
        }
        for (; k < K; k += kWaveSize * 8) {
            float v[8];
            load_x<XT>(x, true, k, K, v);
            const Pack<AT, 8> p = *(const Pack<AT, 8> *)(w + k);
#pragma unroll
            for (int e = 0; e < 8; ++e) part[0] = fmaf(v[e], (float)p.v[e], part[0]);
        }
        sum = wave_sum_f((part[0] + part[1]) + (part[2] + part[3])) * ad.a.scales[slot];
    }
    if (lane == 0) red[wave] = sum;
    __syncthreads();
    if (threadIdx.x < 16) {
        float mx = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) mx = fmaxf(mx, finite_abs(red[i]));
        char *block = ad.h + ((m / kRowsTile) * ad.a.rb + jb) * h_block_bytes(ad.a.dtype);
        put_h<AT>(block, (int)(m % kRowsTile), threadIdx.x, red[threadIdx.x], mx);
    }
}

// Eight of a row's elements from k on as a matrix operand (0 past K, and for no row).
template <typename XT, typename V>
__device__ __forceinline__ V load_operand(const XT *row, bool there, int k, int K)
{
    V v;
    if (there && k + 8 <= K) {
        const Pack<XT, 8> p = *(const Pack<XT, 8> *)(row + k);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = p.v[j];
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = there && k + j < K ? row[k + j] : (XT)0.0f;
    }
    return v;
}

// 32 features' products of 16 rows and twice 16 ranks: in the operands' own 16 bits, else in binary32.
template <typename XT, typename AT>
__device__ __forceinline__ void shrink_step(const XT *x, bool there, const AT *w0, const AT *w1, int k, int K, float4_t (&d)[2])
{
    const AT *const w[2] = {w0, w1};
    if constexpr (__is_same(XT, _Float16) && __is_same(AT, _Float16)) {
        const half8_t v = load_operand<XT, half8_t>(x, there, k, K);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            d[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, load_operand<AT, half8_t>(w[i], true, k, k + 8), d[i], 0, 0, 0);
    } else if constexpr (__is_same(XT, __bf16) && __is_same(AT, __bf16)) {
        const bf8_t v = load_operand<XT, bf8_t>(x, there, k, K);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            d[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, load_operand<AT, bf8_t>(w[i], true, k, k + 8), d[i], 0, 0, 0);
    } else {
        float v[8];
        load_x<XT>(x, there, k, K, v);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const Pack<AT, 8> p = *(const Pack<AT, 8> *)(w[i] + k);
#pragma unroll
            for (int e = 0; e < 8; ++e) d[i] = __builtin_amdgcn_mfma_f32_16x16x4f32(v[e], (float)p.v[e], d[i], 0, 0, 0);
        }
    }
}

constexpr int kShrinkBlocks = 8;               // blocks of 16 ranks at most
constexpr int kShrinkBytes = 4 * kShrinkBlocks * kWaveSize * 16;

// Rows that share ids: a workgroup for 16 rows, once for each slot among them; each
// wavefront takes a quarter of K for all ranks.
template <typename XT, typename AT>
__device__ __forceinline__ void shrink_tile(const LayerCall &c, int32_t K, int64_t tile, float4_t *joint)
{
    const AdaptCall &ad = c.ad;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, quad = lane >> 4;
    const int64_t m = tile * kRowsTile + col;
    const int id = m < c.M && row_active32(c.rows, (uint32_t)m) ? row_adapter(ad, m) : -1;
    const XT *x = (const XT *)c.x + (id >= 0 ? m : 0) * c.x_stride;
    const int kb = ad.a.kp / 32, b0 = kb * wave / 4, b1 = kb * (wave + 1) / 4;
    uint32_t todo = (uint32_t)__ballot(id >= 0) & 0xFFFFu;
    while (todo) {
        const int slot = __builtin_amdgcn_readlane(id, __builtin_ctz(todo));
        const uint32_t mine = (uint32_t)__ballot(id == slot) & 0xFFFFu;
        todo &= ~mine;
        const int rank = ad.a.ranks[slot], nb = (rank + 15) / 16;
        const float scale = ad.a.scales[slot];
        const AT *w = (const AT *)ad.a.down + ((size_t)slot * ad.a.rb * 16 + col) * ad.a.kp;
        for (int jb = 0; jb < nb; jb += 2) {            // (two blocks of ranks share what is read of x)
            float4_t d[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
            const AT *const w0 = w + (size_t)jb * 16 * ad.a.kp, *const w1 = jb + 1 < nb ? w0 + (size_t)16 * ad.a.kp : w0;
            int b = b0;
            for (; b + 4 <= b1; b += 4)
#pragma unroll
                for (int q = 0; q < 4; ++q) shrink_step<XT, AT>(x, id >= 0, w0, w1, (b + q) * 32 + quad * 8, K, d);
            for (; b < b1; ++b) shrink_step<XT, AT>(x, id >= 0, w0, w1, b * 32 + quad * 8, K, d);
            joint[(wave * kShrinkBlocks + jb) * kWaveSize + lane] = d[0];
            joint[(wave * kShrinkBlocks + jb + 1) * kWaveSize + lane] = d[1];
        }
        __syncthreads();
        for (int jb = wave; jb < nb; jb += 4) {
            float4_t d = joint[jb * kWaveSize + lane];
#pragma unroll
            for (int q = 1; q < 4; ++q) d += joint[(q * kShrinkBlocks + jb) * kWaveSize + lane];
            char *block = ad.h + (tile * ad.a.rb + jb) * h_block_bytes(ad.a.dtype);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float v = jb * 16 + col < rank ? d[i] * scale : 0.0f;
                float mx = finite_abs(v);               // over the row's 16 ranks
#pragma unroll
                for (int s = 1; s < 16; s <<= 1) mx = fmaxf(mx, __shfl_xor(mx, s, 64));
                if (mine >> (quad * 4 + i) & 1) put_h<AT>(block, quad * 4 + i, col, v, mx);
            }
        }
        __syncthreads();
    }
}

// Two 16-bit numbers with infinities and NaN as 0: those meet h in its first part
// alone (its other parts may be 0 where h is not).
__device__ __forceinline__ uint32_t finite_pair(uint32_t w, uint32_t exponent, uint32_t one)
{
    const uint32_t bad = ((w & exponent) + one) & 0x80008000u;      // (both halves: the exponent's last value carries)
    return w & ~((bad >> 15) * 0xFFFFu);
}

// The blocks (slot, 16 ranks) that a group of 16, 32 or 64 rows takes, each once, in one
// list for each of the wavefronts that share the group's sums: by the slot's number and
// the block's, so that a row's sum does not depend on the rows beside it. An entry:
// slot | block << 16, the rows it is for (64 bits), 0. One wavefront makes the lists of
// a group, a lane for each row.
__device__ __forceinline__ void make_lists(const LayerCall &c, int64_t group)
{
    const AdaptCall &ad = c.ad;
    const int lane = threadIdx.x & 63, G = ad.group, cap = G * ad.a.rb;
    const int64_t m = group * G + lane;
    const int id = lane < G && m < c.M && row_active32(c.rows, (uint32_t)m) ? row_adapter(ad, m) : -1;
    const int blocks = id >= 0 ? (ad.a.ranks[id] + 15) / 16 : 0;
    uint64_t mine = 0;
    for (int q = 0; q < G; ++q) mine |= (uint64_t)(id == __builtin_amdgcn_readlane(id, q)) << q;
    const bool first = id >= 0 && __builtin_ctzll(mine) == lane;
    uint4 *list = ad.lists + group * ad.parts * cap;
    for (int p = 0; p < ad.parts; ++p, list += cap) {
        const int j0 = (p - id) & (ad.parts - 1);       // the slot's first block of this part, then every parts-th
        const int n = first && blocks > j0 ? (blocks - j0 + ad.parts - 1) / ad.parts : 0;
        int end = n;
#pragma unroll
        for (int d = 1; d < kWaveSize; d <<= 1) {
            const int o = __shfl_up(end, d, kWaveSize);
            end += lane >= d ? o : 0;
        }
        for (int i = 0; i < n; ++i)
            list[end - n + i] = make_uint4((uint32_t)(id | (j0 + i * ad.parts) << 16), (uint32_t)mine, (uint32_t)(mine >> 32), 0);
        if (lane == kWaveSize - 1) ad.counts[group * ad.parts + p] = end;
    }
}

// What the adapters of a group of MT * 16 rows give to NT feature tiles, by the list of
// this wavefront, 64 entries at a time, a lane each. Blocks of up are loaded kAhead
// entries before they are used.
template <int MT, int NT, int kAhead>
struct AdapterTiles {
    const uint4 *list;
    int n, cap;
    uint4 entry;
    uint4 up[kAhead][NT];

    __device__ __forceinline__ void hold(int i)
    {
        if (MT == 1) {
            const uint2 e = *(const uint2 *)(list + i);
            entry = make_uint4(e.x, e.y, 0, 0);
        } else {
            entry = list[i];
        }
    }

    // The list's length and first entries (under way during the layer's product; what
    // lies behind the last entry is not used).
    __device__ __forceinline__ void begin(const AdaptCall &ad, int64_t group, int part)
    {
        cap = ad.group * ad.a.rb;
        list = ad.lists + (group * ad.parts + part) * cap;
        n = ad.counts[group * ad.parts + part];
        hold(min((int)(threadIdx.x & 63), cap - 1));
    }

    // (No branch: the count of loads under way has to be known. 16-bit blocks have 8 bytes
    // a lane, read twice.)
    __device__ __forceinline__ void fetch(const AdaptCall &ad, int nt0, int i, uint4 (&u)[NT]) const
    {
        const uint32_t lane = threadIdx.x & 63, bytes = ad.a.dtype == kF32 ? 16 : 8;
        const uint32_t e = (uint32_t)__builtin_amdgcn_readlane((int)entry.x, i);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const size_t t = ((size_t)(e & 0xFFFFu) * ad.a.nt + min(nt0 + n, ad.a.nt - 1)) * ad.a.rb + (e >> 16);
            const char *from = (const char *)ad.a.up + t * (kWaveSize * bytes) + lane * bytes;
            const uint2 lo = *(const uint2 *)from, hi = *(const uint2 *)(from + bytes - 8);
            u[n] = make_uint4(lo.x, lo.y, hi.x, hi.y);
        }
    }

    __device__ __forceinline__ void block(const AdaptCall &ad, const char *h, int i, const uint4 (&u)[NT], float4_t (&acc)[MT][NT]) const
    {
        const int jb = __builtin_amdgcn_readlane((int)entry.x, i) >> 16;
        const uint32_t rows[2] = {(uint32_t)__builtin_amdgcn_readlane((int)entry.y, i),
                                  MT > 2 ? (uint32_t)__builtin_amdgcn_readlane((int)entry.z, i) : 0u};
        const int lane = threadIdx.x & 63, quad = lane >> 4;
        const float4_t zero = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const uint32_t mine = rows[m / 2] >> (m % 2 * 16) & 0xFFFFu;
            if (!mine) continue;
            const char *b = h + (m * ad.a.rb + jb) * h_block_bytes(ad.a.dtype);
            float4_t d[NT];
            if (ad.a.dtype == kF32) {
                const float4_t a = ((const float4_t *)b)[lane];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const uint32_t w[4] = {u[n].x, u[n].y, u[n].z, u[n].w};
                    d[n] = zero;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        d[n] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[k], __uint_as_float(w[k]), d[n], 0, 0, 0);
                }
            } else if (ad.a.dtype == kF16) {
                const half4_t hi = ((const half4_t *)b)[lane], lo = ((const half4_t *)b)[64 + lane];
                const float4_t f = ((const float4_t *)(b + 1024))[quad];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    union { uint32_t u[2]; half4_t h; } w;
                    w.u[0] = u[n].x;
                    w.u[1] = u[n].y;
                    d[n] = __builtin_amdgcn_mfma_f32_16x16x16f16(hi, w.h, zero, 0, 0, 0);
                    w.u[0] = finite_pair(u[n].x, 0x7C007C00u, 0x04000400u);
                    w.u[1] = finite_pair(u[n].y, 0x7C007C00u, 0x04000400u);
                    const float4_t l = __builtin_amdgcn_mfma_f32_16x16x16f16(lo, w.h, zero, 0, 0, 0);
#pragma unroll
                    for (int i = 0; i < 4; ++i) d[n][i] = fmaf(l[i], 1.0f / 2048.0f, d[n][i]) * f[i];
                }
            } else {
                const short4_t a0 = ((const short4_t *)b)[lane], a1 = ((const short4_t *)b)[64 + lane],
                               a2 = ((const short4_t *)b)[128 + lane];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    union { uint32_t u[2]; short4_t h; } w;
                    w.u[0] = finite_pair(u[n].x, 0x7F807F80u, 0x00800080u);
                    w.u[1] = finite_pair(u[n].y, 0x7F807F80u, 0x00800080u);
                    d[n] = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(a2, w.h, zero, 0, 0, 0);
                    d[n] = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(a1, w.h, d[n], 0, 0, 0);
                    w.u[0] = u[n].x;
                    w.u[1] = u[n].y;
                    d[n] = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(a0, w.h, d[n], 0, 0, 0);
                }
            }
            // only the slot's own rows take it: an infinity in one request's adapter stays in its rows
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[m][n][i] = mine >> (quad * 4 + i) & 1 ? acc[m][n][i] + d[n][i] : acc[m][n][i];
        }
    }

    template <int I>
    __device__ __forceinline__ void step(const AdaptCall &ad, const char *h, int nt0, int i, int end, float4_t (&acc)[MT][NT])
    {
        uint4 u[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) u[n] = up[I][n];
        fetch(ad, nt0, min(i + I + kAhead, end - 1), up[I]);
        if (i + I < end) block(ad, h, i + I, u, acc);
        if constexpr (I + 1 < kAhead) step<I + 1>(ad, h, nt0, i, end, acc);
    }

    // h: the rows' blocks [MT][rb], in LDS.
    __device__ __forceinline__ void add(const AdaptCall &ad, const char *h, int nt0, float4_t (&acc)[MT][NT])
    {
        const int all = __builtin_amdgcn_readfirstlane(n);
        for (int base = 0; base < all; base += kWaveSize) {
            const int end = min(all - base, kWaveSize);
            if (base) hold(min(base + (int)(threadIdx.x & 63), all - 1));
            if (end <= 4) {                             // (filling the ring would cost more than it gains)
                for (int i = 0; i < end; i += 2) {
                    uint4 u[2][NT];
                    fetch(ad, nt0, i, u[0]);
                    fetch(ad, nt0, min(i + 1, end - 1), u[1]);
                    block(ad, h, i, u[0], acc);
                    if (i + 1 < end) block(ad, h, i + 1, u[1], acc);
                }
                continue;
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) fetch(ad, nt0, min(i, end - 1), up[i]);
            for (int i = 0; i < end; i += kAhead) step<0>(ad, h, nt0, i, end, acc);
        }
    }
};

// The blocks of h of `tiles` times 16 rows from a tile on, into LDS (no barrier).
__device__ __forceinline__ void stage_h(const LayerCall &c, int64_t tile, int tiles, char *to)
{
    const int64_t have = (c.M + kRowsTile - 1) / kRowsTile - tile;
    const int each = c.ad.a.rb * h_block_bytes(c.ad.a.dtype) / 16;
    const uint4 *from = (const uint4 *)c.ad.h + tile * each;
    const int n = (int)min((int64_t)tiles, have) * each;
    for (int i = threadIdx.x; i < n; i += blockDim.x) ((uint4 *)to)[i] = from[i];
}

}  // namespace

}  // namespace wfst
