// gfx950 (CDNA4) kernels of the scores of given tokens: log-probability and rank of each, the
// distribution's entropy, the best alternatives.
#include "wfst_score_device.h"

namespace wfst {

namespace {

// m = max x, d = (x - m) / T, S = sum exp d, lz = log S:
// log-probability d - lz, entropy lz - (sum exp(d) d) / S.
//
// A row is read once. Statistics are taken in units of log 2 (y = d log2 e), the
// largest entries (each exactly 1) counted apart so that a dominant label keeps its
// digits (log1p). A rank is a count over ballots. The alternatives: the n-th largest
// of the threads' own largest scores is a bound that n labels reach and few others;
// those it leaves go to a list in LDS, where each counts the ones before it.

typedef unsigned long long u64;

constexpr int kTokenWaves = 4;                 // wavefronts of a row (or of a piece of one)
constexpr int kTokenThreads = kTokenWaves * kWaveSize;
constexpr int kMaxPieces = 64;                 // pieces of one row

// Order of labels as integers: larger scores first, then lower indexes; 0: none
// (-inf, NaN). One zero.
__device__ __forceinline__ uint32_t score_key(float x)
{
    const uint32_t u = __float_as_uint(x + 0.0f);
    return x > -INFINITY ? (u & 0x80000000u ? ~u : u | 0x80000000u) : 0u;
}

__device__ __forceinline__ u64 label_key(float x, int v) { return (u64)score_key(x) << 32 | (uint32_t)~v; }

__device__ __forceinline__ float key_score(uint32_t u) { return __uint_as_float(u & 0x80000000u ? u & 0x7FFFFFFFu : ~u); }

__device__ __forceinline__ int count(bool b) { return __popcll(__ballot(b)); }

// What a row's temperature makes of its distances. Where z - m could pass binary32's
// range, half of it is taken times 2 / T. T below 2^-125 counts as that for the sums.
struct Heat { float t, scale; };

__device__ __forceinline__ Heat row_heat(const TokenCall &c, int64_t r)
{
    float t = c.temperatures ? c.temperatures[r] : c.temperature;
    t = t > 0.0f ? fminf(t, 3.402823466e38f) : 0.0f;
    return {t, 1.44269504088896341f / fmaxf(t, 0x1p-125f)};
}

struct Base { float half, mh, scale; };        // y = (z half - mh) scale

__device__ __forceinline__ Base base_of(float m, const Heat &h)
{
    const float half = m > 0x1p100f ? 0.5f : 1.0f;
    return {half, m * half, h.scale / half};
}

__device__ __forceinline__ float below(float z, const Base &b) { return fmaf(z, b.half, -b.mh) * b.scale; }

// Statistics of a set of z: the largest, how many equal it, and over the others the
// sums of e = 2^y and of e y. +inf as the largest says that the set has a NaN or +inf.
struct TokenStat { float m, ones, sum, ysum; };

__device__ __forceinline__ TokenStat stat_join(const TokenStat &a, const TokenStat &b, const Heat &h)
{
    TokenStat r;
    r.m = fmaxf(a.m, b.m);
    r.ones = r.sum = r.ysum = 0.0f;
    if (r.m == INFINITY || r.m == -INFINITY) return r;
    const Base base = base_of(r.m, h);
    const TokenStat *const s[2] = {&a, &b};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (s[i]->m == r.m) {
            r.ones += s[i]->ones;
            r.sum += s[i]->sum;
            r.ysum += s[i]->ysum;
        } else {
            const float y = fmaxf(below(s[i]->m, base), -200.0f), f = __builtin_amdgcn_exp2f(y);
            const float all = s[i]->sum + s[i]->ones;
            r.sum += f * all;
            r.ysum += f * fmaf(y, all, s[i]->ysum);
        }
    }
    return r;
}

// What a row's results need of its statistics.
struct TokenRow { float m, half, t, lz, entropy; };

__device__ __forceinline__ TokenRow row_result(const TokenStat &s, const Heat &h)
{
    TokenRow r = {s.m, s.m > 0x1p100f ? 0.5f : 1.0f, h.t, 0.0f, 0.0f};
    if (s.m == INFINITY) {
        r.lz = r.entropy = NAN;
    } else if (s.m > -INFINITY && h.t > 0.0f) {
        r.lz = log1pf((s.ones - 1.0f) + s.sum);
        r.entropy = r.lz - 0.693147180559945309f * (s.ysum / (s.ones + s.sum));
    }
    return r;
}

__device__ __forceinline__ float log_prob(const TokenRow &r, float z, int rank)
{
    if (r.lz != r.lz) return NAN;
    if (!(z > -INFINITY)) return -INFINITY;
    if (r.t == 0.0f) return rank == 0 ? 0.0f : -INFINITY;
    return fmaf(z, r.half, -r.m * r.half) / r.t / r.half - r.lz;
}

// The n-th largest (at least) of the keys that WORDS words of each lane hold (0:
// none): the largest prefix of bits that n or more reach, all bits where more than n
// do. reach: how many do. 0 where there are fewer.
template <typename K, int WORDS>
__device__ __forceinline__ K nth_key(const K (&u)[WORDS], int n, int &reach)
{
    K b = 0;
    reach = 0;
    for (int bit = 8 * (int)sizeof(K) - 1; bit >= 0 && reach != n; --bit) {
        const K t = b | (K)1 << bit;
        int got = 0;
#pragma unroll
        for (int w = 0; w < WORDS; ++w) got += count(u[w] >= t);
        if (got >= n) { b = t; reach = got; }
    }
    return b;
}

// LDS of the wavefronts that share a row.
template <int WAVES> struct TokenShared {
    uint32_t top[WAVES > 1 ? WAVES * kWaveSize : 1];    // each thread's largest
    int32_t at[WAVES > 1 ? WAVES * kWaveSize : 1];      // where it stands first
    float red[4 * WAVES];
    int32_t ranks[WAVES > 1 ? kMaxTokens : 1];
    float scores[WAVES > 1 ? kMaxTokens : 1];
    int32_t listed;
};

template <int WAVES>
__device__ __forceinline__ void row_sync()
{
    if constexpr (WAVES > 1) {
        __syncthreads();
    } else {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
}

template <typename XT> constexpr int kTokenVec = 16 / (int)sizeof(XT);

// Sizes of a launch: a row in `pieces` of `subs` runs of WAVES * 64 * VEC * NV labels.
struct TokenPlan { int32_t pieces, subs, list; };       // list: u64 of a row's list in LDS

// What pieces leave for the join: [rows * pieces] statistics, [..][n] sorted keys, [..][C] ranks.
struct TokenWork { TokenStat *stats; u64 *keys; int32_t *ranks; };

__device__ __forceinline__ TokenWork token_work(void *w, int64_t items, int32_t n)
{
    TokenWork r;
    r.stats = (TokenStat *)w;
    r.keys = (u64 *)(r.stats + items);
    r.ranks = (int32_t *)(r.keys + items * n);
    return r;
}

template <typename XT, int WAVES, int NV>
__global__ __launch_bounds__(kTokenThreads) void k_token_rows(TokenCall c, TokenPlan plan)
{
    constexpr int VEC = kTokenVec<XT>;
    constexpr int kSpan = WAVES * kWaveSize * VEC;
    constexpr int kRows = kTokenWaves / WAVES;          // rows of a workgroup
    __shared__ TokenShared<WAVES> shared[kRows];
    extern __shared__ __align__(16) u64 lists[];
    const int lane = threadIdx.x & 63, slot = WAVES > 1 ? 0 : threadIdx.x >> 6;
    const int tid = WAVES > 1 ? threadIdx.x : lane, wave = WAVES > 1 ? threadIdx.x >> 6 : 0;
    TokenShared<WAVES> &sh = shared[slot];
    u64 *list = lists + (size_t)slot * plan.list, *best = list + plan.list - c.top_n;
    const int n = c.top_n, C = c.C;
    const int64_t items = c.rows * plan.pieces;
    const TokenWork work = token_work(c.workspace, items, n);

    for (int64_t w = (int64_t)blockIdx.x * kRows + slot; w < items; w += (int64_t)gridDim.x * kRows) {
        const int64_t r = plan.pieces > 1 ? w / plan.pieces : w;
        const int piece = (int)(w - r * plan.pieces);
        if (!row_active(c.set, r)) continue;
        const XT *x = (const XT *)c.x + r * c.x_stride;
        const int32_t *tokens = c.tokens + r * C;
        const Heat heat = row_heat(c, r);

        // the given tokens, a lane each, and their scores
        int tok = lane < C ? tokens[lane] : -1;
        float zt = tok >= 0 && tok < c.V ? (float)x[tok] : -INFINITY;

        TokenStat all = {-INFINITY, 0.0f, 0.0f, 0.0f};
        int kept = 0;                                   // keys at the head of the list, sorted
        for (int sub = 0; sub < plan.subs; ++sub) {
            const int first = (piece * plan.subs + sub) * (kSpan * NV);
            if (first >= c.V) break;
            const int v0 = first + tid * VEC;
            float z[NV][VEC];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int v = v0 + i * kSpan;
                if (v + VEC <= c.V) {
                    const Pack<XT, VEC> p = *(const Pack<XT, VEC> *)(x + v);
#pragma unroll
                    for (int j = 0; j < VEC; ++j) z[i][j] = (float)p.v[j];
                } else {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) z[i][j] = v + j < c.V ? (float)x[v + j] : -INFINITY;
                }
            }
            TokenStat s = {-INFINITY, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < VEC; ++j) s.m = fmaxf(s.m, z[i][j]);
            const float mine = s.m;
            s.m = wave_max_f(s.m);
            if (WAVES > 1) {
                if (n) sh.top[tid] = score_key(mine);
                if (lane == 0) sh.red[wave] = s.m;
                if (tid == 0) sh.listed = kept;
                if (sub == 0)
                    for (int i = tid; i < C; i += kTokenThreads) sh.ranks[i] = 0;
                row_sync<WAVES>();
#pragma unroll
                for (int q = 0; q < WAVES; ++q) s.m = fmaxf(s.m, sh.red[q]);
            } else if (tid == 0) {
                sh.listed = 0;
            }

            // sums
            if (s.m > -INFINITY && heat.t > 0.0f) {
                const Base base = base_of(s.m, heat);
                uint32_t ones = 0;
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        const float y = below(z[i][j], base), e = __builtin_amdgcn_exp2f(y);
                        const bool top = z[i][j] == s.m;
                        ones += count(top);             // (on the scalar unit)
                        s.sum += top ? 0.0f : e;
                        s.ysum = fmaf(e, fmaxf(y, -200.0f), s.ysum);
                    }
                s.ones = (float)ones;
            } else {
                bool nan = false;
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int j = 0; j < VEC; ++j) nan |= z[i][j] != z[i][j];
                s.sum = nan ? NAN : 0.0f;
            }
            s.sum = wave_sum_f(s.sum);
            s.ysum = wave_sum_f(s.ysum);
            if (WAVES > 1 && lane == 0) {
                sh.red[WAVES + wave] = s.sum;
                sh.red[2 * WAVES + wave] = s.ysum;
                sh.red[3 * WAVES + wave] = s.ones;
            }

            // ranks: labels of this run before each token
            int before = 0;
            for (int i = 0; i < C; ++i) {
                if (i && i % kWaveSize == 0) {          // (the next 64 tokens)
                    tok = i + lane < C ? tokens[i + lane] : -1;
                    zt = tok >= 0 && tok < c.V ? (float)x[tok] : -INFINITY;
                }
                const float a = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(zt), i % kWaveSize));
                const int at = __builtin_amdgcn_readlane(tok, i % kWaveSize);
                int got = 0;
                if (a > -INFINITY) {
#pragma unroll
                    for (int q = 0; q < NV; ++q)
#pragma unroll
                        for (int j = 0; j < VEC; ++j) {
                            got += count(z[q][j] > a);
                            if (__ballot(z[q][j] == a)) got += count(z[q][j] == a && v0 + q * kSpan + j < at);
                        }
                } else {                                // (-inf and NaN stand last, by index)
#pragma unroll
                    for (int q = 0; q < NV; ++q)
#pragma unroll
                        for (int j = 0; j < VEC; ++j)
                            got += count(z[q][j] > -INFINITY || v0 + q * kSpan + j < at);
                }
                before = i % kWaveSize == lane ? got : before;
                if (i % kWaveSize == kWaveSize - 1 || i == C - 1) {
                    const int k = i / kWaveSize * kWaveSize + lane;
                    if (WAVES > 1) {
                        if (k < C) {
                            atomicAdd(&sh.ranks[k], before);
                            if (wave == 0) sh.scores[k] = zt;
                        }
                    } else if (k < C) {
                        TokenStat f = s;
                        if (f.sum != f.sum) f.m = INFINITY;
                        const TokenRow row = row_result(f, heat);
                        const bool is = tok >= 0 && tok < c.V;
                        c.log_probs[r * C + k] = is ? log_prob(row, zt, before) : -INFINITY;
                        c.ranks[r * C + k] = is ? before : -1;
                    }
                }
            }
            if (C > kWaveSize && sub + 1 < plan.subs) {
                tok = tokens[lane];
                zt = tok >= 0 && tok < c.V ? (float)x[tok] : -INFINITY;
            }

            // labels that may be among the n best: those that reach the bound
            if (n) {
                int reach;
                uint32_t bound;
                uint32_t u[WAVES];
#pragma unroll
                for (int q = 0; q < WAVES; ++q) u[q] = WAVES > 1 ? sh.top[q * kWaveSize + lane] : score_key(mine);
                bound = nth_key<uint32_t, WAVES>(u, n, reach);
                // more threads tie at the bound than are needed: those whose largest stands first
                int last = 0x7FFFFFFF;
                const bool tie = reach > n;             // (the same for the whole row)
                if (tie) {
                    int at = 0x7FFFFFFF;
#pragma unroll
                    for (int i = NV - 1; i >= 0; --i)
#pragma unroll
                        for (int j = VEC - 1; j >= 0; --j)
                            if (z[i][j] == mine) at = v0 + i * kSpan + j;
                    if (WAVES > 1) {
                        sh.at[tid] = at;
                        row_sync<WAVES>();
                    }
                    uint32_t late[WAVES];               // (the earliest is the largest)
                    int more = 0;
#pragma unroll
                    for (int q = 0; q < WAVES; ++q) {
                        late[q] = u[q] == bound ? ~(uint32_t)(WAVES > 1 ? sh.at[q * kWaveSize + lane] : at) : 0u;
                        more += count(u[q] > bound);
                    }
                    int got;
                    last = (int)~nth_key<uint32_t, WAVES>(late, n - more, got);
                }
                float lo = key_score(max(bound, 0x00800000u));
                if (kept == n) {                        // (later labels only pass with a larger score)
                    const float run = key_score((uint32_t)(list[n - 1] >> 32));
                    if (run >= lo) { lo = run; last = -1; }
                }
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        const int v = v0 + i * kSpan + j;
                        bool hit = z[i][j] >= lo;
                        u64 mask = __ballot(hit);
                        if (!mask) continue;
                        if (last != 0x7FFFFFFF) {
                            hit = hit && (z[i][j] > lo || v <= last);
                            mask = __ballot(hit);
                            if (!mask) continue;
                        }
                        int base = 0;
                        if (lane == 0) base = atomicAdd(&sh.listed, __popcll(mask));
                        base = __builtin_amdgcn_readfirstlane(base);
                        const int k = base + __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32),
                                                                       __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
                        if (hit) list[k] = label_key(z[i][j], v);
                    }
            }
            row_sync<WAVES>();
            if (WAVES > 1) {
                s.sum = s.ysum = s.ones = 0.0f;
#pragma unroll
                for (int q = 0; q < WAVES; ++q) {
                    s.sum += sh.red[WAVES + q];
                    s.ysum += sh.red[2 * WAVES + q];
                    s.ones += sh.red[3 * WAVES + q];
                }
            }
            if (s.sum != s.sum) s.m = INFINITY;
            all = sub == 0 ? s : stat_join(all, s, heat);

            // the list sorted: each key counts the larger ones
            if (n) {
                const int L = sh.listed;
                const bool more = sub + 1 < plan.subs && first + kSpan * NV < c.V;
                const bool final = plan.pieces == 1 && !more;
                TokenRow row;
                if (final) row = row_result(all, heat);
                for (int i = tid; i < L; i += WAVES * kWaveSize) {
                    const u64 k = list[i];
                    int rank = 0;
                    for (int q = 0; q < L; ++q) rank += list[q] > k;
                    if (rank >= n) continue;
                    if (final) {
                        const float f = key_score((uint32_t)(k >> 32));
                        c.top_tokens[r * n + rank] = (int32_t)~(uint32_t)k;
                        c.top_log_probs[r * n + rank] = log_prob(row, f, rank);
                    } else if (!more) {
                        work.keys[w * n + rank] = k;
                    } else {
                        best[rank] = k;
                    }
                }
                if (!more) {
                    for (int i = L + tid; i < n; i += WAVES * kWaveSize) {
                        if (final) {
                            c.top_tokens[r * n + i] = -1;
                            c.top_log_probs[r * n + i] = -INFINITY;
                        } else {
                            work.keys[w * n + i] = 0;
                        }
                    }
                } else {
                    row_sync<WAVES>();
                    kept = min(L, n);
                    for (int i = tid; i < kept; i += WAVES * kWaveSize) list[i] = best[i];
                }
            }
            if (WAVES > 1) row_sync<WAVES>();
        }

        if (plan.pieces > 1) {
            if (tid == 0) work.stats[w] = all;
            for (int i = tid; i < C; i += WAVES * kWaveSize) work.ranks[w * C + i] = sh.ranks[i];
        } else {
            const TokenRow row = row_result(all, heat);
            if (tid == 0 && c.entropies) c.entropies[r] = row.entropy;
            if (WAVES > 1)
                for (int i = tid; i < C; i += kTokenThreads) {
                    const int t = tokens[i];
                    const bool is = t >= 0 && t < c.V;
                    c.log_probs[r * C + i] = is ? log_prob(row, sh.scores[i], sh.ranks[i]) : -INFINITY;
                    c.ranks[r * C + i] = is ? sh.ranks[i] : -1;
                }
        }
        row_sync<WAVES>();
    }
}

// Joins a row's pieces: one workgroup a row.
constexpr int kJoinList = kMaxTop * ((kMaxPieces * kMaxTop + kTokenThreads - 1) / kTokenThreads);

__global__ __launch_bounds__(kTokenThreads) void k_token_join(TokenCall c, int32_t P, int32_t xcode)
{
    __shared__ u64 top[kTokenThreads], list[kJoinList];
    __shared__ int32_t listed;
    const int tid = threadIdx.x, lane = tid & 63, n = c.top_n, C = c.C;
    const TokenWork work = token_work(c.workspace, c.rows * P, n);
    for (int64_t r = blockIdx.x; r < c.rows; r += gridDim.x) {
        if (!row_active(c.set, r)) continue;
        const Heat heat = row_heat(c, r);
        TokenStat s = {-INFINITY, 0.0f, 0.0f, 0.0f};
        if (lane < P) s = work.stats[r * P + lane];
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) {
            const TokenStat o = {__shfl_xor(s.m, d, 64), __shfl_xor(s.ones, d, 64), __shfl_xor(s.sum, d, 64),
                                 __shfl_xor(s.ysum, d, 64)};
            s = lane & d ? stat_join(o, s, heat) : stat_join(s, o, heat);
        }
        const TokenRow row = row_result(s, heat);
        if (tid == 0 && c.entropies) c.entropies[r] = row.entropy;
        for (int i = tid; i < C; i += kTokenThreads) {
            const int t = c.tokens[r * C + i];
            int before = 0;
            for (int p = 0; p < P; ++p) before += work.ranks[(r * P + p) * C + i];
            float z = -INFINITY;
            const bool is = t >= 0 && t < c.V;
            if (is) {
                const int64_t at = r * c.x_stride + t;
                z = xcode == kF32 ? ((const float *)c.x)[at] : xcode == kF16 ? (float)((const _Float16 *)c.x)[at]
                                                                            : (float)((const __bf16 *)c.x)[at];
            }
            c.log_probs[r * C + i] = is ? log_prob(row, z, before) : -INFINITY;
            c.ranks[r * C + i] = is ? before : -1;
        }
        if (!n) continue;
        const u64 *keys = work.keys + r * P * n;
        u64 mine = 0;
        for (int i = tid; i < P * n; i += kTokenThreads) mine = max(mine, keys[i]);
        top[tid] = mine;
        if (tid == 0) listed = 0;
        __syncthreads();
        u64 u[kTokenWaves];
#pragma unroll
        for (int q = 0; q < kTokenWaves; ++q) u[q] = top[q * kWaveSize + lane];
        int reach;
        const u64 bound = max(nth_key<u64, kTokenWaves>(u, n, reach), (u64)1);
        for (int i = tid; i < P * n; i += kTokenThreads) {
            const u64 k = keys[i];
            if (k >= bound) list[atomicAdd(&listed, 1)] = k;
        }
        __syncthreads();
        const int L = listed;
        for (int i = tid; i < L; i += kTokenThreads) {
            const u64 k = list[i];
            int rank = 0;
            for (int q = 0; q < L; ++q) rank += list[q] > k;
            if (rank >= n) continue;
            c.top_tokens[r * n + rank] = (int32_t)~(uint32_t)k;
            c.top_log_probs[r * n + rank] = log_prob(row, key_score((uint32_t)(k >> 32)), rank);
        }
        for (int i = L + tid; i < n; i += kTokenThreads) {
            c.top_tokens[r * n + i] = -1;
            c.top_log_probs[r * n + i] = -INFINITY;
        }
        __syncthreads();
    }
}

// Runs of a wavefront's or a workgroup's registers that a row takes.
struct TokenShape { int waves, nv, pieces, subs; };

TokenShape token_shape(int64_t rows, int32_t V, int32_t x_dtype)
{
    const int vec = x_dtype == kF32 ? 4 : 8, lane = kWaveSize * vec;
    const auto up = [](int64_t a, int64_t b) { return (int)((a + b - 1) / b); };
    if (V <= 8 * lane) return {1, V <= 2 * lane ? 2 : V <= 4 * lane ? 4 : 8, 1, 1};
    const int span = kTokenWaves * lane;
    if (V <= 8 * span) return {kTokenWaves, std::max(3, up(V, span)), 1, 1};
    const int nv = rows * up(V, 8 * span) >= 512 ? 8 : 2, len = nv * span;
    const int subs = up(up(V, len), kMaxPieces);
    return {kTokenWaves, nv, up(V, (int64_t)len * subs), subs};
}

template <typename XT, int WAVES, int NV>
void rows_launch(const TokenCall &c, const TokenShape &t, hipStream_t s)
{
    const int rows = kTokenWaves / WAVES, each = NV * kTokenVec<XT>;
    const int most = std::min(c.top_n * each, c.V);       // labels that reach the bound
    const TokenPlan plan = {t.pieces, t.subs, c.top_n + most + c.top_n};
    const size_t lds = c.top_n ? (size_t)rows * plan.list * sizeof(u64) : 0;
    const int64_t groups = (c.rows * t.pieces + rows - 1) / rows;
    hipLaunchKernelGGL((k_token_rows<XT, WAVES, NV>), dim3((unsigned)std::min<int64_t>(groups, kMaxRowGrid)),
                       dim3(kTokenThreads), lds, s, c, plan);
}

template <typename XT>
hipError_t token_launch(const TokenCall &c, hipStream_t s)
{
    const TokenShape t = token_shape(c.rows, c.V, c.x_dtype);
    if (t.waves == 1) {
        if (t.nv == 2) rows_launch<XT, 1, 2>(c, t, s);
        else if (t.nv == 4) rows_launch<XT, 1, 4>(c, t, s);
        else rows_launch<XT, 1, 8>(c, t, s);
    } else {
        switch (t.nv) {
        case 2: rows_launch<XT, kTokenWaves, 2>(c, t, s); break;
        case 3: rows_launch<XT, kTokenWaves, 3>(c, t, s); break;
        case 4: rows_launch<XT, kTokenWaves, 4>(c, t, s); break;
        case 5: rows_launch<XT, kTokenWaves, 5>(c, t, s); break;
        case 6: rows_launch<XT, kTokenWaves, 6>(c, t, s); break;
        default: rows_launch<XT, kTokenWaves, 8>(c, t, s); break;
        }
    }
    if (t.pieces > 1)
        hipLaunchKernelGGL(k_token_join, dim3((unsigned)std::min<int64_t>(c.rows, kMaxRowGrid)), dim3(kTokenThreads), 0,
                           s, c, t.pieces, c.x_dtype);
    return hipGetLastError();
}

}  // namespace

size_t token_workspace(int64_t rows, int32_t V, int32_t C, int32_t top_n, int32_t x_dtype)
{
    const TokenShape t = token_shape(rows, V, x_dtype);
    if (t.pieces == 1) return 0;
    return (size_t)rows * t.pieces * (sizeof(TokenStat) + (size_t)top_n * sizeof(u64) + (size_t)C * 4);
}

hipError_t launch_token_scores(const TokenCall &c, hipStream_t s)
{
    if (c.x_dtype == kF32) return token_launch<float>(c, s);
    if (c.x_dtype == kF16) return token_launch<_Float16>(c, s);
    return token_launch<__bf16>(c, s);
}

}  // namespace wfst
