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
//
// What bounds it: the vector instructions, about 16 a label (the exponential counts 4)
// and some 250 a wavefront; binary32 rows without tokens and alternatives run at 5.9 TB/s
// (16000 x 5000 in 54 us), binary16 ones at 4.1 (39 us; one token 49, with 4 alternatives 61).
// Registers decide how many rows are under way at once: loading the next row ahead cost
// more of them than it hid (binary16 107 us).

typedef unsigned long long u64;


constexpr int kTokenWaves = 4;                 // wavefronts of a row (or of a piece of one)
constexpr int kTokenThreads = kTokenWaves * kWaveSize;
constexpr int kMaxPieces = 64;                 // pieces of one row
constexpr int kShortGrid = 4096;               // workgroups of a launch over short rows: each takes several where there are more

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
// range, half of it is taken times 2 / T; where 1 / T could, unit = 2^24 times it and 1 / (unit T).
constexpr float kLog2e = 1.44269504088896341f;

struct Heat { float t, unit, scale; };

__host__ __device__ __forceinline__ Heat heat_of(float t)
{
    const float unit = t < 0x1p-125f ? 0x1p24f : 1.0f, d = t * unit;
    return {t, unit, kLog2e / (d < 0x1p-125f ? 0x1p-125f : d)};        // (T = 0: of no use, but finite)
}

__device__ __forceinline__ Heat row_heat(const TokenCall &c, int64_t r)
{
    if (!c.temperatures) return {c.temperature, c.unit, c.scale};
    const float t = c.temperatures[r];
    return heat_of(t > 0.0f ? fminf(t, 3.402823466e38f) : 0.0f);
}

struct Base { float half, mh, scale; };        // y = (z half - mh) scale, half a power of two

__device__ __forceinline__ Base base_of(float m, const Heat &h)
{
    // (far out distances are 0 or 2^76 and more, whose exponentials are 0 at any T that has a unit)
    const bool far = fabsf(m) > 0x1p100f;
    const float half = far ? 0.5f : h.unit;
    return {half, m * half, far ? 2.0f * h.scale : h.scale};
}

__device__ __forceinline__ float below(float z, const Base &b) { return fmaf(z, b.half, -b.mh) * b.scale; }

// The next smaller number, for a number above -inf.
__device__ __forceinline__ float next_below(float a)
{
    const uint32_t u = __float_as_uint(a);
    return __uint_as_float(u << 1 == 0 ? 0x80000001u : u & 0x80000000u ? u + 1 : u - 1);
}

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

// log(1 + x) for x >= 0: the logarithm of the rounded u = 1 + x and, times 1 / u, what
// the rounding lost (x itself where u is 1).
__device__ __forceinline__ float log1p_of(float x)
{
    const float u = 1.0f + x;
    return fmaf(x - (u - 1.0f), __builtin_amdgcn_rcpf(u), 0.693147180559945309f * __builtin_amdgcn_logf(u));
}

// What a row's results need of its statistics.
struct TokenRow { float m, half, t, lz, entropy; };

__device__ __forceinline__ TokenRow row_result(const TokenStat &s, const Heat &h)
{
    TokenRow r = {s.m, s.m > 0x1p100f ? 0.5f : 1.0f, h.t, 0.0f, 0.0f};
    if (s.m == INFINITY) {
        r.lz = r.entropy = NAN;
    } else if (s.m > -INFINITY && h.t > 0.0f) {
        r.lz = log1p_of((s.ones - 1.0f) + s.sum);
        r.entropy = fmaf(-0.693147180559945309f * s.ysum, __builtin_amdgcn_rcpf(s.ones + s.sum), r.lz);
    }
    return r;
}

__device__ __forceinline__ float log_prob(const TokenRow &r, float z, int rank)
{
    if (r.lz != r.lz) return NAN;
    if (!(z > -INFINITY)) return -INFINITY;
    if (r.t == 0.0f) return rank == 0 ? 0.0f : -INFINITY;
    const float d = fmaf(z, r.half, -r.m * r.half);
    return (r.t == 1.0f ? d : d / r.t) * (r.half == 1.0f ? 1.0f : 2.0f) - r.lz;
}

// How many labels or threads may reach a bound that n have to.
__host__ __device__ constexpr int bound_cap(int n) { return n + n / 4 + 2; }

// A bound that n or more of a set of keys reach: the first prefix of bits, from the
// highest on, that n to bound_cap(n) do, or with all bits the n-th largest key itself
// (more of its kind may reach it). got(t): how many reach t. reach: how many reach the
// result. 0 where there are fewer than n, or few keys at all.
template <typename K, typename F>
__device__ __forceinline__ K nth_key(int n, int all, int &reach, F &&got)
{
    K b = 0;
    reach = all;
    for (int bit = 8 * (int)sizeof(K) - 1; bit >= 0 && reach > bound_cap(n); --bit) {
        const K t = b | (K)1 << bit;
        const int g = got(t);
        if (g >= n) { b = t; reach = g; }
    }
    return b;
}

// LDS of the wavefronts that share a row.
template <int WAVES> struct TokenShared {
    uint32_t top[WAVES > 1 ? WAVES * kWaveSize : 1];    // each thread's largest
    int32_t at[WAVES > 1 ? WAVES * kWaveSize : 1];      // where it stands first
    float red[4 * WAVES];
    int32_t ranks[WAVES > 1 ? kMaxTokens : 1];
    int32_t listed;
};

// All lanes of the row have passed their LDS accesses.
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

__device__ __forceinline__ float read_lane(float v, int lane)
{
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}

// NV packs a thread of a run of labels that begins at `first`; the thread's first
// label is v0. A pack that crosses V is read from V - VEC on, its labels that belong
// to the pack before it are -inf then.
template <typename XT, int WAVES, int NV>
struct TokenRun {
    static constexpr int VEC = kTokenVec<XT>;
    static constexpr int kSpan = WAVES * kWaveSize * VEC;
    float z[NV][VEC], pm[NV];                           // pm: each pack's largest
    float mine;                                         // the thread's
    int first, v0, tid, V;

    // The label of element j of pack i of the thread whose first label is v.
    __device__ __forceinline__ int label(int v, int i, int j) const { return min(v + i * kSpan, max(V - VEC, 0)) + j; }

    // v0 for use in a branch that few threads take: the compiler neither computes what
    // follows from it before the branch nor keeps it from row to row (2.4 registers a label).
    __device__ __forceinline__ int own_v0() const
    {
        int v = v0;
        asm volatile("" : "+v"(v));
        return v;
    }

    // Pack i of this wavefront holds labels (the same for all its lanes).
    __device__ __forceinline__ bool used(int i) const
    {
        return __builtin_amdgcn_readfirstlane(v0) + i * kSpan < V;
    }

    struct __attribute__((packed, aligned(sizeof(XT)))) Raw { uint32_t w[4]; };
    typedef Raw Packs[NV];

    static __device__ __forceinline__ float element(const Raw &p, int j)
    {
        if constexpr (sizeof(XT) == 4) return __uint_as_float(p.w[j]);
        const uint32_t h = j & 1 ? p.w[j / 2] >> 16 : p.w[j / 2] & 0xFFFFu;
        union { uint16_t u; _Float16 f; } c;
        c.u = (uint16_t)h;
        return __is_same(XT, _Float16) ? (float)c.f : __uint_as_float(h << 16);
    }

    static __device__ __forceinline__ void fetch(const XT *x, int V, int first, int tid, Packs &p)
    {
        if (V >= VEC) {
#pragma unroll
            for (int i = 0; i < NV; ++i) p[i] = *(const Raw *)(x + min(first + tid * VEC + i * kSpan, V - VEC));
        } else {
            union { XT v[VEC]; Raw r; } u;
#pragma unroll
            for (int j = 0; j < VEC; ++j) u.v[j] = j < V ? x[j] : (XT)-INFINITY;
#pragma unroll
            for (int i = 0; i < NV; ++i) p[i] = u.r;
        }
    }

    __device__ __forceinline__ TokenRun(const Packs &p, int labels, int f, int t) : first(f), v0(f + t * VEC), tid(t), V(labels)
    {
        const int v = own_v0();
        mine = -INFINITY;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) z[i][j] = element(p[i], j);
            if (first + (i + 1) * kSpan > V) {          // (the last packs of a row)
                const int before = v + i * kSpan - label(v, i, 0);
#pragma unroll
                for (int j = 0; j < VEC; ++j) z[i][j] = j >= before ? z[i][j] : -INFINITY;
            }
            pm[i] = z[i][0];
#pragma unroll
            for (int j = 1; j < VEC; ++j) pm[i] = fmaxf(pm[i], z[i][j]);
            mine = fmaxf(mine, pm[i]);
        }
    }

    // The sums below the row's largest over this wavefront's labels; TOP: it holds that
    // largest, whose entries are counted and left out.
    template <bool TOP>
    __device__ __forceinline__ void add_up(const Base &base, TokenStat &s) const
    {
        uint32_t others = 0, packs = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!used(i)) continue;
            ++packs;
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float y = below(z[i][j], base), e = __builtin_amdgcn_exp2f(y);
                const bool other = !TOP || z[i][j] != s.m;
                if (TOP) others += count(other);        // (on the scalar unit)
                s.sum += other ? e : 0.0f;
                s.ysum = fmaf(e, fmaxf(y, -200.0f), s.ysum);
            }
        }
        if (TOP) s.ones = (float)(packs * VEC * kWaveSize - others);
    }

    // A wavefront's part of the sums below the row's or run's largest, s.m (a NaN as its sum).
    __device__ __forceinline__ void sums(const Heat &heat, float wave_max, TokenStat &s) const
    {
        s.ones = s.sum = s.ysum = 0.0f;
        if (s.m > -INFINITY && heat.t > 0.0f) {
            const Base base = base_of(s.m, heat);
            if (WAVES == 1 || wave_max == s.m) add_up<true>(base, s);
            else add_up<false>(base, s);
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
    }

    // A lane's labels before the token `at` of score a (a label, or a = -inf). Packs
    // before the token's own count its equals too, by the next smaller score as their
    // bound; the wavefront `home` looks at the token's own pack. NaN and -inf stand
    // last, by index.
    __device__ __forceinline__ int before(const XT *x, float a, int at, bool home) const
    {
        int got = 0;
        if (a > -INFINITY) {
            const float down = next_below(a);
#pragma unroll
            for (int q = 0; q < NV; ++q) {
                if (!used(q)) continue;
                const float over = at - v0 >= q * kSpan + VEC ? down : a;
#pragma unroll
                for (int j = 0; j < VEC; ++j) got += z[q][j] > over;
            }
            const int pack = at / VEC * VEC, lane = tid & 63;
            if (home && pack >= first && pack < first + kSpan * NV && lane < VEC && pack + lane < at)
                got += (float)x[pack + lane] == a;
        } else {
            const int v = own_v0();
            float none = -INFINITY;
            asm volatile("" : "+v"(none));              // (else every row compares ahead of this branch)
#pragma unroll
            for (int q = 0; q < NV; ++q)
#pragma unroll
                for (int j = 0; j < VEC; ++j)
                    got += z[q][j] > none || (v + q * kSpan <= label(v, q, j) && label(v, q, j) < at);
        }
        return got;
    }

    // Of m tokens, a lane each, this wavefront's labels before them.
    __device__ __forceinline__ int ranks(const XT *x, float zt, int tok, int m, bool home) const
    {
        const int lane = tid & 63;
        int mine_of = 0;
        for (int k = 0; k < m; k += 2) {                // (two counts below 2^16 in one sum)
            int got = before(x, read_lane(zt, k), __builtin_amdgcn_readlane(tok, k), home);
            if (k + 1 < m) got += before(x, read_lane(zt, k + 1), __builtin_amdgcn_readlane(tok, k + 1), home) << 16;
            got = wave_sum_i(got);
            mine_of = lane == k ? got & 0xFFFF : lane == k + 1 ? got >> 16 : mine_of;
        }
        return mine_of;
    }

    // Appends the labels that may be among the n best to the list (kept of them there,
    // sorted): the ones that reach a bound. sh.top holds the threads' largest and
    // sh.listed is `kept`. The labels of at most bound_cap(n) threads are listed.
    __device__ __forceinline__ void candidates(TokenShared<WAVES> &sh, u64 *list, int n, int kept) const
    {
        const int lane = tid & 63;
        int reach, last = 0x7FFFFFFF;
        uint32_t bound;
        if (WAVES == 1 && n > kWaveSize / 2) {
            // threads are too few to bound with: the labels themselves
            const auto got = [&](uint32_t t) {
                const float lo = key_score(max(t, 0x00800000u));
                int g = 0;
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int j = 0; j < VEC; ++j) g += count(z[i][j] >= lo);
                return g;
            };
            bound = nth_key<uint32_t>(n, V, reach, got);
            if (reach > bound_cap(n) && bound) {        // ties: the first of them
                const float lo = key_score(bound);
                const int v = own_v0();
                const auto first_of = [&](int end) {
                    int g = 0;
#pragma unroll
                    for (int i = 0; i < NV; ++i)
#pragma unroll
                        for (int j = 0; j < VEC; ++j) g += count(z[i][j] > lo || (z[i][j] == lo && label(v, i, j) < end));
                    return g;
                };
                last = 0;                               // (the n-th stands here)
                for (int bit = 23; bit >= 0; --bit)
                    if (first_of(last | 1 << bit) < n) last |= 1 << bit;
            }
        } else {
            uint32_t u[WAVES];
#pragma unroll
            for (int q = 0; q < WAVES; ++q) u[q] = WAVES > 1 ? sh.top[q * kWaveSize + lane] : score_key(mine);
            const auto reach_of = [&](const uint32_t (&k)[WAVES], uint32_t t) {
                int g = 0;
#pragma unroll
                for (int q = 0; q < WAVES; ++q) g += count(k[q] >= t);
                return g;
            };
            bound = nth_key<uint32_t>(n, WAVES * kWaveSize, reach, [&](uint32_t t) { return reach_of(u, t); });
            if (reach > bound_cap(n) && bound) {        // (the same for the whole row)
                // more threads tie at the bound than are needed: those whose largest stands first
                int at = 0x7FFFFFFF;
                const int v = own_v0();
#pragma unroll
                for (int i = NV - 1; i >= 0; --i)
#pragma unroll
                    for (int j = VEC - 1; j >= 0; --j)
                        if (z[i][j] == mine) at = label(v, i, j);
                if (WAVES > 1) {
                    sh.at[tid] = at;
                    row_sync<WAVES>();
                }
                uint32_t early[WAVES];                  // (the earliest is the largest)
                int more = 0, got;
#pragma unroll
                for (int q = 0; q < WAVES; ++q) {
                    early[q] = u[q] == bound ? ~(uint32_t)(WAVES > 1 ? sh.at[q * kWaveSize + lane] : at) : 0u;
                    more += count(u[q] > bound);
                }
                last = (int)~nth_key<uint32_t>(n - more, WAVES * kWaveSize, got,
                                               [&](uint32_t t) { return reach_of(early, t); });
            }
        }
        float lo = key_score(max(bound, 0x00800000u));
        if (kept == n) {                                // (later labels only pass with a larger score)
            const float run = key_score((uint32_t)(list[n - 1] >> 32));
            if (run >= lo) { lo = run; last = -1; }
        }
        if (!__ballot(mine >= lo)) return;
        if (last == 0x7FFFFFFF) append<false>(sh, list, lo, last);
        else append<true>(sh, list, lo, last);
    }

    // Labels above lo, or of lo itself and not behind `last` (FIRST; else all of lo).
    template <bool FIRST>
    __device__ __forceinline__ void append(TokenShared<WAVES> &sh, u64 *list, float lo, int last) const
    {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!__ballot(pm[i] >= lo)) continue;
#pragma unroll
            for (int j = 0; j < VEC; ++j)
                if (z[i][j] >= lo) {
                    const int v = label(own_v0(), i, j);
                    if (!FIRST || z[i][j] > lo || v <= last) list[atomicAdd(&sh.listed, 1)] = label_key(z[i][j], v);
                }
        }
    }
};

// Calls f(place, key) for the first n of a list's L keys in their order, by the threads
// of a row. Each wavefront first ends the list with 8 zeros for itself.
template <int WAVES, typename F>
__device__ __forceinline__ void best_of(u64 *list, int L, int n, int tid, F &&f)
{
    if ((tid & 63) < 8) list[L + (tid & 63)] = 0;
    row_sync<1>();
    for (int i = tid; i < L; i += WAVES * kWaveSize) {
        const u64 k = list[i];
        int place = 0;
        for (int q = 0; q < L; q += 8) {
            u64 o[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = list[q + j];
#pragma unroll
            for (int j = 0; j < 8; ++j) place += o[j] > k;
        }
        if (place < n) f(place, k);
    }
}

__device__ __forceinline__ void write_token(const TokenCall &c, const TokenRow &row, int64_t i, bool is, float z, int before)
{
    c.log_probs[i] = is ? log_prob(row, z, before) : -INFINITY;
    c.ranks[i] = is ? before : -1;
}

__device__ __forceinline__ void write_top(const TokenCall &c, const TokenRow &row, int64_t r, int place, u64 k)
{
    c.top_tokens[r * c.top_n + place] = (int32_t)~(uint32_t)k;
    c.top_log_probs[r * c.top_n + place] = log_prob(row, key_score((uint32_t)(k >> 32)), place);
}

__device__ __forceinline__ void write_no_top(const TokenCall &c, int64_t r, int place)
{
    c.top_tokens[r * c.top_n + place] = -1;
    c.top_log_probs[r * c.top_n + place] = -INFINITY;
}

// The given tokens from the i-th on, a lane each (-1: none), and their scores (-inf: no label).
__device__ __forceinline__ int load_tokens(const int32_t *tokens, int i, int C)
{
    const int lane = threadIdx.x & 63;
    return C ? (i + lane < C ? tokens[min(i + lane, C - 1)] : -1) : -1;
}

template <typename XT>
__device__ __forceinline__ XT gather(const XT *x, int tok, int V) { return x[min(max(tok, 0), V - 1)]; }

template <typename XT>
__device__ __forceinline__ float token_score(XT x, int tok, int V) { return tok >= 0 && tok < V ? (float)x : -INFINITY; }

// A row a wavefront, four to a workgroup, no barriers.
template <typename XT, int NV>
__global__ __launch_bounds__(kTokenThreads) void k_token_short(TokenCall c, int32_t room)
{
    __shared__ TokenShared<1> shared[kTokenWaves];
    extern __shared__ __align__(16) u64 lists[];
    const int lane = threadIdx.x & 63, slot = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    TokenShared<1> &sh = shared[slot];
    u64 *list = lists + (size_t)slot * room;
    typedef TokenRun<XT, 1, NV> Run;
    for (int64_t r = (int64_t)blockIdx.x * kTokenWaves + slot; r < c.rows; r += (int64_t)gridDim.x * kTokenWaves) {
        if (!row_active(c.set, r)) continue;
        const XT *x = (const XT *)c.x + r * c.x_stride;
        const int32_t *tokens = c.tokens + r * c.C;
        int tok = load_tokens(tokens, 0, c.C);
        typename Run::Packs packs;
        Run::fetch(x, c.V, 0, lane, packs);
        XT raw = c.C ? gather(x, tok, c.V) : (XT)0.0f;
        Run run(packs, c.V, 0, lane);
        const Heat heat = row_heat(c, r);
        TokenStat s;
        s.m = wave_max_f(run.mine);
        run.sums(heat, s.m, s);
        if (s.sum != s.sum) s.m = INFINITY;
        const TokenRow row = row_result(s, heat);
        if (lane == 0 && c.entropies) c.entropies[r] = row.entropy;
        for (int i = 0; i < c.C; i += kWaveSize) {
            if (i) {
                tok = load_tokens(tokens, i, c.C);
                raw = gather(x, tok, c.V);
            }
            const float zt = token_score(raw, tok, c.V);
            const int m = min(c.C - i, kWaveSize), before = run.ranks(x, zt, tok, m, true);
            if (lane < m) write_token(c, row, r * c.C + i + lane, tok >= 0 && tok < c.V, zt, before);
        }
        if (c.top_n) {
            if (lane == 0) sh.listed = 0;
            row_sync<1>();
            run.candidates(sh, list, c.top_n, 0);
            row_sync<1>();
            const int L = sh.listed;
            best_of<1>(list, L, c.top_n, lane, [&](int place, u64 k) { write_top(c, row, r, place, k); });
            for (int i = L + lane; i < c.top_n; i += kWaveSize) write_no_top(c, r, i);
            row_sync<1>();
        }
    }
}

// A row, or (CUT) a piece of one, a workgroup.
template <typename XT, int WAVES, int NV, bool CUT>
__global__ __launch_bounds__(WAVES *kWaveSize) void k_token_rows(TokenCall c, TokenPlan plan)
{
    constexpr int kThreads = WAVES * kWaveSize;
    typedef TokenRun<XT, WAVES, NV> Run;
    constexpr int kLen = Run::kSpan * NV;
    __shared__ TokenShared<WAVES> sh;
    extern __shared__ __align__(16) u64 list[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = c.top_n, C = c.C;
    const int64_t items = CUT ? c.rows * plan.pieces : c.rows;
    const TokenWork work = CUT ? token_work(c.workspace, items, n) : TokenWork{};

    for (int64_t w = blockIdx.x; w < items; w += gridDim.x) {
        const int64_t r = CUT ? w / plan.pieces : w;
        const int begin = CUT ? (int)(w - r * plan.pieces) * plan.subs * kLen : 0;
        if (!row_active(c.set, r)) continue;
        const XT *x = (const XT *)c.x + r * c.x_stride;
        const int32_t *tokens = c.tokens + r * C;
        int tok = load_tokens(tokens, 0, C);
        XT raw = (XT)0.0f;
        const Heat heat = row_heat(c, r);

        TokenStat all = {-INFINITY, 0.0f, 0.0f, 0.0f};
        int kept = 0;                                   // keys at the head of the list, sorted
        for (int sub = 0; sub < (CUT ? plan.subs : 1); ++sub) {
            const int first = begin + sub * kLen;
            if (CUT && first >= c.V) break;
            const bool more = CUT && sub + 1 < plan.subs && first + kLen < c.V;
            typename Run::Packs packs;
            Run::fetch(x, c.V, first, tid, packs);
            if (sub == 0 && C) raw = gather(x, tok, c.V);
            Run run(packs, c.V, first, tid);
            TokenStat s;
            const float wave_max = wave_max_f(run.mine);
            s.m = wave_max;
            if (n) sh.top[tid] = score_key(run.mine);
            if (lane == 0) sh.red[wave] = s.m;
            if (tid == 0) sh.listed = kept;
            if (sub == 0)
                for (int i = tid; i < C; i += kThreads) sh.ranks[i] = 0;
            __syncthreads();
#pragma unroll
            for (int q = 0; q < WAVES; ++q) s.m = fmaxf(s.m, sh.red[q]);
            run.sums(heat, wave_max, s);
            if (lane == 0) {
                sh.red[WAVES + wave] = s.sum;
                sh.red[2 * WAVES + wave] = s.ysum;
                sh.red[3 * WAVES + wave] = s.ones;
            }
            for (int i = 0; i < C; i += kWaveSize) {
                if (C > kWaveSize && (i || sub)) {
                    tok = load_tokens(tokens, i, C);
                    raw = gather(x, tok, c.V);
                }
                const int m = min(C - i, kWaveSize);
                const int before = run.ranks(x, token_score(raw, tok, c.V), tok, m, wave == 0);
                if (lane < m) atomicAdd(&sh.ranks[i + lane], before);
            }
            if (n) run.candidates(sh, list, n, kept);
            __syncthreads();
            s.sum = s.ysum = s.ones = 0.0f;
#pragma unroll
            for (int q = 0; q < WAVES; ++q) {
                s.sum += sh.red[WAVES + q];
                s.ysum += sh.red[2 * WAVES + q];
                s.ones += sh.red[3 * WAVES + q];
            }
            if (s.sum != s.sum) s.m = INFINITY;
            all = CUT && sub ? stat_join(all, s, heat) : s;
            const int L = sh.listed;
            if (more && n) {                            // the best so far to the head of the list
                u64 *best = list + plan.list - n;
                best_of<WAVES>(list, L, n, tid, [&](int place, u64 k) { best[place] = k; });
                __syncthreads();
                kept = min(L, n);
                for (int i = tid; i < kept; i += kThreads) list[i] = best[i];
            }
            if (more) __syncthreads();
        }

        const int L = sh.listed;
        if constexpr (CUT) {
            if (n) {
                best_of<WAVES>(list, L, n, tid, [&](int place, u64 k) { work.keys[w * n + place] = k; });
                for (int i = L + tid; i < n; i += kThreads) work.keys[w * n + i] = 0;
            }
            if (tid == 0) work.stats[w] = all;
            for (int i = tid; i < C; i += kThreads) work.ranks[w * C + i] = sh.ranks[i];
        } else {
            const TokenRow row = row_result(all, heat);
            if (n) {
                best_of<WAVES>(list, L, n, tid, [&](int place, u64 k) { write_top(c, row, r, place, k); });
                for (int i = L + tid; i < n; i += kThreads) write_no_top(c, r, i);
            }
            if (tid == 0 && c.entropies) c.entropies[r] = row.entropy;
            if (wave == WAVES - 1)                      // (the list's first keys lie with the first)
                for (int i = 0; i < C; i += kWaveSize) {
                    if (C > kWaveSize) {
                        tok = load_tokens(tokens, i, C);
                        raw = gather(x, tok, c.V);
                    }
                    if (i + lane < C)
                        write_token(c, row, r * C + i + lane, tok >= 0 && tok < c.V, token_score(raw, tok, c.V),
                                    sh.ranks[i + lane]);
                }
        }
        __syncthreads();
    }
}

// Joins a row's pieces: one workgroup a row.
constexpr int kJoinList = bound_cap(kMaxTop) * ((kMaxTop + kTokenThreads / kMaxPieces - 1) / (kTokenThreads / kMaxPieces));

__global__ __launch_bounds__(kTokenThreads) void k_token_join(TokenCall c, int32_t P, int32_t xcode)
{
    __shared__ u64 top[kTokenThreads];
    __shared__ __align__(16) u64 list[kJoinList + 8];
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
            write_token(c, row, r * C + i, is, z, before);
        }
        if (!n) continue;
        const u64 *keys = work.keys + r * P * n;
        // a piece's keys over `share` threads in turn, so that the best of all lie far apart
        const int share = kTokenThreads / P, piece = tid / share;
        const int i0 = piece < P ? piece * n + tid % share : 0, end = piece < P ? piece * n + n : 0;
        u64 mine = 0;
        for (int i = i0; i < end; i += share) mine = max(mine, keys[i]);
        top[tid] = mine;
        if (tid == 0) listed = 0;
        __syncthreads();
        u64 u[kTokenWaves];
#pragma unroll
        for (int q = 0; q < kTokenWaves; ++q) u[q] = top[q * kWaveSize + lane];
        int reach;
        const u64 bound = max(nth_key<u64>(n, kTokenThreads, reach, [&](u64 t) {
            int g = 0;
#pragma unroll
            for (int q = 0; q < kTokenWaves; ++q) g += count(u[q] >= t);
            return g;
        }), (u64)1);
        for (int i = i0; i < end; i += share) {
            const u64 k = keys[i];
            if (k >= bound) list[atomicAdd(&listed, 1)] = k;
        }
        __syncthreads();
        const int L = listed;
        best_of<kTokenWaves>(list, L, n, tid, [&](int place, u64 k) { write_top(c, row, r, place, k); });
        for (int i = L + tid; i < n; i += kTokenThreads) write_no_top(c, r, i);
        __syncthreads();
    }
}

// Wavefronts and packs a thread of a row (or a run of one), its pieces and their runs.
// One wavefront a row up to 2048 labels, two up to 5120, four up to 8192, pieces of that
// beyond. 16000 rows, one given token and no / 4 / 20 / 64 alternatives, us: 2000 binary16
// labels on 1 / 2 wavefronts 23 / 30, 32 / 41, 41 / 48, 129 / 74; 5000 on 2 / 4 46 / 55, 60 /
// 79, 72 / 92, 147 / 117 (binary32 68 / 81, 83 / 107, 97 / 120, 155 / 148), 3000 82 / 129 with
// 64: many alternatives take more wavefronts where a thread holds many labels. Fewer rows
// than fill the card take about as long either way. Pieces of 8192 labels, or of 2048 and more of
// them, us, without tokens and alternatives, with one token and 20, with 16 and 64, binary32:
// 131072 labels, 1 row 13 / 14, 17 / 19, 30 / 34; 16 rows 13 / 13, 18 / 22, 32 / 38; 64 rows 13 /
// 15, 21 / 34, 41 / 64; 256 rows 27 / 36, 46 / 83, 105 / 164. 32003 labels, 1 row 12 / 12, 16 / 15, 27
// / 23; 48 rows 13 / 13, 17 / 17, 28 / 26; 256 rows 13 / 15, 21 / 30, 38 / 54. 16384 labels, 1 to 64
// rows 13 / 14, 16 / 17, 26 to 28 / 21 to 22. So short pieces pay for a few rows with many given
// tokens alone (up to 7 us), and the rule does not look at either.
struct TokenShape { int waves, nv, pieces, subs; };

TokenShape token_shape(int32_t V, int32_t top_n, int32_t x_dtype)
{
    const bool f32 = x_dtype == kF32, many = top_n > kMaxTop / 2;
    const int vec = f32 ? 4 : 8, most = 32 / vec, lane = kWaveSize * vec;
    const auto up = [](int64_t a, int64_t b) { return (int)((a + b - 1) / b); };
    if (V <= (many ? most / 2 : most) * lane) return {1, up(V, lane) <= 4 ? up(V, lane) : most, 1, 1};
    if (V <= 2 * lane * (many ? most : most + most / 4)) {
        const int nv = f32 ? std::max(3, up(V, 4 * lane)) * 2 : std::max(3, up(V, 2 * lane));
        return {2, nv, 1, 1};
    }
    const int len = kTokenWaves * lane * most;
    if (V <= len) return {kTokenWaves, f32 ? most : std::max(3, up(V, kTokenWaves * lane)), 1, 1};
    const int subs = up(up(V, len), kMaxPieces);
    return {kTokenWaves, most, up(V, (int64_t)len * subs), subs};
}

// u64 of a row's list in LDS: the labels that may reach the bound, 8 zeros, and twice
// the n best so far. Room for the worst case (all of bound_cap(n) threads' labels), where about
// n are listed. It takes workgroups off a CU that the registers leave room for in three cases: 3
// instead of 4 with 31 or 32 alternatives of the longest rows of one wavefront (41 to 43 KiB), 5
// instead of 7 with 64 of 1000 16-bit labels (32 KiB), 7 instead of 8 with 64 of two wavefronts'
// rows (23 KiB).
int token_list(const TokenCall &c, int nv, int vec, bool cut)
{
    return c.top_n ? (std::min(bound_cap(c.top_n) * nv * vec, c.V) + 8 + (cut ? 2 * c.top_n : 0) + 1) / 2 * 2 : 0;
}

template <typename XT, int NV>
void short_launch(const TokenCall &c, hipStream_t s)
{
    const int room = token_list(c, NV, kTokenVec<XT>, false);
    const int64_t groups = (c.rows + kTokenWaves - 1) / kTokenWaves;
    hipLaunchKernelGGL((k_token_short<XT, NV>), dim3((unsigned)std::min<int64_t>(groups, kShortGrid)),
                       dim3(kTokenThreads), (size_t)kTokenWaves * room * sizeof(u64), s, c, room);
}

template <typename XT, int WAVES, int NV, bool CUT>
void rows_launch(const TokenCall &c, const TokenShape &t, hipStream_t s)
{
    const TokenPlan plan = {t.pieces, t.subs, token_list(c, NV, kTokenVec<XT>, CUT)};
    const int64_t groups = c.rows * t.pieces;
    hipLaunchKernelGGL((k_token_rows<XT, WAVES, NV, CUT>), dim3((unsigned)std::min<int64_t>(groups, kMaxRowGrid)),
                       dim3(WAVES * kWaveSize), (size_t)plan.list * sizeof(u64), s, c, plan);
}

template <typename XT>
hipError_t token_launch(const TokenCall &c, hipStream_t s)
{
    constexpr int kMost = 32 / kTokenVec<XT>;
    const TokenShape t = token_shape(c.V, c.top_n, c.x_dtype);
    if (t.waves == 1) {
        switch (t.nv) {
        case 1: short_launch<XT, 1>(c, s); break;
        case 2: short_launch<XT, 2>(c, s); break;
        case 3: short_launch<XT, 3>(c, s); break;
        case 4: short_launch<XT, 4>(c, s); break;
        default: short_launch<XT, kMost>(c, s); break;
        }
    } else if (t.pieces > 1) {
        rows_launch<XT, kTokenWaves, kMost, true>(c, t, s);
    } else if constexpr (kMost == 8) {
        if (t.waves == kTokenWaves) rows_launch<XT, kTokenWaves, 8, false>(c, t, s);
        else if (t.nv == 6) rows_launch<XT, 2, 6, false>(c, t, s);
        else if (t.nv == 8) rows_launch<XT, 2, 8, false>(c, t, s);
        else rows_launch<XT, 2, 10, false>(c, t, s);
    } else if (t.waves == kTokenWaves) {
        if (t.nv == 3) rows_launch<XT, kTokenWaves, 3, false>(c, t, s);
        else rows_launch<XT, kTokenWaves, 4, false>(c, t, s);
    } else {
        if (t.nv == 3) rows_launch<XT, 2, 3, false>(c, t, s);
        else if (t.nv == 4) rows_launch<XT, 2, 4, false>(c, t, s);
        else rows_launch<XT, 2, 5, false>(c, t, s);
    }
    if (t.pieces > 1)
        hipLaunchKernelGGL(k_token_join, dim3((unsigned)std::min<int64_t>(c.rows, kMaxRowGrid)), dim3(kTokenThreads), 0,
                           s, c, t.pieces, c.x_dtype);
    return hipGetLastError();
}

}  // namespace

size_t token_workspace(int64_t rows, int32_t V, int32_t C, int32_t top_n, int32_t x_dtype)
{
    const TokenShape t = token_shape(V, top_n, x_dtype);
    if (t.pieces == 1) return 0;
    return (size_t)rows * t.pieces * (sizeof(TokenStat) + (size_t)top_n * sizeof(u64) + (size_t)C * 4);
}

hipError_t launch_token_scores(const TokenCall &call, hipStream_t s)
{
    TokenCall c = call;
    const Heat h = heat_of(c.temperature);
    c.unit = h.unit;
    c.scale = h.scale;
    if (c.x_dtype == kF32) return token_launch<float>(c, s);
    if (c.x_dtype == kF16) return token_launch<_Float16>(c, s);
    return token_launch<__bf16>(c, s);
}

}  // namespace wfst
