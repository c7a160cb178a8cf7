// gfx950 (CDNA4) kernels of the draw of tokens from scores.
#include <type_traits>

#include "wfst_score_device.h"

namespace wfst {

// mass_i = exp((x_i - max) / T). Kept: the top_k largest (among equal scores the
// lowest indices), of these the shortest run of the largest whose mass reaches
// top_p of theirs, of these the ones with mass >= min_p. The token is the first
// kept i, in index order, whose running mass exceeds u times the kept mass.
//
// Nothing is sorted. Labels are ordered by one integer, (max key - key) << bits
// of an index | index, key being the score's bits in an order that integers
// compare: top_k and top_p each cut at one value of it, `last`, found digit by
// digit (8 bits at a time) from histograms of counts or masses. Masses are
// binary64 powers rounded to multiples of 2^-unit and added as integers, so no
// sum depends on the order in which threads add, and sums of any two groupings
// agree. V roundings leave a sum off by at most V 2^-(unit+1) of the largest
// mass: 2^-41 up to 2048 labels (unit 51), 2^-29 at 131072 (45), 2^-23 at 2^20 (42),
// for a row all of whose masses are rounded the same way; a draw or a cut next to a
// border by less than that may fall on its other side. Past 2^20 labels, where V
// masses of 1 would leave fewer bits still, a row's unit comes from a bound on its
// own total (row_unit).

namespace {

constexpr uint32_t kKeyNegInf = 0x007FFFFFu;

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

// The coefficients of 2^f on [-1/2, 1/2] (degree 10, interpolating at Chebyshev
// nodes; relative error below 2^-51), in scalar registers: the compiler would
// otherwise copy each into the accumulator of every multiply-add.
struct Exp2Poly {
    double c[10];
    __device__ __forceinline__ Exp2Poly()
    {
        const double k[10] = {7.072585949269224e-09, 1.0208690299958306e-07, 1.321544258792169e-06,
                              1.5252657260200837e-05, 1.540353044173605e-04, 1.3333558230164974e-03,
                              9.618129107606888e-03, 5.550410866444772e-02, 2.4022650695910097e-01,
                              6.9314718055995e-01};
#pragma unroll
        for (int i = 0; i < 10; ++i) {
            c[i] = k[i];
            asm("" : "+s"(c[i]));
        }
    }
};

// The mass of a score, times 2^unit. A row whose choice is already made (greedy,
// or +inf scores, which leave only each other) is read with its largest scores
// as 0 and all others as -inf, and keeps this one form.
struct MassOf {
    double m, a;       // the row's maximum; log2(e) / T
    double t;          // T
    double one, base;  // 2^unit; 1.5 * 2^52 + unit
    double lim;        // min_p * 2^unit (0: no limit)
    float top;         // the largest score as stored
    bool pick;         // read as above
    bool greedy;

    __device__ __forceinline__ MassOf(float top_, float T, float minp, int unit, bool greedy_)
    {
        greedy = greedy_;
        one = (double)(1ull << unit);
        base = 6755399441055744.0 + (double)unit;
        top = top_ > -INFINITY ? top_ : NAN;             // (an empty row: nothing is picked)
        pick = greedy || top_ == INFINITY;
        m = pick ? 0.0 : (double)top_;
        t = greedy ? 1.0 : (double)T;
        a = 1.4426950408889634 / t;
        lim = minp > 0.0f ? (minp < 1.0f ? (double)minp : 1.0) * one : 0.0;
    }
    // A score below which no label passes min_p (a little low, for the roundings on the way).
    __device__ __forceinline__ float least_score() const
    {
        if (!(lim > 0.0)) return -INFINITY;
        const double y = m + t * log(lim / one);
        const double low = y - 1e-6 * (fabs(y) + fabs(m)) - 1e-12 * t;      // (t: a mass is off by 2^-51 of itself)
        return low > -INFINITY ? (float)low : -INFINITY;       // (also where an infinite T leaves a NaN)
    }
    __device__ __forceinline__ float read(float x) const { return pick ? (x == top ? 0.0f : -INFINITY) : x; }
    // 2^(t + unit), t = (x - m) a <= 0 (below -1000: as -1000): adding `base`
    // rounds t to an integer, leaves unit + that integer in the low bits and f in
    // [-1/2, 1/2]; the polynomial gives 2^f, the low bits go to its exponent.
    __device__ __forceinline__ double operator()(float x, const Exp2Poly &k) const
    {
        const double e = fmax(((double)x - m) * a, -1000.0);
        const double r = e + base;
        const double f = e - (r - base);
        double p = k.c[0];
#pragma unroll
        for (int i = 1; i < 10; ++i) p = fma(p, f, k.c[i]);
        p = fma(p, f, 1.0);
        return __hiloint2double(__double2hiint(p) + (__double2loint(r) << 20), __double2loint(p));
    }
    // As an integer (one < 2^52: adding 2^52 leaves it in the low bits), first with the bits of 2^52 itself.
    static constexpr uint64_t kRaw = 0x4330000000000000ull;
    static __device__ __forceinline__ uint64_t raw(double w) { return (uint64_t)__double_as_longlong(w + 4503599627370496.0); }
    static __device__ __forceinline__ uint64_t fixed(double w) { return raw(w) - kRaw; }
    __device__ __forceinline__ float log_prob(float y, uint64_t total) const
    {
        return (float)(((double)y - m) / t - log((double)total / one));
    }
};

// The running mass that the token is the first to reach: above u times the total.
__device__ __forceinline__ uint64_t draw_goal(float u, uint64_t total)
{
    const double t = u > 0.0f ? floor((double)u * (double)total) : 0.0;
    return t < (double)total ? min((uint64_t)t + 1, total) : total;
}

__device__ __forceinline__ void emit(const SampleCall &c, int64_t r, int token, float lp, uint32_t kept)
{
    c.token[r] = token;
    if (c.log_prob) c.log_prob[r] = lp;
    if (c.kept) c.kept[r] = (int32_t)kept;
}

// Labels v .. v + VEC - 1 of a row of V (-inf past its end).
template <typename XT, int VEC>
__device__ __forceinline__ void load_scores(const XT *x, int V, int v, float (&y)[VEC])
{
    if (v + VEC <= V) {
        const Pack<XT, VEC> p = *(const Pack<XT, VEC> *)(x + v);
#pragma unroll
        for (int j = 0; j < VEC; ++j) y[j] = (float)p.v[j];
    } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) y[j] = v + j < V ? (float)x[v + j] : -INFINITY;
    }
}

template <int CTRL, int ROWS>
__device__ __forceinline__ uint64_t dpp_u64(uint64_t v)
{
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)v, CTRL, ROWS, 0xf, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(v >> 32), CTRL, ROWS, 0xf, false);
    return (uint64_t)hi << 32 | lo;
}

// Inclusive running sum over the wavefront (all lanes active).
__device__ __forceinline__ uint64_t wave_scan_u64(uint64_t v)
{
    v += dpp_u64<0x111, 0xf>(v);
    v += dpp_u64<0x112, 0xf>(v);
    v += dpp_u64<0x114, 0xf>(v);
    v += dpp_u64<0x118, 0xf>(v);
    v += dpp_u64<0x142, 0xa>(v);
    v += dpp_u64<0x143, 0xc>(v);
    return v;
}

__device__ __forceinline__ uint64_t lane_u64(uint64_t v, int lane)
{
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, lane);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), lane);
    return (uint64_t)hi << 32 | lo;
}

__device__ __forceinline__ uint64_t wave_sum_u64(uint64_t v) { return lane_u64(wave_scan_u64(v), 63); }

// The unit of a row of more than kUnitLabels labels, by the WAVES wavefronts of a
// workgroup: its total is at most `each` (the labels a thread reads) times the sum
// of the threads' largest masses, and 2^unit times that stays below 2^63. A row
// with few large masses then gets nearly all bits, and a level one loses no more
// than the bound exceeds its total: sums are off by at most V each 2^-63 of the
// total, 2^-23 for 2^24 labels on 256 threads. (By V alone 2^-15.)
constexpr int kUnitLabels = 1 << 20;

template <int WAVES>
__device__ __forceinline__ int row_unit(float own, float top, float T, bool greedy, int each, int least, const Exp2Poly &poly,
                                        unsigned long long *sum)
{
    constexpr int kUnit = 50;                        // 1024 masses stay below 2^62
    const MassOf mass(top, T, 0.0f, kUnit, greedy);
    const uint64_t w = wave_sum_u64(MassOf::fixed(mass(mass.read(own), poly)) + 1);       // (+ 1: rounded up)
    if ((threadIdx.x & 63) == 0) sum[threadIdx.x >> 6] = w;
    __syncthreads();
    uint64_t all = 0;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) all += sum[i];
    __syncthreads();                                 // (sum may be written again)
    const double bound = (double)all * (double)each;      // < 2^e: the total is below 2^(e - kUnit)
    const int e = (int)((uint32_t)__double2hiint(bound) >> 20) - 1022;
    return min(51, max(least, 63 + kUnit - e));
}

// f(v, scores v .. v + VEC - 1) for the lane's packs of labels v0 .. v1 - 1 of a row
// of V, a wavefront taking 64 * VEC labels at once: AHEAD packs are loaded before
// the first is used. v0 is the wavefront's; packs may reach past v1 (to V).
template <typename XT, int AHEAD, typename F>
__device__ __forceinline__ void each_pack(const XT *x, int V, int v0, int v1, F f)
{
    constexpr int VEC = 16 / sizeof(XT);
    constexpr int kStepW = 64 * VEC;
    const int lane = threadIdx.x & 63;
    int v = v0;
    for (; v + AHEAD * kStepW <= v1; v += AHEAD * kStepW) {
        Pack<XT, VEC> p[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) p[i] = *(const Pack<XT, VEC> *)(x + v + i * kStepW + lane * VEC);
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            float y[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) y[j] = (float)p[i].v[j];
            f(v + i * kStepW + lane * VEC, y);
        }
    }
    for (; v < v1; v += kStepW) {
        if (v + lane * VEC >= v1) continue;
        float y[VEC];
        load_scores<XT, VEC>(x, V, v + lane * VEC, y);
        f(v + lane * VEC, y);
    }
}

// LDS of draw_row.
template <int WAVES> struct RowSums {
    unsigned long long sum[WAVES];
    uint32_t kept[WAVES];
};

// Draw from the scores x[0 .. V) (labels base ..) by the WAVES wavefronts of a
// workgroup (or each wavefront on a row of its own). Every wavefront owns one
// contiguous run of packs of 64 * VEC labels; the sums of the wavefronts, then of
// their packs, then of the lanes say where the token lies. raw_of(score, label,
// kept) is a label's MassOf::raw, counting it if it is kept. span: the token is
// known to lie here, where the running mass is span.goal, and the row's mass and
// count are known.
struct DrawSpan {
    uint64_t goal, total;      // goal 0: not known
    uint32_t kept;
};

template <typename XT, int WAVES, typename Mass>
__device__ __forceinline__ void draw_row(const SampleCall &c, int64_t r, const XT *x, int V, int base, const MassOf &mass,
                                         float u, RowSums<WAVES> &s, const DrawSpan &span, Mass raw_of)
{
    constexpr int VEC = 16 / sizeof(XT);
    constexpr int kPackW = 64 * VEC;
    const int lane = threadIdx.x & 63, wave = WAVES == 1 ? 0 : threadIdx.x >> 6;
    const int packs = (V + WAVES * kPackW - 1) / (WAVES * kPackW);       // of one wavefront
    const int group = (packs + 63) / 64;                                 // packs whose sum one lane keeps
    const int v0 = wave * packs * kPackW;
    uint64_t part = 0, own = 0;                      // of the lane's group of packs; of the wavefront
    uint32_t kept = 0;
    for (int i = 0, g = 0, in = 0; i < packs && v0 + i * kPackW < V; ++i) {
        const int v = v0 + i * kPackW + lane * VEC;
        float y[VEC];
        load_scores<XT, VEC>(x, V, v, y);
        uint64_t w = (uint64_t)0 - VEC * MassOf::kRaw;
#pragma unroll
        for (int j = 0; j < VEC; ++j) w += raw_of(y[j], base + v + j, kept);
        w = wave_sum_u64(w);
        part += lane == g ? w : 0;
        own += w;
        if (++in == group) { in = 0; ++g; }
    }
    kept = (uint32_t)wave_sum_u64(kept);
    uint64_t total = own, before = 0;                // `before`: the wavefronts in front
    if (WAVES > 1) {
        if (lane == 0) { s.sum[wave] = own; s.kept[wave] = kept; }
        __syncthreads();
        total = 0;
        kept = 0;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            before += w < wave ? (uint64_t)s.sum[w] : 0;
            total += s.sum[w];
            kept += s.kept[w];
        }
    }
    uint64_t goal = span.goal;
    if (goal) {
        total = span.total;
        kept = span.kept;
    } else {
        if (total == 0) {                            // (no label with a score above -inf)
            if (lane == 0 && wave == 0) emit(c, r, -1, -INFINITY, 0);
            return;
        }
        goal = mass.greedy ? 1 : draw_goal(u, total);
    }
    if (goal <= before || goal > before + own) return;       // (one wavefront goes on)
    const uint64_t run = before + wave_scan_u64(part);
    const int at = __ffsll((unsigned long long)__ballot(run >= goal)) - 1;
    before = lane_u64(run - part, at);
    for (int i = at * group; i < packs; ++i) {
        const int v = v0 + i * kPackW + lane * VEC;
        float y[VEC];
        load_scores<XT, VEC>(x, V, v, y);
        uint64_t w[VEC], mine = 0;
        uint32_t n = 0;
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            w[j] = raw_of(y[j], base + v + j, n) - MassOf::kRaw;
            mine += w[j];
        }
        const uint64_t upto = before + wave_scan_u64(mine);
        const uint64_t hit = __ballot(upto >= goal);
        if (hit) {
            if (lane == __ffsll((unsigned long long)hit) - 1) {
                uint64_t acc = upto - mine;
                int found = -1;
                float score = 0.0f;
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    acc += w[j];
                    if (found < 0 && acc >= goal) { found = j; score = mass.read(y[j]); }
                }
                emit(c, r, base + v + found, mass.greedy ? 0.0f : mass.log_prob(score, total), mass.greedy ? 1 : kept);
            }
            return;
        }
        before = lane_u64(upto, 63);
    }
}

// Rows without top_k and top_p. A workgroup of one-wavefront rows holds four of
// them and no barrier.
template <typename XT, int WAVES>
__global__ __launch_bounds__(WAVES == 1 ? 256 : WAVES * 64) void k_draw_all(SampleCall c, int unit)
{
    constexpr int VEC = 16 / sizeof(XT);
    constexpr int kRows = WAVES == 1 ? 4 : 1;
    constexpr int kPackW = 64 * VEC;
    __shared__ RowSums<WAVES> s;
    __shared__ float red[WAVES];
    const int lane = threadIdx.x & 63, wave = WAVES == 1 ? 0 : threadIdx.x >> 6;
    const int64_t step = (int64_t)gridDim.x * kRows;
    const Exp2Poly poly;
    for (int64_t r = (int64_t)blockIdx.x * kRows + (WAVES == 1 ? threadIdx.x >> 6 : 0); r < c.rows; r += step) {
        if (!row_active(c.set, r)) continue;
        const XT *x = (const XT *)c.x + r * c.x_stride;
        const float T = c.temperatures ? c.temperatures[r] : c.temperature;
        const float minp = c.min_ps ? c.min_ps[r] : c.min_p;
        const float u = c.u[r];
        float top = -INFINITY;
        const int packs = (c.V + WAVES * kPackW - 1) / (WAVES * kPackW);
        const int p0 = min(c.V, wave * packs * kPackW);
        each_pack<XT, 4>(x, c.V, p0, min(c.V, p0 + packs * kPackW), [&](int, const float (&y)[VEC]) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) top = fmaxf(top, y[j]);        // (NaN leaves it)
        });
        const float own = top;
        top = wave_max_f(top);
        if (WAVES > 1) {
            if (lane == 0) red[wave] = top;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < WAVES; ++w) top = fmaxf(top, red[w]);
        }
        const bool greedy = !(T > 0.0f);
        int bits = unit;
        if constexpr (WAVES > 1) {
            if (c.V > kUnitLabels) bits = row_unit<WAVES>(own, top, T, greedy, packs * VEC, unit, poly, s.sum);
        }
        const MassOf mass(top, T, greedy ? 0.0f : minp, bits, greedy);
        // Two forms: the tests of the general one, as selects, take half as long again as the sum itself.
        // Without them -inf and NaN have the mass 2^-1000, which rounds to 0. With min_p most labels fail a test
        // of their score and need no mass.
        if (__builtin_amdgcn_readfirstlane(mass.pick || mass.lim > 0.0)) {
            const float least = mass.pick ? 0.0f : mass.least_score();
            draw_row<XT, WAVES>(c, r, x, c.V, 0, mass, u, s, {0, 0, 0}, [&](float y, int, uint32_t &n) {
                y = mass.read(y);
                if (!(y >= least)) return MassOf::kRaw;
                const double w = mass(y, poly);
                const bool keep = y > -INFINITY && w >= mass.lim;
                n += keep ? 1u : 0u;
                return MassOf::raw(keep ? w : 0.0);
            });
        } else {
            draw_row<XT, WAVES>(c, r, x, c.V, 0, mass, u, s, {0, 0, 0}, [&](float y, int, uint32_t &n) {
                n += y > -INFINITY ? 1u : 0u;
                return MassOf::raw(mass(y, poly));
            });
        }
        if (WAVES > 1) __syncthreads();
    }
}

// Among the THREADS threads that work on a list: a workgroup, or (64) one
// wavefront of it, whose LDS operations are in order by themselves.
template <int THREADS>
__device__ __forceinline__ void sync_list()
{
    if (THREADS > 64) {
        __syncthreads();
    } else {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
}

struct Digit {
    uint32_t digit, count;
    uint64_t before, mine;
};

// Histograms of 256 digits, three in turn: a round adds to one while the next is
// cleared, and the third may still be read for the round before.
struct Hist {
    unsigned long long mass[3][256];
    uint32_t cnt[3][256];
    Digit found;
};

template <int THREADS>
__device__ __forceinline__ void clear_hist(Hist &h, int slot)
{
    for (int i = threadIdx.x & (THREADS - 1); i < 256; i += THREADS) { h.mass[slot][i] = 0; h.cnt[slot][i] = 0; }
}

// The digit in which the running sum over 256 bins, from `above`, reaches target:
// the sum before it, its own, its count; digit 256 if none does. By one wavefront,
// four digits to a lane.

__device__ __forceinline__ Digit find_digit(const unsigned long long *mass, const uint32_t *cnt, bool by_mass,
                                            uint64_t above, uint64_t target)
{
    const int lane = threadIdx.x & 63;
    uint32_t c[4];
    uint64_t w[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        c[i] = cnt[lane * 4 + i];
        w[i] = by_mass ? (uint64_t)mass[lane * 4 + i] : c[i];
        sum += w[i];
    }
    uint64_t acc = above + wave_scan_u64(sum) - sum;
    int d = 4;
    Digit r = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool hit = d == 4 && acc + w[i] >= target;
        d = hit ? i : d;
        r.before = hit ? acc : r.before;
        r.mine = hit ? w[i] : r.mine;
        r.count = hit ? c[i] : r.count;
        acc += w[i];
    }
    const uint64_t hit = __ballot(d < 4);
    const int src = hit ? __ffsll((unsigned long long)hit) - 1 : 63;
    r.digit = __builtin_amdgcn_readlane(src * 4 + d, src);
    r.before = lane_u64(r.before, src);
    r.mine = lane_u64(r.mine, src);
    r.count = __builtin_amdgcn_readlane(r.count, src);
    return r;
}

// The value `last` at which the elements, taken in ascending order of their
// numbers, reach `target` (in masses, or in counts): the one that reaches it and
// all before are <= last, the others are not. each(f) calls f(number, mass) for
// the thread's elements; digits is the position of the highest bit set in any
// number, plus one. The search goes down by digits of 8 bits until a digit holds
// one element, or (counts) the elements up to its end are at most `enough`.
// `round` counts the histograms used in this workgroup; its slot is clear on
// entry and on return. target must not pass the elements' total. The first
// wavefront looks for the digit: all sixteen at once would take its time four
// times over.
template <int THREADS, typename Each>
__device__ __forceinline__ uint64_t select_last(Hist &h, uint32_t &round, Each each, bool by_mass, int digits,
                                                uint64_t target, uint64_t enough)
{
    uint64_t prefix = 0, above = 0;
    int shift = digits;                                // the digits above it are fixed
    for (;;) {
        const int width = min(8, shift), next = shift - width;
        const int slot = round % 3;
        clear_hist<THREADS>(h, (round + 1) % 3);
        each([&](uint64_t num, uint64_t w) {
            if (num >> shift == prefix) {
                const uint32_t d = (uint32_t)(num >> next) & ((1u << width) - 1u);
                atomicAdd(&h.cnt[slot][d], 1u);
                if (by_mass) atomicAdd(&h.mass[slot][d], (unsigned long long)w);
            }
        });
        sync_list<THREADS>();
        if (threadIdx.x < 64) {
            const Digit d = find_digit(h.mass[slot], h.cnt[slot], by_mass, above, target);
            if (threadIdx.x == 0) h.found = d;
        }
        sync_list<THREADS>();
        ++round;
        const Digit d = h.found;
        prefix = prefix << width | (d.digit & 255u);
        above = d.before;
        shift = next;
        const bool whole = !by_mass && above + d.mine <= enough;
        if (d.count <= 1 || whole || shift == 0) return ((prefix + 1) << shift) - 1;
    }
}

// A row's settings.
struct RowRules {
    float T, topp, minp, u;
    int topk;
    bool greedy, cut_k, cut_p;

    __device__ __forceinline__ RowRules(const SampleCall &c, int64_t r)
    {
        T = c.temperatures ? c.temperatures[r] : c.temperature;
        topk = c.top_ks ? c.top_ks[r] : c.top_k;
        topp = c.top_ps ? c.top_ps[r] : c.top_p;
        minp = c.min_ps ? c.min_ps[r] : c.min_p;
        u = c.u[r];
        greedy = !(T > 0.0f);
        if (greedy) minp = 0.0f;
        cut_k = !greedy && topk > 0 && topk < c.V;
        cut_p = !greedy && topp < 1.0f;
    }
};

// The mass to reach for top_p of `total`.
__device__ __forceinline__ uint64_t top_p_goal(float topp, uint64_t total)
{
    const double t = ceil((double)topp * (double)total);
    return min(t >= 1.0 ? (uint64_t)t : (uint64_t)1, total);
}

// What a workgroup of THREADS threads keeps of a row, with a list of labels that
// may be kept, E a thread.
template <int THREADS> struct ListShared {
    Hist hist;
    unsigned long long sum[THREADS / 64];
    uint32_t a[THREADS / 64], b[THREADS / 64];
};

template <int THREADS, int E, bool HOLD> struct DrawShared : ListShared<THREADS> {
    RowSums<THREADS / 64> row;
    ListShared<64> small;                              // of the first wavefront alone
    uint32_t settled;
    uint32_t count, first;
    unsigned long long list[HOLD ? 1 : E * THREADS];
};

// Count and mass of the elements that each() gives, in the whole workgroup.
template <int THREADS, typename Each>
__device__ __forceinline__ void element_totals(ListShared<THREADS> &s, Each each, uint32_t &n, uint64_t &w)
{
    constexpr int WAVES = THREADS / 64;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint64_t tn = 0, tw = 0;
    each([&](uint64_t, uint64_t m) { ++tn; tw += m; });
    tn = wave_sum_u64(tn);
    tw = wave_sum_u64(tw);
    n = (uint32_t)tn;
    w = tw;
    if (WAVES == 1) return;
    sync_list<THREADS>();
    if (lane == 0) { s.sum[wave] = tw; s.b[wave] = (uint32_t)tn; }
    sync_list<THREADS>();
    n = 0;
    w = 0;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) { n += s.b[i]; w += s.sum[i]; }
}

// Cut by top_k and top_p among the elements that each(last, f) gives.
template <int THREADS, typename Each>
__device__ __forceinline__ void cut_elements(ListShared<THREADS> &s, uint32_t &round, const RowRules &row, Each each, int digits,
                                             uint64_t &last)
{
    const auto now = [&](auto f) { each(last, f); };
#pragma unroll 1
    for (int rule = 0; rule < 2; ++rule) {
        if (!(rule ? row.cut_p : row.cut_k)) continue;
        uint32_t n;
        uint64_t w;
        element_totals<THREADS>(s, now, n, w);
        if (!rule && (uint32_t)row.topk >= n) continue;
        const uint64_t target = rule ? top_p_goal(row.topp, w) : (uint64_t)row.topk;
        // (the search may end above what top_k left: at the end of a digit that held one label)
        last = min(last, select_last<THREADS>(s.hist, round, now, rule, digits, target, (uint64_t)row.topk));
    }
}

// Cut a list of elements (number, mass; ~0: none) that holds all labels which may
// be kept, n of them, and draw from it. total_p: the mass top_p is a share of where that is
// not the elements' own (0 otherwise); false, and nothing written, if their mass
// falls short of it. The three searches (top_k, top_p, the draw by index) share
// one piece of code: a row's time here is latency, and code that runs once is
// fetched as it runs.
template <int THREADS, int E>
__device__ __forceinline__ bool draw_list(const SampleCall &c, int64_t r, const RowRules &row, const MassOf &mass,
                                          const Exp2Poly &poly, uint32_t kmax, int ibits, uint64_t (&el)[E],
                                          const uint64_t (&ew)[E], uint32_t n, int digits, uint64_t total_p, ListShared<THREADS> &s,
                                          uint32_t &round)
{
    constexpr int WAVES = THREADS / 64;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint64_t imask = ((uint64_t)1 << ibits) - 1;
    uint64_t last = ~0ull - 1, mask = ~0ull, total = 0;
#pragma unroll 1
    for (int rule = 0; rule < 3; ++rule) {
        if (rule == 0 ? !row.cut_k : rule == 1 ? !row.cut_p : false) continue;
        if (rule == 2) {
            if (mass.lim > 0.0) {
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    const double w = mass(key_score(kmax - (uint32_t)(el[i] >> ibits)), poly);
                    el[i] = w >= mass.lim ? el[i] : ~0ull;
                }
            }
#pragma unroll
            for (int i = 0; i < E; ++i) el[i] = el[i] <= last ? el[i] : ~0ull;
            last = ~0ull - 1;
            mask = imask;
            digits = max(ibits, 1);
        }
        if (rule > 0)
            element_totals<THREADS>(
                s,
                [&](auto f) {
#pragma unroll
                    for (int i = 0; i < E; ++i)
                        if (el[i] <= last) f(el[i], ew[i]);
                },
                n, total);
        if (rule == 0 && (uint32_t)row.topk >= n) continue;
        uint64_t target = (uint64_t)row.topk;
        if (rule == 1) {
            target = top_p_goal(row.topp, total_p ? total_p : total);
            if (target > total) return false;
        }
        if (rule == 2) target = row.greedy ? 1 : draw_goal(row.u, total);
        // (the search may end above what top_k left: at the end of a digit that held one label)
        last = min(last, select_last<THREADS>(
                             s.hist, round,
                             [&](auto f) {
#pragma unroll
                                 for (int i = 0; i < E; ++i)
                                     if (el[i] <= last && (rule < 2 || ew[i])) f(el[i] & mask, ew[i]);
                             },
                             rule > 0, digits, target, target));
    }
    // the last label with mass at or before `last`: no other shares its digits
    uint32_t at = 0;
    float y = 0.0f;
    bool have = false;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const uint32_t v = (uint32_t)(el[i] & imask);
        const bool later = el[i] != ~0ull && ew[i] && v <= last && (!have || v > at);
        at = later ? v : at;
        y = later ? key_score(kmax - (uint32_t)(el[i] >> ibits)) : y;
        have = have || later;
    }
    uint32_t best = have ? at + 1 : 0;
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) best = max(best, (uint32_t)__shfl_xor((int)best, d, 64));
    if (WAVES > 1) {
        if (lane == 0) s.a[wave] = best;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < WAVES; ++i) best = max(best, s.a[i]);
    }
    if (have && at + 1 == best) emit(c, r, (int)at, row.greedy ? 0.0f : mass.log_prob(y, total), row.greedy ? 1 : n);
    return true;
}

// draw_list on the first n labels of s.list, by the first wavefront where it can
// hold them: alone it needs no barriers, and does not share its SIMD's issue slots
// with three others that do the same. For the whole workgroup; n <= E * THREADS.
template <int THREADS, int E>
__device__ __forceinline__ bool draw_listed(const SampleCall &c, int64_t r, const RowRules &row, const MassOf &mass,
                                            const Exp2Poly &poly, uint32_t kmax, int ibits, uint32_t n, int digits,
                                            uint64_t total_p, DrawShared<THREADS, E, false> &s, uint32_t &round,
                                            uint32_t &round_small)
{
    constexpr int kSmall = 4;
    const auto take = [&](int at, uint64_t &num, uint64_t &w) {
        const uint64_t v = s.list[at];                 // (past the count: whatever the list held)
        const uint64_t m = MassOf::fixed(mass(key_score(kmax - (uint32_t)(v >> ibits)), poly));
        num = (uint32_t)at < n ? v : ~0ull;
        w = (uint32_t)at < n ? m : 0;
    };
    if (n <= kSmall * 64) {
        if (threadIdx.x < 64) {
            uint64_t el[kSmall], ew[kSmall];
#pragma unroll
            for (int i = 0; i < kSmall; ++i) take(i * 64 + threadIdx.x, el[i], ew[i]);
            const bool ok = draw_list<64, kSmall>(c, r, row, mass, poly, kmax, ibits, el, ew, n, digits, total_p, s.small,
                                                  round_small);
            if (threadIdx.x == 0) s.settled = ok;
        }
        __syncthreads();
        return s.settled;
    }
    uint64_t el[E], ew[E];
#pragma unroll
    for (int i = 0; i < E; ++i) take(i * THREADS + threadIdx.x, el[i], ew[i]);
    return draw_list<THREADS, E>(c, r, row, mass, poly, kmax, ibits, el, ew, n, digits, total_p, s, round);
}

// One row by one workgroup. HOLD: the row in registers, E scores a thread (rows
// of at most E * THREADS labels), all of them elements. Otherwise a short list of
// labels that are sure to hold the kept ones is tried first.
template <typename XT, int THREADS, int E, bool HOLD>
__device__ __forceinline__ void draw_one(const SampleCall &c, int64_t r, const RowRules &row, const Exp2Poly &poly,
                                         int unit, int ibits, DrawShared<THREADS, E, HOLD> &s, uint32_t &round,
                                         uint32_t &round_small)
{
    constexpr int WAVES = THREADS / 64;
    constexpr int VEC = 16 / sizeof(XT);
    constexpr int kStepW = 64 * VEC;                   // labels a wavefront takes at once
    constexpr int kCap = E * THREADS;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int V = c.V;
    const XT *x = (const XT *)c.x + r * c.x_stride;
    // each wavefront owns one contiguous piece of the row
    const int seg = (V + WAVES * kStepW - 1) / (WAVES * kStepW) * kStepW;
    const int v0 = min(V, wave * seg), v1 = min(V, v0 + seg);

    // the row's largest score, and each thread's own
    float own = -INFINITY;
    each_pack<XT, 8>(x, V, v0, v1, [&](int, const float (&y)[VEC]) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) own = fmaxf(own, y[j]);       // (NaN leaves it)
    });
    float top = wave_max_f(own);
    __syncthreads();
    if (lane == 0) s.a[wave] = __float_as_uint(top);
    if (tid == 0) { s.count = 0; s.first = 0xFFFFFFFFu; }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WAVES; ++w) top = fmaxf(top, __uint_as_float(s.a[w]));
    if (top == -INFINITY) {
        if (tid == 0) emit(c, r, -1, -INFINITY, 0);
        return;
    }
    if (row.greedy) {
        // the first label with the largest score
        uint32_t at = 0xFFFFFFFFu;
        if (own == top)                                            // (one thread, as a rule)
            for (int v = v0 + lane * VEC; v < v1 && at == 0xFFFFFFFFu; v += kStepW) {
                float y[VEC];
                load_scores<XT, VEC>(x, V, v, y);
#pragma unroll
                for (int j = VEC - 1; j >= 0; --j)
                    if (y[j] == top) at = v + j;
            }
        if (at != 0xFFFFFFFFu) atomicMin(&s.first, at);
        __syncthreads();
        if (tid == 0) emit(c, r, (int)s.first, 0.0f, 1);
        return;
    }

    if constexpr (WAVES == 16) {
        if (V > kUnitLabels) unit = row_unit<WAVES>(own, top, row.T, false, seg / 64, unit, poly, s.sum);
    }
    const MassOf mass(top, row.T, row.minp, unit, false);
    const float high = mass.read(top);                 // the largest score as it is read
    const uint32_t kmax = score_key(high);
    own = mass.read(own);
    const auto load = [&](int v, float (&y)[VEC]) {
        load_scores<XT, VEC>(x, V, v, y);
        if (mass.pick) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) y[j] = mass.read(y[j]);
        }
    };
    const auto each = [&](auto ahead, auto f) {
        each_pack<XT, decltype(ahead)::value>(x, V, v0, v1, [&](int v, float (&y)[VEC]) {
            if (mass.pick) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) y[j] = mass.read(y[j]);
            }
            f(v, y);
        });
    };
    using Ahead2 = std::integral_constant<int, 2>;
    using Ahead4 = std::integral_constant<int, 4>;
    const auto number = [&](float y, uint32_t i) { return (uint64_t)(kmax - score_key(y)) << ibits | i; };
    uint64_t last = ~0ull;                             // kept: number <= last

    if (row.cut_k || row.cut_p) {
        uint64_t el[E], ew[E];                         // the thread's elements: number, mass
        if (HOLD) {
#pragma unroll
            for (int i = 0; i < E / VEC; ++i) {
                const int v = (i * THREADS + tid) * VEC;
                float y[VEC];
                load(v, y);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    el[i * VEC + j] = y[j] > -INFINITY ? number(y[j], v + j) : ~0ull;
                    ew[i * VEC + j] = MassOf::fixed(mass(y[j], poly));      // (0 for -inf and NaN)
                }
            }
            uint32_t n = 0, far = 0;                   // labels; the lowest one's distance from the top
#pragma unroll
            for (int i = 0; i < E; ++i) {
                n += el[i] != ~0ull ? 1u : 0u;
                far = max(far, el[i] != ~0ull ? (uint32_t)(el[i] >> ibits) : 0u);
            }
            n = (uint32_t)wave_sum_u64(n);             // (a held row has one wavefront)
#pragma unroll
            for (int d = 32; d >= 1; d >>= 1) far = max(far, (uint32_t)__shfl_xor((int)far, d, 64));
            draw_list<THREADS, E>(c, r, row, mass, poly, kmax, ibits, el, ew, n, ibits + (far ? 32 - __clz((int)far) : 1),
                                  0, s, round);
            return;
        }
        // the list's labels become the threads' elements
        const auto take = [&](uint32_t count) {
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const uint32_t at = i * THREADS + tid;
                const uint64_t n = s.list[at];                 // (past the count: whatever the list held)
                const uint64_t w = MassOf::fixed(mass(key_score(kmax - (uint32_t)(n >> ibits)), poly));
                el[i] = at < count ? n : ~0ull;
                ew[i] = at < count ? w : 0;
            }
        };
        bool done = false;
        if (row.cut_k && row.topk <= THREADS * 7 / 8) {
            // A bound that at least top_k threads' largest scores reach: the labels that reach it are that many or
            // more, and among labels in random order not many more than that
            const uint32_t want = (uint32_t)row.topk;
            const uint32_t mine = own > -INFINITY ? kmax - score_key(own) : 0xFFFFFFFFu;
            uint32_t far = mine == 0xFFFFFFFFu ? 0 : mine, n = __popcll(__ballot(mine != 0xFFFFFFFFu));
#pragma unroll
            for (int d = 32; d >= 1; d >>= 1) far = max(far, (uint32_t)__shfl_xor((int)far, d, 64));
            if (lane == 0) { s.b[wave] = far; s.sum[wave] = n; }
            __syncthreads();
            n = 0;
            for (int w = 0; w < WAVES; ++w) { far = max(far, s.b[w]); n += (uint32_t)s.sum[w]; }
            __syncthreads();
            uint32_t bound = kmax - kKeyNegInf - 1u;                    // all labels above -inf
            if (n > want) {
                const int bits = far ? 32 - __clz((int)far) : 1;
                const uint64_t b = select_last<THREADS>(
                    s.hist, round,
                    [&](auto f) {
                        if (mine != 0xFFFFFFFFu) f((uint64_t)mine, (uint64_t)1);
                    },
                    false, bits, want, want + want / 4 + 8);
                bound = (uint32_t)min(b, (uint64_t)bound);
            }
            const float floor_x = key_score(kmax - bound);
            each(Ahead4{}, [&](int v, const float (&y)[VEC]) {
                uint32_t hits = 0;
#pragma unroll
                for (int j = 0; j < VEC; ++j) hits |= (y[j] >= floor_x ? 1u : 0u) << j;
                if (hits) {
                    uint32_t at = atomicAdd(&s.count, (uint32_t)__popc(hits));
#pragma unroll
                    for (int j = 0; j < VEC; ++j)
                        if (hits >> j & 1u) {
                            if (at < kCap) s.list[at] = number(y[j], v + j);
                            ++at;
                        }
                }
            });
            __syncthreads();
            const uint32_t count = s.count;
            if (count <= kCap) {
                const int digits = ibits + (bound ? 32 - __clz((int)bound) : 1);
                if constexpr (!HOLD)
                    draw_listed<THREADS, E>(c, r, row, mass, poly, kmax, ibits, count, digits, 0, s, round, round_small);
                return;
            }
            __syncthreads();
        } else if (!row.cut_k) {
            // top_p alone. In one pass the mass of all labels and, by 256 equal steps of the score and each
            // wavefront's piece, of those that may be kept: the others weigh less than 1 - top_p even all together
            // (all labels weighing no less than the threads' largest ones). The steps say in which the nucleus ends;
            // a list of that step's labels, exactly where; the pieces' masses, in which piece the token lies.
            uint64_t some = own > -INFINITY ? MassOf::fixed(mass(own, poly)) : 0;
            some = wave_sum_u64(some);
            if (lane == 0) s.sum[wave] = some;
            __syncthreads();
            some = 0;
            for (int w = 0; w < WAVES; ++w) some += s.sum[w];
            const double least = (1.0 - (double)row.topp) * ((double)some / mass.one) / (double)V;
            double low = mass.m + mass.t * log(least);
            low -= 1e-6 * (fabs(low) + fabs(mass.m));
            const float y_low = low > -3.4028234663852886e38 ? (float)low : -3.4028234663852886e38f;
            const float steps = 255.9f / (high - y_low);
            const float scale = steps < INFINITY && steps > 0.0f ? steps : 0.0f;
            const auto step_of = [&](float y) { return min(255u, (uint32_t)((high - y) * scale)); };
            // (the list's room serves as the pieces' histograms first)
            unsigned long long *piece = s.list;
            static_assert(HOLD || WAVES * 256 <= kCap, "histograms fit the list's room");
            for (int i = tid; i < WAVES * 256; i += THREADS) piece[i] = 0;
            __syncthreads();
            uint64_t z = 0;
            each(Ahead2{}, [&](int, const float (&y)[VEC]) {
                z -= VEC * MassOf::kRaw;
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    // (-inf and NaN have the mass 2^-1000, which rounds to 0)
                    const uint64_t w = MassOf::raw(mass(y[j], poly));
                    z += w;
                    if (y[j] >= y_low) atomicAdd(&piece[wave * 256 + step_of(y[j])], (unsigned long long)(w - MassOf::kRaw));
                }
            });
            z = wave_sum_u64(z);
            if (lane == 0) s.sum[wave] = z;
            if (tid == 0) { s.count = 0; s.first = 0; }
            __syncthreads();
            z = 0;
            for (int w = 0; w < WAVES; ++w) z += s.sum[w];
            const uint64_t target = top_p_goal(row.topp, z);
            const int slot = round % 3;
            for (int i = tid; i < 256; i += THREADS) {
                unsigned long long w = 0;
                for (int q = 0; q < WAVES; ++q) w += piece[q * 256 + i];
                s.hist.mass[slot][i] = w;
            }
            clear_hist<THREADS>(s.hist, (round + 1) % 3);
            __syncthreads();
            if (wave == 0) {
                const Digit d = find_digit(s.hist.mass[slot], s.hist.cnt[slot], true, 0, target);
                if (tid == 0) s.hist.found = d;
            }
            __syncthreads();
            ++round;
            const Digit d = s.hist.found;
            if (d.digit < 256) {
                // each wavefront's mass above the step
                uint64_t over = 0;
                for (uint32_t i = lane; i < d.digit; i += 64) over += piece[wave * 256 + i];
                over = wave_sum_u64(over);
                __syncthreads();                           // (the list's room is free)
                uint32_t kept = 0;
                each(Ahead4{}, [&](int v, const float (&y)[VEC]) {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        if (!(y[j] >= y_low)) continue;
                        const uint32_t t = step_of(y[j]);
                        kept += t < d.digit ? 1u : 0u;
                        if (t == d.digit) {
                            const uint64_t n = number(y[j], v + j);
                            const uint32_t at = atomicAdd(&s.count, 1u);
                            if (at < kCap) s.list[at] = n;
                            atomicMax(&s.first, (uint32_t)(n >> ibits));
                        }
                    }
                });
                __syncthreads();
                const uint32_t far = s.first, count = s.count;
                if (count <= kCap) {
                    take(count);
                    // (scores below the step lie below `far`, the search's end need not)
                    last = min(((uint64_t)far << ibits) + (((uint64_t)1 << ibits) - 1),
                               select_last<THREADS>(
                                   s.hist, round,
                                   [&](auto f) {
#pragma unroll
                                       for (int i = 0; i < E; ++i)
                                           if (el[i] != ~0ull) f(el[i], ew[i]);
                                   },
                                   true, ibits + (far ? 32 - __clz((int)far) : 1), target - d.before, 0));
                    done = true;
                    if (!(mass.lim > 0.0)) {
                        // the step's kept labels to their pieces; then the piece that holds the token
                        kept = (uint32_t)wave_sum_u64(kept);
                        if (lane == 0) { s.sum[wave] = over; s.b[wave] = kept; }
                        if (tid == 0) s.first = 0;
                        __syncthreads();
#pragma unroll
                        for (int i = 0; i < E; ++i)
                            if (el[i] <= last) {
                                const uint32_t v = (uint32_t)(el[i] & (((uint64_t)1 << ibits) - 1));
                                atomicAdd(&s.sum[v / (uint32_t)seg], (unsigned long long)ew[i]);
                                atomicAdd(&s.first, 1u);
                            }
                        __syncthreads();
                        uint64_t total = 0, before = 0, goal;
                        kept = s.first;
                        for (int w = 0; w < WAVES; ++w) { total += s.sum[w]; kept += s.b[w]; }
                        goal = draw_goal(row.u, total);
                        int at = 0;
                        while (at < WAVES - 1 && before + s.sum[at] < goal) before += s.sum[at++];
                        const int p0 = at * seg;
                        const float least = key_score(kmax - (uint32_t)(last >> ibits));
                        draw_row<XT, WAVES>(c, r, x + p0, min(seg, V - p0), p0, mass, row.u, s.row,
                                            {goal - before, total, kept}, [&](float y, int v, uint32_t &) {
                                                y = mass.read(y);
                                                if (!(y >= least)) return MassOf::kRaw;
                                                return MassOf::raw(number(y, v) <= last ? mass(y, poly) : 0.0);
                                            });
                        return;
                    }
                }
            }
        }
        if (!done)
            cut_elements<THREADS>(
                s, round, row,
                [&](uint64_t upto, auto f) {
                    each(Ahead2{}, [&](int v, const float (&y)[VEC]) {
#pragma unroll
                        for (int j = 0; j < VEC; ++j) {
                            if (!(y[j] > -INFINITY)) continue;
                            const uint64_t n = number(y[j], v + j);
                            if (n <= upto) f(n, MassOf::fixed(mass(y[j], poly)));
                        }
                    });
                },
                ibits + 32, last);
    }

    __syncthreads();
    const float cut_score = last == ~0ull ? -INFINITY : key_score(kmax - (uint32_t)(last >> ibits));
    const float least = fmaxf(cut_score, mass.least_score());
    draw_row<XT, WAVES>(c, r, x, V, 0, mass, row.u, s.row, {0, 0, 0}, [&](float y, int v, uint32_t &n) {
        y = mass.read(y);
        if (!(y >= least)) return MassOf::kRaw;
        const double w = mass(y, poly);
        const bool keep = y > -INFINITY && w >= mass.lim && (last == ~0ull || number(y, v) <= last);
        n += keep ? 1u : 0u;
        return MassOf::raw(keep ? w : 0.0);
    });
}

template <typename XT, int THREADS, int E, bool HOLD>
__global__ __launch_bounds__(THREADS) void k_draw(SampleCall c, int unit, int ibits, const uint32_t *open)
{
    __shared__ DrawShared<THREADS, E, HOLD> s;
    const Exp2Poly poly;
    uint32_t round = 0, round_small = 0;
    clear_hist<THREADS>(s.hist, 0);
    clear_hist<THREADS>(s.small.hist, 0);
    for (int64_t r = blockIdx.x; r < c.rows; r += gridDim.x) {
        if (!row_active(c.set, r) || (open && !open[r])) continue;
        __syncthreads();
        const RowRules row(c, r);
        draw_one<XT, THREADS, E, HOLD>(c, r, row, poly, unit, ibits, s, round, round_small);
    }
}

// Few long rows: a first launch cuts each row into chunks of kChunkPacks packs a
// thread of 256, one workgroup each, which reads its chunk once and leaves its
// largest score, its mass relative to that (where a row needs its whole mass),
// its number of labels above -inf, and a list of its labels above a bound of its
// own. A second launch joins a row's chunks: labels at or above the largest of the
// chunks' bounds are in the lists for certain, and draw_list works on those. Rows
// that they do not settle are left to a third launch, which takes them from their
// scores (in the second its code and registers would slow every row).
constexpr int kChunkThreads = 256;
constexpr int kChunkPacks = 2;
constexpr int kChunkList = 256;                        // entries of a chunk's list
constexpr int kJoinThreads = 256;
constexpr int kMaxChunks = kJoinThreads;               // of a row: one a thread of the join

struct ChunkStat {
    unsigned long long mass;                           // relative to `top`
    float top;
    uint32_t bound;                                    // key: all labels with a key above or at it are listed
    uint32_t listed;                                   // may pass kChunkList: the list does not hold
    uint32_t labels;                                   // above -inf
};

// What a row needs of its chunks.
__device__ __forceinline__ bool row_needs_mass(const RowRules &row) { return !row.greedy && !row.cut_k; }
__device__ __forceinline__ bool row_needs_list(const RowRules &row)
{
    return row.greedy || row.cut_k || row.cut_p || row.minp > 0.0f;
}

template <typename XT>
__global__ __launch_bounds__(kChunkThreads) void k_draw_chunk(SampleCall c, int unit, int chunks, ChunkStat *stats,
                                                              unsigned long long *lists)
{
    constexpr int VEC = 16 / sizeof(XT);
    constexpr int WAVES = kChunkThreads / 64;
    constexpr int kSpan = kChunkThreads * VEC;
    __shared__ Hist hist;
    __shared__ unsigned long long sum[WAVES];
    __shared__ uint32_t a[WAVES], b[WAVES], n_list;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const Exp2Poly poly;
    uint32_t round = 0;
    clear_hist<kChunkThreads>(hist, 0);
    for (int64_t w = blockIdx.x; w < c.rows * chunks; w += gridDim.x) {
        const int64_t r = w / chunks;
        if (!row_active(c.set, r)) continue;
        const int v0 = (int)(w - r * chunks) * (kSpan * kChunkPacks);
        const XT *x = (const XT *)c.x + r * c.x_stride;
        const RowRules row(c, r);
        float y[kChunkPacks][VEC];
        float own = -INFINITY;
#pragma unroll
        for (int i = 0; i < kChunkPacks; ++i) load_scores<XT, VEC>(x, c.V, v0 + i * kSpan + tid * VEC, y[i]);
        uint32_t labels = 0;
#pragma unroll
        for (int i = 0; i < kChunkPacks; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                own = fmaxf(own, y[i][j]);
                labels += y[i][j] > -INFINITY ? 1u : 0u;
            }
        float top = wave_max_f(own);
        labels = (uint32_t)wave_sum_u64(labels);
        const bool have = own > -INFINITY;
        const uint32_t key = score_key(own);
        uint32_t low = have ? key : 0xFFFFFFFFu;           // the smallest of the threads' largest
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) low = min(low, (uint32_t)__shfl_xor((int)low, d, 64));
        const uint32_t threads = __popcll(__ballot(have));
        __syncthreads();
        if (lane == 0) { a[wave] = __float_as_uint(top); b[wave] = low; sum[wave] = (unsigned long long)threads << 32 | labels; }
        if (tid == 0) n_list = 0;
        __syncthreads();
        uint64_t both = 0;
#pragma unroll
        for (int i = 0; i < WAVES; ++i) {
            top = fmaxf(top, __uint_as_float(a[i]));
            low = min(low, b[i]);
            both += sum[i];
        }
        labels = (uint32_t)both;
        uint64_t mass_sum = 0;
        if (row_needs_mass(row) && top > -INFINITY) {
            const MassOf mass(top, row.T, 0.0f, unit, false);
            mass_sum -= kChunkPacks * VEC * MassOf::kRaw;
#pragma unroll
            for (int i = 0; i < kChunkPacks; ++i)
#pragma unroll
                for (int j = 0; j < VEC; ++j) mass_sum += MassOf::raw(mass(mass.read(y[i][j]), poly));
        }
        mass_sum = wave_sum_u64(mass_sum);
        uint32_t bound = kKeyNegInf + 1u;                  // all labels above -inf
        if (row_needs_list(row) && top > -INFINITY) {
            // enough labels of every chunk that a row's lists together hold about 1536; for top_k twice a chunk's
            // share of it and 8, which the largest bound then rarely lies above (once in 10^4 rows in random order)
            const uint32_t share = row.greedy ? 1u
                                   : row.cut_k ? (uint32_t)min((int64_t)192, 8 + 2 * (int64_t)row.topk / chunks)
                                               : (uint32_t)min(192, max(8, 1536 / chunks));
            const uint32_t kmax = score_key(top);
            if ((uint32_t)(both >> 32) > share) {
                const uint32_t far = kmax - low;
                const uint64_t d = select_last<kChunkThreads>(
                    hist, round,
                    [&](auto f) {
                        if (have) f((uint64_t)(kmax - key), (uint64_t)1);
                    },
                    false, far ? 32 - __clz((int)far) : 1, share, share + share / 4 + 4);
                bound = max(bound, d < kmax ? kmax - (uint32_t)d : 0u);
            }
            const float floor_x = key_score(bound);
            unsigned long long *list = lists + w * kChunkList;
#pragma unroll
            for (int i = 0; i < kChunkPacks; ++i)
#pragma unroll
                for (int j = 0; j < VEC; ++j)
                    if (y[i][j] >= floor_x) {
                        const uint32_t at = atomicAdd(&n_list, 1u);
                        if (at < kChunkList)
                            list[at] = (unsigned long long)score_key(y[i][j]) << 32 | (uint32_t)(v0 + i * kSpan + tid * VEC + j);
                    }
        }
        __syncthreads();
        if (lane == 0) sum[wave] = mass_sum;
        __syncthreads();
        if (tid == 0) {
            ChunkStat st = {0, top, bound, n_list, labels};
#pragma unroll
            for (int i = 0; i < WAVES; ++i) st.mass += sum[i];
            stats[w] = st;
        }
    }
}

// Exclusive running sum over a workgroup, and its total.
template <int WAVES>
__device__ __forceinline__ uint64_t block_before(uint64_t v, unsigned long long *sum, uint64_t &total)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint64_t run = wave_scan_u64(v);
    __syncthreads();
    if (lane == 63) sum[wave] = run;
    __syncthreads();
    uint64_t before = run - v;
    total = 0;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) {
        before += i < wave ? (uint64_t)sum[i] : 0;
        total += sum[i];
    }
    return before;
}

template <typename XT>
__global__ __launch_bounds__(kJoinThreads) void k_draw_join(SampleCall c, int unit, int ibits, int chunks,
                                                           const ChunkStat *stats, const unsigned long long *lists,
                                                           uint32_t *open)
{
    constexpr int THREADS = kJoinThreads, WAVES = THREADS / 64, E = 8;
    constexpr int VEC = 16 / sizeof(XT);
    constexpr int kChunk = kChunkThreads * VEC * kChunkPacks;
    constexpr int kEach = kChunk / THREADS;
    __shared__ DrawShared<THREADS, E, false> s;
    __shared__ uint16_t n_listed[kMaxChunks];
    __shared__ uint32_t longest[WAVES];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const Exp2Poly poly;
    uint32_t round = 0, round_small = 0;
    clear_hist<THREADS>(s.hist, 0);
    clear_hist<THREADS>(s.small.hist, 0);
    for (int64_t r = blockIdx.x; r < c.rows; r += gridDim.x) {
        if (!row_active(c.set, r)) continue;
        __syncthreads();
        const RowRules row(c, r);
        const XT *x = (const XT *)c.x + r * c.x_stride;
        if (tid == 0) open[r] = 0;
        const bool mine = tid < chunks;
        ChunkStat st = {0, -INFINITY, kKeyNegInf + 1u, 0, 0};
        if (mine) st = stats[r * chunks + tid];
        float top = wave_max_f(st.top);
        uint32_t bound = st.bound;
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) bound = max(bound, (uint32_t)__shfl_xor((int)bound, d, 64));
        // s.a, s.b and s.sum: the row before has been read by all (the barrier above). Read here, s.sum and s.b are
        // written again behind a barrier only (block_before, element_totals, draw_list); a row that needs no masses
        // reaches its lists without one, so what it passes there, `longest` and n_listed, is read nowhere else.
        const uint64_t spilt = __ballot(st.listed > kChunkList);
        if (lane == 0) { s.a[wave] = __float_as_uint(top); s.b[wave] = bound; s.sum[wave] = spilt; }
        if (tid == 0) s.count = 0;
        __syncthreads();
        bool whole = true;                                 // every chunk's list holds
#pragma unroll
        for (int i = 0; i < WAVES; ++i) {
            top = fmaxf(top, __uint_as_float(s.a[i]));
            bound = max(bound, s.b[i]);
            whole = whole && s.sum[i] == 0;
        }
        if (top == -INFINITY) {
            if (tid == 0) emit(c, r, -1, -INFINITY, 0);
            continue;
        }
        const bool all = bound == kKeyNegInf + 1u;         // the lists hold the whole row
        const MassOf mass(top, row.T, row.minp, unit, row.greedy);
        const uint32_t kmax = score_key(mass.read(top));
        // the chunks' masses, brought to the row's largest score
        uint64_t z = 0, before = 0;
        if (row_needs_mass(row)) {
            const double w = mass(mass.read(st.top), poly) * ((double)st.mass / mass.one);
            const uint64_t m = st.top > -INFINITY ? (uint64_t)rint(w) : 0;
            before = block_before<WAVES>(m, s.sum, z);
            st.mass = m;
        }
        if (!row_needs_list(row)) {
            // no rule but the temperature: the chunk that holds the token, then its labels
            uint64_t labels;
            (void)block_before<WAVES>(mass.pick ? 0 : st.labels, s.sum, labels);
            const uint64_t goal = draw_goal(row.u, z);
            __syncthreads();
            if (before < goal && goal <= before + st.mass) { s.first = (uint32_t)tid; s.sum[0] = before; }
            __syncthreads();
            const int v = (int)s.first * kChunk + tid * kEach;
            const uint64_t front = s.sum[0];
            float y[kEach];
            uint64_t w[kEach], own = 0, total;
#pragma unroll
            for (int j = 0; j < kEach; ++j) {
                y[j] = v + j < c.V ? mass.read((float)x[v + j]) : -INFINITY;
                w[j] = MassOf::fixed(mass(y[j], poly));
                own += w[j];
            }
            uint64_t run = block_before<WAVES>(own, s.sum, total);
            // (the chunk's own sum differs from its share of z by roundings)
            const uint64_t left = min(goal - front, total);
            uint32_t found = 0xFFFFFFFFu;
            float score = 0.0f;
#pragma unroll
            for (int j = 0; j < kEach; ++j) {
                if (run < left && left <= run + w[j]) { found = v + j; score = y[j]; }
                run += w[j];
            }
            if (mass.pick) labels = (uint64_t)rint((double)z / mass.one);
            if (found != 0xFFFFFFFFu) emit(c, r, (int)found, mass.log_prob(score, z), (uint32_t)labels);
            if (total) continue;                           // (0 only where the chunk's whole share was one rounding)
        } else if (whole && (all || row.greedy || row.cut_k || row.cut_p ||
                             mass(mass.read(key_score(bound)), poly) < mass.lim)) {
            // all lists at once, as many places of each as the longest fills (a power of two)
            uint32_t most = st.listed;
#pragma unroll
            for (int d = 32; d >= 1; d >>= 1) most = max(most, (uint32_t)__shfl_xor((int)most, d, 64));
            if (lane == 0) longest[wave] = most;
            n_listed[tid] = (uint16_t)st.listed;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < WAVES; ++i) most = max(most, longest[i]);
            const int places = most > 1 ? 32 - __clz((int)most - 1) : 0;
            const unsigned long long *list = lists + r * chunks * kChunkList;
            constexpr int kAhead = 4;                          // loads in flight (those past a list's end are dropped)
            for (int i0 = tid; i0 - tid < chunks << places; i0 += kAhead * THREADS) {
                uint64_t e[kAhead], hit[kAhead];
                uint32_t hits = 0;
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    const int i = min(i0 + k * THREADS, (chunks << places) - 1);
                    e[k] = list[(size_t)(i >> places) * kChunkList + (i & ((1 << places) - 1))];
                }
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    const int i = min(i0 + k * THREADS, (chunks << places) - 1);
                    const float y = mass.read(key_score((uint32_t)(e[k] >> 32)));
                    const bool take = i == i0 + k * THREADS && (uint32_t)(i & ((1 << places) - 1)) < n_listed[i >> places] &&
                                      (uint32_t)(e[k] >> 32) >= bound && y > -INFINITY;
                    e[k] = (uint64_t)(kmax - score_key(y)) << ibits | (uint32_t)e[k];
                    hit[k] = __ballot(take);
                    hits += __popcll(hit[k]);
                }
                uint32_t at = 0;
                if (lane == 0 && hits) at = atomicAdd(&s.count, hits);
                at = __builtin_amdgcn_readfirstlane(at);
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    const uint32_t p = at + __popcll(hit[k] & ((1ull << lane) - 1ull));
                    if ((hit[k] >> lane & 1ull) && p < E * THREADS) s.list[p] = e[k];
                    at += __popcll(hit[k]);
                }
            }
            __syncthreads();
            const uint32_t n = s.count;
            if (n <= E * THREADS && (all || row.greedy || !row.cut_k || n >= (uint32_t)row.topk)) {
                const uint32_t far = mass.pick ? 0u : kmax - bound;
                const int digits = ibits + (far ? 32 - __clz((int)far) : 1);
                if (draw_listed<THREADS, E>(c, r, row, mass, poly, kmax, ibits, n, digits, all || row.cut_k ? 0 : z, s,
                                            round, round_small))
                    continue;
            }
        }
        if (tid == 0) open[r] = 1;
    }
}

// Wavefronts a row: one for short rows (the fixed work of a row, its scans and its
// logarithm, is then done once), more for long ones or where few rows would leave
// the card idle. 1 / 4 / 16 wavefronts, binary16, us: 500 labels, 4096 rows 12 / 25 / 84;
// 5000 labels, 256 rows 12 / 11 / 11, 1024 rows 13 / 15 / 27, 16000 rows 104 / 153 / 375;
// 32003 labels, 256 rows 50 / 19 / 17, 1024 rows 67 / 49 / 61, 2048 rows 94 / 81 / 115.
template <typename XT>
void draw_all(const SampleCall &c, int unit, hipStream_t s)
{
    constexpr int kPackW = 64 * (16 / (int)sizeof(XT));
    const int64_t packs = (c.V + kPackW - 1) / kPackW;
    const auto grid = [&](int64_t n) { return dim3((unsigned)std::min<int64_t>(n, kMaxRowGrid)); };
    if (packs >= 16 && c.rows <= 256) hipLaunchKernelGGL((k_draw_all<XT, 16>), grid(c.rows), dim3(1024), 0, s, c, unit);
    else if (packs >= 32 || (packs >= 4 && c.rows <= 512))
        hipLaunchKernelGGL((k_draw_all<XT, 4>), grid(c.rows), dim3(256), 0, s, c, unit);
    else hipLaunchKernelGGL((k_draw_all<XT, 1>), grid((c.rows + 3) / 4), dim3(256), 0, s, c, unit);
}

template <typename XT>
hipError_t sample_xt(const SampleCall &c, hipStream_t s)
{
    // V masses of at most 2^unit each stay below 2^62
    int ibits = 0;
    while ((1ll << ibits) < (long long)c.V) ++ibits;
    const int unit = std::min(51, 62 - ibits);
    const dim3 g((unsigned)std::min<int64_t>(c.rows, kMaxRowGrid));
    const int chunks = sample_chunks(c.rows, c.V, c.x_dtype);
    if (chunks) {
        ChunkStat *stats = (ChunkStat *)c.workspace;
        unsigned long long *lists = (unsigned long long *)(stats + c.rows * chunks);
        uint32_t *open = (uint32_t *)(lists + c.rows * chunks * kChunkList);
        const dim3 gc((unsigned)std::min<int64_t>(c.rows * chunks, kMaxRowGrid));
        hipLaunchKernelGGL(k_draw_chunk<XT>, gc, dim3(kChunkThreads), 0, s, c, unit, chunks, stats, lists);
        hipLaunchKernelGGL(k_draw_join<XT>, g, dim3(kJoinThreads), 0, s, c, unit, ibits, chunks, stats, lists, open);
        hipLaunchKernelGGL((k_draw<XT, 1024, 4, false>), g, dim3(1024), 0, s, c, unit, ibits, (const uint32_t *)open);
    } else if (c.top_k == 0 && !c.top_ks && c.top_p >= 1.0f && !c.top_ps) draw_all<XT>(c, unit, s);
    else if (c.V <= 512) hipLaunchKernelGGL((k_draw<XT, 64, 8, true>), g, dim3(64), 0, s, c, unit, ibits, (const uint32_t *)nullptr);
    else if (c.V <= 1024) hipLaunchKernelGGL((k_draw<XT, 64, 16, true>), g, dim3(64), 0, s, c, unit, ibits, (const uint32_t *)nullptr);
    else if (c.V <= 8192) hipLaunchKernelGGL((k_draw<XT, 256, 4, false>), g, dim3(256), 0, s, c, unit, ibits, (const uint32_t *)nullptr);
    else hipLaunchKernelGGL((k_draw<XT, 1024, 4, false>), g, dim3(1024), 0, s, c, unit, ibits, (const uint32_t *)nullptr);
    return hipGetLastError();
}

}  // namespace

// Chunks a row is cut into, 0 for rows that stay whole. Three launches pay for
// long rows only, and for few of them: 131072 bfloat16 labels, whole / in chunks,
// one row 34 / 19 us without cuts, 24 / 21 with top_k 50, 60 / 28 with top_p 0.9 (67 /
// 85 where the nucleus outgrows the lists); 32 rows 34 / 20, 24 / 24, 61 / 36; 64 rows
// 35 / 25, 24 / 30, 60 / 44; 32003 binary32 labels, one row 14 / 19, 18 / 19, 29 / 26.
// Next to the border, 70003 binary32 labels, whole / in chunks: one row 26 / 12 without
// cuts, 21 / 18 with top_k 50, 41 / 25 with top_p 0.9, 19 / 20 with min_p 0.05, 18 / 15
// greedy; 32 rows 27 / 16, 22 / 22, 44 / 31, 20 / 25, 18 / 17. By shape alone, so that the
// workspace does not depend on settings that live on the device: rows with min_p alone
// (131072 bfloat16, 32 rows 22 / 28) and nuclei that outgrow the lists pay for it.
int sample_chunks(int64_t rows, int32_t V, int32_t x_dtype)
{
    const int chunk = kChunkThreads * kChunkPacks * (16 / (int)dtype_size(x_dtype));
    const int chunks = (V + chunk - 1) / chunk;
    return rows <= 32 && V > 65536 && chunks <= kMaxChunks ? chunks : 0;
}

size_t sample_workspace(int64_t rows, int32_t V, int32_t x_dtype)
{
    const int chunks = sample_chunks(rows, V, x_dtype);
    if (!chunks) return 0;
    return (size_t)rows * chunks * (sizeof(ChunkStat) + kChunkList * 8) + (size_t)rows * 4;
}

hipError_t launch_sample(const SampleCall &c, hipStream_t s)
{
    if (c.x_dtype == kF32) return sample_xt<float>(c, s);
    if (c.x_dtype == kF16) return sample_xt<_Float16>(c, s);
    return sample_xt<__bf16>(c, s);
}

}  // namespace wfst
