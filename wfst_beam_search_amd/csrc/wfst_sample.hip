// gfx950 (CDNA4) kernels of the draw of tokens from scores.
#include "wfst_score_device.h"

namespace wfst {

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
