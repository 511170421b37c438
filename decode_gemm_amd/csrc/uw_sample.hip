// Sampling from logits: temperature, top-k, top-p, min-p and the draw with a given uniform
// number, one token per row.
//
// Mathematics. With tokens ordered by (logit descending, index ascending), every filter keeps
// a beginning of the order, and the draw asks where a running mass crosses a number. So no row is
// ever sorted: each question is "the first token in the order at which the running count or mass
// reaches t", and it is answered from a histogram over the exponent y = (l - max) log2(e) / T
// (monotone in l, so bins are in order), then among the tokens of one bin. Masses are
// integers, round(2^43 * 2^y) from a 64-bit exponential, so sums are exact, the same in any order
// (atomics included), and two questions about the same tokens never contradict each other.
#include <hip/hip_runtime.h>

#include <cmath>

#include "uw_internal.h"

namespace uw {

namespace {

typedef unsigned long long u64;

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr int kBins = 2048;            // 46 per unit of y: the 44 units that have mass fill 2024 of them
constexpr double kBinsPerUnit = 46.0;
constexpr double kDeepest = -44.0;     // 2^43 * 2^y rounds to 0 from here down
constexpr int kList = 2048;            // tokens of the questioned bins that are sorted in LDS
constexpr u64 kOne = u64{1} << 43;     // mass of the row's largest token

struct SampleArgs {
    const void* x;
    int64_t ld, M;
    int32_t V;
    const float* u;
    const float* temperature;
    const int32_t* top_k;
    const float* top_p;
    const float* min_p;
    int32_t* token;
    float* prob;
};

__device__ __forceinline__ float value(const float* x, int i) { return x[i]; }
__device__ __forceinline__ float value(const uint16_t* x, int i) { return __uint_as_float(static_cast<uint32_t>(x[i]) << 16); }

// 2^f for f in [-0.5, 0.5] by its series in (f ln 2), twelve terms: the first one left out is
// below 2e-16 of the result.
__device__ __forceinline__ double exp2_poly(double f)
{
    const double t = f * 0.69314718055994530942;
    double p = 1.0 / 479001600.0;
    p = __builtin_fma(p, t, 1.0 / 39916800.0);
    p = __builtin_fma(p, t, 1.0 / 3628800.0);
    p = __builtin_fma(p, t, 1.0 / 362880.0);
    p = __builtin_fma(p, t, 1.0 / 40320.0);
    p = __builtin_fma(p, t, 1.0 / 5040.0);
    p = __builtin_fma(p, t, 1.0 / 720.0);
    p = __builtin_fma(p, t, 1.0 / 120.0);
    p = __builtin_fma(p, t, 1.0 / 24.0);
    p = __builtin_fma(p, t, 1.0 / 6.0);
    p = __builtin_fma(p, t, 0.5);
    p = __builtin_fma(p, t, 1.0);
    return __builtin_fma(p, t, 1.0);
}

// 2^43 * 2^y as a double, for y in (-44, 0].
__device__ __forceinline__ double weight(double y)
{
    const double n = __builtin_rint(y);
    return __builtin_ldexp(exp2_poly(y - n), static_cast<int>(n) + 43);
}

// Nearest whole number (ties to even) of 0 <= w < 2^52.
__device__ __forceinline__ u64 whole(double w)
{
    return static_cast<u64>(__double_as_longlong(w + 4503599627370496.0)) & ((u64{1} << 52) - 1);
}

// A row's scale of exponents.
struct Scale {
    float top;  // largest logit
    double c;   // log2(e) / T
    // y of logit l; anything at or below kDeepest has no mass
    __device__ __forceinline__ double y(float l) const
    {
        if (l == top) return 0.0;                    // also +inf - +inf
        if (!(l < top) || top == INFINITY || l == -INFINITY) return -INFINITY;  // NaN; finite beside +inf; masked
        return (static_cast<double>(l) - static_cast<double>(top)) * c;
    }
};

__device__ __forceinline__ int bin_of(double y) { return static_cast<int>(-y * kBinsPerUnit); }

// Sort key of (logit, index): ascending keys are the order. -0 and +0 are equal logits.
__device__ __forceinline__ uint32_t order_bits(float l)
{
    const uint32_t b = __float_as_uint(l + 0.0f);
    return (b & 0x80000000u) ? b : ~(b | 0x80000000u);  // larger logits get smaller bits
}
__device__ __forceinline__ float order_value(uint32_t o) { return __uint_as_float((o & 0x80000000u) ? o : ~o & 0x7FFFFFFFu); }

struct Shared {
    u64 H[kBins + 1];       // mass before each bin (while the histogram is made: mass of it)
    uint32_t C[kBins + 1];  // tokens before each bin
    u64 base[kBins];        // list path: H[bin] - mass in the list before the bin
    uint32_t cbase[kBins];  // likewise for counts (mod 2^32); slow path: digit histogram
    u64 list[kList];
    uint32_t take[kBins / 32];  // bins whose tokens go to the list
    u64 wsum[kWaves];
    uint32_t wcnt[kWaves];
    float wmax[kWaves];
    uint32_t n;
    int found[4];
    u64 mass[4];
    u64 drawn;
};

__device__ __forceinline__ u64 shfl_up64(u64 v, int d)
{
    const uint32_t lo = __shfl_up(static_cast<uint32_t>(v), d), hi = __shfl_up(static_cast<uint32_t>(v >> 32), d);
    return (static_cast<u64>(hi) << 32) | lo;
}

// Exclusive sums over the workgroup's threads.
__device__ void block_scan(Shared& S, u64 m, uint32_t c, u64& em, uint32_t& ec)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    u64 im = m;
    uint32_t ic = c;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const u64 a = shfl_up64(im, d);
        const uint32_t b = __shfl_up(ic, d);
        if (lane >= d) {
            im += a;
            ic += b;
        }
    }
    __syncthreads();
    if (lane == 63) {
        S.wsum[wave] = im;
        S.wcnt[wave] = ic;
    }
    __syncthreads();
    em = im - m;
    ec = ic - c;
    for (int w = 0; w < wave; w++) {
        em += S.wsum[w];
        ec += S.wcnt[w];
    }
}

// Smallest bin b with H[b + 1] >= t (1 <= t <= H[kBins]); all threads get it.
__device__ int find_mass(Shared& S, u64 t, int slot)
{
    for (int b = threadIdx.x; b < kBins; b += kThreads)
        if (S.H[b] < t && t <= S.H[b + 1]) S.found[slot] = b;
    __syncthreads();
    return S.found[slot];
}

// Where the running count (by_count) or mass reaches t inside bin b, found without a list: four
// passes over the row, each a histogram of the next eight bits of the order among the tokens that
// share those already known, leave one logit; its tokens weigh the same, so the crossing
// one is found by division. Returns the mass up to and with the crossing token; if `index`, also
// the token (a pass that counts that logit's tokens in order of index).
template <class T>
__device__ u64 search_row(Shared& S, const T* x, int V, const Scale& sc, int b, bool by_count, u64 t, bool index)
{
    u64 m0 = S.H[b];
    uint32_t c0 = S.C[b];
    uint32_t prefix = 0;
    u64* const dm = S.base;         // 256 digits' masses
    uint32_t* const dc = S.cbase;   // and counts
    for (int level = 0; level < 4; level++) {
        const int shift = 24 - 8 * level;
        __syncthreads();
        if (threadIdx.x < 256) {
            dm[threadIdx.x] = 0;
            dc[threadIdx.x] = 0;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < V; i += kThreads) {
            const float l = value(x, i);
            const double y = sc.y(l);
            if (!(y > kDeepest) || bin_of(y) != b) continue;
            const uint32_t o = order_bits(l);
            if (level && (o >> (shift + 8)) != prefix) continue;
            const uint32_t d = (o >> shift) & 255u;
            atomicAdd(&dm[d], whole(weight(y)));
            atomicAdd(&dc[d], 1u);
        }
        __syncthreads();
        const u64 m = threadIdx.x < 256 ? dm[threadIdx.x] : 0;
        const uint32_t c = threadIdx.x < 256 ? dc[threadIdx.x] : 0;
        u64 em;
        uint32_t ec;
        block_scan(S, m, c, em, ec);
        const bool here = by_count ? c0 + ec < t && t <= c0 + ec + c : m0 + em < t && t <= m0 + em + m;
        if (here) {
            S.found[3] = static_cast<int>(threadIdx.x);
            S.mass[3] = m0 + em;
            S.n = c0 + ec;
        }
        __syncthreads();
        prefix = (prefix << 8) | static_cast<uint32_t>(S.found[3]);
        m0 = S.mass[3];
        c0 = S.n;
    }
    const float l = order_value(prefix);
    const u64 w = whole(weight(sc.y(l)));
    const u64 j = by_count ? t - c0 : (t - m0 + w - 1) / w;  // the j-th token of this logit, from 1
    if (index) {
        const int chunk = (V + kThreads - 1) / kThreads;
        const int i0 = threadIdx.x * chunk, i1 = i0 + chunk < V ? i0 + chunk : V;
        uint32_t mine = 0;
        for (int i = i0; i < i1; i++) mine += value(x, i) == l;
        u64 em;
        uint32_t ec;
        block_scan(S, 0, mine, em, ec);
        if (ec < j && j <= ec + mine) {
            uint32_t seen = ec;
            for (int i = i0; i < i1; i++)
                if (value(x, i) == l && ++seen == j) S.drawn = (static_cast<u64>(prefix) << 32) | static_cast<uint32_t>(i);
        }
        __syncthreads();
    }
    return m0 + j * w;
}

template <class T>
__global__ void __launch_bounds__(kThreads) sample_rows(SampleArgs a)
{
    __shared__ Shared S;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t row = blockIdx.x;
    const T* const x = static_cast<const T*>(a.x) + row * a.ld;
    const int V = a.V;

    // the row's settings
    const float temp = a.temperature ? a.temperature[row] : 1.0f;
    const bool greedy = !(temp > 0.0f);
    int64_t k = greedy ? 1 : a.top_k ? a.top_k[row] : 0;
    const float p = a.top_p ? a.top_p[row] : 1.0f;
    const float mp = a.min_p ? a.min_p[row] : 0.0f;
    float u = a.u[row];
    u = u > 0.0f ? fminf(u, 0x1.fffffep-1f) : 0.0f;

    // the largest logit
    float top = -INFINITY;
    for (int i = tid; i < V; i += kThreads) top = fmaxf(top, value(x, i));
#pragma unroll
    for (int d = 32; d; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
    if (lane == 0) S.wmax[wave] = top;
    for (int b = tid; b < kBins; b += kThreads) {
        S.H[b] = 0;
        S.C[b] = 0;
    }
    if (tid < kBins / 32) S.take[tid] = 0;
    if (tid == 0) {
        S.n = 0;
        S.drawn = 0;
    }
    __syncthreads();
    for (int w = 0; w < kWaves; w++) top = fmaxf(top, S.wmax[w]);
    if (top == -INFINITY) {  // nothing to draw
        if (tid == 0) {
            a.token[row] = -1;
            if (a.prob) a.prob[row] = 0.0f;
        }
        return;
    }
    const Scale sc{top, 1.4426950408889634074 / (greedy ? 1.0 : static_cast<double>(temp))};

    // histogram of counts and masses
    for (int i = tid; i < V; i += kThreads) {
        const double y = sc.y(value(x, i));
        if (!(y > kDeepest)) continue;
        const int b = bin_of(y);
        atomicAdd(&S.H[b], whole(weight(y)));
        atomicAdd(&S.C[b], 1u);
    }
    __syncthreads();
    {
        const u64 m0 = S.H[2 * tid], m1 = S.H[2 * tid + 1];
        const uint32_t c0 = S.C[2 * tid], c1 = S.C[2 * tid + 1];
        u64 em;
        uint32_t ec;
        block_scan(S, m0 + m1, c0 + c1, em, ec);
        S.H[2 * tid] = em;
        S.H[2 * tid + 1] = em + m0;
        S.C[2 * tid] = ec;
        S.C[2 * tid + 1] = ec + c0;
        if (tid == kThreads - 1) {
            S.H[kBins] = em + m0 + m1;
            S.C[kBins] = ec + c0 + c1;
        }
    }
    __syncthreads();
    const u64 Z = S.H[kBins];
    const uint32_t tokens = S.C[kBins];

    // Bins in which each question's answer lies. Later questions depend on earlier answers,
    // which are known so far to a bin: they get the range of bins that the bounds allow.
    const bool by_k = k > 0 && k < static_cast<int64_t>(tokens);
    int b1 = 0;
    u64 lo = Z, hi = Z;  // bounds of the mass kept
    if (by_k) {
        for (int b = tid; b < kBins; b += kThreads)
            if (S.C[b] < k && k <= S.C[b + 1]) S.found[0] = b;
        __syncthreads();
        b1 = S.found[0];
        lo = S.H[b1];
        hi = S.H[b1 + 1];
        if (lo < 1) lo = 1;
        if (tid == 0) atomicOr(&S.take[b1 >> 5], 1u << (b1 & 31));
    }
    const bool by_p = p < 1.0f;
    auto p_target = [&](u64 m) {
        const double t = ceil(static_cast<double>(p) * static_cast<double>(m));
        const u64 v = t >= 1.0 ? static_cast<u64>(t) : 1;
        return v < m ? v : m;
    };
    if (by_p) {
        const int f = find_mass(S, p_target(lo), 1), g = find_mass(S, p_target(hi), 2);
        lo = S.H[f] < 1 ? 1 : S.H[f];
        if (S.H[g + 1] < hi) hi = S.H[g + 1];
        for (int b = f + tid; b <= g; b += kThreads) atomicOr(&S.take[b >> 5], 1u << (b & 31));
    }
    const bool by_m = mp > 0.0f && mp >= 0x1p-44f;
    const float least = fminf(mp, 1.0f);
    int q0 = 0, q1 = 0;
    if (by_m) {
        const int c = bin_of(log2(static_cast<double>(least)));
        q0 = c > 0 ? c - 1 : 0;
        q1 = c + 1 < kBins - 1 ? c + 1 : kBins - 1;
        if (S.H[q0] < lo) lo = S.H[q0] < 1 ? 1 : S.H[q0];
        if (S.H[q1 + 1] < hi) hi = S.H[q1 + 1];
        for (int b = q0 + tid; b <= q1; b += kThreads) atomicOr(&S.take[b >> 5], 1u << (b & 31));
    }
    auto u_target = [&](u64 m) { return static_cast<u64>(static_cast<double>(u) * static_cast<double>(m)) + 1; };
    {
        __syncthreads();
        const int f = find_mass(S, u_target(lo), 1), g = find_mass(S, u_target(hi), 2);
        for (int b = f + tid; b <= g; b += kThreads) atomicOr(&S.take[b >> 5], 1u << (b & 31));
    }
    __syncthreads();
    uint32_t n = 0;
    {
        uint32_t c = 0;
        for (int b = 2 * tid; b < 2 * tid + 2; b++)
            if ((S.take[b >> 5] >> (b & 31)) & 1u) c += S.C[b + 1] - S.C[b];
        if (c) atomicAdd(&S.n, c);
        __syncthreads();
        n = S.n;
        __syncthreads();
        if (tid == 0) S.n = 0;
    }
    __syncthreads();

    u64 kept = Z;
    if (n <= kList) {
        // their tokens, sorted
        for (int i = tid; i < V; i += kThreads) {
            const float l = value(x, i);
            const double y = sc.y(l);
            if (!(y > kDeepest)) continue;
            const int b = bin_of(y);
            if (!((S.take[b >> 5] >> (b & 31)) & 1u)) continue;
            const uint32_t at = atomicAdd(&S.n, 1u);
            S.list[at] = (static_cast<u64>(order_bits(l)) << 32) | static_cast<uint32_t>(i);
        }
        __syncthreads();
        int size = 64;
        while (size < static_cast<int>(n)) size <<= 1;
        for (int i = n + tid; i < size; i += kThreads) S.list[i] = ~u64{0};
        __syncthreads();
        for (int span = 2; span <= size; span <<= 1)
            for (int d = span >> 1; d; d >>= 1) {
                for (int i = tid; i < size / 2; i += kThreads) {
                    const int a0 = 2 * i - (i & (d - 1)), a1 = a0 + d;
                    const u64 v0 = S.list[a0], v1 = S.list[a1];
                    if ((v0 > v1) == ((a0 & span) == 0)) {
                        S.list[a0] = v1;
                        S.list[a1] = v0;
                    }
                }
                __syncthreads();
            }
        // mass before each of a thread's two tokens
        u64 key[2], mass[2], before[2];
        int bin[2];
        double w[2];
        for (int e = 0; e < 2; e++) {
            const int i = 2 * tid + e;
            key[e] = i < static_cast<int>(n) ? S.list[i] : ~u64{0};
            mass[e] = 0;
            bin[e] = -1;
            w[e] = 0;
            if (i < static_cast<int>(n)) {
                const double y = sc.y(order_value(static_cast<uint32_t>(key[e] >> 32)));
                w[e] = weight(y);
                mass[e] = whole(w[e]);
                bin[e] = bin_of(y);
            }
        }
        uint32_t unused;
        block_scan(S, mass[0] + mass[1], 0, before[0], unused);
        before[1] = before[0] + mass[0];
        for (int e = 0; e < 2; e++) {
            const int i = 2 * tid + e;
            if (bin[e] < 0) continue;
            const int prev = i == 0 ? -1 : e ? bin[0] : bin_of(sc.y(order_value(static_cast<uint32_t>(S.list[i - 1] >> 32))));
            if (prev != bin[e]) {
                S.base[bin[e]] = S.H[bin[e]] - before[e];
                S.cbase[bin[e]] = S.C[bin[e]] - i;
            }
        }
        __syncthreads();
        uint32_t rank[2];
        for (int e = 0; e < 2; e++)
            if (bin[e] >= 0) {
                before[e] += S.base[bin[e]];
                rank[e] = S.cbase[bin[e]] + 2 * tid + e;
            }
        if (by_k) {
            for (int e = 0; e < 2; e++)
                if (bin[e] >= 0 && rank[e] == k - 1) S.mass[0] = before[e] + mass[e];
            __syncthreads();
            kept = S.mass[0];
        }
        if (by_p) {
            const u64 t = p_target(kept);
            for (int e = 0; e < 2; e++)
                if (bin[e] >= 0 && before[e] < t && t <= before[e] + mass[e]) S.mass[1] = before[e] + mass[e];
            __syncthreads();
            kept = S.mass[1];
        }
        if (by_m) {
            if (tid == 0) S.mass[2] = S.H[q0] > kOne ? S.H[q0] : kOne;
            __syncthreads();
            const double wl = static_cast<double>(least) * static_cast<double>(kOne);
            for (int e = 0; e < 2; e++)
                if (bin[e] >= q0 && bin[e] <= q1 && w[e] >= wl) atomicMax(&S.mass[2], before[e] + mass[e]);
            __syncthreads();
            if (mp > 1.0f) kept = kOne;
            else if (S.mass[2] < kept) kept = S.mass[2];
        }
        const u64 t = u_target(kept);
        for (int e = 0; e < 2; e++)
            if (bin[e] >= 0 && before[e] < t && t <= before[e] + mass[e]) S.drawn = key[e];
        __syncthreads();
    } else {
        // too many tokens in those bins (long runs of equal logits): passes over the row
        if (by_k) kept = search_row(S, x, V, sc, b1, true, static_cast<u64>(k), false);
        if (by_p) {
            const u64 t = p_target(kept);
            __syncthreads();
            const int b = find_mass(S, t, 1);
            kept = search_row(S, x, V, sc, b, false, t, false);
        }
        if (by_m) {
            const double wl = static_cast<double>(least) * static_cast<double>(kOne);
            u64 m = 0;
            for (int i = tid; i < V; i += kThreads) {
                const double y = sc.y(value(x, i));
                if (!(y > kDeepest)) continue;
                const double w = weight(y);
                if (w >= wl) m += whole(w);
            }
            if (tid == 0) S.mass[2] = 0;
            __syncthreads();
            if (m) atomicAdd(&S.mass[2], m);
            __syncthreads();
            if (mp > 1.0f) kept = kOne;
            else if (S.mass[2] < kept) kept = S.mass[2];
        }
        const u64 t = u_target(kept);
        __syncthreads();
        const int b = find_mass(S, t, 1);
        search_row(S, x, V, sc, b, false, t, true);
        __syncthreads();
    }
    if (tid == 0) {
        const u64 d = S.drawn;
        a.token[row] = static_cast<int32_t>(d & 0xFFFFFFFFu);
        if (a.prob)
            a.prob[row] = static_cast<float>(weight(sc.y(order_value(static_cast<uint32_t>(d >> 32)))) / static_cast<double>(kept));
    }
}

uw_status check_sample(const uw_sample_args* p)
{
    if (!p) return fail(UW_EINVAL, "NULL argument");
    if (p->M < 0 || p->V < 1) return fail(UW_ESHAPE, "bad shape %lld x %lld", (long long)p->M, (long long)p->V);
    if (p->type != UW_F32 && p->type != UW_BF16) return fail(UW_EINVAL, "bad type %d", p->type);
    if (p->V > UW_SAMPLE_MAX_V) return fail(UW_EUNSUPPORTED, "V > %d", UW_SAMPLE_MAX_V);
    if (p->M >= (1 << 24)) return fail(UW_EUNSUPPORTED, "M >= 2^24");
    if (p->M == 0) return UW_OK;
    if (!p->d_logits || !p->d_u || !p->d_token) return fail(UW_EINVAL, "NULL device pointer");
    if (p->ld < p->V) return fail(UW_EINVAL, "ld must be >= V");
    if (!aligned(p->d_logits, p->type == UW_F32 ? 4 : 2)) return fail(UW_EINVAL, "d_logits misaligned");
    if (!aligned(p->d_u, 4) || !aligned(p->d_token, 4) || !aligned(p->d_temperature, 4) || !aligned(p->d_top_k, 4) ||
        !aligned(p->d_top_p, 4) || !aligned(p->d_min_p, 4) || !aligned(p->d_prob, 4))
        return fail(UW_EINVAL, "settings and outputs must be 4-byte aligned");
    const size_t need = uw_sample_workspace(p->M, p->V);
    if (need) {
        if (!p->d_ws || !aligned(p->d_ws, 16)) return fail(UW_EINVAL, "d_ws must be 16-byte aligned and not NULL");
        if (p->ws_bytes < need) return fail(UW_ENOSPACE, "workspace of %zu bytes needed", need);
    }
    return UW_OK;
}

}  // namespace

}  // namespace uw

using namespace uw;

size_t uw_sample_workspace(int64_t M, int64_t V)
{
    (void)M;
    (void)V;
    return 0;
}

uw_status uw_sample(const uw_sample_args* args, void* stream)
{
    clear_error();
    uw_status st = check_sample(args);
    if (st != UW_OK || args->M == 0) return st;
    SampleArgs a{};
    a.x = args->d_logits;
    a.ld = args->ld;
    a.M = args->M;
    a.V = static_cast<int32_t>(args->V);
    a.u = args->d_u;
    a.temperature = args->d_temperature;
    a.top_k = args->d_top_k;
    a.top_p = args->d_top_p;
    a.min_p = args->d_min_p;
    a.token = args->d_token;
    a.prob = args->d_prob;
    const dim3 grid(static_cast<uint32_t>(a.M));
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (args->type == UW_F32)
        hipLaunchKernelGGL(sample_rows<float>, grid, dim3(kThreads), 0, s, a);
    else
        hipLaunchKernelGGL(sample_rows<uint16_t>, grid, dim3(kThreads), 0, s, a);
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? UW_OK : fail(UW_EHIP, "sample launch failed: %s", hipGetErrorString(e));
}
