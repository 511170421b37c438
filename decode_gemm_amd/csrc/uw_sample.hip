// Sampling from logits: temperature, top-k, top-p, min-p and the draw with a given uniform
// number, one token per row.
//
// Mathematics. With tokens ordered by (logit descending, index ascending), every filter keeps
// a beginning of the order, and the draw asks where a running mass crosses a number. So each
// question is "the first token in the order at which the running count or mass reaches t", and no
// row is ever sorted as a whole:
//   - the beginning of the order, a few hundred tokens, is gathered and sorted. Its lower end tau
//     comes from the largest logit of each thread's share: the q-th largest of those is reached
//     by at least q tokens, and hardly more while q is well below the number of threads.
//   - a question that reaches past it is answered from a histogram of masses over the
//     exponent y = (l - max) log2(e) / T (monotone in l, so bins are in order), and then among the
//     tokens of one bin.
// Masses are integers, round(2^43 2^y) from a 64-bit exponential, so sums are exact, the same in
// any order (atomics included), and two questions about the same tokens never contradict each
// other.
#include <hip/hip_runtime.h>

#include <cfloat>
#include <cmath>

#include "uw_internal.h"
#include "uw_order.h"
#include "uw_recon.h"

namespace uw {

namespace {

// A token's mass is worked out in several places and has to come out the same in all of them.
#pragma clang fp contract(off)

constexpr int kBins = 2048;            // 46 per unit of y: the 44 units that have mass fill 2025 of them
constexpr double kBinsPerUnit = 46.0, kUnitPerBin = 1.0 / 46.0;
constexpr double kDeepest = -44.0;     // 2^43 * 2^y rounds to 0 from here down
constexpr int kList = 4096;            // tokens that are sorted in LDS
constexpr uint32_t kAim = 256;         // tokens that the gathered beginning of the order has at least
constexpr uint32_t kCrowd = 255;       // most tokens of a sort bin that are compared with one another
// Largest k that it is made to hold, for `parts` workgroups of nt threads: of s = parts * nt maxima the q-th
// largest is reached by s ln(s / (s - q)) tokens or so, which leaves three tenths of the list free. (k = 1000
// of 131072: 1 row 20 us from the list, 51 by counting all tokens; 850 in 256 rows 59 and 87.)
__host__ __device__ constexpr int64_t short_most(uint32_t parts, int nt)
{
    return parts == 1 ? 7 * nt / 8 : parts * nt / 2 < kList / 2 ? parts * nt / 2 : kList / 2;
}
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

// Adding kRound to a double of less than 2^31 leaves its nearest whole number in the low 32 bits: two
// additions in place of a rounding and a conversion, which take four times an addition's time each.
constexpr double kRound = 6755399441055744.0;  // 3 * 2^51
__device__ __forceinline__ int low_bits(double v) { return static_cast<int>(__double_as_longlong(v)); }

// Bin b holds the y nearest to -b / 46; the sum's low bits are b.
__device__ __forceinline__ double bin_sum(double y) { return __builtin_fma(y, -kBinsPerUnit, kRound); }
__device__ __forceinline__ int bin_of(double y) { return low_bits(bin_sum(y)); }

// 2^43 * 2^y for y in (-44.5, 0] is that of the bin's middle times 2^d for the distance d from it; both
// are polynomials 1 + f q(f) where q meets (2^f - 1) / f at Chebyshev points (nine for |f| <= 1/2 with
// the whole part in the exponent bits, four for |d| <= 1/92), together within 7e-14 of the value, and
// exact at 0. Over whole rows the middles come from a table in LDS: the pass of 256 rows of 131072
// takes 28 us, 32 with one long polynomial for all of y.
__device__ __forceinline__ double middle(int b)
{
    const double y = static_cast<double>(b) * -kUnitPerBin, t = y + kRound, f = y - (t - kRound);
    double q = 0x1.b63880a30ec15p-24;
    q = __builtin_fma(q, f, 0x1.63d136366db24p-20);
    q = __builtin_fma(q, f, 0x1.ffcb9515a8013p-17);
    q = __builtin_fma(q, f, 0x1.4308ac85aa947p-13);
    q = __builtin_fma(q, f, 0x1.5d87fe86fe88ep-10);
    q = __builtin_fma(q, f, 0x1.3b2ab7181b755p-7);
    q = __builtin_fma(q, f, 0x1.c6b08d7047e52p-5);
    q = __builtin_fma(q, f, 0x1.ebfbdff823cedp-3);
    q = __builtin_fma(q, f, 0x1.62e42fefa39efp-1);
    const u64 v = static_cast<u64>(__double_as_longlong(__builtin_fma(q, f, 1.0)));
    return __longlong_as_double(static_cast<long long>(v + (static_cast<u64>(static_cast<uint32_t>(low_bits(t) + 43) << 20) << 32)));
}
__device__ __forceinline__ double weight(double y, double bin, double mid)
{
    const double d = __builtin_fma(bin - kRound, kUnitPerBin, y);
    double q = 0x1.3b2ade109790cp-7;
    q = __builtin_fma(q, d, 0x1.c6b0e2036dc06p-5);
    q = __builtin_fma(q, d, 0x1.ebfbdff829fbbp-3);
    q = __builtin_fma(q, d, 0x1.62e42fef9e814p-1);
    return mid * __builtin_fma(q, d, 1.0);
}
__device__ __forceinline__ double weight(double y)
{
    const double bin = bin_sum(y);
    return weight(y, bin, middle(low_bits(bin)));
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
    // y of logit l. Masked logits come out as -inf or NaN, and finite ones beside an infinite top
    // too: callers take y > kDeepest only.
    __device__ __forceinline__ double y(float l) const
    {
        return l == top ? 0.0 : (static_cast<double>(l) - static_cast<double>(top)) * c;
    }
};

// Bins in which the answers of a row's questions lie, and the logits of each range of bins (a little
// widened): 0 top-k, 1 top-p, 2 min-p, 3 the draw.
struct Marks {
    u64 Z;              // mass of the row
    float from[4], to[4];
    uint32_t by_k;      // top-k cuts, in bin b1, before which are c1 tokens
    uint32_t by_p, by_m;  // top-p and min-p may decide
    int32_t b1;
    uint32_t c1;
    int32_t q0, q1;     // bins that min-p's cut may be in
    uint32_t take[kBins / 32];    // all these bins
    uint32_t before[kBins / 32];  // how many of them lie before each word's
    uint32_t bins;                // and in all
};

template <int NT>
struct Shared {
    u64 H[kBins + 1];       // mass before each bin (while the histogram is made: mass of it)
    uint32_t C[kBins + 1];  // tokens before each bin, likewise
    double mid[kBins];      // middle(b), filled where a row's masses are summed
    u64 list[kList];
    u64 upto[kList];        // mass up to and with each token of the sorted list; scratch before that
    Marks marks;
    u64 wsum[NT / 64];
    uint32_t wcnt[NT / 64];
    float wmax[NT / 64];
    uint32_t spare[64];  // where lanes add what counts nowhere
    uint32_t n, first, last, crowd;
    int found[4];
    u64 mass[4];
    u64 drawn, kept;
};

// Inclusive sums over a wave's lanes (DPP: shifts within rows of 16, then row ends broadcast).
__device__ __forceinline__ uint32_t dpp_from(uint32_t v, int step)
{
    switch (step) {
    case 0: return __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);
    case 1: return __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
    case 2: return __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
    case 3: return __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
    case 4: return __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);
    default: return __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);
    }
}
__device__ __forceinline__ uint32_t wave_sums(uint32_t v)
{
#pragma unroll
    for (int s = 0; s < 6; s++) v += dpp_from(v, s);
    return v;
}
__device__ __forceinline__ u64 wave_sums(u64 v)
{
#pragma unroll
    for (int s = 0; s < 6; s++)
        v += (static_cast<u64>(dpp_from(static_cast<uint32_t>(v >> 32), s)) << 32) | dpp_from(static_cast<uint32_t>(v), s);
    return v;
}

// Exclusive sums over the workgroup's threads.
template <int NT>
__device__ void block_sums(Shared<NT>& S, u64 m, uint32_t c, u64& em, uint32_t& ec)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const u64 im = wave_sums(m);
    const uint32_t ic = wave_sums(c);
    __syncthreads();
    if (lane == 63) {
        S.wsum[wave] = im;
        S.wcnt[wave] = ic;
    }
    __syncthreads();
    em = im - m;
    ec = ic - c;
#pragma unroll
    for (int w = 0; w < NT / 64 - 1; w++) {
        const u64 a = S.wsum[w];
        const uint32_t b = S.wcnt[w];
        em += w < wave ? a : 0;
        ec += w < wave ? b : 0;
    }
}

// Largest of the threads' values, for all of them.
template <int NT>
__device__ __forceinline__ float block_max(Shared<NT>& S, float v)
{
#pragma unroll
    for (int d = 32; d; d >>= 1) v = fmaxf(v, __shfl_xor(v, d));
    __syncthreads();
    if ((threadIdx.x & 63) == 0) S.wmax[threadIdx.x >> 6] = v;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NT / 64; w++) v = fmaxf(v, S.wmax[w]);
    return v;
}

// test(logit) for the logits i0 .. i1-1 of a row, once each, by all threads of the workgroup (NaN must
// not pass). 16-byte loads between the 16-byte boundaries, up to 32 logits on the way per thread. What
// passes is noted in a mask, which goes to act(mask, index) by the batch, index(b) being the place of
// the logit that bit b stands for: most code here runs once or twice per launch, and fetching
// instructions costs more than running them, so only the test is unrolled.
template <int NT, int L, class T, class Test, class Act>
__device__ __forceinline__ void each_batch(const T* x, int i0, int i1, Test test, Act act)
{
    constexpr int W = 16 / sizeof(T), U = L / W;  // logits per load, loads on the way
    static_assert(L <= 32 && U >= 1, "mask");
    const int tid = threadIdx.x;
    int head = static_cast<int>((16 - (reinterpret_cast<uintptr_t>(x + i0) & 15)) & 15) / static_cast<int>(sizeof(T));
    head = head < i1 - i0 ? head : i1 - i0;
    const int a = i0 + head, nv = (i1 - a) / W, tail = a + nv * W;
    const u32x4* v = reinterpret_cast<const u32x4*>(x + a);
    for (int j0 = 0; j0 < nv; j0 += U * NT) {
        u32x4 q[U];
#pragma unroll
        for (int e = 0; e < U; e++) {
            const int j = j0 + e * NT + tid;
            q[e] = u32x4{~0u, ~0u, ~0u, ~0u};  // NaN
            if (j < nv) q[e] = v[j];
        }
        uint32_t passed = 0;
#pragma unroll
        for (int e = 0; e < U; e++)
#pragma unroll
            for (int c = 0; c < 4; c++) {
                if constexpr (W == 4) {
                    passed |= test(__uint_as_float(q[e][c])) ? 1u << (W * e + c) : 0u;
                } else {
                    passed |= test(__uint_as_float(q[e][c] << 16)) ? 1u << (W * e + 2 * c) : 0u;
                    passed |= test(__uint_as_float(q[e][c] & 0xFFFF0000u)) ? 1u << (W * e + 2 * c + 1) : 0u;
                }
            }
        act(passed, [&](int b) { return a + W * (j0 + b / W * NT + tid) + b % W; });
    }
    // the logits beside the boundaries
    const bool mine = tid < head + (i1 - tail);
    const int at = tid < head ? i0 + tid : tail + tid - head;
    if (head + (i1 - tail) > 0) act(mine && test(value(x, at)) ? 1u : 0u, [&](int) { return at; });
}

// act(logit, index) for those that pass.
template <int NT, int L, class T, class Test, class Act>
__device__ __forceinline__ void each_if(const T* x, int i0, int i1, Test test, Act act)
{
    each_batch<NT, L>(x, i0, i1, test, [&](uint32_t passed, auto index) {
        while (passed) {
            const int at = index(__ffs(passed) - 1);
            passed &= passed - 1;
            act(value(x, at), at);
        }
    });
}

// The indexes of those that pass go to the list, counted in S.n, which may pass kList. A wave reserves
// room for its batch at once; the logits are read again behind that (to_keys), all at the same time.
template <int NT, int L, class T, class Test>
__device__ __forceinline__ void collect(Shared<NT>& S, const T* x, int i0, int i1, Test test)
{
    each_batch<NT, L>(x, i0, i1, test, [&](uint32_t passed, auto index) {
        if (!__any(passed)) return;
        const uint32_t c = __popc(passed), upto = wave_sums(c);
        uint32_t at = 0;
        if ((threadIdx.x & 63) == 63) at = atomicAdd(&S.n, upto);
        at = __builtin_amdgcn_readlane(at, 63) + upto - c;
        while (passed) {
            if (at < kList) S.list[at] = static_cast<u64>(index(__ffs(passed) - 1));
            at++;
            passed &= passed - 1;
        }
    });
}

template <int NT>
__device__ __forceinline__ void fill_middles(Shared<NT>& S)
{
    for (int b = threadIdx.x; b < kBins; b += NT) S.mid[b] = middle(b);
}

// A row's settings, brought into range.
struct Row {
    bool by_k, by_p, by_m;
    bool short_k;  // the beginning of the order answers top-k: then no masses of other tokens are needed
    int64_t k;
    float temp;  // 1 for the greedy choice, which is k = 1
    float p, least, u;
    bool only_first;  // min-p above 1

    __device__ __forceinline__ Row(const SampleArgs& a, int64_t row, int64_t most)
    {
        const float t = a.temperature ? a.temperature[row] : 1.0f;
        const int32_t kk = a.top_k ? a.top_k[row] : 0;
        const float m = a.min_p ? a.min_p[row] : 0.0f, v = a.u[row];
        p = a.top_p ? a.top_p[row] : 1.0f;
        const bool greedy = !(t > 0.0f);
        temp = greedy ? 1.0f : t;
        k = greedy ? 1 : kk;
        by_k = k > 0 && k < a.V;
        short_k = by_k && k <= most;
        by_p = p < 1.0f;
        by_m = m > 0.0f && m >= 0x1p-44f;
        only_first = m > 1.0f;
        least = fminf(m, 1.0f);
        u = v > 0.0f ? fminf(v, 0x1.fffffep-1f) : 0.0f;
    }
    // the mass that top-p asks of m, and the one that the draw asks of m
    __device__ __forceinline__ u64 p_target(u64 m) const
    {
        const double t = ceil(static_cast<double>(p) * static_cast<double>(m));
        const u64 v = t >= 1.0 ? static_cast<u64>(t) : 1;
        return v < m ? v : m;
    }
    __device__ __forceinline__ u64 u_target(u64 m) const { return static_cast<u64>(static_cast<double>(u) * static_cast<double>(m)) + 1; }
    // the least whole mass that min-p keeps
    __device__ __forceinline__ u64 least_mass() const { return static_cast<u64>(ceil(static_cast<double>(least) * static_cast<double>(kOne))); }
    __device__ __forceinline__ Scale scale(float top) const { return Scale{top, 1.4426950408889634074 / static_cast<double>(temp)}; }
};

// Smallest bin b with H[b + 1] >= t (1 <= t <= H[kBins]); all threads get it.
template <int NT>
__device__ int find_mass(Shared<NT>& S, u64 t, int slot)
{
    for (int b = threadIdx.x; b < kBins; b += NT)
        if (S.H[b] < t && t <= S.H[b + 1]) S.found[slot] = b;
    __syncthreads();
    return S.found[slot];
}

// The same for two masses at once.
template <int NT>
__device__ void find_two(Shared<NT>& S, u64 t, u64 u, int& f, int& g)
{
    for (int b = threadIdx.x; b < kBins; b += NT) {
        const u64 from = S.H[b], to = S.H[b + 1];
        if (from < t && t <= to) S.found[1] = b;
        if (from < u && u <= to) S.found[2] = b;
    }
    __syncthreads();
    f = S.found[1];
    g = S.found[2];
}

// H and (counts) C from contents of bins to sums before each bin.
template <int NT>
__device__ void bins_to_sums(Shared<NT>& S, bool masses, bool counts)
{
    constexpr int B = kBins / NT;
    const int b0 = B * threadIdx.x;
    u64 m[B], mt = 0;
    uint32_t c[B], ct = 0;
    __syncthreads();
#pragma unroll
    for (int b = 0; b < B; b++) {
        m[b] = masses ? S.H[b0 + b] : 0;
        c[b] = counts ? S.C[b0 + b] : 0;
        mt += m[b];
        ct += c[b];
    }
    u64 em;
    uint32_t ec;
    block_sums(S, mt, ct, em, ec);
#pragma unroll
    for (int b = 0; b < B; b++) {
        if (masses) S.H[b0 + b] = em;
        if (counts) S.C[b0 + b] = ec;
        em += m[b];
        ec += c[b];
    }
    if (threadIdx.x == NT - 1) {
        if (masses) S.H[kBins] = em;
        if (counts) S.C[kBins] = ec;
    }
    __syncthreads();
}

template <int NT>
__device__ __forceinline__ void clear_bins(Shared<NT>& S, bool masses, bool counts)
{
    for (int b = threadIdx.x; b < kBins; b += NT) {
        if (masses) S.H[b] = 0;
        if (counts) S.C[b] = 0;
    }
}

// A logit at or below the lower end of bin b (bins of smaller number hold larger logits).
__device__ __forceinline__ float below_bin(const Scale& sc, int b)
{
    if (sc.top == INFINITY) return INFINITY;
    const float t = static_cast<float>(static_cast<double>(sc.top) - (static_cast<double>(b) + 0.5) / kBinsPerUnit / sc.c);
    // a little less, for the roundings (of the difference, too); -inf where all logits weigh the same
    return t - fabsf(t) * 0x1p-22f - fabsf(sc.top) * 0x1p-48f - FLT_MIN;
}

// A logit at or above the upper end of bin b.
__device__ __forceinline__ float above_bin(const Scale& sc, int b)
{
    if (b == 0) return INFINITY;
    // (-inf where a bin ends within the margin of the lowest number: kept from becoming NaN, which no logit
    // would reach; the logits there are then looked at for more bins than their own)
    const float t = fmaxf(below_bin(sc, b - 1), -FLT_MAX);
    return t + fabsf(t) * 0x1p-20f + fabsf(sc.top) * 0x1p-46f + 3 * FLT_MIN;
}

// f(logit, bin, mass) for the logits of a row in the bins b0 .. b1 (with S.mid filled).
template <int NT, class T, class F>
__device__ __forceinline__ void each_mass(const Shared<NT>& S, const T* x, int V, const Scale& sc, int b0, int b1, F f)
{
    const float from = fmaxf(below_bin(sc, b1), -FLT_MAX), to = above_bin(sc, b0);
    each_if<NT, 32>(
        x, 0, V, [&](float l) { return (l >= from) & (l <= to); },
        [&](float l, int) {
            const double y = sc.y(l), bin = bin_sum(y);
            const int b = low_bits(bin);
            if (y > kDeepest && b >= b0 && b <= b1) f(l, b, whole(weight(y, bin, S.mid[b])));
        });
}

// A logit that at least q of the threads' maxima `mine` reach; -inf if fewer than q have mass.
template <int NT>
__device__ float reached_by(Shared<NT>& S, float mine, const Scale& sc, uint32_t q)
{
    clear_bins(S, false, true);
    if (threadIdx.x == 0) S.found[0] = -1;
    __syncthreads();
    const double y = sc.y(mine);
    if (y > kDeepest) atomicAdd(&S.C[bin_of(y)], 1u);
    bins_to_sums(S, false, true);
    for (int b = threadIdx.x; b < kBins; b += NT)
        if (S.C[b] < q && q <= S.C[b + 1]) S.found[0] = b;
    __syncthreads();
    const int b = S.found[0];
    return b < 0 ? -INFINITY : below_bin(sc, b);
}

// Keys in place of the indexes in the list.
template <int NT, class T>
__device__ __forceinline__ void to_keys(Shared<NT>& S, const T* x, int n)
{
    for (int i = threadIdx.x; i < n; i += NT) {
        const int at = static_cast<int>(S.list[i]);
        S.list[i] = key_of(value(x, at), at);
    }
    __syncthreads();
}

// The masses of all tokens of i0 .. i1-1 go to the histogram (COUNT: and their number), and the indexes of
// those that reach tau to the list. Without branches, so that the exponentials of several logits
// overlap: what has no mass (NaN too) adds to a place of its lane's own, and masses a little below
// the end are 0.
template <int NT, bool COUNT, class T>
__device__ __forceinline__ void add_masses(Shared<NT>& S, const T* x, int i0, int i1, const Scale& sc, float end, float tau)
{
    const double top = static_cast<double>(sc.top);
    collect<NT, 16>(S, x, i0, i1, [&](float l) {
        double y = fmax((static_cast<double>(l) - top) * sc.c, kDeepest - 0.49);
        if (COUNT && l == sc.top) y = 0.0;  // an infinite one too
        const double bin = bin_sum(y);
        const int b = low_bits(bin);
        atomicAdd(l >= end ? &S.H[b] : &S.upto[threadIdx.x & 63], whole(weight(y, bin, S.mid[b])));
        if (COUNT) atomicAdd(((l >= end) & (y > kDeepest)) ? &S.C[b] : &S.spare[threadIdx.x & 63], 1u);
        return l >= tau;
    });
}

// What has no mass ends below this logit.
__device__ __forceinline__ float mass_end(const Scale& sc)
{
    return fmaxf(below_bin(sc, static_cast<int>(-kDeepest * kBinsPerUnit)), -FLT_MAX);
}

// The indexes of the tokens of i0 .. i1-1 that reach tau go to the list (those that have no mass only
// if they come within the rounding of its end); with `masses` all tokens' masses go to the histogram,
// with `counts` their numbers too.
template <int NT, class T>
__device__ void gather(Shared<NT>& S, const T* x, int i0, int i1, const Scale& sc, float tau, bool masses, bool counts)
{
    const float end = mass_end(sc);
    tau = fmaxf(tau, end);
    if (counts)
        add_masses<NT, true>(S, x, i0, i1, sc, end, tau);
    else if (masses)
        add_masses<NT, false>(S, x, i0, i1, sc, end, tau);
    else
        collect<NT, 32>(S, x, i0, i1, [&](float l) { return l >= tau; });
}

// The place of a token's bin among the marked ones, drawn out to `sub` sort bins each by its place
// within it. A token of no marked bin, there by rounding alone, goes before the next one.
template <int NT>
__device__ __forceinline__ int marked_place(const Shared<NT>& S, const Scale& sc, u64 key, int sub)
{
    const Marks& K = S.marks;
    const double v = fmin(sc.y(key_value(key)) * -kBinsPerUnit, kBins - 1.0);  // -inf and the like of y too
    const int b = low_bits(v + kRound);
    const uint32_t w = K.take[b >> 5], bit = 1u << (b & 31);
    int at = static_cast<int>(K.before[b >> 5] + __popc(w & (bit - 1))) * sub;
    if (w & bit) {
        const int f = static_cast<int>((v - b + 0.5) * sub);
        at += f < sub - 1 ? f : sub - 1;
    }
    return at < kBins - 1 ? at : kBins - 1;
}

// Sort the n (1 .. kList) tokens of the list: into bins that share out the range between its largest
// and smallest logit (or, of marked bins, those), then by comparing within a bin. Lists that crowd a bin
// (ties) go through a bitonic network instead: 512 tokens in 10 us. Uses C.
template <int NT>
__device__ void sort_list(Shared<NT>& S, const Scale& sc, int n, bool marked)
{
    const int tid = threadIdx.x;
    uint32_t lo = ~0u, hi = 0;
    if (tid == 0) {
        S.first = ~0u;
        S.last = 0;
        S.crowd = 0;
    }
    clear_bins(S, false, true);
    float top = 0.f, scale = 0.f;
    int sub = 0;
    if (marked) {
        sub = kBins / static_cast<int>(S.marks.bins);
    } else {
        for (int i = tid; i < n; i += NT) {
            const uint32_t o = static_cast<uint32_t>(S.list[i] >> 32);
            lo = o < lo ? o : lo;
            hi = o > hi ? o : hi;
        }
#pragma unroll
        for (int d = 32; d; d >>= 1) {
            const uint32_t a = __shfl_xor(lo, d), b = __shfl_xor(hi, d);
            lo = a < lo ? a : lo;
            hi = b > hi ? b : hi;
        }
        __syncthreads();
        if ((tid & 63) == 0) {
            atomicMin(&S.first, lo);
            atomicMax(&S.last, hi);
        }
    }
    __syncthreads();
    if (!marked) {
        top = order_value(S.first);
        const float span = top - order_value(S.last);
        scale = span > 0.f && span < INFINITY ? (kBins - 1) / span : 0.f;
    }
    auto bin = [&](u64 k) {
        if (marked) return marked_place(S, sc, k, sub);
        const int b = scale > 0.f ? static_cast<int>((top - key_value(k)) * scale) : 0;
        return b < kBins - 1 ? b : kBins - 1;
    };
    for (int i = tid; i < n; i += NT)
        if (atomicAdd(&S.C[bin(S.list[i])], 1u) == kCrowd) S.crowd = 1;
    __syncthreads();
    if (!S.crowd) {
        bins_to_sums(S, false, true);
        for (int i = tid; i < n; i += NT) {
            const u64 k = S.list[i];
            S.upto[atomicAdd(&S.C[bin(k)], 1u)] = k;
        }
        __syncthreads();
        // C[b] has come to the end of bin b
        for (int i = tid; i < n; i += NT) {
            const u64 k = S.upto[i];
            const int b = bin(k), i0 = b ? S.C[b - 1] : 0, i1 = S.C[b];
            int at = i0;
            for (int e = i0; e < i1; e++) at += S.upto[e] < k;
            S.list[at] = k;
        }
        __syncthreads();
        return;
    }
    int size = 64;
    while (size < n) size <<= 1;
    for (int i = n + tid; i < size; i += NT) S.list[i] = ~u64{0};
    __syncthreads();
    for (int width = 2; width <= size; width <<= 1)
        for (int d = width >> 1; d; d >>= 1) {
            for (int i = tid; i < size / 2; i += NT) {
                const int a0 = 2 * i - (i & (d - 1)), a1 = a0 + d;
                const u64 v0 = S.list[a0], v1 = S.list[a1];
                if ((v0 > v1) == ((a0 & width) == 0)) {
                    S.list[a0] = v1;
                    S.list[a1] = v0;
                }
            }
            __syncthreads();
        }
}

// y of a token of the list, and its mass: 0 from kDeepest down, where weight() ends.
__device__ __forceinline__ double listed_y(const Scale& sc, u64 key) { return fmax(sc.y(key_value(key)), kDeepest - 0.49); }
__device__ __forceinline__ u64 mass_of(const Scale& sc, u64 key) { return whole(weight(listed_y(sc, key))); }

// upto[] of the sorted list: masses summed within the list (rows == false), or over the row by the
// sums in H, where the list holds whole bins (H of those bins is used up; tokens of other bins, there
// by rounding alone, get sums between those of the marked bins around them). Returns the place of the
// first token of bin b1 in the list (rows only).
template <int NT>
__device__ int sum_list(Shared<NT>& S, int n, const Scale& sc, bool rows, int b1)
{
    const int tid = threadIdx.x, share = (n + NT - 1) / NT;
    const int from = tid * share < n ? tid * share : n, to = from + share < n ? from + share : n;
    u64 total = 0, before;
    for (int i = from; i < to; i++) {
        const u64 m = mass_of(sc, S.list[i]);
        S.upto[i] = m;
        total += m;
    }
    uint32_t unused;
    if (tid == 0) S.found[3] = 0;
    block_sums(S, total, 0, before, unused);
    u64 m = before;
    auto bin = [&](int i) { return bin_of(listed_y(sc, S.list[i])); };
    for (int i = from; i < to; i++) {
        if (rows) {
            const int b = bin(i);
            if (i == 0 || bin(i - 1) != b) {
                S.H[b] -= m;  // what comes before the bin and is not in the list
                if (b == b1) S.found[3] = i;
            }
        }
        m += S.upto[i];
        S.upto[i] = m;
    }
    __syncthreads();
    if (rows) {
        for (int i = from; i < to; i++) S.upto[i] += S.H[bin(i)];
        __syncthreads();
    }
    return S.found[3];
}

// First i < n with reached(i), which once true stays true; n if none. By one wave, two looks of 64.
template <class F>
__device__ __forceinline__ int first_that(int n, F reached)
{
    const int lane = threadIdx.x & 63, stride = (n + 63) / 64;  // n <= 64 * 64
    const int end = (lane + 1) * stride < n ? (lane + 1) * stride : n;
    const u64 a = __ballot(reached(end - 1));
    if (!a) return n;
    const int from = (__ffsll(static_cast<long long>(a)) - 1) * stride;
    const u64 b = __ballot(lane < stride && (from + lane >= n || reached(from + lane)));
    return from + __ffsll(static_cast<long long>(b)) - 1;
}

// Whether the list that tau gives has every token with mass.
__device__ __forceinline__ bool holds_all(const Scale& sc, float tau) { return tau == -INFINITY || sc.top == INFINITY; }

// Whether min-p's cut is above tau by a margin in y.
__device__ __forceinline__ bool cuts_above(const Row& r, const Scale& sc, float tau, double margin)
{
    return r.only_first || sc.y(tau) < log2(static_cast<double>(r.least)) - margin;
}

// Whether the masses of all tokens are needed beside the list that tau gives.
__device__ __forceinline__ bool needs_masses(const Row& r, const Scale& sc, float tau)
{
    if (holds_all(sc, tau)) return false;  // the list answers, or from_row counts for itself
    if (r.by_k) return !r.short_k;
    if (r.by_p || !r.by_m) return true;
    return !cuts_above(r, sc, tau, 0.01);  // min-p alone, and its cut lies in the list
}

// Answer from the beginning of the order (n tokens, those that reach tau; all: every token with mass is in it; Z: the
// row's mass, 0 if not known). Leaves the token in S.drawn and returns the mass kept; 0 if a
// question reaches past the list.
template <int NT>
__device__ u64 from_list(Shared<NT>& S, const Row& r, const Scale& sc, int n, float tau, u64 Z)
{
    const bool all = holds_all(sc, tau);
    if (Z && !(r.by_m && cuts_above(r, sc, tau, -0.01))) {
        // the first question decides: does it reach past the list? (min-p does unless it cuts in the list)
        u64 m = 0, before;
        uint32_t unused;
        for (int i = threadIdx.x; i < n; i += NT) m += mass_of(sc, S.list[i]);
        block_sums(S, m, 0, before, unused);
        if (threadIdx.x == NT - 1) S.mass[0] = before + m;
        __syncthreads();
        if ((r.by_p ? r.p_target(Z) : r.by_m ? Z : r.u_target(Z)) > S.mass[0]) return 0;
    }
    sort_list(S, sc, n, false);
    sum_list(S, n, sc, false, 0);
    if (threadIdx.x < 64) {
        const u64 L = S.upto[n - 1];
        u64 kept = all ? L : Z;  // 0: not known, but more than the list
        bool open = false;       // a question reaches past the list
        if (r.by_k && r.k <= n)
            kept = S.upto[r.k - 1];
        else if (r.by_k && !all)
            open = true;
        if (r.by_p) {
            const u64 t = kept ? r.p_target(kept) : ~u64{0};
            kept = t <= L ? S.upto[first_that(n, [&](int i) { return S.upto[i] >= t; })] : 0;
        }
        if (r.by_m) {
            const u64 w = r.least_mass();
            const int i = r.only_first ? 1 : first_that(n, [&](int j) { return mass_of(sc, S.list[j]) < w; });
            const u64 m = i > 0 ? S.upto[i - 1] : S.upto[0];
            if (i < n || all)
                kept = kept && kept < m ? kept : m;
            else if (kept > L)
                kept = 0;  // the cut may lie past the list
        }
        const u64 t = kept ? r.u_target(kept) : ~u64{0};
        open |= t > L;
        if (!open) {
            const int i = first_that(n, [&](int j) { return S.upto[j] >= t; });
            if (threadIdx.x == 0) S.drawn = S.list[i];
        }
        if (threadIdx.x == 0) S.kept = open ? 0 : kept;
    }
    __syncthreads();
    return S.kept;
}

// Where the running count (by_count) or mass reaches t inside bin b, found without a list: four
// passes over the row, each a histogram of the next eight bits of the order among the tokens that
// share those already known, leave one logit; its tokens weigh the same, so the crossing
// one is found by division. Returns the mass up to and with the crossing token; if `index`, also
// the token (a pass that counts that logit's tokens in order of index).
template <int NT, class T>
__device__ u64 search_row(Shared<NT>& S, const T* x, int V, const Scale& sc, int b, bool by_count, u64 t, bool index)
{
    u64 m0 = S.H[b];
    uint32_t c0 = by_count ? S.C[b] : 0;
    uint32_t prefix = 0;
    u64* const dm = S.upto;                                      // 256 digits' masses
    uint32_t* const dc = reinterpret_cast<uint32_t*>(S.list);    // and counts
#pragma unroll 1
    for (int level = 0; level < 4; level++) {
        const int shift = 24 - 8 * level;
        __syncthreads();
        if (threadIdx.x < 256) {
            dm[threadIdx.x] = 0;
            dc[threadIdx.x] = 0;
        }
        __syncthreads();
        each_mass<NT>(S, x, V, sc, b, b, [&](float l, int, u64 mass) {
            const uint32_t o = order_bits(l);
            if (level && (o >> (shift + 8)) != prefix) return;
            const uint32_t d = (o >> shift) & 255u;
            atomicAdd(&dm[d], mass);
            atomicAdd(&dc[d], 1u);
        });
        __syncthreads();
        const u64 m = threadIdx.x < 256 ? dm[threadIdx.x] : 0;
        const uint32_t c = threadIdx.x < 256 ? dc[threadIdx.x] : 0;
        u64 em;
        uint32_t ec;
        block_sums(S, m, c, em, ec);
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
        const int chunk = (V + NT - 1) / NT;
        const int i0 = threadIdx.x * chunk, i1 = i0 + chunk < V ? i0 + chunk : V;
        uint32_t mine = 0;
        for (int i = i0; i < i1; i++) mine += value(x, i) == l;
        u64 em;
        uint32_t ec;
        block_sums(S, 0, mine, em, ec);
        if (ec < j && j <= ec + mine) {
            uint32_t seen = ec;
            for (int i = i0; i < i1; i++)
                if (value(x, i) == l && ++seen == j) S.drawn = key_of(l, i);
        }
        __syncthreads();
    }
    return m0 + j * w;
}

// The row's histogram of masses and counts, as sums.
template <int NT, class T>
__device__ void count_row(Shared<NT>& S, const T* x, int V, const Scale& sc)
{
    __syncthreads();
    clear_bins(S, true, true);
    fill_middles(S);
    __syncthreads();
    gather(S, x, 0, V, sc, INFINITY, true, true);
    bins_to_sums(S, true, true);
}

// S.marks from the histogram (H as sums, and C if top-k is set). Later questions depend on earlier
// answers, which are known so far to a bin: they get the range of bins that the bounds allow.
template <int NT>
__device__ void mark_bins(Shared<NT>& S, const Row& r, const Scale& sc)
{
    const int tid = threadIdx.x;
    Marks& K = S.marks;
    const u64 Z = S.H[kBins];
    const bool by_k = r.by_k && r.k < static_cast<int64_t>(S.C[kBins]);
    if (tid < kBins / 32) K.take[tid] = 0;
    if (tid < 4) {
        K.from[tid] = INFINITY;
        K.to[tid] = -INFINITY;
    }
    if (tid == 0) {
        K.Z = Z;
        K.by_k = by_k;
        S.n = 0;
    }
    __syncthreads();
    u64 lo = Z, hi = Z;  // bounds of the mass kept
    auto mark = [&](int w, int f, int g) {
        for (int b = f + tid; b <= g; b += NT) atomicOr(&K.take[b >> 5], 1u << (b & 31));
        if (tid == 0) {
            K.from[w] = fmaxf(below_bin(sc, g), -FLT_MAX);
            K.to[w] = above_bin(sc, f);
        }
    };
    if (by_k) {
        for (int b = tid; b < kBins; b += NT)
            if (S.C[b] < r.k && r.k <= S.C[b + 1]) S.found[0] = b;
        __syncthreads();
        const int b1 = S.found[0];
        lo = S.H[b1] < 1 ? 1 : S.H[b1];
        hi = S.H[b1 + 1];
        mark(0, b1, b1);
        if (tid == 0) {
            K.b1 = b1;
            K.c1 = S.C[b1];
        }
    }
    // of top-p and min-p, one that surely keeps no less than the other decides nothing
    bool by_p = r.by_p, by_m = r.by_m;
    int f1 = 0, g1 = 0, q0 = 0, q1 = 0;
    if (by_p) {
        find_two(S, r.p_target(lo), r.p_target(hi), f1, g1);
    }
    if (by_m) {
        // where a mass is r.least to within the rounding to whole ones
        const double y = log2(static_cast<double>(r.least)), d = 1e-6 + 1.5 / static_cast<double>(r.least_mass());
        q0 = bin_of(fmin(y + d, 0.0));
        q1 = bin_of(fmax(y - d, kDeepest));
        if (by_p && S.H[q0] >= S.H[g1 + 1]) by_m = false;
        if (by_p && S.H[q1 + 1] <= S.H[f1] && S.H[q1 + 1] >= kOne) by_p = false;
    }
    if (by_p) {
        lo = S.H[f1] < 1 ? 1 : S.H[f1];
        hi = S.H[g1 + 1] < hi ? S.H[g1 + 1] : hi;
        mark(1, f1, g1);
    }
    if (by_m) {
        if (S.H[q0] < lo) lo = S.H[q0] < 1 ? 1 : S.H[q0];
        hi = S.H[q1 + 1] < hi ? S.H[q1 + 1] : hi;
        mark(2, q0, q1);
    }
    if (tid == 0) {
        K.by_p = by_p;
        K.by_m = by_m;
        K.q0 = q0;
        K.q1 = q1;
    }
    __syncthreads();
    int f, g;
    find_two(S, r.u_target(lo), r.u_target(hi), f, g);
    mark(3, f, g);
    __syncthreads();
    if (tid < kBins / 32) {
        static_assert(kBins / 32 == 64, "one wave");
        const uint32_t c = __popc(K.take[tid]), upto = wave_sums(c);
        K.before[tid] = upto - c;
        if (tid == 63) K.bins = upto;
    }
    __syncthreads();
}

// The tokens of the marked bins go to the list (counted in S.n, which may pass kList), told by their
// logits: the draw's range alone, or top-p's or min-p's too, or all.
template <int NT, class T>
__device__ void gather_marked(Shared<NT>& S, const T* x, int V)
{
    const Marks& K = S.marks;
    const float f0 = K.from[0], f1 = K.from[1], f2 = K.from[2], f3 = K.from[3];
    const float t0 = K.to[0], t1 = K.to[1], t2 = K.to[2], t3 = K.to[3];
    const float fa = K.by_p ? f1 : f2, ta = K.by_p ? t1 : t2;
    if (K.by_k || (K.by_p && K.by_m))
        collect<NT, 32>(S, x, 0, V, [&](float l) {
            return ((l >= f0) & (l <= t0)) | ((l >= f1) & (l <= t1)) | ((l >= f2) & (l <= t2)) | ((l >= f3) & (l <= t3));
        });
    else if (K.by_p || K.by_m)
        collect<NT, 32>(S, x, 0, V, [&](float l) { return ((l >= fa) & (l <= ta)) | ((l >= f3) & (l <= t3)); });
    else
        collect<NT, 32>(S, x, 0, V, [&](float l) { return (l >= f3) & (l <= t3); });
    __syncthreads();
}

// Answer from the marked bins: from their n tokens in the list, or, where more than fit (long runs of
// equal logits), by passes over the row. H holds sums, C too if top-k cuts and n > kList. Leaves the
// token in S.drawn and returns the mass kept.
template <int NT, class T>
__device__ u64 from_marked(Shared<NT>& S, const T* x, int V, const Row& r, const Scale& sc, int n)
{
    const int tid = threadIdx.x;
    const Marks& K = S.marks;
    const bool by_k = K.by_k;
    __syncthreads();
    if (n <= kList) {
        to_keys(S, x, n);
        sort_list(S, sc, n, true);
        const u64 before_m = K.by_m ? S.H[K.q0] : 0;  // mass before min-p's bins
        const int before_b1 = sum_list(S, n, sc, true, by_k ? K.b1 : -2);
        if (tid < 64) {
            u64 kept = by_k ? S.upto[r.k - 1 - K.c1 + before_b1] : K.Z;
            if (K.by_p) {
                const u64 t = r.p_target(kept);
                kept = S.upto[first_that(n, [&](int i) { return S.upto[i] >= t; })];
            }
            if (K.by_m) {
                u64 m = kOne;  // the first token is never left out
                if (!r.only_first) {
                    const u64 w = r.least_mass();
                    const int i = first_that(n, [&](int j) { return mass_of(sc, S.list[j]) < w; });
                    m = i > 0 && bin_of(sc.y(key_value(S.list[i - 1]))) >= K.q0 ? S.upto[i - 1] : before_m;
                    m = m > kOne ? m : kOne;
                }
                kept = m < kept ? m : kept;
            }
            const u64 t = r.u_target(kept);
            const int i = first_that(n, [&](int j) { return S.upto[j] >= t; });
            if (tid == 0) {
                S.drawn = S.list[i];
                S.kept = kept;
            }
        }
        __syncthreads();
        return S.kept;
    }
    u64 kept = K.Z;
    if (by_k) kept = search_row(S, x, V, sc, K.b1, true, static_cast<u64>(r.k), false);
    if (K.by_p) {
        const u64 t = r.p_target(kept);
        __syncthreads();
        const int b = find_mass(S, t, 1);
        kept = search_row(S, x, V, sc, b, false, t, false);
    }
    if (K.by_m) {
        const u64 w = r.least_mass();
        u64 m = 0;
        each_mass<NT>(S, x, V, sc, K.q0, K.q1, [&](float, int, u64 mass) {
            if (mass >= w) m += mass;
        });
        if (tid == 0) S.mass[2] = S.H[K.q0];
        __syncthreads();
        if (m) atomicAdd(&S.mass[2], m);
        __syncthreads();
        m = r.only_first || S.mass[2] < kOne ? kOne : S.mass[2];
        kept = m < kept ? m : kept;
    }
    const u64 t = r.u_target(kept);
    __syncthreads();
    const int b = find_mass(S, t, 1);
    search_row(S, x, V, sc, b, false, t, true);
    __syncthreads();
    return kept;
}

// All of that for a row in one workgroup; the histogram of masses may be there already.
template <int NT, class T>
__device__ u64 from_row(Shared<NT>& S, const T* x, int V, const Row& r, const Scale& sc, bool have_masses)
{
    if (!have_masses) count_row(S, x, V, sc);
    __syncthreads();
    mark_bins(S, r, sc);
    gather_marked(S, x, V);
    return from_marked(S, x, V, r, sc, static_cast<int>(S.n));
}

__device__ __forceinline__ void write_row(const SampleArgs& a, int64_t row, int32_t token, float prob)
{
    if (threadIdx.x == 0) {
        a.token[row] = token;
        if (a.prob) a.prob[row] = prob;
    }
}

__device__ __forceinline__ void write_drawn(const SampleArgs& a, int64_t row, const Scale& sc, u64 drawn, u64 kept)
{
    write_row(a, row, static_cast<int32_t>(drawn & 0xFFFFFFFFu),
              static_cast<float>(weight(sc.y(key_value(drawn))) / static_cast<double>(kept)));
}

constexpr uint32_t kMostParts = 32;
struct alignas(16) RowSpace {
    uint32_t n;        // tokens in the list
    uint32_t arrived;  // workgroups done with the row
    u64 Z[kMostParts];  // the parts' masses
    float top[kMostParts], tau[kMostParts];
    u64 list[kList];
};
static_assert(sizeof(RowSpace) % 16 == 0, "layout");

// Data that workgroups of one launch hand to another. Atomics of agent scope, so that the compiler marks the
// accesses (sc1): on gfx950 such a store is written through the XCD's own L2, and such a load does not
// take what that L2 may hold of an older value.
template <class U>
__device__ __forceinline__ void put(U* p, U v)
{
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <class U>
__device__ __forceinline__ U got(const U* p)
{
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The part's list (S.n tokens, of which kList at most are there) is added to the row's; true for the
// workgroup that is the row's last. The order that this needs is gfx950's, not the language's (all atomics here
// are relaxed): a store that put() made has left the counter vmcnt only when it is where the whole
// device sees it; every wave waits for that before the barrier, behind which one thread counts the
// workgroup as arrived; and the last workgroup's got() come behind the barrier that its own count went
// through. So it finds all that the others put. What they put goes through put() and got() alone. (A release in
// the language's sense writes back the whole L2, which holds nothing of it: with 512 workgroups 10 us.)
template <int NT, class T>
__device__ bool hand_over(Shared<NT>& S, const T* x, RowSpace& R, uint32_t part, uint32_t parts, bool masses)
{
    const uint32_t mine = S.n < kList ? S.n : kList;
    if (threadIdx.x == 0) S.found[0] = static_cast<int>(atomicAdd(&R.n, S.n));
    to_keys(S, x, static_cast<int>(mine));
    const uint32_t at = static_cast<uint32_t>(S.found[0]);
    for (uint32_t i = threadIdx.x; i < mine; i += NT)
        if (at + i < kList) put(&R.list[at + i], S.list[i]);
    if (masses && threadIdx.x == 0) {
        u64 m = 0;
#pragma unroll
        for (int w = 0; w < NT / 64; w++) m += S.wsum[w];
        put(&R.Z[part], m);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (threadIdx.x == 0) S.found[1] = __hip_atomic_fetch_add(&R.arrived, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1 == parts;
    __syncthreads();
    return S.found[1];
}

// The parts' bins, summed; 16 loads on the way at a time.
template <int NT, class U>
__device__ __forceinline__ void join_parts(U* to, const U* from, uint32_t parts)
{
    constexpr int B = kBins / NT, E = 16 / B;
    U m[B] = {};
    for (uint32_t s = 0; s < parts; s += E) {
        U v[E][B];
#pragma unroll
        for (uint32_t e = 0; e < E; e++)
#pragma unroll
            for (int b = 0; b < B; b++) v[e][b] = s + e < parts ? got(&from[(s + e) * kBins + b * NT + threadIdx.x]) : 0;
#pragma unroll
        for (uint32_t e = 0; e < E; e++)
#pragma unroll
            for (int b = 0; b < B; b++) m[b] += v[e][b];
    }
#pragma unroll
    for (int b = 0; b < B; b++) to[b * NT + threadIdx.x] = m[b];
}

__device__ __forceinline__ int part_begin(int V, uint32_t part, uint32_t parts)
{
    return static_cast<int>(static_cast<int64_t>(V) * part / parts);
}

// One workgroup per row. 256 rows of 131072 (134 MB) take 77 us: 18 the first pass (7.4 TB/s), 6 the beginning's
// lower end, 14 the second pass or, with masses, 28 (bound by the 64-bit operations and LDS atomics),
// 5 the list, and 17 to 20 in rows whose answers lie past it.
template <class T, int NT>
__global__ void __launch_bounds__(NT) sample_rows(SampleArgs a)
{
    __shared__ Shared<NT> S;
    const int64_t row = blockIdx.x;
    const T* const x = static_cast<const T*>(a.x) + row * a.ld;
    const Row r(a, row, short_most(1, NT));
    float mine = -INFINITY;
    each_if<NT, 32>(
        x, 0, a.V,
        [&](float l) {
            mine = fmaxf(mine, l);
            return false;
        },
        [](float, int) {});
    const float top = block_max(S, mine);
    if (top == -INFINITY) return write_row(a, row, -1, 0.0f);  // nothing to draw
    const Scale sc = r.scale(top);
    const bool listed = !r.by_k || r.short_k;
    // room for the tokens that share the last one's bin
    const float tau = listed ? reached_by(S, mine, sc, r.by_k ? (r.k > 32 ? static_cast<uint32_t>(r.k) : 32u) : kAim) : INFINITY;
    const bool masses = needs_masses(r, sc, tau), counts = masses && !listed;
    clear_bins(S, masses, counts);
    if (masses) fill_middles(S);
    if (threadIdx.x == 0) S.n = 0;
    __syncthreads();
    if (listed || masses) gather(S, x, 0, a.V, sc, tau, masses, counts);
    __syncthreads();
    const int n = static_cast<int>(S.n);
    if (masses) bins_to_sums(S, true, counts);
    u64 kept = 0;
    if (listed && n <= kList) {
        to_keys(S, x, n);
        kept = from_list(S, r, sc, n, tau, masses ? S.H[kBins] : 0);
    }
    if (!kept) kept = from_row(S, x, a.V, r, sc, masses);
    write_drawn(a, row, sc, S.drawn, kept);
}

// Few rows: `parts` workgroups per row, in two launches. The first finds each part's largest logit and
// a logit that enough of its threads reach. The second gathers the beginning of the order and, where
// it is needed, the histogram; the workgroup that is last to do so for a row answers, from the list or
// with passes over the whole row. (A third launch that shared those passes out over the CUs took
// longer than it saved, 14% at 64 rows of 50257 and at 256 of 131072.)
// What bounds it is latency: 64 rows of 50257 take 34 to 39 us by their settings, of which the loads of
// the two launches are 4; a row answered from the beginning of the order is through 15 us after the
// second launch starts, one that needs the marked bins 12 to 14 us later (joining the histograms 2.6,
// marking 2.5, the pass over the row 5, sorting 2.5, sums and search 2.5).
template <class T, int NT>
__global__ void __launch_bounds__(NT) sample_tops(SampleArgs a, RowSpace* space, uint32_t parts)
{
    __shared__ Shared<NT> S;
    const int64_t row = blockIdx.x / parts;
    const uint32_t part = blockIdx.x % parts;
    const T* const x = static_cast<const T*>(a.x) + row * a.ld;
    const Row r(a, row, short_most(parts, NT));
    float mine = -INFINITY;
    each_if<NT, 32>(
        x, part_begin(a.V, part, parts), part_begin(a.V, part + 1, parts),
        [&](float l) {
            mine = fmaxf(mine, l);
            return false;
        },
        [](float, int) {});
    const float top = block_max(S, mine);
    float tau = -INFINITY;
    const uint32_t aim = r.short_k ? static_cast<uint32_t>(r.k) + 32 : kAim;
    if (top > -INFINITY) tau = reached_by(S, mine, r.scale(top), (aim + parts - 1) / parts);
    if (threadIdx.x == 0) {
        space[row].top[part] = top;
        space[row].tau[part] = tau == -INFINITY ? INFINITY : tau;  // a part with few tokens has no say
        if (part == 0) {
            RowSpace& R = space[row];
            R.n = R.arrived = 0;
        }
    }
}

template <class T, int NT>
__global__ void __launch_bounds__(NT) sample_parts(SampleArgs a, RowSpace* space, u64* hist, uint32_t parts)
{
    __shared__ Shared<NT> S;
    const int tid = threadIdx.x, lane = tid & 63;
    const int64_t row = blockIdx.x / parts;
    const uint32_t part = blockIdx.x % parts;
    const T* const x = static_cast<const T*>(a.x) + row * a.ld;
    RowSpace& R = space[row];
    float top = lane < static_cast<int>(parts) ? R.top[lane] : -INFINITY;
    float tau = lane < static_cast<int>(parts) ? R.tau[lane] : INFINITY;
    const Row r(a, row, short_most(parts, NT));
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        top = fmaxf(top, __shfl_xor(top, d));
        tau = fminf(tau, __shfl_xor(tau, d));
    }
    if (top == -INFINITY) {  // nothing to draw
        if (part == 0) write_row(a, row, -1, 0.0f);
        return;
    }
    const Scale sc = r.scale(top);
    // no part had enough tokens: all of them (tau is +inf also where the largest logits are)
    if (tau == INFINITY && top < INFINITY) tau = -INFINITY;
    const bool listed = !r.by_k || r.short_k;
    const bool masses = needs_masses(r, sc, tau), counts = masses && !listed;
    clear_bins(S, masses, counts);
    if (masses) fill_middles(S);
    if (tid == 0) S.n = 0;
    __syncthreads();
    if (listed || masses)
        gather(S, x, part_begin(a.V, part, parts), part_begin(a.V, part + 1, parts), sc, listed ? tau : INFINITY, masses, counts);
    __syncthreads();
    // this part's tokens, mass and histogram go to the row's space
    u64* const H = hist + row * parts * kBins;
    uint32_t* const C = reinterpret_cast<uint32_t*>(hist + a.M * parts * kBins) + row * parts * kBins;
    if (masses) {
        u64 m = 0;
        for (int b = tid; b < kBins; b += NT) {
            put(&H[part * kBins + b], S.H[b]);
            if (counts) put(&C[part * kBins + b], S.C[b]);
            m += S.H[b];
        }
        m = wave_sums(m);
        if (lane == 63) S.wsum[tid >> 6] = m;
    }
    if (!hand_over(S, x, R, part, parts, masses)) return;
    const uint32_t n = got(&R.n);
    u64 Z = 0;
    if (masses) {
        Z = wave_sums(lane < static_cast<int>(parts) ? got(&R.Z[lane]) : u64{0});
        Z = __shfl(Z, 63);
    }
    u64 kept = 0;
    if (listed && n <= kList) {
        for (uint32_t i = tid; i < n; i += NT) S.list[i] = got(&R.list[i]);
        __syncthreads();
        kept = from_list(S, r, sc, static_cast<int>(n), tau, Z);
    }
    if (!kept) {
        if (masses) {
            __syncthreads();
            join_parts<NT>(S.H, H, parts);
            if (counts) join_parts<NT>(S.C, C, parts);
            bins_to_sums(S, true, counts);
        }
        kept = from_row(S, x, a.V, r, sc, masses);
    }
    write_drawn(a, row, sc, S.drawn, kept);
}

// How a call is launched: workgroups per row and their threads. With few rows 512 threads pass their
// barriers sooner (1 row of 131072: 15.3 us, 17.8 with 1024 threads, 18.7 in one workgroup of those); with more
// rows 1024 threads and one workgroup for each of 256 CUs do well (64 rows of 131072: 43.5 us, 48.4 with 512
// threads, 49.5 with two workgroups a row, 52.6 with eight; 64 rows of 50257: 33.5, 32.8, 35.5 and 49.6 us). In
// between the rule is not the best: 8 rows of 131072 take 42.7 us, with 8 workgroups of 1024 threads each they
// would take 36.5. No part has less than 2048 logits. The whole device is meant: on a stream of fewer CUs the
// choice is the same.
struct Launch {
    uint32_t parts, threads;
};

Launch plan_launch(int64_t M, int64_t V)
{
    const bool few = M <= 8;
    int64_t p = (few ? 512 : 256) / (M > 0 ? M : 1);
    p = p < V / 2048 ? p : V / 2048;
    return {static_cast<uint32_t>(p < 1 ? 1 : p > kMostParts ? kMostParts : p), few ? 512u : 1024u};
}

template <class T, int NT>
void launch_rows(const SampleArgs& a, RowSpace* space, u64* hist, const Launch& l, hipStream_t s)
{
    const uint32_t M = static_cast<uint32_t>(a.M);
    if (l.parts == 1) {
        hipLaunchKernelGGL((sample_rows<T, NT>), dim3(M), dim3(NT), 0, s, a);
    } else {
        hipLaunchKernelGGL((sample_tops<T, NT>), dim3(M * l.parts), dim3(NT), 0, s, a, space, l.parts);
        hipLaunchKernelGGL((sample_parts<T, NT>), dim3(M * l.parts), dim3(NT), 0, s, a, space, hist, l.parts);
    }
}

constexpr int64_t kRowsMost = kThreadsMost / 1024;  // a workgroup per row

uw_status check_sample(const uw_sample_args* p)
{
    if (!p) return fail(UW_EINVAL, "NULL argument");
    if (p->M < 0 || p->V < 1) return fail(UW_ESHAPE, "bad shape %lld x %lld", (long long)p->M, (long long)p->V);
    if (p->type != UW_F32 && p->type != UW_BF16) return fail(UW_EINVAL, "bad type %d", p->type);
    if (p->V > UW_SAMPLE_MAX_V) return fail(UW_EUNSUPPORTED, "V > %d", UW_SAMPLE_MAX_V);
    if (p->M > kRowsMost) return fail(UW_EUNSUPPORTED, "M >= 2^22");
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
    if (M < 1 || V < 1 || V > UW_SAMPLE_MAX_V || M > kRowsMost) return 0;
    const Launch l = plan_launch(M, V);
    return l.parts == 1 ? 0 : static_cast<size_t>(M) * (sizeof(RowSpace) + l.parts * kBins * (sizeof(u64) + sizeof(uint32_t)));
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
    hipStream_t s = static_cast<hipStream_t>(stream);
    const Launch l = plan_launch(a.M, a.V);
    RowSpace* space = l.parts > 1 ? static_cast<RowSpace*>(args->d_ws) : nullptr;
    u64* hist = reinterpret_cast<u64*>(space + a.M);
    if (args->type == UW_F32)
        l.threads == 512 ? launch_rows<float, 512>(a, space, hist, l, s) : launch_rows<float, 1024>(a, space, hist, l, s);
    else
        l.threads == 512 ? launch_rows<uint16_t, 512>(a, space, hist, l, s) : launch_rows<uint16_t, 1024>(a, space, hist, l, s);
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? UW_OK : fail(UW_EHIP, "sample launch failed: %s", hipGetErrorString(e));
}
