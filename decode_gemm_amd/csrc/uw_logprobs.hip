// Log probabilities of given tokens, their ranks, rows' entropies and the first tokens of the order, from
// logits.
//
// Mathematics. With y_i = (l_i - max) log2(e) / T, S = sum 2^y_i and H = sum y_i 2^y_i: log p_t = (l_t - max) / T - log S
// and the entropy is log S - log(2) H / S. One pass over the row keeps a running maximum with the sums below it: a
// maximum that grows by d (in units of y) turns S into 2^-d S and H into 2^-d (H - d S). Sums of 128 of a thread's values are fp32, sums
// of these and over threads fp64. The rank counts l_i > l_t, and l_i >= l_t before t, in the same pass.
// The first n tokens are not sorted out of the row: of the maxima of 256 shares of the row, the n-th largest is
// reached by at least n tokens and hardly more, and these, found by looking again into the shares of the threads
// whose maximum reaches it, are sorted in LDS. Where ties make them too many, a search over the digits of
// (logit, index) finds the n-th token itself.
// Bound by the row's bytes for many rows (1024 x 131072 fp32 with one first token 102 us, 5.3 TB/s, part of it from the cache behind
// the L2; bf16 55 us), a row alone by its two launches and their chains of barriers (131072 tokens, 20 first ones: 14 us).
#include <hip/hip_runtime.h>

#include <cfloat>
#include <cmath>

#include "uw_internal.h"
#include "uw_order.h"
#include "uw_recon.h"

namespace uw {

namespace {

constexpr int kParts = 256;   // shares of a slice whose maxima are compared
constexpr int kList = 2048;   // tokens that are sorted in LDS
constexpr int kCounted = 512;  // as many are ordered by counting
constexpr int kMostSlices = 8;
constexpr int kRun = 8;  // steps of a thread whose sums are fp32: equal logits round the same way in every step
constexpr double kLn2 = 0x1.62e42fefa39efp-1;
constexpr u64 kNoKey = ~u64{0};

// What is known of a row or of one workgroup's slice of it.
struct Part {
    double S, H;     // relative to `top`
    float top;
    float given;     // logit of the given token, -inf where it has no place in the order
    int32_t before;  // tokens before it
    int32_t unused;
};

struct LogprobArgs {
    const void* x;
    int64_t ld, M;
    int32_t V, n_top;
    const int32_t* token;
    const float* temperature;
    float* logprob;
    int32_t* rank;
    float* entropy;
    int32_t* top_token;
    float* top_logprob;
    Part* part;  // [M][slices], then keys
    u64* keys;   // [M][slices][n_top]
    uint32_t slices;
};

template <class T>
struct Row;
template <>
struct Row<float> {
    static constexpr int VEC = 4;
};
template <>
struct Row<uint16_t> {
    static constexpr int VEC = 8;
};

__device__ __forceinline__ void unpack(const u32x4& w, float (&v)[4])
{
#pragma unroll
    for (int i = 0; i < 4; i++) v[i] = __uint_as_float(w[i]);
}
__device__ __forceinline__ void unpack(const u32x4& w, float (&v)[8])
{
#pragma unroll
    for (int i = 0; i < 4; i++) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

// The 16-byte words of memory that hold a row: word i holds tokens i * VEC - skip and on. What is not of the row
// reads as -inf and is not touched.
template <class T>
struct Words {
    static constexpr int VEC = Row<T>::VEC;
    const T* x;
    int V, skip, n;
    __device__ __forceinline__ Words(const T* row, int V_) : x(row), V(V_)
    {
        skip = static_cast<int>((reinterpret_cast<uintptr_t>(row) / sizeof(T)) % VEC);
        n = (V + skip + VEC - 1) / VEC;
    }
    __device__ __forceinline__ int first(int i) const { return i * VEC - skip; }
    // As it lies in memory: with the conversion apart, the branch has nothing in it that waits.
    __device__ __forceinline__ u32x4 raw(int i) const
    {
        const int e = first(i);
        if (e >= 0 && e + VEC <= V) return *reinterpret_cast<const u32x4*>(x + e);
        u32x4 w = nothing();
#pragma unroll
        for (int k = 0; k < VEC; k++)
            if (e + k >= 0 && e + k < V) put(w, k, x[e + k]);
        return w;
    }
    static __device__ __forceinline__ u32x4 nothing()
    {
        constexpr uint32_t kNone = VEC == 4 ? 0xFF800000u : 0xFF80FF80u;
        return u32x4{kNone, kNone, kNone, kNone};
    }
    static __device__ __forceinline__ void put(u32x4& w, int k, float v) { w[k] = __float_as_uint(v); }
    static __device__ __forceinline__ void put(u32x4& w, int k, uint16_t v)
    {
        w[k / 2] = k & 1 ? (w[k / 2] & 0xFFFFu) | static_cast<uint32_t>(v) << 16 : (w[k / 2] & 0xFFFF0000u) | v;
    }
    __device__ __forceinline__ void load(int i, float (&v)[VEC]) const { unpack(raw(i), v); }
};

// log2(e) / T as two factors: y = (unit (l - top)) slope. The unit is 1/2, so that differences cannot overflow; at temperatures below
// 2^-100, where the slope would, it is 2^23 beside a maximum below 1 (what is then past fp32's range has no mass), and beside a larger one
// still 1/2, whose product with any difference that is not 0 is past the mass too.
// The slope is 0 where all tokens weigh the same or (T <= 0, NaN) the sums are not used.
__device__ __forceinline__ bool tiny(float T) { return T < 0x1p-100f && T > 0.f; }
__device__ __forceinline__ float unit(float top, bool tiny) { return tiny && fabsf(top) < 1.f ? 0x1p23f : 0.5f; }
__device__ __forceinline__ float slope(float T)
{
    if (!(T > 0.f) || T > FLT_MAX) return 0.f;
    return static_cast<float>(1.4426950408889634 / static_cast<double>(T) * (tiny(T) ? 0x1p-23 : 2.0));
}

// Sums below a maximum `from` as sums below `top`, in units of its exponential; h is top's unit. An infinite maximum leaves what is
// finite no mass.
template <class V>
__device__ __forceinline__ void rebase(V& S, V& H, float from, float top, float c, float h)
{
    if (from == top) return;
    const float y = fmaxf(__builtin_fmaf(from, h, -h * top) * c, -200.f);  // NaN too
    const float f = top == INFINITY ? 0.f : __builtin_amdgcn_exp2f(y);
    H = f * (H + y * S);
    S *= f;
}

// Maximum and sum over the lanes of a wave, the same bits in all of them: rotations within 16 lanes, then across.
template <int CTRL>
__device__ __forceinline__ float rotated(float v)
{
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, false));
}
template <int CTRL>
__device__ __forceinline__ double rotated(double v)
{
    const long long b = __double_as_longlong(v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(b), CTRL, 0xF, 0xF, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(b >> 32), CTRL, 0xF, 0xF, false);
    return __longlong_as_double(static_cast<long long>(static_cast<u64>(hi) << 32 | lo));
}
template <int CTRL>
__device__ __forceinline__ int rotated(int v)
{
    return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, false);
}
template <class V>
__device__ __forceinline__ V wave_sum(V v)
{
    v += rotated<0x128>(v);
    v += rotated<0x124>(v);
    v += rotated<0x122>(v);
    v += rotated<0x121>(v);
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}
__device__ __forceinline__ float wave_max(float v)
{
    v = fmaxf(v, rotated<0x128>(v));
    v = fmaxf(v, rotated<0x124>(v));
    v = fmaxf(v, rotated<0x122>(v));
    v = fmaxf(v, rotated<0x121>(v));
    v = fmaxf(v, __shfl_xor(v, 16));
    return fmaxf(v, __shfl_xor(v, 32));
}

// The greatest number below v (v not NaN or -inf).
__device__ __forceinline__ float below(float v)
{
    const uint32_t b = __float_as_uint(v);
    return v == 0.f ? -0x1p-149f : __uint_as_float(v > 0.f ? b - 1 : b + 1);
}

// Answers of a row from what is known of all of it.
__device__ __forceinline__ double log_share(float l, const Part& p, double logS, float T)
{
    if (p.top == INFINITY) return l == p.top ? -logS : -INFINITY;
    return (l == p.top ? 0.0 : (static_cast<double>(l) - static_cast<double>(p.top)) / static_cast<double>(T)) - logS;
}
__device__ __forceinline__ bool greedy(float T) { return !(T > 0.f); }

__device__ __forceinline__ void answer_row(const LogprobArgs& a, int64_t m, const Part& p, double logS, float T)
{
    const bool placed = p.given > -INFINITY;
    if (a.rank) a.rank[m] = placed ? p.before : -1;
    if (a.logprob) {
        const double v = !placed ? -INFINITY : greedy(T) ? (p.before == 0 ? 0.0 : -INFINITY) : log_share(p.given, p, logS, T);
        a.logprob[m] = static_cast<float>(v);
    }
    if (a.entropy) {
        const double e = p.top == -INFINITY || greedy(T) ? 0.0 : logS - kLn2 * (p.H / p.S);
        a.entropy[m] = static_cast<float>(e > 0.0 ? e : 0.0);
    }
}
__device__ __forceinline__ void answer_top(const LogprobArgs& a, int64_t m, uint32_t place, u64 key, const Part& p, double logS, float T)
{
    const int64_t o = m * a.n_top + place;
    if (a.top_token) a.top_token[o] = key == kNoKey ? -1 : static_cast<int32_t>(key & 0xFFFFFFFFu);
    if (a.top_logprob) {
        const double v = key == kNoKey ? -INFINITY : greedy(T) ? (place == 0 ? 0.0 : -INFINITY) : log_share(key_value(key), p, logS, T);
        a.top_logprob[o] = static_cast<float>(v);
    }
}

__device__ __forceinline__ uint32_t wave_min(uint32_t v)
{
    auto less = [](uint32_t a, uint32_t b) { return a < b ? a : b; };
    v = less(v, static_cast<uint32_t>(rotated<0x128>(static_cast<int>(v))));
    v = less(v, static_cast<uint32_t>(rotated<0x124>(static_cast<int>(v))));
    v = less(v, static_cast<uint32_t>(rotated<0x122>(static_cast<int>(v))));
    v = less(v, static_cast<uint32_t>(rotated<0x121>(static_cast<int>(v))));
    v = less(v, __shfl_xor(v, 16));
    v = less(v, __shfl_xor(v, 32));
    return __builtin_amdgcn_readfirstlane(v);
}

template <int NT>
struct Shared {
    u64 list[kList];
    uint32_t share[kParts];
    uint32_t hist[256];
    uint16_t flagged[NT];
    float top[NT / 64];
    double S[NT / 64], H[NT / 64];
    int before[NT / 64];
    uint32_t n_flagged, n_list;
    u64 prefix;
    uint32_t taken, shift, done;
};

template <int NT>
__device__ __forceinline__ void put(Shared<NT>& sh, float l, int i)
{
    const uint32_t at = atomicAdd(&sh.n_list, 1u);
    if (at < kList) sh.list[at] = key_of(l, i);
}

// Ties made the tokens from tau on too many for the list: the n-th key digit by digit, 8 bits at a time, until
// what is left up to it fits.
template <class T, int NT>
__device__ __noinline__ void search_keys(Shared<NT>& sh, const Words<T>& w, int first, int end, int n)
{
    constexpr int VEC = Words<T>::VEC;
    const int tid = threadIdx.x;
    if (tid == 0) {
        sh.prefix = 0;
        sh.taken = 0;
        sh.shift = 64;
        sh.done = 0;
    }
    __syncthreads();
    while (!sh.done) {
        const uint32_t shift = sh.shift;
        const u64 prefix = sh.prefix;
        if (tid < 256) sh.hist[tid] = 0;
        __syncthreads();
        for (int i = first + tid; i < end; i += NT) {
            float v[VEC];
            w.load(i, v);
#pragma unroll
            for (int k = 0; k < VEC; k++)
                if (v[k] > -INFINITY) {
                    const u64 key = key_of(v[k], w.first(i) + k);
                    if (shift == 64 || key >> shift == prefix) atomicAdd(&sh.hist[(key >> (shift - 8)) & 255], 1u);
                }
        }
        __syncthreads();
        if (tid == 0) {
            uint32_t c = sh.taken;
            int d = 0;
            while (d < 255 && c + sh.hist[d] < static_cast<uint32_t>(n)) c += sh.hist[d++];
            sh.taken = c;
            sh.prefix = (shift == 64 ? 0 : prefix << 8) | static_cast<u64>(d);
            sh.shift = shift - 8;
            sh.done = c + sh.hist[d] <= kList || shift == 8;
            sh.n_list = 0;
        }
        __syncthreads();
    }
    const uint32_t shift = sh.shift;
    const u64 prefix = sh.prefix;
    for (int i = first + tid; i < end; i += NT) {
        float v[VEC];
        w.load(i, v);
#pragma unroll
        for (int k = 0; k < VEC; k++)
            if (v[k] > -INFINITY && key_of(v[k], w.first(i) + k) >> shift <= prefix) put(sh, v[k], w.first(i) + k);
    }
    __syncthreads();
}

// A number that at least n of the shares' maxima reach, but not many more; -inf where fewer than n have one. By halving, in
// the order of numbers, between the least and the largest of them, each wave for itself: the counts are those of its lanes'
// comparisons. A quarter more, or eight, are near enough: a few more candidates cost less than another turn.
__device__ __forceinline__ float threshold(const uint32_t* share, float top, uint32_t n)
{
    constexpr uint32_t kNone = 0x007FFFFFu;  // -inf in that order
    const int lane = threadIdx.x & 63;
    uint32_t v[kParts / 64], least;
#pragma unroll
    for (int i = 0; i < kParts / 64; i++) {
        v[i] = share[lane + 64 * i];
        least = i == 0 || v[i] < least ? v[i] : least;
    }
    least = wave_min(least);
    const uint32_t most = n + (n / 4 > 8 ? n / 4 : 8);
    uint32_t lo = least > kNone ? least : kNone, hi = __builtin_amdgcn_readfirstlane(top > -INFINITY ? ~order_bits(top) : kNone);
    while (lo < hi) {
        const uint32_t mid = lo + (hi - lo + 1) / 2;
        uint32_t c = 0;
#pragma unroll
        for (int i = 0; i < kParts / 64; i++) c += __popcll(__ballot(v[i] >= mid));
        if (c < n) {
            hi = mid - 1;
        } else {
            lo = mid;
            if (c <= most) break;
        }
    }
    return lo == kNone ? -INFINITY : order_value(~lo);
}

// Place of a wave's key among the keys that its first `count` lanes hold.
__device__ __forceinline__ int place_in_wave(u64 key, int count)
{
    const uint32_t lo = static_cast<uint32_t>(key), hi = static_cast<uint32_t>(key >> 32);
    int place = 0;
    for (int o = 0; o < count; o++) {
        const u64 other = static_cast<u64>(static_cast<uint32_t>(__builtin_amdgcn_readlane(hi, o))) << 32 |
                          static_cast<uint32_t>(__builtin_amdgcn_readlane(lo, o));
        place += other < key;
    }
    return place;
}

// One slice of a row (all of it with slices = 1) per workgroup; thread t has the words first + t + NT i.
template <class T, int NT, int EL>
__global__ void __launch_bounds__(NT) logprobs_rows(LogprobArgs a)
{
    constexpr int VEC = Words<T>::VEC, U = EL / VEC;  // EL values per thread and step
    constexpr int PER = NT / kParts;                  // threads per share
    static_assert(PER == 1 || PER == 2 || PER == 4, "threads per share");
    __shared__ Shared<NT> sh;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const uint32_t z = blockIdx.x % a.slices;
    const int64_t m = blockIdx.x / a.slices;
    const T* x = static_cast<const T*>(a.x) + m * a.ld;
    const Words<T> w(x, a.V);
    const int per = (w.n + static_cast<int>(a.slices) - 1) / static_cast<int>(a.slices);
    const int first = per * static_cast<int>(z), end = first + per < w.n ? first + per : w.n;
    u32x4 next[U];  // the next step's words, on the way
#pragma unroll
    for (int u = 0; u < U; u++) next[u] = first + tid + u * NT < end ? w.raw(first + tid + u * NT) : Words<T>::nothing();
    const float temp = a.temperature ? a.temperature[m] : 1.f, c2 = slope(temp);
    const bool small = tiny(temp);
    const int t = a.token ? a.token[m] : -1;
    const float lt = t >= 0 && t < a.V ? value(x, t) : -INFINITY;
    const bool placed = lt > -INFINITY;
    const float lt_before = placed ? below(lt) : INFINITY, lt_after = placed ? lt : INFINITY;

    float top = -INFINITY, S = 0.f, H = 0.f, v[U][VEC];
    double dS = 0.0, dH = 0.0;  // of kRun steps and kRun more ...
    int before = 0, steps = 0;
    const bool counts = a.rank || greedy(temp);
    for (int i = first + tid; i < end; i += NT * U) {
#pragma unroll
        for (int u = 0; u < U; u++) unpack(next[u], v[u]);
        if (i + NT * U < end)
#pragma unroll
            for (int u = 0; u < U; u++) next[u] = i + (U + u) * NT < end ? w.raw(i + (U + u) * NT) : Words<T>::nothing();
        float now = top;
#pragma unroll
        for (int u = 0; u < U; u++)
#pragma unroll
            for (int k = 0; k < VEC; k++) now = fmaxf(now, v[u][k]);
        if (steps == kRun) {
            steps = 0;
            dS += S;
            dH += H;
            S = H = 0.f;
        }
        steps++;
        if (now > top) {
            rebase(S, H, top, now, c2, unit(now, small));
            if (i >= first + kRun * NT * U) rebase(dS, dH, top, now, c2, unit(now, small));
        }
        top = now;
        if (top == INFINITY) {
#pragma unroll
            for (int u = 0; u < U; u++)
#pragma unroll
                for (int k = 0; k < VEC; k++) S += v[u][k] == top ? 1.f : 0.f;
        } else {
            const float h2 = unit(top, small), scaled = h2 * top;
            float s = 0.f, h = 0.f;
#pragma unroll
            for (int u = 0; u < U; u++)
#pragma unroll
                for (int k = 0; k < VEC; k++) {
                    const float y = fmaxf(__builtin_fmaf(v[u][k], h2, -scaled) * c2, -200.f);  // a mask's NaN too
                    const float e = __builtin_amdgcn_exp2f(y);
                    s += e;
                    h = __builtin_fmaf(y, e, h);
                }
            S += s;
            H += h;
        }
        if (counts)
#pragma unroll
            for (int u = 0; u < U; u++) {
                const float than = w.first(i + u * NT) < t ? lt_before : lt_after;
#pragma unroll
                for (int k = 0; k < VEC; k++) before += v[u][k] > than;
            }
    }
    {   // In the word that t lies in, but does not begin, tokens that equal it were counted from t on too.
        const int word = (t + w.skip) / VEC, e = w.first(word) + tid;
        if (counts && placed && first <= word && word < end && w.first(word) < t && tid < VEC && e >= t && e < a.V) before -= value(x, e) == lt;
    }
    // The row's maximum ...
    const int n = a.n_top;
    {
        const float m_wave = wave_max(top);
        if (lane == 0) sh.top[wave] = m_wave;
        float share = top;
        if (PER > 1) share = fmaxf(share, __shfl_xor(share, 1));
        if (PER > 2) share = fmaxf(share, __shfl_xor(share, 2));
        if (tid % PER == 0) sh.share[tid / PER] = share > -INFINITY ? ~order_bits(share) : 0u;
        if (tid == 0) {
            sh.n_flagged = 0;
            sh.n_list = 0;
        }
    }
    __syncthreads();
    Part p{};
    p.top = sh.top[0];
#pragma unroll
    for (int i = 1; i < NT / 64; i++) p.top = fmaxf(p.top, sh.top[i]);
    p.given = lt;
    // ... and the sums below that maximum.
    dS += S;
    dH += H;
    rebase(dS, dH, top, p.top, c2, unit(p.top, small));
    dS = wave_sum(dS);
    dH = wave_sum(dH);
    before = wave_sum(before);
    if (lane == 0) {
        sh.S[wave] = dS;
        sh.H[wave] = dH;
        sh.before[wave] = before;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NT / 64; i++) {
        p.S += sh.S[i];
        p.H += sh.H[i];
        p.before += sh.before[i];
    }
    const double logS = a.slices > 1 ? 0.0 : log(p.S);
    if (tid == 0) {
        if (a.slices > 1)
            a.part[m * a.slices + z] = p;
        else
            answer_row(a, m, p, logS, temp);
    }
    if (n == 0) return;
    // Tokens from tau on: a number that at least n shares reach and few more, or -inf.
    const float tau = n == 1 ? p.top : threshold(sh.share, p.top, static_cast<uint32_t>(n));
    const bool mine = top > -INFINITY && top >= tau;
    if (end - first <= NT * U) {  // they are in registers still
        if (mine) {
#pragma unroll
            for (int u = 0; u < U; u++)
#pragma unroll
                for (int k = 0; k < VEC; k++)
                    if (v[u][k] > -INFINITY && v[u][k] >= tau) put(sh, v[u][k], w.first(first + tid + u * NT) + k);
        }
    } else {  // a wave looks through a thread's words
        if (mine) sh.flagged[atomicAdd(&sh.n_flagged, 1u)] = static_cast<uint16_t>(tid);
        __syncthreads();
        const int nf = static_cast<int>(sh.n_flagged);
        for (int f = wave; f < nf; f += NT / 64)
            for (int i = first + sh.flagged[f] + NT * lane; i < end; i += NT * 64) {
                float c[VEC];
                w.load(i, c);
#pragma unroll
                for (int k = 0; k < VEC; k++)
                    if (c[k] > -INFINITY && c[k] >= tau) put(sh, c[k], w.first(i) + k);
            }
    }
    __syncthreads();
    if (sh.n_list > kList) search_keys<T, NT>(sh, w, first, end, n);
    // Keys are all different, so a key's place is the number of smaller ones; many are sorted instead.
    const int C = static_cast<int>(sh.n_list);
    u64* keys = a.slices > 1 ? a.keys + (m * a.slices + z) * n : nullptr;
    auto answer = [&](int place, u64 key) {
        if (keys)
            keys[place] = key;
        else
            answer_top(a, m, static_cast<uint32_t>(place), key, p, logS, temp);
    };
    if (C <= 64) {  // a wave has them all; the others fill the places past the last key
        if (wave == 0) {
            const u64 key = lane < C ? sh.list[lane] : kNoKey;
            const int place = lane < C ? place_in_wave(key, C) : n;
            if (place < n) answer(place, key);
        } else {
            for (int c = C + tid - 64; c < n; c += NT - 64) answer(c, kNoKey);
        }
        return;
    }
    if (C > kCounted) {
        int size = 2 * kCounted;
        while (size < C) size *= 2;
        for (int c = C + tid; c < size; c += NT) sh.list[c] = kNoKey;
        __syncthreads();
        for (int run = 2; run <= size; run *= 2)
            for (int d = run / 2; d > 0; d /= 2) {
                for (int q = tid; q < size / 2; q += NT) {
                    const int i = 2 * q - (q & (d - 1)), j = i + d;
                    const u64 x0 = sh.list[i], x1 = sh.list[j];
                    if ((x0 > x1) == ((i & run) == 0)) {
                        sh.list[i] = x1;
                        sh.list[j] = x0;
                    }
                }
                __syncthreads();
            }
    }
    for (int c = tid; c < n || (c < C && C <= kCounted); c += NT) {
        u64 key = kNoKey;
        int place = c;
        if (c < C) {
            key = sh.list[c];
            if (C <= kCounted) {
                place = 0;
#pragma unroll 4
                for (int o = 0; o < C; o++) place += sh.list[o] < key;
            }
        }
        if (place < n) answer(place, key);
    }
}

// A row's answers from its slices: sums in slice order, and each key's place among all slices' sorted
// keys, the sum of its places in each list.
constexpr int kJoinThreads = 512;
template <class T>
__global__ void __launch_bounds__(kJoinThreads) logprobs_join(LogprobArgs a)
{
    __shared__ u64 keys[kMostSlices * UW_LOGPROBS_MAX_TOP];
    __shared__ int place[kMostSlices * UW_LOGPROBS_MAX_TOP], count;
    __shared__ uint16_t list[kMostSlices * UW_LOGPROBS_MAX_TOP];
    static_assert(kMostSlices <= 64, "one lane per slice");
    const int64_t m = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 63, n = a.n_top, slices = static_cast<int>(a.slices);
    for (int i = tid; i < n * slices; i += kJoinThreads) {
        keys[i] = a.keys[m * slices * n + i];
        place[i] = 0;
    }
    if (tid == 0) count = 0;
    const float temp = a.temperature ? a.temperature[m] : 1.f, c2 = slope(temp);
    Part p{};
    p.top = p.given = -INFINITY;
    if (lane < slices) p = a.part[m * slices + lane];
    const float top = wave_max(p.top);
    if (p.top != top) {
        const double h = unit(top, tiny(temp)), y = fmax((h * p.top - h * top) * c2, -1100.0);  // NaN too
        const double f = top == INFINITY ? 0.0 : exp2(y);
        p.H = f * (p.H + y * p.S);
        p.S *= f;
    }
    p.S = wave_sum(p.S);
    p.H = wave_sum(p.H);
    p.before = wave_sum(p.before);
    p.given = __shfl(p.given, 0);
    p.top = top;
    const double logS = log(p.S);
    if (tid == 0) answer_row(a, m, p, logS, temp);
    if (n == 0) return;
    __syncthreads();
    // Of the lists' q-th keys the r-th smallest has q r >= n keys up to it, and not many more with q near 2 n / slices:
    // only these are looked at.
    const int q = 2 * n < slices ? 1 : (2 * n + slices - 1) / slices < n ? (2 * n + slices - 1) / slices : n, r = (n + q - 1) / q;
    const u64 mine = lane < slices ? keys[lane * n + q - 1] : kNoKey;
    int below_mine = 0;
    for (int z = 0; z < slices; z++) {
        const u64 other = keys[z * n + q - 1];
        below_mine += other < mine || (other == mine && z < lane);
    }
    const u64 at = __ballot(lane < slices && below_mine == r - 1);
    const u64 most = __shfl(mine, static_cast<int>(__builtin_ctzll(at)));
    for (int i = tid; i < n * slices; i += kJoinThreads)
        if (keys[i] <= most && keys[i] != kNoKey) list[atomicAdd(&count, 1)] = static_cast<uint16_t>(i);
    __syncthreads();
    const int C = count;
    for (int i = tid; i < C * slices; i += kJoinThreads) {
        const int c = list[i / slices], z = i % slices;
        const u64 key = keys[c];
        int lo = 0, hi = n;  // keys of list z below this one
        while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if (keys[z * n + mid] < key)
                lo = mid + 1;
            else
                hi = mid;
        }
        if (lo) atomicAdd(&place[c], lo);
    }
    __syncthreads();
    for (int i = tid; i < C; i += kJoinThreads) {
        const int c = list[i];
        if (place[c] < n) answer_top(a, m, static_cast<uint32_t>(place[c]), keys[c], p, logS, temp);
    }
    // (with fewer than n keys in the row all of them are in the list)
    for (int i = C + tid; i < n; i += kJoinThreads) answer_top(a, m, static_cast<uint32_t>(i), kNoKey, p, logS, temp);
}

// Workgroups of `threads`, `slices` of them per row. Measured (us, fp32, 20 first tokens):
//   slices cost a second launch and pay for a few long rows: 1 x 131072 takes 23.6, 19.9, 16.7 and 15.0 with 1, 2, 4 and 8, 64 x
//   131072 27.6, 23.6, 19.1 and 20.5, 1 x 64000 14.5 with 4 and 13.3 with 8; 1 x 32000 13.4 with one, 13.0 with 4, 64 x 32000
//   13.7 and 13.8, 200 x 131072 30.4 with one and 32.0 with two;
//   threads, 256 / 512 / 1024: 1 x 4000 8.4 8.6 11.0, 200 x 32000 18.5 14.9 15.8, 200 x 131072 - 30.4 27.7, 500 x 131072 59.0 55.1
//   59.5, and with many rows, where ends of small workgroups meet others' beginnings, 1024 x 32000 34.5 38.4 56.9.
struct Shape {
    int threads;
    uint32_t slices;
};

Shape shape_of(int64_t M, int64_t V)
{
    if (V <= 4096 || M >= 768) return {256, 1};
    if (M >= 128) return {V >= 100000 && M <= 320 ? 1024 : 512, 1};
    if (V < 48000) return {512, 1};
    int64_t s = V / 8192;  // a step's tokens at the shortest
    if (s > 256 / M) s = 256 / M;
    return {512, static_cast<uint32_t>(s < kMostSlices ? s : kMostSlices)};
}

bool sizes_ok(int64_t M, int64_t V, int32_t n_top)
{
    return M >= 0 && V >= 1 && V <= UW_SAMPLE_MAX_V && M < (int64_t{1} << 22) && n_top >= 0 && n_top <= UW_LOGPROBS_MAX_TOP;
}

size_t workspace(int64_t M, int64_t V, int32_t n_top)
{
    const Shape h = shape_of(M, V);
    return h.slices > 1 ? static_cast<size_t>(M) * h.slices * (sizeof(Part) + static_cast<size_t>(n_top) * sizeof(u64)) : 0;
}

uw_status check(const uw_logprobs_args* p)
{
    if (!p) return fail(UW_EINVAL, "args is NULL");
    if (p->M < 0 || p->V < 1) return fail(UW_ESHAPE, "bad shape %lld x %lld", (long long)p->M, (long long)p->V);
    if (p->n_top < 0) return fail(UW_EINVAL, "n_top must be >= 0");
    if (!sizes_ok(p->M, p->V, p->n_top)) return fail(UW_EUNSUPPORTED, "V over %d, M over 2^22 - 1 or n_top over %d", UW_SAMPLE_MAX_V, UW_LOGPROBS_MAX_TOP);
    if (p->type != UW_F32 && p->type != UW_BF16) return fail(UW_EINVAL, "bad type %d", p->type);
    if (p->M == 0) return UW_OK;
    if (!p->d_logits) return fail(UW_EINVAL, "d_logits is NULL");
    if (!aligned(p->d_logits, p->type == UW_F32 ? 4 : 2)) return fail(UW_EINVAL, "d_logits must be aligned to its elements");
    if (p->ld < p->V) return fail(UW_EINVAL, "ld must be >= V");
    for (const void* q : {static_cast<const void*>(p->d_token), static_cast<const void*>(p->d_temperature), static_cast<const void*>(p->d_logprob),
                          static_cast<const void*>(p->d_rank), static_cast<const void*>(p->d_entropy), static_cast<const void*>(p->d_top_token),
                          static_cast<const void*>(p->d_top_logprob)})
        if (!aligned(q, 4)) return fail(UW_EINVAL, "arrays must be 4-byte aligned");
    if ((p->d_logprob || p->d_rank) && !p->d_token) return fail(UW_EINVAL, "d_logprob and d_rank need d_token");
    const bool top = p->d_top_token || p->d_top_logprob;
    if (top != (p->n_top > 0)) return fail(UW_EINVAL, "n_top and the top lists belong together");
    if (!p->d_logprob && !p->d_rank && !p->d_entropy && !top) return fail(UW_EINVAL, "no output");
    const size_t need = workspace(p->M, p->V, p->n_top);
    if (need && (p->ws_bytes < need || !p->d_ws)) return fail(UW_ENOSPACE, "workspace of %zu bytes needed", need);
    if (need && !aligned(p->d_ws, 16)) return fail(UW_EINVAL, "d_ws must be 16-byte aligned");
    return UW_OK;
}

template <class T>
void launch(const LogprobArgs& a, const Shape& h, hipStream_t s)
{
    const dim3 grid(static_cast<uint32_t>(a.M * h.slices)), block(h.threads);
    if (h.threads == 256)
        hipLaunchKernelGGL((logprobs_rows<T, 256, 16>), grid, block, 0, s, a);
    else if (h.threads == 512)
        hipLaunchKernelGGL((logprobs_rows<T, 512, 16>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((logprobs_rows<T, 1024, 16>), grid, block, 0, s, a);
    if (h.slices > 1) hipLaunchKernelGGL(logprobs_join<T>, dim3(static_cast<uint32_t>(a.M)), dim3(kJoinThreads), 0, s, a);
}

}  // namespace

}  // namespace uw

using namespace uw;

size_t uw_logprobs_workspace(int64_t M, int64_t V, int32_t n_top)
{
    clear_error();
    return M > 0 && sizes_ok(M, V, n_top) ? workspace(M, V, n_top) : 0;
}

uw_status uw_logprobs(const uw_logprobs_args* p, void* stream)
{
    clear_error();
    const uw_status st = check(p);
    if (st != UW_OK || p->M == 0) return st;
    const Shape h = shape_of(p->M, p->V);
    LogprobArgs a{};
    a.x = p->d_logits;
    a.ld = p->ld;
    a.M = p->M;
    a.V = static_cast<int32_t>(p->V);
    a.n_top = p->n_top;
    a.token = p->d_token;
    a.temperature = p->d_temperature;
    a.logprob = p->d_logprob;
    a.rank = p->d_rank;
    a.entropy = p->d_entropy;
    a.top_token = p->d_top_token;
    a.top_logprob = p->d_top_logprob;
    a.slices = h.slices;
    if (h.slices > 1) {
        a.part = static_cast<Part*>(p->d_ws);
        a.keys = reinterpret_cast<u64*>(a.part + a.M * h.slices);
    }
    hipStream_t s = static_cast<hipStream_t>(stream);
    p->type == UW_F32 ? launch<float>(a, h, s) : launch<uint16_t>(a, h, s);
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? UW_OK : fail(UW_EHIP, "logprobs launch failed: %s", hipGetErrorString(e));
}
