// Log probabilities of given tokens, their ranks, rows' entropies and the first tokens of the order, from
// logits.
//
// Mathematics. With y_i = (l_i - max) log2(e) / T, S = sum 2^y_i and H = sum y_i 2^y_i: log p_t = (l_t - max) / T - log S
// and the entropy is log S - log(2) H / S. One pass over the row keeps a running maximum with the sums below it: a
// maximum that grows by d (in units of y) turns S into 2^-d S and H into 2^-d (H - d S). Sums of a thread's values are fp32, sums
// over threads fp64. The rank counts l_i > l_t, and l_i >= l_t before t, in the same pass.
// The first n tokens are not sorted out of the row: of the maxima of 256 shares of the row, the n-th largest is
// reached by at least n tokens and hardly more, and these, found by looking again into the shares of the threads
// whose maximum reaches it, are sorted in LDS. Where ties make them too many, a search over the digits of
// (logit, index) finds the n-th token itself.
// Bound by the row's bytes for many rows; a row alone by its two launches and their chains of barriers.
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
constexpr int kMostSlices = 32;
constexpr double kLn2 = 0x1.62e42fefa39efp-1;
constexpr u64 kNoKey = ~u64{0};

// What one workgroup knows of its slice of a row.
struct Part {
    double S, H;  // relative to `top`
    float top;
    int32_t before;  // tokens before the given one
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
    __device__ __forceinline__ void load(int i, float (&v)[VEC]) const
    {
        const int e = first(i);
        if (e >= 0 && e + VEC <= V) {
            unpack(*reinterpret_cast<const u32x4*>(x + e), v);
        } else {
#pragma unroll
            for (int k = 0; k < VEC; k++) v[k] = e + k >= 0 && e + k < V ? value(x, e + k) : -INFINITY;
        }
    }
};

// Running maximum and sums.
struct Sums {
    float top, S, H;
};

// 2 log2(e) / T, of halved differences, which cannot overflow; 0 where all tokens weigh the same or (T <= 0, NaN)
// the sums are not used.
__device__ __forceinline__ float slope(float T)
{
    if (!(T > 0.f) || T > FLT_MAX) return 0.f;
    return static_cast<float>(fmin(2.8853900817779268 / static_cast<double>(T), 3.0e38));
}

__device__ __forceinline__ double from(float lower, float top, float c2)  // y of `lower` below `top`
{
    if (lower == top) return 0.0;
    const double y = (static_cast<double>(lower) - static_cast<double>(top)) * 0.5 * static_cast<double>(c2);
    return y > -1100.0 ? y : -1100.0;  // NaN too
}

// Adds sums below another maximum.
__device__ __forceinline__ void join(Part& a, double S, double H, float top, float c2)
{
    const float m = fmaxf(a.top, top);
    const double ya = a.top == -INFINITY ? 0.0 : from(a.top, m, c2), yb = top == -INFINITY ? 0.0 : from(top, m, c2);
    const double fa = exp2(ya), fb = exp2(yb);
    // an infinite maximum leaves what is finite no mass
    const bool inf = m == INFINITY;
    const double A = inf && a.top != m ? 0.0 : fa, B = inf && top != m ? 0.0 : fb;
    a.H = A * (a.H + ya * a.S) + B * (H + yb * S);
    a.S = A * a.S + B * S;
    a.top = m;
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

__device__ __forceinline__ void answer_row(const LogprobArgs& a, int64_t m, const Part& p, double logS, float T, bool placed, float lt)
{
    if (a.rank) a.rank[m] = placed ? p.before : -1;
    if (a.logprob) {
        const double v = !placed ? -INFINITY : greedy(T) ? (p.before == 0 ? 0.0 : -INFINITY) : log_share(lt, p, logS, T);
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

// The given token of a row: whether it has a place in the order, and its logit.
template <class T>
__device__ __forceinline__ bool given(const LogprobArgs& a, const T* x, int64_t m, int& t, float& l)
{
    t = a.token ? a.token[m] : -1;
    l = t >= 0 && t < a.V ? value(x, t) : -INFINITY;
    return l > -INFINITY;
}

template <int NT>
struct Shared {
    u64 list[kList];
    uint32_t share[kParts];
    uint32_t better[kParts];
    uint32_t hist[256];
    uint16_t flagged[NT];
    uint32_t n_flagged, n_list, bound_tau;
    Part part[NT / 64];
    u64 prefix;
    uint32_t taken, shift, done;
};

// The slice's first n keys, in order, into out (kNoKey past the last one); every thread's words are first + tid + NT i
// below `end`, and `top` is its largest logit.
template <class T, int NT, class Out>
__device__ void first_keys(Shared<NT>& sh, const Words<T>& w, int first, int end, float top, int n, Out out)
{
    constexpr int VEC = Words<T>::VEC, QUAD = NT / kParts;
    static_assert(QUAD == 1 || QUAD == 2 || QUAD == 4, "threads per share");
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    float share = top;
    if (QUAD > 1) share = fmaxf(share, __shfl_xor(share, 1));
    if (QUAD > 2) share = fmaxf(share, __shfl_xor(share, 2));
    // larger is better; 0 = nothing with a place
    const uint32_t mine = share > -INFINITY ? ~order_bits(share) : 0u;
    if (tid % QUAD == 0) sh.share[tid / QUAD] = mine;
    if (tid < kParts) sh.better[tid] = 0;
    if (tid == 0) {
        sh.n_flagged = 0;
        sh.n_list = 0;
        sh.bound_tau = 0;
    }
    __syncthreads();
    {
        const int p = tid % kParts, q0 = tid / kParts * (kParts / QUAD);
        const uint32_t own = sh.share[p];
        uint32_t c = 0;
        for (int q = q0; q < q0 + kParts / QUAD; q++) {
            const uint32_t o = sh.share[q];
            c += o > own || (o == own && q < p);
        }
        if (c) atomicAdd(&sh.better[p], c);
    }
    __syncthreads();
    if (tid < kParts && sh.better[tid] == static_cast<uint32_t>(n - 1)) sh.bound_tau = sh.share[tid];
    __syncthreads();
    const uint32_t tau = sh.bound_tau;
    const bool any = top > -INFINITY;
    if (any && ~order_bits(top) >= tau) sh.flagged[atomicAdd(&sh.n_flagged, 1u)] = static_cast<uint16_t>(tid);
    __syncthreads();
    const int nf = static_cast<int>(sh.n_flagged);
    for (int f = wave; f < nf; f += NT / 64) {
        const int t = sh.flagged[f];
        for (int i = first + t + NT * lane; i < end; i += NT * 64) {
            float v[VEC];
            w.load(i, v);
#pragma unroll
            for (int k = 0; k < VEC; k++)
                if (v[k] > -INFINITY && ~order_bits(v[k]) >= tau) {
                    const uint32_t at = atomicAdd(&sh.n_list, 1u);
                    if (at < kList) sh.list[at] = key_of(v[k], w.first(i) + k);
                }
        }
    }
    __syncthreads();
    if (sh.n_list > kList) {
        // Ties: the n-th key digit by digit, 8 bits at a time, until what is left up to it fits the list.
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
                if (v[k] > -INFINITY) {
                    const u64 key = key_of(v[k], w.first(i) + k);
                    if (key >> shift <= prefix) {
                        const uint32_t at = atomicAdd(&sh.n_list, 1u);
                        if (at < kList) sh.list[at] = key;
                    }
                }
        }
        __syncthreads();
    }
    // Keys are all different, so a key's place is the number of smaller ones.
    const int C = static_cast<int>(sh.n_list);
    for (int c = tid; c < C; c += NT) {
        const u64 key = sh.list[c];
        int place = 0;
        for (int o = 0; o < C; o++) place += sh.list[o] < key;
        if (place < n) out(place, key);
    }
    for (int c = C + tid; c < n; c += NT) out(c, kNoKey);
}

// One slice of a row (all of it with slices = 1) per workgroup.
template <class T, int NT>
__global__ void __launch_bounds__(NT) logprobs_rows(LogprobArgs a)
{
    constexpr int VEC = Words<T>::VEC, U = 16 / VEC;  // 16 values per thread and step
    __shared__ Shared<NT> sh;
    const int tid = threadIdx.x;
    const uint32_t z = blockIdx.x % a.slices;
    const int64_t m = blockIdx.x / a.slices;
    const T* x = static_cast<const T*>(a.x) + m * a.ld;
    const Words<T> w(x, a.V);
    const int per = (w.n + static_cast<int>(a.slices) - 1) / static_cast<int>(a.slices);
    const int first = per * static_cast<int>(z), end = first + per < w.n ? first + per : w.n;
    const float temp = a.temperature ? a.temperature[m] : 1.f, c2 = slope(temp);
    int t;
    float lt;
    const bool placed = given(a, x, m, t, lt);
    const float lt_before = placed ? below(lt) : INFINITY, lt_after = placed ? lt : INFINITY;

    Sums s = {-INFINITY, 0.f, 0.f};
    int before = 0;
    for (int i = first + tid; i < end; i += NT * U) {
        float v[U][VEC];
#pragma unroll
        for (int u = 0; u < U; u++) {
            if (i + u * NT < end) {
                w.load(i + u * NT, v[u]);
            } else {
#pragma unroll
                for (int k = 0; k < VEC; k++) v[u][k] = -INFINITY;
            }
        }
        float top = s.top;
#pragma unroll
        for (int u = 0; u < U; u++)
#pragma unroll
            for (int k = 0; k < VEC; k++) top = fmaxf(top, v[u][k]);
        if (top == INFINITY) {
            float c = s.top == top ? s.S : 0.f;
#pragma unroll
            for (int u = 0; u < U; u++)
#pragma unroll
                for (int k = 0; k < VEC; k++) c += v[u][k] == top ? 1.f : 0.f;
            s.S = c;
            s.H = 0.f;
        } else {
            const float half = 0.5f * top;
            if (top > s.top) {
                const float y = fmaxf(__builtin_fmaf(s.top, 0.5f, -half) * c2, -200.f), f = __builtin_amdgcn_exp2f(y);
                s.H = f * __builtin_fmaf(y, s.S, s.H);
                s.S *= f;
            }
            float S = 0.f, H = 0.f;
#pragma unroll
            for (int u = 0; u < U; u++)
#pragma unroll
                for (int k = 0; k < VEC; k++) {
                    const float y = fmaxf(__builtin_fmaf(v[u][k], 0.5f, -half) * c2, -200.f);  // a mask's NaN too
                    const float e = __builtin_amdgcn_exp2f(y);
                    S += e;
                    H = __builtin_fmaf(y, e, H);
                }
            s.S += S;
            s.H += H;
        }
        s.top = top;
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int e = w.first(i + u * NT);
            if (e < t && t < e + VEC) {
#pragma unroll
                for (int k = 0; k < VEC; k++) before += v[u][k] > (e + k < t ? lt_before : lt_after);
            } else {
                const float than = e < t ? lt_before : lt_after;
#pragma unroll
                for (int k = 0; k < VEC; k++) before += v[u][k] > than;
            }
        }
    }
    // threads, then waves
    Part p = {s.S, s.H, s.top, before};
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const double S = __shfl_xor(p.S, d), H = __shfl_xor(p.H, d);
        const float o = __shfl_xor(p.top, d);
        const int b = __shfl_xor(p.before, d);
        join(p, S, H, o, c2);
        p.before += b;
    }
    if ((tid & 63) == 0) sh.part[tid >> 6] = p;
    __syncthreads();
    p = sh.part[0];
    for (int i = 1; i < NT / 64; i++) {
        join(p, sh.part[i].S, sh.part[i].H, sh.part[i].top, c2);
        p.before += sh.part[i].before;
    }
    if (a.slices > 1) {
        if (tid == 0) a.part[m * a.slices + z] = p;
        if (a.n_top) {
            u64* keys = a.keys + (m * a.slices + z) * a.n_top;
            first_keys<T, NT>(sh, w, first, end, s.top, a.n_top, [&](int place, u64 key) { keys[place] = key; });
        }
    } else {
        const double logS = log(p.S);
        if (tid == 0) answer_row(a, m, p, logS, temp, placed, lt);
        if (a.n_top)
            first_keys<T, NT>(sh, w, first, end, s.top, a.n_top, [&](int place, u64 key) { answer_top(a, m, static_cast<uint32_t>(place), key, p, logS, temp); });
    }
}

// A row's answers from its slices: sums in slice order, and each key's place among all slices' sorted
// keys, by a search in each list.
template <class T>
__global__ void __launch_bounds__(256) logprobs_join(LogprobArgs a)
{
    __shared__ u64 keys[kMostSlices * UW_LOGPROBS_MAX_TOP];
    const int64_t m = blockIdx.x;
    const int tid = threadIdx.x, n = a.n_top, S = static_cast<int>(a.slices);
    for (int i = tid; i < n * S; i += 256) keys[i] = a.keys[m * S * n + i];
    const float temp = a.temperature ? a.temperature[m] : 1.f, c2 = slope(temp);
    Part p = a.part[m * S];
    for (int z = 1; z < S; z++) {
        const Part o = a.part[m * S + z];
        join(p, o.S, o.H, o.top, c2);
        p.before += o.before;
    }
    const double logS = log(p.S);
    if (tid == 0) {
        int t;
        float lt;
        const bool placed = given(a, static_cast<const T*>(a.x) + m * a.ld, m, t, lt);
        answer_row(a, m, p, logS, temp, placed, lt);
    }
    __syncthreads();
    for (int i = tid; i < n * S; i += 256) {
        const u64 key = keys[i];
        if (key == kNoKey) continue;
        int place = 0;
        for (int z = 0; z < S && place < n; z++) {
            int lo = 0, hi = n;  // keys of list z below this one
            while (lo < hi) {
                const int mid = (lo + hi) / 2;
                if (keys[z * n + mid] < key)
                    lo = mid + 1;
                else
                    hi = mid;
            }
            place += lo;
        }
        if (place < n) answer_top(a, m, static_cast<uint32_t>(place), key, p, logS, temp);
    }
    // places past the last token of the row
    __shared__ int have;
    if (tid == 0) have = 0;
    __syncthreads();
    int c = 0;
    for (int i = tid; i < n * S; i += 256) c += keys[i] != kNoKey;
    if (c) atomicAdd(&have, c);
    __syncthreads();
    for (int i = have + tid; i < n; i += 256) answer_top(a, m, static_cast<uint32_t>(i), kNoKey, p, logS, temp);
}

// Workgroups of NT threads, `slices` of them per row.
struct Shape {
    int threads;
    uint32_t slices;
};

Shape shape_of(int64_t M, int64_t V)
{
    // slices of 4096 tokens at the shortest, about 1024 workgroups of 256 threads in all
    int64_t s = (V + 4095) / 4096, want = (1024 + M - 1) / M;
    if (s > want) s = want;
    if (s > kMostSlices) s = kMostSlices;
    return {256, static_cast<uint32_t>(s < 1 ? 1 : s)};
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
    const dim3 grid(static_cast<uint32_t>(a.M * h.slices));
    hipLaunchKernelGGL((logprobs_rows<T, 256>), grid, dim3(256), 0, s, a);
    if (h.slices > 1) hipLaunchKernelGGL(logprobs_join<T>, dim3(static_cast<uint32_t>(a.M)), dim3(256), 0, s, a);
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
