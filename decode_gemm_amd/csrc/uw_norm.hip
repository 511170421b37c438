// The norm after a block, its gate and scale, the residual stream and the norm before the next block,
// in one pass: v = post(y), r' = scale_r r + scale_y gate v, h = pre(r').
//
// Mathematics. Up to 16384 values a row lies in the registers of its threads from the first load to the last store, so y and r
// are read once and r' and h written once, which is all that the step has to move (longer rows: see launch_shape); the sums that a norm needs
// are reduced over lanes by rotations, over waves in LDS. A layer norm takes the mean first and then the squares of
// the differences from it (two reductions): the difference of two sums of squares would lose the variance of a
// row whose mean is large. HBM-bound for many rows (4096 x 4096 of fp32 y and bf16 r into bf16 r' and h 34.2 us, 168 MB, 4.9 TB/s; into
// codes 35.8, 151 MB, with a gate 37.5 to 40.7; a large copy reaches 5.1), a launch, the loads and two reductions for few (1 x 4096 3.8 us).
#include <hip/hip_runtime.h>

#include <cmath>

#include "uw_codes.h"
#include "uw_internal.h"

namespace uw {

namespace {

struct NormArgs {
    const void *y, *r;
    void *r_out, *h;
    const void *post_w, *post_b, *pre_w, *pre_b, *gate;
    float* s;
    int64_t M, K, ldy, ldr, ldr_out, ldh, lds, ldgate;
    uint32_t gate_rows;  // 0: one gate row for all
    int32_t y_type, r_type, w_type, h_type, post, pre;
    float w_add, scale_y, scale_r, eps;
};

// Eight consecutive values as they lie in memory. Loading is kept apart from reading them, so that the branch on the type
// has nothing in it that waits, and all of a thread's loads are on the way together (4096 x 4096, 16 values per thread: 37.5 us when this
// was brought in, 46.0 with the conversion beside each load).
struct Raw {
    u32x4 a, b;  // bf16: b is unused
};
__device__ __forceinline__ Raw load_raw(const void* p, int32_t type, int64_t row, int64_t k, int64_t K)
{
    Raw w;
    w.a = w.b = u32x4{0, 0, 0, 0};
    if (k + 8 <= K) {
        const uint8_t* at = static_cast<const uint8_t*>(p) + (row + k) * (type == UW_BF16 ? 2 : 4);
        w.a = *reinterpret_cast<const u32x4*>(at);
        if (type != UW_BF16) w.b = *reinterpret_cast<const u32x4*>(at + 16);
    } else if (k < K) {  // values past K are 0 and not read
        if (type == UW_BF16) {
#pragma unroll
            for (int i = 0; i < 8; i++)
                if (k + i < K) w.a[i / 2] |= static_cast<uint32_t>(static_cast<const uint16_t*>(p)[row + k + i]) << (16 * (i & 1));
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++)
                if (k + i < K) (i < 4 ? w.a : w.b)[i & 3] = static_cast<const uint32_t*>(p)[row + k + i];
        }
    }
    return w;
}
__device__ __forceinline__ void read(const Raw& w, int32_t type, float (&v)[8])
{
    if (type == UW_BF16) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            v[2 * i] = __uint_as_float(w.a[i] << 16);
            v[2 * i + 1] = __uint_as_float(w.a[i] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            v[i] = __uint_as_float(w.a[i]);
            v[4 + i] = __uint_as_float(w.b[i]);
        }
    }
}

typedef float floatx2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ void store8(void* p, int32_t type, int64_t row, int64_t k, int64_t K, const float (&v)[8])
{
    if (type == UW_BF16) {
        uint16_t* o = static_cast<uint16_t*>(p) + row + k;
        u32x4 w;  // the one rounding, to nearest even
#pragma unroll
        for (int i = 0; i < 4; i++) w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(floatx2{v[2 * i], v[2 * i + 1]}, bf16x2));
        if (k + 8 <= K) {
            *reinterpret_cast<u32x4*>(o) = w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++)
                if (k + i < K) o[i] = static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1)));
        }
    } else {
        float* o = static_cast<float*>(p) + row + k;
        if (k + 8 <= K) {
            *reinterpret_cast<floatx4*>(o) = floatx4{v[0], v[1], v[2], v[3]};
            *reinterpret_cast<floatx4*>(o + 4) = floatx4{v[4], v[5], v[6], v[7]};
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++)
                if (k + i < K) o[i] = v[i];
        }
    }
}

// Sum over a row's threads, the same bits in all of them: every step adds two values that each other's
// lanes add too.
template <int WAVES>
__device__ __forceinline__ float row_sum(float a, float* red)
{
#define UW_ROW_ADD(ctrl) \
    a += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(a), ctrl, 0xF, 0xF, false))
    UW_ROW_ADD(0x128);
    UW_ROW_ADD(0x124);
    UW_ROW_ADD(0x122);
    UW_ROW_ADD(0x121);
#undef UW_ROW_ADD
    a += __shfl_xor(a, 16);
    a += __shfl_xor(a, 32);
    if constexpr (WAVES > 1) {
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = a;
        __syncthreads();
        a = red[0];
#pragma unroll
        for (int w = 1; w < WAVES; w++) a += red[w];
    }
    return a;
}

// A norm's vectors, on the way beside the row where registers allow it.
template <int E>
struct Vectors {
    const void *w, *b;
    int32_t type;
    float add;
    Raw rw[E], rb[E];
    __device__ __forceinline__ void load(int64_t k0, int64_t step, int64_t K)
    {
#pragma unroll
        for (int e = 0; e < E; e++) {
            if (w) rw[e] = load_raw(w, type, 0, k0 + e * step, K);
            if (b) rb[e] = load_raw(b, type, 0, k0 + e * step, K);
        }
    }
    // v <- v (w + add) + b
    __device__ __forceinline__ void apply(int e, float (&v)[8]) const
    {
        if (w) {
            float x[8];
            read(rw[e], type, x);
#pragma unroll
            for (int i = 0; i < 8; i++) v[i] *= x[i] + add;
        }
        if (b) {
            float x[8];
            read(rb[e], type, x);
#pragma unroll
            for (int i = 0; i < 8; i++) v[i] += x[i];
        }
    }
};

// v <- norm(v); red: two rows of LDS, one for each sum (the next norm's are others).
template <int WAVES, int E>
__device__ __forceinline__ void norm(float (&v)[E][8], int kind, const Vectors<E>& vectors, int64_t k0, const NormArgs& a, float (*red)[16])
{
    constexpr int STEP = WAVES * 64 * 8;
    const float n = static_cast<float>(a.K);
    if (kind == UW_NORM_LAYER) {
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; e++)
#pragma unroll
            for (int i = 0; i < 8; i++) s += v[e][i];
        const float mean = row_sum<WAVES>(s, red[0]) / n;
#pragma unroll
        for (int e = 0; e < E; e++)
#pragma unroll
            for (int i = 0; i < 8; i++) v[e][i] = k0 + e * STEP + i < a.K ? v[e][i] - mean : 0.f;
    }
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; e++)
#pragma unroll
        for (int i = 0; i < 8; i++) s = __builtin_fmaf(v[e][i], v[e][i], s);
    // 1 / sqrt(ms) in two parts: f and the rest that its residual 1 - ms f^2, in which f^2 counts in two parts too, tells. So a value
    // times the factor is off by its own rounding alone, not by the factor's as well.
    const float ms = row_sum<WAVES>(s, red[1]) / n + a.eps;
    const float f = 1.0f / sqrtf(ms), ff = f * f;
    const float rest = __builtin_fmaf(-ms, ff, 1.0f) - ms * __builtin_fmaf(f, f, -ff);
    const float low = fabsf(rest) < 1.0f ? 0.5f * f * rest : 0.f;  // (0, infinities and NaN have none)
#pragma unroll
    for (int e = 0; e < E; e++) {
#pragma unroll
        for (int i = 0; i < 8; i++) v[e][i] = __builtin_fmaf(v[e][i], f, v[e][i] * low);
        vectors.apply(e, v[e]);
    }
}

// Values k .. k + 7 of a row of h; 16 lanes hold a group of 128 values, or nothing of the row.
__device__ __forceinline__ void store_h(const NormArgs& a, int64_t m, int64_t k, float (&v)[8])
{
    if (a.h_type != UW_E4M3) {
        store8(a.h, a.h_type, m * a.ldh, k, a.K, v);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = k + i < a.K ? v[i] : 0.f;
    const float s = scale_of(row_max16(amax8(v)));
    const uint2 c = codes8(v, s);
    store8(static_cast<uint8_t*>(a.h) + m * a.ldh, k, a.K, c);
    if ((threadIdx.x & 15) == 0 && k < a.K) a.s[k / kG * a.lds + m] = s;
}

// One row per WAVES waves, E times eight values per thread; with WAVES = 1 four rows share a workgroup.
template <int WAVES, int E>
__global__ void __launch_bounds__(WAVES == 1 ? 256 : 64 * WAVES) block_norm_kernel(NormArgs a)
{
    constexpr int STEP = WAVES * 64 * 8;
    // Vectors are loaded with the row, for the latency, where that leaves registers for other rows (4096 x 4096 of 16 values per thread:
    // 36.8 us with them late, 40.0 early).
    constexpr bool EARLY = E == 1;
    __shared__ float red[WAVES > 1 ? 4 : 1][16];
    const int t = WAVES == 1 ? threadIdx.x & 63 : threadIdx.x;
    const int64_t m = WAVES == 1 ? static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6) : blockIdx.x;
    if (WAVES == 1 && m >= a.M) return;
    const int64_t k0 = 8 * t;
    const bool posts = a.y && a.post != UW_NORM_NONE, pres = a.h && a.pre != UW_NORM_NONE, gates = a.y && a.gate;
    const int64_t gate_row = gates && a.gate_rows ? static_cast<uint32_t>(m) / a.gate_rows : 0;
    Raw y[E], r[E], g[E];
    Vectors<E> post{posts ? a.post_w : nullptr, posts ? a.post_b : nullptr, a.w_type, a.w_add};
    Vectors<E> pre{pres ? a.pre_w : nullptr, pres ? a.pre_b : nullptr, a.w_type, a.w_add};
    auto load_gate = [&]() {
#pragma unroll
        for (int e = 0; e < E; e++)
            if (gates) g[e] = load_raw(a.gate, a.w_type, gate_row * a.ldgate, k0 + e * STEP, a.K);
    };
#pragma unroll
    for (int e = 0; e < E; e++)
        if (a.y) y[e] = load_raw(a.y, a.y_type, m * a.ldy, k0 + e * STEP, a.K);
#pragma unroll
    for (int e = 0; e < E; e++)
        if (a.r) r[e] = load_raw(a.r, a.r_type, m * a.ldr, k0 + e * STEP, a.K);
    if (EARLY) {
        post.load(k0, STEP, a.K);
        load_gate();
        pre.load(k0, STEP, a.K);
    }
    float v[E][8];
    if (a.y) {
#pragma unroll
        for (int e = 0; e < E; e++) read(y[e], a.y_type, v[e]);
        if (posts) {
            if (!EARLY) post.load(k0, STEP, a.K);
            norm<WAVES, E>(v, a.post, post, k0, a, red);
        }
        if (gates) {
            if (!EARLY) load_gate();
#pragma unroll
            for (int e = 0; e < E; e++) {
                float x[8];
                read(g[e], a.w_type, x);
#pragma unroll
                for (int i = 0; i < 8; i++) v[e][i] *= x[i];
            }
        }
#pragma unroll
        for (int e = 0; e < E; e++)
#pragma unroll
            for (int i = 0; i < 8; i++) v[e][i] *= a.scale_y;
    } else {
#pragma unroll
        for (int e = 0; e < E; e++)
#pragma unroll
            for (int i = 0; i < 8; i++) v[e][i] = 0.f;
    }
#pragma unroll
    for (int e = 0; e < E; e++) {
        if (a.r) {
            float x[8];
            read(r[e], a.r_type, x);
#pragma unroll
            for (int i = 0; i < 8; i++) v[e][i] = a.y ? __builtin_fmaf(a.scale_r, x[i], v[e][i]) : a.scale_r * x[i];
        }
        if (a.r_out) store8(a.r_out, a.r_type, m * a.ldr_out, k0 + e * STEP, a.K, v[e]);
    }
    if (!a.h) return;
    if (pres) {
        if (!EARLY) pre.load(k0, STEP, a.K);
        norm<WAVES, E>(v, a.pre, pre, k0, a, red + (WAVES > 1 ? 2 : 0));
    }
#pragma unroll
    for (int e = 0; e < E; e++) store_h(a, m, k0 + e * STEP, v[e]);
}

template <int WAVES, int E>
uw_status launch(const NormArgs& a, hipStream_t s)
{
    const int64_t blocks = WAVES == 1 ? (a.M + 3) / 4 : a.M;
    constexpr int threads = WAVES == 1 ? 256 : 64 * WAVES;
    if (blocks > kThreadsMost / threads) return fail(UW_EUNSUPPORTED, "too many rows for one launch");
    hipLaunchKernelGGL((block_norm_kernel<WAVES, E>), dim3(static_cast<uint32_t>(blocks)), dim3(threads), 0, s, a);
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? UW_OK : fail(UW_EHIP, "block norm launch failed: %s", hipGetErrorString(e));
}

// How many waves share a row: with few rows as many as keep eight values per thread, for the latency; with many rows four, and more
// values per thread, so that more rows are in a CU at once (us, cold, y fp32, r bf16 and h in codes; few- and many-row shape:
// 1 x 4096 3.8 and 5.0, 64 x 8192 6.5 and 9.5, 512 x 4096 9.2 and 9.2, 4096 x 4096 40.5 and 35.8, 4096 x 8192 100 and 72). Workgroups
// that stay, keep the vectors and have the next row on the way took 38.1 and 78 for the last two.
// Past 16384 values a thread of a workgroup of 1024 has more of them than its 128 registers hold, and part goes through scratch memory (212
// bytes per thread up to 32768, 848 past that): fp32 y, bf16 r, r' and h, 4096 x 16384 157 us (4.3 TB/s), 2048 x 28672 254 (2.3), 1024 x 65536 865 (0.8),
// one row of 28672 20.7, of 65536 123.
uw_status launch_shape(const NormArgs& a, hipStream_t s)
{
    if (a.K <= 512) return launch<1, 1>(a, s);
    if (a.K <= 1024) return launch<2, 1>(a, s);
    if (a.K <= 2048) return launch<4, 1>(a, s);
    if (a.M >= 512) {
        if (a.K <= 4096) return launch<4, 2>(a, s);
        if (a.K <= 6144) return launch<4, 3>(a, s);
        if (a.K <= 8192) return launch<4, 4>(a, s);
        if (a.K <= 16384) return launch<8, 4>(a, s);
    } else {
        if (a.K <= 4096) return launch<8, 1>(a, s);
        if (a.K <= 8192) return launch<16, 1>(a, s);
        if (a.K <= 16384) return launch<16, 2>(a, s);
    }
    if (a.K <= 32768) return launch<16, 4>(a, s);
    return launch<16, 8>(a, s);
}

// The rows [M][K] of `type` at p, `ld` elements apart, start at 16-byte boundaries.
uw_status check_rows(const char* name, const void* p, int32_t type, int64_t ld, int64_t K)
{
    if (type != UW_F32 && type != UW_BF16) return fail(UW_EINVAL, "bad type %d of %s", type, name);
    if (!aligned(p, 16)) return fail(UW_EINVAL, "%s must be 16-byte aligned", name);
    if (ld < K || ld % (type == UW_BF16 ? 8 : 4)) return fail(UW_EINVAL, "the leading dimension of %s must be >= K and keep rows 16-byte aligned", name);
    return UW_OK;
}

}  // namespace

}  // namespace uw

using namespace uw;

uw_status uw_block_norm(const uw_block_norm_args* p, void* stream)
{
    clear_error();
    if (!p) return fail(UW_EINVAL, "args is NULL");
    if (p->M < 0 || p->K < 1) return fail(UW_ESHAPE, "bad shape %lld x %lld", (long long)p->M, (long long)p->K);
    if (p->K > UW_NORM_MAX_K || p->M > INT32_MAX) return fail(UW_EUNSUPPORTED, "K over %d or M over 2^31 - 1", UW_NORM_MAX_K);
    if (p->post < UW_NORM_NONE || p->post > UW_NORM_LAYER || p->pre < UW_NORM_NONE || p->pre > UW_NORM_LAYER)
        return fail(UW_EINVAL, "bad norm %d / %d", p->post, p->pre);
    if (!(p->eps >= 0.f) || std::isinf(p->eps)) return fail(UW_EINVAL, "eps must be a finite number >= 0");
    if (p->gate_rows < 0) return fail(UW_EINVAL, "gate_rows must be >= 0");
    if (p->M == 0) return UW_OK;
    if (!p->d_y && !p->d_r) return fail(UW_EINVAL, "d_y and d_r are both NULL");
    if (!p->d_r_out && !p->d_h) return fail(UW_EINVAL, "d_r_out and d_h are both NULL");
    if (p->w_type != UW_F32 && p->w_type != UW_BF16) return fail(UW_EINVAL, "bad w_type %d", p->w_type);
    if ((p->d_post_b && p->post != UW_NORM_LAYER) || (p->d_pre_b && p->pre != UW_NORM_LAYER))
        return fail(UW_EINVAL, "biases belong to UW_NORM_LAYER");
    uw_status st = UW_OK;
    if (p->d_y && (st = check_rows("d_y", p->d_y, p->y_type, p->ldy, p->K)) != UW_OK) return st;
    if (p->d_r && (st = check_rows("d_r", p->d_r, p->r_type, p->ldr, p->K)) != UW_OK) return st;
    if (p->d_r_out && (st = check_rows("d_r_out", p->d_r_out, p->r_type, p->ldr_out, p->K)) != UW_OK) return st;
    if (p->d_gate && (st = check_rows("d_gate", p->d_gate, p->w_type, p->ldgate, p->K)) != UW_OK) return st;
    for (const void* w : {p->d_post_w, p->d_post_b, p->d_pre_w, p->d_pre_b})
        if (!aligned(w, 16)) return fail(UW_EINVAL, "weights and biases must be 16-byte aligned");
    const bool codes = p->d_h && p->h_type == UW_E4M3;
    if (codes) {
        if (!p->d_s || !aligned(p->d_s, 4) || !aligned(p->d_h, 16)) return fail(UW_EINVAL, "codes must be 16-byte aligned, d_s 4-byte aligned and not NULL");
        if (p->ldh < p->K || p->ldh % 16) return fail(UW_EINVAL, "ldh must be >= K and a multiple of 16 for codes");
        if (p->lds < p->M) return fail(UW_EINVAL, "lds must be >= M");
    } else if (p->d_h && (st = check_rows("d_h", p->d_h, p->h_type, p->ldh, p->K)) != UW_OK) {
        return st;
    }
    // in place: the same elements at the same places
    auto same = [](const void* o, int32_t ot, int64_t ol, const void* i, int32_t it, int64_t il) { return !o || o != i || (ot == it && ol == il); };
    if (!same(p->d_r_out, p->r_type, p->ldr_out, p->d_y, p->y_type, p->ldy) || !same(p->d_r_out, p->r_type, p->ldr_out, p->d_r, p->r_type, p->ldr) ||
        !same(p->d_h, p->h_type, p->ldh, p->d_y, p->y_type, p->ldy) || !same(p->d_h, p->h_type, p->ldh, p->d_r, p->r_type, p->ldr) ||
        (p->d_h && p->d_h == p->d_r_out))
        return fail(UW_EINVAL, "an output in place of an input must have its type and leading dimension; d_h and d_r_out must differ");
    NormArgs a{};
    a.y = p->d_y;
    a.r = p->d_r;
    a.r_out = p->d_r_out;
    a.h = p->d_h;
    a.post_w = p->d_post_w;
    a.post_b = p->d_post_b;
    a.pre_w = p->d_pre_w;
    a.pre_b = p->d_pre_b;
    a.gate = p->d_gate;
    a.s = p->d_s;
    a.M = p->M;
    a.K = p->K;
    a.ldy = p->ldy;
    a.ldr = p->ldr;
    a.ldr_out = p->ldr_out;
    a.ldh = p->ldh;
    a.lds = p->lds;
    a.gate_rows = static_cast<uint32_t>(p->gate_rows < INT32_MAX ? p->gate_rows : INT32_MAX);
    a.ldgate = p->ldgate;
    a.y_type = p->y_type;
    a.r_type = p->r_type;
    a.w_type = p->w_type;
    a.h_type = p->h_type;
    a.post = p->post;
    a.pre = p->pre;
    a.w_add = p->w_add;
    a.scale_y = p->scale_y;
    a.scale_r = p->scale_r;
    a.eps = p->eps;
    return launch_shape(a, static_cast<hipStream_t>(stream));
}
