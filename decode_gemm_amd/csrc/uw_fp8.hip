// The 8-bit block-scaled path: quantizers to e4m3 codes with one fp32 scale per 128 values of
// a row or per 128 x 128 block, and the activation between the MLP projections that ends in
// such codes. (The matrix product that reads them is in uw_fp8_gemm.hip.)
#include <hip/hip_runtime.h>

#include <cfloat>
#include <type_traits>

#include "uw_internal.h"
#include "uw_recon.h"

namespace uw {

namespace {

typedef float floatx4 __attribute__((ext_vector_type(4)));

constexpr int kG = UW_FP8_GROUP;
constexpr float kTop = 448.0f;  // largest e4m3 value

// 8 consecutive values of a row, from k on; values at and past K read as 0.
__device__ __forceinline__ void load8(const uint16_t* p, int64_t k, int64_t K, float (&v)[8])
{
    if (k + 8 <= K) {
        const u32x4 w = *reinterpret_cast<const u32x4*>(p + k);
#pragma unroll
        for (int i = 0; i < 4; i++) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = k + i < K ? __uint_as_float(static_cast<uint32_t>(p[k + i]) << 16) : 0.f;
    }
}

__device__ __forceinline__ void load8(const float* p, int64_t k, int64_t K, float (&v)[8])
{
    if (k + 8 <= K) {
        const floatx4 a = *reinterpret_cast<const floatx4*>(p + k), b = *reinterpret_cast<const floatx4*>(p + k + 4);
#pragma unroll
        for (int i = 0; i < 4; i++) {
            v[i] = a[i];
            v[4 + i] = b[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = k + i < K ? p[k + i] : 0.f;
    }
}

// Largest |v| among the finite values (0 if there is none): NaN and infinities are passed over,
// so one of them does not change what the other values of its group become.
__device__ __forceinline__ float amax8(const float (&v)[8])
{
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const float t = fabsf(v[i]);
        a = fmaxf(a, t <= FLT_MAX ? t : 0.f);
    }
    return a;
}

// Maximum over the 16 lanes of a DPP row (rotations by 8, 4, 2 and 1 within the row).
__device__ __forceinline__ float row_max16(float a)
{
#define UW_ROW_MAX(ctrl) \
    a = fmaxf(a, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(a), ctrl, 0xF, 0xF, false)))
    UW_ROW_MAX(0x128);
    UW_ROW_MAX(0x124);
    UW_ROW_MAX(0x122);
    UW_ROW_MAX(0x121);
#undef UW_ROW_MAX
    return a;
}

__device__ __forceinline__ float scale_of(float a) { return a == 0.f ? 1.f : fmaxf(a / kTop, FLT_MIN); }

// Eight codes of v / s. The quotient is the correctly rounded one: r = 1 / s is, and one
// residual step (y s - x, exact in an fma) corrects y = x r by the last bit where it is off.
// Taken that way round the residual of a zero is +0, and the zero keeps its sign. Three
// operations instead of a division's ten. The one rounding to fewer bits is the conversion's, to
// nearest even.
// The residual's last bit, 2^-57 of s or so for the smallest quotients that get a code, is a number of
// fp32 only while s is not too small: with SMALL x and s are taken 2^64 times as large, which changes
// no quotient.
template <bool SMALL>
__device__ __forceinline__ uint2 codes8(const float (&v)[8], float s, float r)
{
    constexpr float k = SMALL ? 0x1p64f : 1.0f;
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const float x = v[i] * k;
        const float q = x * r;
        const float e = __builtin_fmaf(q, s, -x);
        const float t = __builtin_amdgcn_fmed3f(__builtin_fmaf(-e, r, q), -kTop, kTop);
        y[i] = fabsf(x) <= FLT_MAX ? t : __uint_as_float(0x7FC00000u);
    }
    uint2 o;
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
    o.x = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], w, true);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(y[4], y[5], 0, false);
    o.y = __builtin_amdgcn_cvt_pk_fp8_f32(y[6], y[7], w, true);
    return o;
}

// The wave tells whether it has a small scale at all, so that the others jump over that code: no slower than
// without (4096 x 4096 bf16 12.6 us; 13.5 with a factor chosen for every value).
__device__ __forceinline__ bool small_scale(float s) { return s < 0x1p-80f; }
__device__ __forceinline__ uint2 codes8(const float (&v)[8], float s)
{
    if (__builtin_expect(__any(small_scale(s)), 0) && small_scale(s)) return codes8<true>(v, s * 0x1p64f, 1.0f / (s * 0x1p64f));
    return codes8<false>(v, s, 1.0f / s);
}

// Codes k .. k+7 of a row (those before K).
__device__ __forceinline__ void store8(uint8_t* q, int64_t k, int64_t K, const uint2& c)
{
    if (k + 8 <= K) {
        *reinterpret_cast<uint2*>(q + k) = c;
    } else {
        for (int i = 0; i < 8; i++)
            if (k + i < K) q[k + i] = static_cast<uint8_t>((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
    }
}

struct QuantArgs {
    const void* x;   // values (gate for the activation)
    const float* u;  // up (activation only)
    int64_t ldx, ldu, M, K;
    uint8_t* q;
    float* s;
    int64_t ldq, lds;
    uint32_t tiles_k;  // workgroups along K
};

template <class T>
struct LoadX {
    __device__ static void row(const QuantArgs& a, int64_t m, int64_t k, float (&v)[8])
    {
        load8(static_cast<const T*>(a.x) + m * a.ldx, k, a.K, v);
    }
};

// silu(g) = g / (1 + e^-g), for negative g as g e^g / (1 + e^g): z = e^-|g| never overflows, and the sum
// lies in [1, 2]. z is 2^(n + r) for the least whole n above -|g| log2(e), whose constant is in two parts, so
// that 2^r lies in (1/2, 1] and g 2^r cannot overflow; the quotient is corrected by its residual, in which the
// sum's rounding error counts too, and the power 2^n of a negative g comes last: below -87 e^g is subnormal, and
// |g| times its rounding would be up to 50 steps of the result. So the result is within 2.5 steps of fp32 plus,
// where it is subnormal itself, its one rounding to that grid (half of 2^-149). 512 x 14336, where the arithmetic
// is as long as the transfers, takes 12.4 us: 12.1 with the power taken first, 14.1 with the library's exponential
// and division. 4096 x 14336 does not notice.
__device__ __forceinline__ float silu(float g)
{
    constexpr float kHi = 0x1.7154760000000p+0f, kLo = 0x1.4ae0c00000000p-26f;  // log2(e)
    const float m = fmaxf(-fabsf(g), -200.0f), n = __builtin_ceilf(m * kHi);  // silu(-200) is 0
    const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(m, kLo, __builtin_fmaf(m, kHi, -n)));
    const float z = __builtin_amdgcn_ldexpf(e, static_cast<int>(n));
    const float d = 1.0f + z, low = z - (d - 1.0f), r = __builtin_amdgcn_rcpf(d);
    const float x = g < 0.0f ? g * e : g;
    const float q = x * r;
    // (the residual's sign as in codes8, for a g of -0)
    return __builtin_amdgcn_ldexpf(__builtin_fmaf(-__builtin_fmaf(q, low, __builtin_fmaf(q, d, -x)), r, q), g < 0.0f ? static_cast<int>(n) : 0);
}

struct LoadSwiglu {
    __device__ static void row(const QuantArgs& a, int64_t m, int64_t k, float (&v)[8])
    {
        float g[8], u[8];
        load8(static_cast<const float*>(a.x) + m * a.ldx, k, a.K, g);
        load8(a.u + m * a.ldu, k, a.K, u);
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = silu(g[i]) * u[i];
    }
};

// Row groups: 16 lanes hold one group's 128 values, eight each, so the group's maximum is a DPP row
// reduction and nothing passes through LDS. A workgroup of 256 threads covers ROWS rows x 16 / ROWS
// groups, one group per 16 lanes: more per thread is slower at every size (2 groups 4%, 4 groups 15%
// at 4096 x 14336), as the registers then hold fewer waves. HBM-bound: the activation of 4096 x 14336
// moves 530 MB in 93 to 95 us (5.6 TB/s, part of it from the cache behind the L2), bf16 to codes at
// 4096 x 4096 51 MB in 11.2 us.
template <class Load, int ROWS>
__global__ void __launch_bounds__(256) quantize_rows(QuantArgs a)
{
    constexpr int GC = 16 / ROWS;  // groups side by side
    const uint32_t tk = blockIdx.x % a.tiles_k, tm = blockIdx.x / a.tiles_k;
    const int sub = threadIdx.x >> 4, l = threadIdx.x & 15;
    const int64_t m = static_cast<int64_t>(tm) * ROWS + sub % ROWS, g = static_cast<int64_t>(tk) * GC + sub / ROWS;
    if (m >= a.M || g * kG >= a.K) return;
    float v[8];
    Load::row(a, m, g * kG + 8 * l, v);
    const float s = scale_of(row_max16(amax8(v)));
    store8(a.q + m * a.ldq, g * kG + 8 * l, a.K, codes8(v, s));
    if (l == 0) a.s[g * a.lds + m] = s;
}

// 128 x 128 blocks, one workgroup each: the block stays in registers between the maximum, joined over
// the waves in LDS, and the codes. HBM-bound: bf16 to codes at 14336 x 4096 moves 176 MB in 37.8 us (4.7
// TB/s; 38.8 with 512 threads, 43.2 with 256). A matrix of few blocks waits for one block's loads and
// barrier: 1000 x 1000 4.1 us, 4.6 with 512 threads, 7.0 with 256.
constexpr int kBlockThreads = 1024;
template <class T>
__global__ void __launch_bounds__(kBlockThreads) quantize_blocks(QuantArgs a)
{
    constexpr int STEP = kBlockThreads / 16, N = kG / STEP;  // rows per step, steps
    __shared__ float part[kBlockThreads / 64];
    const uint32_t g = blockIdx.x % a.tiles_k;
    const int64_t nb = blockIdx.x / a.tiles_k;
    const int64_t m0 = nb * kG + (threadIdx.x >> 4), k = static_cast<int64_t>(g) * kG + 8 * (threadIdx.x & 15);
    float v[N][8];
    float top = 0.f;
#pragma unroll
    for (int t = 0; t < N; t++) {
        const int64_t m = m0 + STEP * t;
        if (m < a.M) {
            LoadX<T>::row(a, m, k, v[t]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++) v[t][i] = 0.f;
        }
    }
#pragma unroll
    for (int t = 0; t < N; t++) top = fmaxf(top, amax8(v[t]));
    top = row_max16(top);
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kBlockThreads / 64; w++) top = fmaxf(top, part[w]);
    const float s = scale_of(top);
    auto store = [&](auto small, float su, float r) {
#pragma unroll
        for (int t = 0; t < N; t++) {
            const int64_t m = m0 + STEP * t;
            if (m < a.M) store8(a.q + m * a.ldq, k, a.K, codes8<decltype(small)::value>(v[t], su, r));
        }
    };
    if (__builtin_expect(__builtin_amdgcn_readfirstlane(small_scale(s)), 0))
        store(std::true_type(), s * 0x1p64f, 1.0f / (s * 0x1p64f));
    else
        store(std::false_type(), s, 1.0f / s);
    if (threadIdx.x == 0) a.s[nb * a.lds + g] = s;
}

// Checks that the two quantizers share.
uw_status check_quant(int64_t K, const void* q, int64_t ldq, const void* s, int64_t lds, int64_t lds_least)
{
    if (!q || !s) return fail(UW_EINVAL, "NULL device pointer");
    if (!aligned(q, 16) || !aligned(s, 4)) return fail(UW_EINVAL, "codes must be 16-byte aligned, scales 4-byte aligned");
    if (ldq < K || ldq % 16) return fail(UW_EINVAL, "ldq must be >= K and a multiple of 16");
    if (lds < lds_least) return fail(UW_EINVAL, "lds too small");
    return UW_OK;
}

template <class Load, int ROWS>
uw_status launch_rows(QuantArgs& a, hipStream_t s)
{
    const int64_t G = (a.K + kG - 1) / kG, wide = 16 / ROWS;
    const int64_t tk = (G + wide - 1) / wide, tm = (a.M + ROWS - 1) / ROWS;
    if (tk > kThreadsMost / 256 || tm > kThreadsMost / 256 / tk) return fail(UW_EUNSUPPORTED, "too many groups for one launch");
    a.tiles_k = static_cast<uint32_t>(tk);
    hipLaunchKernelGGL((quantize_rows<Load, ROWS>), dim3(static_cast<uint32_t>(tk * tm)), dim3(256), 0, s, a);
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? UW_OK : fail(UW_EHIP, "quantize launch failed: %s", hipGetErrorString(e));
}

// Eight rows side by side fill 32 bytes of a scale row per store; one or two rows take groups instead
// (1 x 4096: 2.3 us, 2.7 with eight).
template <class Load>
uw_status launch_rows(QuantArgs& a, hipStream_t s)
{
    return a.M <= 2 ? launch_rows<Load, 1>(a, s) : launch_rows<Load, 8>(a, s);
}

template <class T>
uw_status launch_blocks(QuantArgs& a, hipStream_t s)
{
    const int64_t G = (a.K + kG - 1) / kG, nb = (a.M + kG - 1) / kG;
    if (G > kThreadsMost / kBlockThreads || nb > kThreadsMost / kBlockThreads / G) return fail(UW_EUNSUPPORTED, "too many blocks for one launch");
    a.tiles_k = static_cast<uint32_t>(G);
    hipLaunchKernelGGL(quantize_blocks<T>, dim3(static_cast<uint32_t>(G * nb)), dim3(kBlockThreads), 0, s, a);
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? UW_OK : fail(UW_EHIP, "quantize launch failed: %s", hipGetErrorString(e));
}

}  // namespace

}  // namespace uw

using namespace uw;

uw_status uw_fp8_quantize(const void* d_x, int32_t x_type, int64_t M, int64_t K, int64_t ldx, int32_t block_rows,
                          uint8_t* d_q, int64_t ldq, float* d_s, int64_t lds, void* stream)
{
    clear_error();
    if (M < 0 || K < 1) return fail(UW_ESHAPE, "bad shape %lld x %lld", (long long)M, (long long)K);
    if (x_type != UW_F32 && x_type != UW_BF16) return fail(UW_EINVAL, "bad x_type %d", x_type);
    if (block_rows != 1 && block_rows != kG) return fail(UW_EINVAL, "block_rows must be 1 or %d", kG);
    if (M == 0) return UW_OK;
    if (!d_x || !aligned(d_x, 16)) return fail(UW_EINVAL, "d_x must be 16-byte aligned and not NULL");
    if (ldx < K || ldx % (x_type == UW_BF16 ? 8 : 4)) return fail(UW_EINVAL, "ldx must be >= K and keep rows 16-byte aligned");
    uw_status st = check_quant(K, d_q, ldq, d_s, lds, block_rows == 1 ? M : (K + kG - 1) / kG);
    if (st != UW_OK) return st;
    QuantArgs a{};
    a.x = d_x;
    a.ldx = ldx;
    a.M = M;
    a.K = K;
    a.q = d_q;
    a.ldq = ldq;
    a.s = d_s;
    a.lds = lds;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (block_rows == 1) return x_type == UW_BF16 ? launch_rows<LoadX<uint16_t>>(a, s) : launch_rows<LoadX<float>>(a, s);
    return x_type == UW_BF16 ? launch_blocks<uint16_t>(a, s) : launch_blocks<float>(a, s);
}

uw_status uw_fp8_swiglu(const float* d_g, int64_t ldg, const float* d_u, int64_t ldu, int64_t M, int64_t K,
                        uint8_t* d_q, int64_t ldq, float* d_s, int64_t lds, void* stream)
{
    clear_error();
    if (M < 0 || K < 1) return fail(UW_ESHAPE, "bad shape %lld x %lld", (long long)M, (long long)K);
    if (M == 0) return UW_OK;
    if (!d_g || !d_u || !aligned(d_g, 16) || !aligned(d_u, 16)) return fail(UW_EINVAL, "d_g and d_u must be 16-byte aligned and not NULL");
    if (ldg < K || ldu < K || ldg % 4 || ldu % 4) return fail(UW_EINVAL, "ldg and ldu must be >= K and multiples of 4");
    uw_status st = check_quant(K, d_q, ldq, d_s, lds, M);
    if (st != UW_OK) return st;
    QuantArgs a{};
    a.x = d_g;
    a.ldx = ldg;
    a.u = d_u;
    a.ldu = ldu;
    a.M = M;
    a.K = K;
    a.q = d_q;
    a.ldq = ldq;
    a.s = d_s;
    a.lds = lds;
    return launch_rows<LoadSwiglu>(a, static_cast<hipStream_t>(stream));
}
