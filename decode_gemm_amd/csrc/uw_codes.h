// Device helpers of the kernels that end in e4m3 codes: eight values of a row, a group's largest
// magnitude, its scale and the codes.
#pragma once

#include <hip/hip_runtime.h>

#include <cfloat>
#include <cstdint>

#include "uw.h"
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

}  // namespace

}  // namespace uw
