// 4-bit weights with a scale and a zero point per group of values: the quantizer, the way back, and the
// product of few rows with such a plane (also as the two products of an MLP with their activation).
//
// Mathematics of the product. A group's sum is s (sum x q - z sum x), so no weight is ever rounded: the
// codes go into the matrix unit as the bf16 numbers 1 + q / 16 (the code in the top four mantissa bits, made with a
// shift and an and-or per two codes), and the group's sum of x comes out of the matrix unit too, from a B operand of
// ones, once for all rows of W: D - (1 + z / 16) S = (sum x q - z sum x) / 16, scaled by s into the fp32
// accumulator, and by 16 at the end.
//
// X is the A operand and W the B operand of v_mfma_f32_16x16x32_bf16: the result's column, a lane's low four bits, is
// the row n, so a lane needs one scale for all four of its results. A lane's 16 bytes of a 16 x 128 tile of
// W are its four 8-value operands of four MFMAs.
#include <hip/hip_runtime.h>

#include <cfloat>

#include "uw_codes.h"
#include "uw_internal.h"
#include "uw_recon.h"

namespace uw {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int64_t kMostNK = int64_t{1} << 24;

__host__ __device__ __forceinline__ int64_t tiles16(int64_t n) { return (n + 15) / 16; }
__host__ __device__ __forceinline__ int64_t tiles128(int64_t k) { return (k + 127) / 128; }

// ------------------------------------------------------------------ quantizer and the way back
struct PlaneArgs {
    const void* w;   // quantizer: in
    void* out;       // expansion: out
    uint32_t* plane;
    int64_t N, K, ldw, J, meta;  // K tiles; words before the scales
};

// The nearest number of 20 significant bits, as fp32, ties to even; v > 0 is a normal number of fp64.
__device__ __forceinline__ float round20(double v)
{
    const unsigned long long b = static_cast<unsigned long long>(__double_as_longlong(v));
    const unsigned long long r = (b + 0xFFFFFFFFull + ((b >> 33) & 1)) & ~0x1FFFFFFFFull;
    return static_cast<float>(__longlong_as_double(static_cast<long long>(r)));
}

template <int LANES>
__device__ __forceinline__ uint32_t lanes_max(uint32_t a)
{
#pragma unroll
    for (int d = 1; d < LANES; d *= 2) {
        const uint32_t o = __shfl_xor(a, d);
        a = a > o ? a : o;
    }
    return a;
}
template <int LANES>
__device__ __forceinline__ float lanes_maxf(float a)
{
#pragma unroll
    for (int d = 1; d < LANES; d *= 2) a = fmaxf(a, __shfl_xor(a, d));
    return a;
}

// w / s rounded to the nearest whole number, ties to even, for s of 20 bits and |w / s| <= 15.5: the product with 1 / s is
// at most one off, and the residual w - i s, exact, tells.
__device__ __forceinline__ float whole_quotient(float w, float s, float inv)
{
    const float i = __builtin_rintf(w * inv), e = __builtin_fmaf(-i, s, w), h = 0.5f * s;
    const bool odd = (static_cast<int>(i) & 1) != 0;
    return fabsf(e) > h || (fabsf(e) == h && odd) ? i + __builtin_copysignf(1.0f, e) : i;
}

// One 16 x 128 tile per workgroup, 8 values per thread: row threadIdx / 16, octet threadIdx % 16.
template <class T, int GROUP, bool ZEROS>
__global__ void __launch_bounds__(256) w4_quantize_kernel(PlaneArgs a)
{
    constexpr int LANES = GROUP / 8, PER = 128 / GROUP;
    const int64_t tile = blockIdx.x, t = tile / a.J, j = tile % a.J;
    const int r = threadIdx.x >> 4, o = threadIdx.x & 15;
    const int64_t n = 16 * t + r, k = 128 * j + 8 * o;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = 0.f;
    if (n < a.N && k < a.K) load8(static_cast<const T*>(a.w) + n * a.ldw, k, a.K, v);
    uint32_t top = 0;  // of |v|; infinities and NaN are the largest
    float hi = 0.f, lo = 0.f;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const uint32_t b = __float_as_uint(v[i]) & 0x7FFFFFFFu;
        top = top > b ? top : b;
        hi = fmaxf(hi, v[i]);
        lo = fmaxf(lo, -v[i]);
    }
    top = lanes_max<LANES>(top);
    float s = 1.f, z = 8.f;
    if constexpr (ZEROS) {
        hi = lanes_maxf<LANES>(hi);
        lo = lanes_maxf<LANES>(lo);
        const double d = (static_cast<double>(hi) + static_cast<double>(lo)) / 15.0;
        if (top != 0) s = fmaxf(round20(d), FLT_MIN);
        z = fminf(whole_quotient(lo, s, 1.0f / s), 15.f);
    } else {
        if (top != 0) s = fmaxf(round20(static_cast<double>(__uint_as_float(top)) / 7.0), FLT_MIN);
    }
    const bool broken = top >= 0x7F800000u;
    const float inv = 1.0f / s;
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const float q = broken ? 0.f : fminf(fmaxf(whole_quotient(v[i], s, inv) + z, 0.f), 15.f);
        if (n < a.N && k + i < a.K) word |= static_cast<uint32_t>(static_cast<int>(q)) << (4 * (i / 2) + 16 * (i & 1));
    }
    a.plane[tile * 256 + 4 * (16 * (o & 3) + r) + (o >> 2)] = word;
    if (o % LANES == 0) {
        const uint32_t bits = broken ? 0x7FC00000u : __float_as_uint(s);
        a.plane[a.meta + (tile * PER + o / LANES) * 16 + r] =
            n < a.N && k < a.K ? bits | static_cast<uint32_t>(broken ? 0 : static_cast<int>(z)) : 0u;
    }
}

__device__ __forceinline__ void store_values(uint16_t* w, int64_t k, int64_t K, const float (&v)[8])
{
    if (k + 8 <= K) {
        u32x4 p;
#pragma unroll
        for (int i = 0; i < 4; i++) p[i] = f32_to_bf16_rne(v[2 * i]) | (f32_to_bf16_rne(v[2 * i + 1]) << 16);
        *reinterpret_cast<u32x4*>(w + k) = p;
    } else {
        for (int i = 0; i < 8; i++)
            if (k + i < K) w[k + i] = static_cast<uint16_t>(f32_to_bf16_rne(v[i]));
    }
}
__device__ __forceinline__ void store_values(float* w, int64_t k, int64_t K, const float (&v)[8])
{
    if (k + 8 <= K) {
        *reinterpret_cast<floatx4*>(w + k) = floatx4{v[0], v[1], v[2], v[3]};
        *reinterpret_cast<floatx4*>(w + k + 4) = floatx4{v[4], v[5], v[6], v[7]};
    } else {
        for (int i = 0; i < 8; i++)
            if (k + i < K) w[k + i] = v[i];
    }
}

// s (q - z): a 20-bit number times a 4-bit one, exact in fp32.
template <class T, int GROUP>
__global__ void __launch_bounds__(256) w4_expand_kernel(PlaneArgs a)
{
    constexpr int PER = 128 / GROUP, LANES = GROUP / 8;
    const int64_t tile = blockIdx.x, t = tile / a.J, j = tile % a.J;
    const int r = threadIdx.x >> 4, o = threadIdx.x & 15;
    const int64_t n = 16 * t + r, k = 128 * j + 8 * o;
    if (n >= a.N || k >= a.K) return;
    const uint32_t word = a.plane[tile * 256 + 4 * (16 * (o & 3) + r) + (o >> 2)];
    const uint32_t meta = a.plane[a.meta + (tile * PER + o / LANES) * 16 + r];
    const float s = __uint_as_float(meta & ~15u);
    const int z = static_cast<int>(meta & 15u);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = static_cast<float>(static_cast<int>((word >> (4 * (i / 2) + 16 * (i & 1))) & 15u) - z) * s;
    store_values(static_cast<T*>(a.out) + n * a.ldw, k, a.K, v);
}

// ------------------------------------------------------------------------------ product
struct W4Args {
    const uint16_t* x;
    const uint32_t *w, *up;
    void* y;
    int64_t M, N, K, ldx, ldy, J, meta;
    int32_t bf16;
};

// Four MFMA operands of a lane from its 16 bytes: word p holds the codes of operand p, a pair of them in
// the halves of each bf16 pair. 1 + q / 16 in bf16 is 0x3F80 | q << 3.
__device__ __forceinline__ bf16x8 operand(uint32_t w)
{
    constexpr uint32_t kMask = 0x00780078u, kOne = 0x3F803F80u;
    const u32x4 o = {((w << 3) & kMask) | kOne, ((w >> 1) & kMask) | kOne, ((w >> 5) & kMask) | kOne, ((w >> 9) & kMask) | kOne};
    return __builtin_bit_cast(bf16x8, o);
}

// Eight values of a row of X from k on; what is past K is 0 and not read.
__device__ __forceinline__ u32x4 load_x(const uint16_t* p, int64_t k, int64_t K)
{
    if (k + 8 <= K) return *reinterpret_cast<const u32x4*>(p + k);
    u32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; i++)
        if (k + i < K) v[i / 2] |= static_cast<uint32_t>(p[k + i]) << (16 * (i & 1));
    return v;
}

// 16 RT rows of W (with UP: of each of the two planes) x 16 CT rows of X per workgroup, whose NW waves take the K
// tiles in turn and meet in LDS. FEW: at most four rows of X, in the operand's rows 0, 4, 8 and 12, so that a
// lane's first result is the only one that counts.
template <int CT, int RT, int U, int NW, int PER, bool FEW, bool UP>
__global__ void __launch_bounds__(64 * NW) w4_skinny(W4Args a)
{
    static_assert(!FEW || CT == 1, "few rows are one tile");
    constexpr int RW = UP ? 2 * RT : RT, RES = FEW ? 1 : 4;
    __shared__ float red[NW][RW * CT][RES][64];
    const int lane = threadIdx.x & 63, r = lane & 15, c4 = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t T = static_cast<uint32_t>(tiles16(a.N)), J = static_cast<uint32_t>(a.J);
    const uint32_t tiles_n = (T + RT - 1) / RT;
    const uint32_t t0 = blockIdx.x % tiles_n * RT;
    const int64_t m0 = static_cast<int64_t>(blockIdx.x / tiles_n) * (FEW ? 4 : 16 * CT);

    const uint32_t *wp[RW], *sp[RW];
#pragma unroll
    for (int i = 0; i < RW; i++) {
        const uint32_t* plane = UP && i >= RT ? a.up : a.w;
        const uint32_t t = t0 + i % RT < T ? t0 + i % RT : T - 1;
        wp[i] = plane + static_cast<int64_t>(t) * J * 256 + 4 * lane;
        sp[i] = plane + a.meta + static_cast<int64_t>(t) * J * PER * 16 + r;
    }
    const uint16_t* xp[CT];
    bool has[CT];
#pragma unroll
    for (int c = 0; c < CT; c++) {
        const int64_t m = FEW ? m0 + (r >> 2) : m0 + 16 * c + r;
        has[c] = m < a.M && (!FEW || (r & 3) == 0);
        xp[c] = a.x + (has[c] ? m : 0) * a.ldx + 8 * c4;
    }
    floatx4 acc[RW][CT];
#pragma unroll
    for (int i = 0; i < RW; i++)
#pragma unroll
        for (int c = 0; c < CT; c++) acc[i][c] = floatx4{0.f, 0.f, 0.f, 0.f};

    u32x4 wv[U][RW], xv[U][CT][4];
    uint32_t sv[U][RW][PER];
    auto load_w = [&](int u, uint32_t j) {
#pragma unroll
        for (int i = 0; i < RW; i++) {
            wv[u][i] = *reinterpret_cast<const u32x4*>(wp[i] + static_cast<int64_t>(j) * 256);
#pragma unroll
            for (int g = 0; g < PER; g++) sv[u][i][g] = sp[i][(j * PER + g) * 16];
        }
    };
    auto load = [&](int u, uint32_t j) {
        load_w(u, j);
#pragma unroll
        for (int c = 0; c < CT; c++)
#pragma unroll
            for (int p = 0; p < 4; p++) {
                xv[u][c][p] = u32x4{0, 0, 0, 0};
                if (has[c]) xv[u][c][p] = *reinterpret_cast<const u32x4*>(xp[c] + static_cast<int64_t>(j) * 128 + 32 * p);
            }
    };
    auto multiply = [&](int u) {
        constexpr int P = 4 / PER;  // operands per group
        const u32x4 kOnes = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
#pragma unroll
        for (int g = 0; g < PER; g++) {
            floatx4 sum[CT], d[RW][CT];
#pragma unroll
            for (int c = 0; c < CT; c++) {
                sum[c] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int p = 0; p < P; p++)
                    sum[c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, xv[u][c][g * P + p]),
                                                                     __builtin_bit_cast(bf16x8, kOnes), sum[c], 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < RW; i++) {
#pragma unroll
                for (int c = 0; c < CT; c++) d[i][c] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int p = 0; p < P; p++) {
                    const bf16x8 b = operand(wv[u][i][g * P + p]);
#pragma unroll
                    for (int c = 0; c < CT; c++)
                        d[i][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, xv[u][c][g * P + p]), b, d[i][c], 0, 0, 0);
                }
                const uint32_t meta = sv[u][i][g];
                const float s = __uint_as_float(meta & ~15u), z = __uint_as_float(0x3F800000u | (meta & 15u) << 19);
#pragma unroll
                for (int c = 0; c < CT; c++)
#pragma unroll
                    for (int q = 0; q < RES; q++) acc[i][c][q] = __builtin_fmaf(s, __builtin_fmaf(-z, sum[c][q], d[i][c][q]), acc[i][c][q]);
            }
        }
    };
    const uint32_t full = static_cast<uint32_t>(a.K / 128);
    if (static_cast<uint32_t>(wave) < full) {
        const uint32_t last = full - 1;
#pragma unroll
        for (int u = 0; u < U; u++) {
            const uint32_t j = wave + u * NW;
            load(u, j < last ? j : last);
        }
        for (uint32_t j = wave; j < full; j += U * NW)
#pragma unroll
            for (int u = 0; u < U; u++) {
                if (j + u * NW < full) multiply(u);
                const uint32_t next = j + (u + U) * NW;
                load(u, next < last ? next : last);
            }
    }
    if (J > full && full % NW == static_cast<uint32_t>(wave)) {  // the tile that K ends inside
        load_w(0, full);
#pragma unroll
        for (int c = 0; c < CT; c++)
#pragma unroll
            for (int p = 0; p < 4; p++) {
                xv[0][c][p] = u32x4{0, 0, 0, 0};
                if (has[c]) xv[0][c][p] = load_x(xp[c] - 8 * c4, static_cast<int64_t>(full) * 128 + 32 * p + 8 * c4, a.K);
            }
        multiply(0);
    }
#pragma unroll
    for (int i = 0; i < RW; i++)
#pragma unroll
        for (int c = 0; c < CT; c++)
#pragma unroll
            for (int q = 0; q < RES; q++) red[wave][i * CT + c][q][lane] = acc[i][c][q];
    __syncthreads();
    for (int e = threadIdx.x; e < RT * CT * RES * 64; e += 64 * NW) {
        const int l = e & 63, q = (e >> 6) % RES, tc = (e >> 6) / RES;  // tc = i * CT + c
        const int64_t n = 16 * (static_cast<int64_t>(t0) + tc / CT) + (l & 15);
        const int64_t m = FEW ? m0 + (l >> 4) : m0 + 16 * (tc % CT) + 4 * (l >> 4) + q;
        if (n >= a.N || m >= a.M) continue;
        float v = red[0][tc][q][l];
#pragma unroll
        for (int w = 1; w < NW; w++) v += red[w][tc][q][l];
        v *= 16.f;
        if constexpr (UP) {
            float u = red[0][RT * CT + tc][q][l];
#pragma unroll
            for (int w = 1; w < NW; w++) u += red[w][RT * CT + tc][q][l];
            v = silu_mul(v, 16.f * u);
        }
        if (a.bf16)
            static_cast<uint16_t*>(a.y)[m * a.ldy + n] = static_cast<uint16_t>(f32_to_bf16_rne(v));
        else
            static_cast<float*>(a.y)[m * a.ldy + n] = v;
    }
}

template <int CT, int RT, int U, int NW, bool FEW, bool UP>
uw_status launch_skinny(const W4Args& a, int32_t group, hipStream_t s)
{
    const int64_t blocks = ((tiles16(a.N) + RT - 1) / RT) * ((a.M + (FEW ? 4 : 16 * CT) - 1) / (FEW ? 4 : 16 * CT));
    if (blocks > kThreadsMost / (64 * NW)) return fail(UW_EUNSUPPORTED, "M x N too large for one launch");
    const dim3 grid(static_cast<uint32_t>(blocks)), block(64 * NW);
    if (group == 128)
        hipLaunchKernelGGL((w4_skinny<CT, RT, U, NW, 1, FEW, UP>), grid, block, 0, s, a);
    else if (group == 64)
        hipLaunchKernelGGL((w4_skinny<CT, RT, U, NW, 2, FEW, UP>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((w4_skinny<CT, RT, U, NW, 4, FEW, UP>), grid, block, 0, s, a);
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? UW_OK : fail(UW_EHIP, "4-bit product launch failed: %s", hipGetErrorString(e));
}

template <bool UP>
uw_status run_product(const W4Args& a, int32_t group, hipStream_t s)
{
    if (a.M <= 4) return launch_skinny<1, 1, 2, 8, true, UP>(a, group, s);
    if (a.M <= 16) return launch_skinny<1, 1, 2, 8, false, UP>(a, group, s);
    if (a.M <= 32) return launch_skinny<2, UP ? 1 : 2, 1, 8, false, UP>(a, group, s);
    return launch_skinny<4, UP ? 1 : 2, 1, 4, false, UP>(a, group, s);
}

uw_status check_plane(int64_t N, int64_t K, int32_t group)
{
    if (N < 1 || K < 1) return fail(UW_ESHAPE, "bad shape N=%lld K=%lld", (long long)N, (long long)K);
    if (group != 32 && group != 64 && group != 128) return fail(UW_EINVAL, "group must be 32, 64 or 128");
    if (N > kMostNK || K > kMostNK || tiles16(N) * tiles128(K) > kThreadsMost / 256) return fail(UW_EUNSUPPORTED, "N or K too large");
    return UW_OK;
}

uw_status check_weights(const void* w, int32_t type, int64_t ld, int64_t K)
{
    if (type != UW_F32 && type != UW_BF16) return fail(UW_EINVAL, "bad w_type %d", type);
    if (!w || !aligned(w, 16)) return fail(UW_EINVAL, "d_w must be 16-byte aligned and not NULL");
    if (ld < K || ld % (type == UW_BF16 ? 8 : 4)) return fail(UW_EINVAL, "ldw must be >= K and keep rows 16-byte aligned");
    return UW_OK;
}

PlaneArgs plane_args(const void* plane, int64_t N, int64_t K, int64_t ldw)
{
    PlaneArgs a{};
    a.plane = static_cast<uint32_t*>(const_cast<void*>(plane));
    a.N = N;
    a.K = K;
    a.ldw = ldw;
    a.J = tiles128(K);
    a.meta = tiles16(N) * a.J * 256;
    return a;
}

template <class T, int GROUP>
void launch_quantize(const PlaneArgs& a, bool zeros, hipStream_t s)
{
    const dim3 grid(static_cast<uint32_t>(tiles16(a.N) * a.J));
    if (zeros)
        hipLaunchKernelGGL((w4_quantize_kernel<T, GROUP, true>), grid, dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((w4_quantize_kernel<T, GROUP, false>), grid, dim3(256), 0, s, a);
}
template <class T>
void launch_quantize(const PlaneArgs& a, int32_t group, bool zeros, hipStream_t s)
{
    if (group == 128)
        launch_quantize<T, 128>(a, zeros, s);
    else if (group == 64)
        launch_quantize<T, 64>(a, zeros, s);
    else
        launch_quantize<T, 32>(a, zeros, s);
}

template <class T>
void launch_expand(const PlaneArgs& a, int32_t group, hipStream_t s)
{
    const dim3 grid(static_cast<uint32_t>(tiles16(a.N) * a.J));
    if (group == 128)
        hipLaunchKernelGGL((w4_expand_kernel<T, 128>), grid, dim3(256), 0, s, a);
    else if (group == 64)
        hipLaunchKernelGGL((w4_expand_kernel<T, 64>), grid, dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((w4_expand_kernel<T, 32>), grid, dim3(256), 0, s, a);
}

uw_status product(const uw_w4_args* p, bool up, void* stream)
{
    if (!p) return fail(UW_EINVAL, "args is NULL");
    if (p->M < 0) return fail(UW_ESHAPE, "M < 0");
    uw_status st = check_plane(p->N, p->K, p->group);
    if (st != UW_OK) return st;
    if (p->M > INT32_MAX) return fail(UW_EUNSUPPORTED, "M too large");
    if (p->y_type != UW_F32 && p->y_type != UW_BF16) return fail(UW_EINVAL, "bad y_type %d", p->y_type);
    if (up && p->y_type != UW_BF16) return fail(UW_EINVAL, "h is bf16");
    if (p->M == 0) return UW_OK;
    if (!p->d_x || !p->d_plane || !p->d_y || (up && !p->d_up)) return fail(UW_EINVAL, "NULL device pointer");
    if (!aligned(p->d_x, 16) || !aligned(p->d_plane, 16) || (up && !aligned(p->d_up, 16)) || (p->d_ws && !aligned(p->d_ws, 16)))
        return fail(UW_EINVAL, "X, planes and workspace must be 16-byte aligned");
    if (!aligned(p->d_y, p->y_type == UW_BF16 ? 2 : 4)) return fail(UW_EINVAL, "d_y must be aligned to its elements");
    if (p->ldx < p->K || p->ldx % 8) return fail(UW_EINVAL, "ldx must be >= K and a multiple of 8");
    if (p->ldy < p->N) return fail(UW_EINVAL, "ldy must be >= N");
    W4Args a{};
    a.x = p->d_x;
    a.w = static_cast<const uint32_t*>(p->d_plane);
    a.up = static_cast<const uint32_t*>(p->d_up);
    a.y = p->d_y;
    a.M = p->M;
    a.N = p->N;
    a.K = p->K;
    a.ldx = p->ldx;
    a.ldy = p->ldy;
    a.J = tiles128(p->K);
    a.meta = tiles16(p->N) * a.J * 256;
    a.bf16 = p->y_type == UW_BF16;
    hipStream_t s = static_cast<hipStream_t>(stream);
    return up ? run_product<true>(a, p->group, s) : run_product<false>(a, p->group, s);
}

}  // namespace

}  // namespace uw

using namespace uw;

size_t uw_w4_plane_bytes(int64_t N, int64_t K, int32_t group)
{
    clear_error();
    if (check_plane(N, K, group) != UW_OK) return 0;
    return static_cast<size_t>(tiles16(N) * tiles128(K)) * (1024 + 64 * (128 / group));
}

uw_status uw_w4_quantize(const void* d_w, int32_t w_type, int64_t N, int64_t K, int64_t ldw, int32_t group, int32_t zeros,
                         void* d_plane, void* stream)
{
    clear_error();
    uw_status st = check_plane(N, K, group);
    if (st == UW_OK) st = check_weights(d_w, w_type, ldw, K);
    if (st != UW_OK) return st;
    if (zeros != 0 && zeros != 1) return fail(UW_EINVAL, "zeros must be 0 or 1");
    if (!d_plane || !aligned(d_plane, 16)) return fail(UW_EINVAL, "d_plane must be 16-byte aligned and not NULL");
    PlaneArgs a = plane_args(d_plane, N, K, ldw);
    a.w = d_w;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (w_type == UW_BF16)
        launch_quantize<uint16_t>(a, group, zeros != 0, s);
    else
        launch_quantize<float>(a, group, zeros != 0, s);
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? UW_OK : fail(UW_EHIP, "4-bit quantize launch failed: %s", hipGetErrorString(e));
}

uw_status uw_w4_expand(const void* d_plane, int64_t N, int64_t K, int32_t group, void* d_w, int32_t w_type, int64_t ldw,
                       void* stream)
{
    clear_error();
    uw_status st = check_plane(N, K, group);
    if (st == UW_OK) st = check_weights(d_w, w_type, ldw, K);
    if (st != UW_OK) return st;
    if (!d_plane || !aligned(d_plane, 16)) return fail(UW_EINVAL, "d_plane must be 16-byte aligned and not NULL");
    PlaneArgs a = plane_args(d_plane, N, K, ldw);
    a.out = d_w;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (w_type == UW_BF16)
        launch_expand<uint16_t>(a, group, s);
    else
        launch_expand<float>(a, group, s);
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? UW_OK : fail(UW_EHIP, "4-bit expand launch failed: %s", hipGetErrorString(e));
}

uw_status uw_w4_gemm(const uw_w4_args* args, void* stream)
{
    clear_error();
    return product(args, false, stream);
}

uw_status uw_w4_gate_up(const uw_w4_args* args, void* stream)
{
    clear_error();
    return product(args, true, stream);
}

size_t uw_w4_gemm_workspace(int64_t M, int64_t N, int64_t K)
{
    clear_error();
    (void)M;
    (void)N;
    (void)K;
    return 0;
}
