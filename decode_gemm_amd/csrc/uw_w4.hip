// 4-bit weights with a scale and a zero point per group of values: the quantizer, the way back, and the
// product of few rows with such a plane (also as the two products of an MLP with their activation).
//
// Mathematics of the product. A group's sum is s (sum x q - z sum x), so no weight is ever rounded: the
// codes go into the matrix unit as the bf16 numbers 1 + q / 16 (the code in the top four mantissa bits, made with a
// shift and an and-or per two codes), and the group's sum of x comes out of the matrix unit too, from a B operand of
// ones, once for all rows of W: D - (1 + z / 16) S = (sum x q - z sum x) / 16, scaled by s into the fp32
// accumulator, and by 16 at the end.
// D and S are rounded apart. For a group whose codes are all its zero point (weights that are 0) what is left between them would be
// multiplied by a scale that says nothing (1 where the quantizer found only zeros). So a wave that may have met such a group
// goes through its tiles once more and takes each row's S with an operand of its 1 + z / 16: for such a group the same
// operations as D, and D - S is 0. (So they are with ones where the zero point is 0.) What it looks for in the first pass is a
// word of eight like codes, not 0, in each of a row's four lanes. (Rows' own sums in the first pass take 10% longer for M = 1 gate and up and 20% for M = 16, an exact
// comparison of the codes 8% and 7%.)
//
// X is the A operand and W the B operand of v_mfma_f32_16x16x32_bf16: the result's column, a lane's low four bits, is
// the row n, so a lane needs one scale for all four of its results. A lane's 16 bytes of a 16 x 128 tile of
// W are its four 8-value operands of four MFMAs.
#include <hip/hip_runtime.h>

#include <cfloat>

#include "uw_codes.h"
#include "uw_internal.h"
#include "uw_recon.h"
#include "uw_tiles.h"

namespace uw {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int64_t kMostNK = int64_t{1} << 24;
constexpr int64_t kMostLd = int64_t{1} << 25;  // 64 rows of X and K values more lie within 32-bit byte offsets

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

// Maximum over 4, 8 or 16 neighbouring lanes: pairs, quads, then mirrored halves and rows.
template <int CTRL>
__device__ __forceinline__ uint32_t moved(uint32_t v)
{
    return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xF, 0xF, false));
}
template <int CTRL>
__device__ __forceinline__ uint32_t larger(uint32_t v)
{
    const uint32_t o = moved<CTRL>(v);
    return v > o ? v : o;
}
template <int CTRL>
__device__ __forceinline__ float larger(float v)
{
    return fmaxf(v, __uint_as_float(moved<CTRL>(__float_as_uint(v))));
}
template <int LANES, class V>
__device__ __forceinline__ V lanes_max(V v)
{
    v = larger<0xB1>(v);
    v = larger<0x4E>(v);
    if constexpr (LANES > 4) v = larger<0x141>(v);
    if constexpr (LANES > 8) v = larger<0x140>(v);
    return v;
}

// a / 7 to 20 significant bits, the nearest, ties to even, for a >= 2^-100: the product with 1 / 7 rounded to 20 bits is at most
// one step off, and the residual a - 7 c, exact, tells. Below a power of two the step is half as long (with that of the power itself
// one mantissa in 2^23, 7 - 2^-18, came out one step too large).
__device__ __forceinline__ float seventh20(float a)
{
    const uint32_t c = (__float_as_uint(a * (1.0f / 7.0f)) + 8) & ~15u;
    const float v = __uint_as_float(c), e = __builtin_fmaf(-7.0f, v, a);
    const float u = __uint_as_float((c & 0x7F800000u) - ((e < 0.f && !(c & 0x7FFFFFu) ? 20u : 19u) << 23)), h = 3.5f * u;  // a step of 20 bits
    return fabsf(e) > h || (fabsf(e) == h && (c & 16)) ? v + __builtin_copysignf(u, e) : v;
}

// w / s rounded to fp32 and then, by adding 1.5 * 2^23, to the nearest whole number, ties to even, which is left with that
// number. The quotient is the correctly rounded one (inv = 1 / s is, and one residual step corrects it; s is not so small that the
// residual underflows). Rounding twice is no loss, as no quotient but T itself becomes a T = t / 2 halfway between two whole numbers up to
// 15. s is S 2^a with S < 2^20, so T s is the whole number t S of at most 25 bits times 2^(a-1), and a w beside it lies at least
// that unit away, or, with fewer than 24 bits in t S, one of w's own steps. Over s that is more than 2^-21 in the first case and more than
// 2^-24 T in the other: more than half of T's step.
constexpr float kWhole = 12582912.0f;
__device__ __forceinline__ float whole_quotient(float w, float s, float inv)
{
    const float q = w * inv;
    return __builtin_fmaf(__builtin_fmaf(-q, s, w), inv, q) + kWhole;
}

// Eight codes of values v as a plane's word. A word's sum takes over each whole number with the bits of 1.5 * 2^23 above it, the
// same for every value and taken off at once.
__device__ __forceinline__ uint32_t codes_of(const float (&v)[8], float s, float inv, float z)
{
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const int at = 4 * (i / 2) + 16 * (i & 1);
        word += __float_as_uint(__builtin_amdgcn_fmed3f(whole_quotient(v[i], s, inv) + z, kWhole, kWhole + 15.0f)) << at;
        word -= 0x4B400000u << at;
    }
    return word;
}

// TJ 16 x 128 tiles, one after another in K, per workgroup, 8 values of each per thread: row threadIdx / 16, octet
// threadIdx % 16. Bound by HBM: bf16 weights of 14336 x 4096 take 33.1 us with a
// scale per 128 (148 MB, 4.5 TB/s; 34.9 with one tile per workgroup, which is as good for a matrix of few tiles), 40 with zero
// points, whose fp64 quotients show; fp32 weights with zero points 42.3 (272 MB).
template <class T, int GROUP, bool ZEROS, int TJ>
__global__ void __launch_bounds__(256) w4_quantize_kernel(PlaneArgs a)
{
    constexpr int LANES = GROUP / 8, PER = 128 / GROUP;
    const uint32_t runs = static_cast<uint32_t>((a.J + TJ - 1) / TJ);
    const int64_t t = blockIdx.x / runs, j0 = static_cast<int64_t>(blockIdx.x % runs) * TJ;
    const int r = threadIdx.x >> 4, o = threadIdx.x & 15;
    const int64_t n = 16 * t + r;
    float v[TJ][8];
#pragma unroll
    for (int u = 0; u < TJ; u++) {
        const int64_t k = 128 * (j0 + u) + 8 * o;
#pragma unroll
        for (int i = 0; i < 8; i++) v[u][i] = 0.f;
        if (n < a.N && k < a.K) load8(static_cast<const T*>(a.w) + n * a.ldw, k, a.K, v[u]);
    }
#pragma unroll
    for (int u = 0; u < TJ; u++) {
        if (j0 + u >= a.J) break;
        const int64_t tile = t * a.J + j0 + u, k = 128 * (j0 + u) + 8 * o;
        uint32_t top = 0;  // of |v|; infinities and NaN are the largest
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const uint32_t b = __float_as_uint(v[u][i]) & 0x7FFFFFFFu;
            top = top > b ? top : b;
        }
        top = lanes_max<LANES>(top);
        float s = 1.f, z = 8.f, lowest = 0.f;
        if constexpr (ZEROS) {
            float hi = 0.f, lo = 0.f;
#pragma unroll
            for (int i = 0; i < 8; i++) {
                hi = fmaxf(hi, v[u][i]);
                lo = fmaxf(lo, -v[u][i]);
            }
            hi = lanes_max<LANES>(hi);
            lowest = lo = lanes_max<LANES>(lo);
            if (top != 0) s = fmaxf(round20((static_cast<double>(hi) + static_cast<double>(lo)) / 15.0), FLT_MIN);
        } else if (top != 0) {
            const float a7 = __uint_as_float(top);
            s = seventh20(a7);
            if (__builtin_expect(a7 < 0x1p-100f, 0)) s = fmaxf(round20(static_cast<double>(a7) / 7.0), FLT_MIN);
        }
        const bool broken = top >= 0x7F800000u;
        // below 2^-80 all is taken 2^64 times as large, which changes no quotient
        const bool small = s < 0x1p-80f;
        const float k64 = small ? 0x1p64f : 1.0f, sk = s * k64, inv = 1.0f / sk;
        if (__builtin_expect(__any(small), 0))
#pragma unroll
            for (int i = 0; i < 8; i++) v[u][i] *= k64;
        if constexpr (ZEROS) z = fminf(whole_quotient(lowest * k64, sk, inv) - kWhole, 15.f);
        uint32_t word = broken ? 0u : codes_of(v[u], sk, inv, z);
        if (n >= a.N || k + 8 > a.K) {  // what is past the matrix is 0
            uint32_t keep = 0;
#pragma unroll
            for (int i = 0; i < 8; i++)
                if (n < a.N && k + i < a.K) keep |= 15u << (4 * (i / 2) + 16 * (i & 1));
            word &= keep;
        }
        a.plane[tile * 256 + 4 * (16 * (o & 3) + r) + (o >> 2)] = word;
        if (o % LANES == 0) {
            const uint32_t bits = broken ? 0x7FC00000u : __float_as_uint(s) | static_cast<uint32_t>(static_cast<int>(z));
            a.plane[a.meta + (tile * PER + o / LANES) * 16 + r] = n < a.N && k < a.K ? bits : 0u;
        }
    }
}

typedef float floatx2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ void store_values(uint16_t* w, int64_t k, int64_t K, const float (&v)[8])
{
    u32x4 p;
#pragma unroll
    for (int i = 0; i < 4; i++) p[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(floatx2{v[2 * i], v[2 * i + 1]}, bf16x2));
    if (k + 8 <= K) {
        *reinterpret_cast<u32x4*>(w + k) = p;
    } else {
        for (int i = 0; i < 8; i++)
            if (k + i < K) w[k + i] = static_cast<uint16_t>(p[i / 2] >> (16 * (i & 1)));
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

// s q - z s: z s is a 20-bit number times a 4-bit one, exact in fp32, and so is the difference: the fma rounds nothing. One tile per
// workgroup, a thread as in the quantizer. Bound by HBM's writes: 14336 x 4096 to bf16 takes 22.5 us, to fp32 45.7 (148 and 272 MB,
// part of them in the cache behind the L2); with four tiles per workgroup 23.7 and 48.4.
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
    const float s = __uint_as_float(meta & ~15u), zs = -static_cast<float>(meta & 15u) * s;
    const uint32_t even = word & 0x0F0F0F0Fu, odd = (word >> 4) & 0x0F0F0F0Fu;  // values 0 4 1 5 and 2 6 3 7
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = __builtin_fmaf(static_cast<float>(((i & 2 ? odd : even) >> (8 * (i / 4) + 16 * (i & 1))) & 255u), s, zs);
    store_values(static_cast<T*>(a.out) + n * a.ldw, k, a.K, v);
}

// ------------------------------------------------------------------------------ product
struct W4Args {
    const uint16_t* x;
    const uint32_t *w, *up;
    void* y;
    int64_t M, N, K, ldx, ldy, J, meta;
    int32_t bf16;
    float* part;      // K slices: partial sums [slice][plane][M][N], in units of 1/16
    uint32_t slices;  // slice z takes every slices-th turn of the waves
};

// Four MFMA operands of a lane from its 16 bytes: word p holds the codes of operand p, a pair of them in
// the halves of each bf16 pair. 1 + q / 16 in bf16 is 0x3F80 | q << 3: a shift and an and-or per two codes. The and-or takes
// both constants from registers, where the compiler, left to itself, would use literals and two operations.
struct Codes {
    uint32_t mask = 0x00780078u, one = 0x3F803F80u;
    __device__ __forceinline__ Codes() { asm volatile("" : "+v"(mask), "+v"(one)); }
    __device__ __forceinline__ bf16x8 operand(uint32_t w) const
    {
        const u32x4 o = {((w << 3) & mask) | one, ((w >> 1) & mask) | one, ((w >> 5) & mask) | one, ((w >> 9) & mask) | one};
        return __builtin_bit_cast(bf16x8, o);
    }
    // an operand all of whose codes are q
    __device__ __forceinline__ bf16x8 all_of(uint32_t q) const
    {
        const uint32_t two = __umul24(q, 0x00080008u) | one;
        return __builtin_bit_cast(bf16x8, u32x4{two, two, two, two});
    }
};

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

// Sum over k of a tile's values with the codes, by groups, scaled into the accumulators. x[c][p]: operands of X. RES: results of
// a lane that count. OWN: the sums of x are taken for each row of W, with its 1 + z / 16; else with ones, and multiplied by that.
template <int RW, int CT, int PER, int RES, bool OWN>
__device__ __forceinline__ void multiply_tile(const Codes& k, const u32x4 (&x)[CT][4], const u32x4 (&w)[RW], const uint32_t (&meta)[RW][PER], floatx4 (&acc)[RW][CT])
{
    constexpr int P = 4 / PER;  // operands per group
#pragma unroll
    for (int g = 0; g < PER; g++) {
        floatx4 sum[CT];
        auto sums = [&](const bf16x8& b) {
#pragma unroll
            for (int c = 0; c < CT; c++) {
                sum[c] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int p = 0; p < P; p++)
                    sum[c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x[c][g * P + p]), b, sum[c], 0, 0, 0);
            }
        };
        if constexpr (!OWN) sums(k.all_of(0));
#pragma unroll
        for (int i = 0; i < RW; i++) {
            if constexpr (OWN) sums(k.all_of(meta[i][g] & 15u));
            floatx4 d[CT];
#pragma unroll
            for (int c = 0; c < CT; c++) d[c] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int p = 0; p < P; p++) {
                const bf16x8 b = k.operand(w[i][g * P + p]);
#pragma unroll
                for (int c = 0; c < CT; c++) d[c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x[c][g * P + p]), b, d[c], 0, 0, 0);
            }
            const float s = __uint_as_float(meta[i][g] & ~15u), z = OWN ? 1.f : __uint_as_float(0x3F800000u | (meta[i][g] & 15u) << 19);
#pragma unroll
            for (int c = 0; c < CT; c++)
#pragma unroll
                for (int q = 0; q < RES; q++) acc[i][c][q] = __builtin_fmaf(s, __builtin_fmaf(-z, sum[c][q], d[c][q]), acc[i][c][q]);
        }
    }
}

// The pointer in scalar registers, where a transfer's base belongs.
__device__ __forceinline__ const uint8_t* uniform(const void* p)
{
    const uint64_t v = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v)), hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32));
    return reinterpret_cast<const uint8_t*>(static_cast<uint64_t>(hi) << 32 | lo);
}

__device__ __forceinline__ void store_y(const W4Args& a, int64_t m, int64_t n, float v)
{
    if (a.bf16)
        static_cast<uint16_t*>(a.y)[m * a.ldy + n] = static_cast<uint16_t>(f32_to_bf16_rne(v));
    else
        static_cast<float*>(a.y)[m * a.ldy + n] = v;
}

// 16 RT rows of W (with UP: of each of the two planes) x XR rows of X per workgroup, whose NW waves take the K tiles in
// turn and meet in LDS; U tiles of a wave are on the way, W's in registers and X's, sent there by DMA, in LDS that the wave
// has for itself. XR is 16 CT, or 4 or 1 rows, which then stand in the operand's rows 0, 4, 8 and 12 (the rows between
// repeat them), so that a lane's first result is the only one that counts.
// An X tile in LDS: row i's 16-byte chunk c at 256 i + 16 (c ^ i mod 16), so that 16 lanes that read one chunk of 16 rows hit
// all banks. Transfer q covers rows 4 q .. 4 q + 3, lane l landing at 16 l.
// Order: a tile's transfers are issued before its load of W, loads and transfers return in order, so a wait for W (an empty
// asm that uses it) is one for X; reads of a slot are waited for before it is filled again.
// Measured, W from memory (24 matrices in turn) and from the cache behind the L2: M = 1, N = 4096, K = 14336 8.7 and 6.6 us (31 MB, 3.6 and 4.7
// TB/s), gate and up of N = 14336, K = 4096 with the activation 13.6 and 12.5 (62 MB, 4.6 and 5.0); N = 14336, K = 4096 with M = 16 11.3 and 8.6,
// M = 32 12.7 and 10.6, M = 64 18.5 and 16.4, gate and up of it 22.1 and 20.2 with M = 32, 32.4 and 30.5 with M = 64. W's stream bounds it up to 16
// rows, vector operations and matrix cores, one after the other, at 64.
// Planes that have groups of zeros (1% of all, or 48 rows) take the second pass, tile by tile: M = 1 9 -> 10 to 13 us, M = 32 12.7 -> 20, M = 64 18.4 -> 33.
template <int XR, int RT, int U, int NW, bool UP>
struct Skinny {
    static constexpr int RW = UP ? 2 * RT : RT, CT = XR >= 16 ? XR / 16 : 1, RES = XR >= 16 ? 4 : 1;
    static constexpr int SLOT = XR * 256, RING = NW * U * SLOT, RED = NW * RW * CT * RES * 64 * 4;
    static constexpr int LDS = RING > RED ? RING : RED, SENDS = XR >= 16 ? XR / 4 : 1;
};

template <int XR, int RT, int U, int NW, int PER, bool UP>
// (16 rows with two groups a tile: held to the registers of two workgroups per CU, which it would miss by two)
__global__ void __launch_bounds__(64 * NW, (XR == 16 && PER == 2 ? 4 : 1)) w4_skinny(W4Args a)
{
    typedef Skinny<XR, RT, U, NW, UP> C;
    constexpr int RW = C::RW, CT = C::CT, RES = C::RES, SLOT = C::SLOT;
    extern __shared__ __align__(16) uint8_t lds[];
    const int lane = threadIdx.x & 63, r = lane & 15, c4 = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t T = static_cast<uint32_t>(tiles16(a.N)), J = static_cast<uint32_t>(a.J);
    const uint32_t tiles_n = (T + RT - 1) / RT;
    const uint32_t t0 = blockIdx.x % tiles_n * RT;
    const int64_t m0 = static_cast<int64_t>(blockIdx.x / tiles_n) * XR;
    const int rows = a.M - m0 < XR ? static_cast<int>(a.M - m0) : XR;  // rows past M repeat the last one

    const uint32_t *wp[RW], *sp[RW];
#pragma unroll
    for (int i = 0; i < RW; i++) {
        const uint32_t* plane = UP && i >= RT ? a.up : a.w;
        const uint32_t t = t0 + i % RT < T ? t0 + i % RT : T - 1;
        wp[i] = plane + static_cast<int64_t>(t) * J * 256;
        sp[i] = plane + a.meta + static_cast<int64_t>(t) * J * PER * 16;
    }
    const uint16_t* x0 = a.x + m0 * a.ldx;
    const Codes k;
    const uint8_t* xbase = uniform(x0);
    const uint32_t ring = lds_offset(lds) + static_cast<uint32_t>(wave * U * SLOT);
    // what a lane sends: one row's chunk per transfer, or with one row a dword of it
    uint32_t xoff[C::SENDS];
#pragma unroll
    for (int q = 0; q < C::SENDS; q++) {
        const int i = 4 * q + (lane >> 4), row = i < rows ? i : rows - 1;
        xoff[q] = XR == 1 ? 4 * lane : static_cast<uint32_t>(row * a.ldx * 2) + 16 * ((lane & 15) ^ (i & 15));
    }
    // and reads: row r's chunk 4 p + c4 (of the first 16 rows; the others lie 4096 bytes apart)
    const int xrow = XR >= 16 ? r : XR == 4 ? r >> 2 : 0;
    uint32_t rd[4];
#pragma unroll
    for (int p = 0; p < 4; p++) rd[p] = 256 * xrow + 16 * ((4 * p + c4) ^ xrow);
    const uint8_t* mine = lds + wave * U * SLOT;

    floatx4 acc[RW][CT];
    auto clear = [&]() {
#pragma unroll
        for (int i = 0; i < RW; i++)
#pragma unroll
            for (int c = 0; c < CT; c++) acc[i][c] = floatx4{0.f, 0.f, 0.f, 0.f};
    };
    clear();
    u32x4 wv[U][RW];
    uint32_t sv[U][RW][PER];
    uint64_t alike = 0;  // lanes that met a word of eight like codes other than 0 (of zero point 0, or of a row past N)
    auto load_w = [&](int u, uint32_t j) {
#pragma unroll
        for (int i = 0; i < RW; i++) {
            wv[u][i] = *reinterpret_cast<const u32x4*>(wp[i] + static_cast<int64_t>(j) * 256 + 4 * lane);
#pragma unroll
            for (int g = 0; g < PER; g++) sv[u][i][g] = sp[i][(j * PER + g) * 16 + r];
        }
    };
    auto issue = [&](int u, uint32_t j) {
        if constexpr (XR == 1)
            dma4(xbase, xoff[0] + 256 * j, ring + u * SLOT);
        else
#pragma unroll
            for (int q = 0; q < C::SENDS; q++) dma16(xbase, xoff[q] + 256 * j, ring + u * SLOT + q * 1024);
        load_w(u, j);
    };
    auto step = [&](int u) {
        asm volatile("" : "+v"(wv[u][0])::"memory");  // W has come, and with it X
        u32x4 x[CT][4];
#pragma unroll
        for (int c = 0; c < CT; c++)
#pragma unroll
            for (int p = 0; p < 4; p++) x[c][p] = *reinterpret_cast<const u32x4*>(mine + u * SLOT + c * 4096 + rd[p]);
#pragma unroll
        for (int i = 0; i < RW; i++)
#pragma unroll
            for (int g = 0; g < PER; g++) {
                const uint32_t w = wv[u][i][g * (4 / PER)];
                alike |= __ballot(w == __builtin_amdgcn_alignbit(w, w, 4)) & __ballot(w != 0);
            }
        multiply_tile<RW, CT, PER, RES, false>(k, x, wv[u], sv[u], acc);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    };
    const uint32_t full = static_cast<uint32_t>(a.K / 128);
    // tiles first, first + stride, ...: the waves of all slices take neighbouring ones
    const uint32_t first = blockIdx.z * NW + wave, stride = NW * a.slices;
    const uint32_t count = full > first ? (full - first + stride - 1) / stride : 0;
    uint32_t slow = count;
    if (count > 0) {
        auto tile = [&](uint32_t i) { return first + stride * (i < count ? i : count - 1); };
#pragma unroll
        for (int u = 0; u < U; u++) issue(u, tile(u));
        uint32_t done = 0;
        for (; done + U < count; done += U)
#pragma unroll
            for (int u = 0; u < U; u++) {
                step(u);
                issue(u, tile(done + U + u));
            }
#pragma unroll
        for (int u = 0; u < U; u++)
            if (done + u < count) step(u);
        // A row whose four lanes (r, 16 + r, 32 + r, 48 + r) have all met like codes may have a group of zeros: from the beginning, with sums of
        // each row's own.
        const uint64_t half = alike & alike >> 32;
        if (__builtin_expect((half & half >> 16 & 0xFFFFu) != 0, 0)) {
            slow = 0;
            clear();
        }
    }
    // What is left: the tile that K ends inside, whose codes past K are 0 whatever the zero point.
    const uint32_t left = J > full && full % stride == first ? count + 1 : count;
    for (; slow < left; slow++) {
        const uint32_t j = first + stride * slow;
        load_w(0, j);
        u32x4 x[CT][4];
#pragma unroll
        for (int c = 0; c < CT; c++)
#pragma unroll
            for (int p = 0; p < 4; p++) {
                const int row = 16 * c + xrow < rows ? 16 * c + xrow : rows - 1;
                x[c][p] = load_x(x0 + static_cast<int64_t>(row) * a.ldx, static_cast<int64_t>(j) * 128 + 32 * p + 8 * c4, a.K);
            }
        multiply_tile<RW, CT, PER, RES, true>(k, x, wv[0], sv[0], acc);
    }
    // every transfer has landed before the ring becomes the waves' meeting place
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    float* red = reinterpret_cast<float*>(lds);
#pragma unroll
    for (int i = 0; i < RW; i++)
#pragma unroll
        for (int c = 0; c < CT; c++)
#pragma unroll
            for (int q = 0; q < RES; q++) red[(((wave * RW + i) * CT + c) * RES + q) * 64 + lane] = acc[i][c][q];
    __syncthreads();
    for (int e = threadIdx.x; e < RT * CT * RES * 64; e += 64 * NW) {
        const int l = e & 63, q = (e >> 6) % RES, c = (e >> 6) / RES % CT, i = (e >> 6) / (RES * CT);
        const int64_t n = 16 * (static_cast<int64_t>(t0) + i) + (l & 15);
        const int row = XR >= 16 ? 16 * c + 4 * (l >> 4) + q : l >> 4;
        if (n >= a.N || row >= rows) continue;
        float v = 0.f, u = 0.f;
#pragma unroll
        for (int w = 0; w < NW; w++) {
            v += red[(((w * RW + i) * CT + c) * RES + q) * 64 + l];
            if constexpr (UP) u += red[(((w * RW + RT + i) * CT + c) * RES + q) * 64 + l];
        }
        if (a.part) {
            float* part = a.part + (blockIdx.z * (UP ? 2 : 1) * a.M + m0 + row) * a.N + n;
            part[0] = v;
            if constexpr (UP) part[a.M * a.N] = u;
        } else {
            store_y(a, m0 + row, n, UP ? silu_mul(16.f * v, 16.f * u) : 16.f * v);
        }
    }
}

// Sum of the K slices' partial results, in slice order.
template <bool UP>
__global__ void __launch_bounds__(256) w4_join(W4Args a)
{
    const int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, mn = a.M * a.N;
    if (e >= mn) return;
    float v = 0.f, u = 0.f;
    for (uint32_t z = 0; z < a.slices; z++) {
        v += a.part[z * (UP ? 2 : 1) * mn + e];
        if constexpr (UP) u += a.part[(2 * z + 1) * mn + e];
    }
    store_y(a, e / a.N, e % a.N, UP ? silu_mul(16.f * v, 16.f * u) : 16.f * v);
}

template <int XR, int RT, int U, int NW, int PER, bool UP>
hipError_t launch_skinny(const W4Args& a, uint32_t blocks, hipStream_t s)
{
    constexpr size_t lds = Skinny<XR, RT, U, NW, UP>::LDS;
    static_assert(lds <= 160 * 1024, "LDS");
    static uint64_t attr_done = 0;  // devices the LDS limit was raised on
    const auto fn = w4_skinny<XR, RT, U, NW, PER, UP>;
    const hipError_t e = allow_lds(reinterpret_cast<const void*>(fn), lds, attr_done);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(fn, dim3(blocks, 1, a.slices), dim3(64 * NW), lds, s, a);
    return hipGetLastError();
}

template <int XR, int RT, int U, int NW, bool UP>
hipError_t launch_skinny(const W4Args& a, int32_t group, hipStream_t s)
{
    const uint32_t blocks = static_cast<uint32_t>(((tiles16(a.N) + RT - 1) / RT) * ((a.M + XR - 1) / XR));
    return group == 128  ? launch_skinny<XR, RT, U, NW, 1, UP>(a, blocks, s)
           : group == 64 ? launch_skinny<XR, RT, U, NW, 2, UP>(a, blocks, s)
                         : launch_skinny<XR, RT, U, NW, 4, UP>(a, blocks, s);
}

// Row tiles per workgroup and K slices of a product with more than four rows.
//   (Figures of the kernels before they looked for groups of zeros, which takes 2 to 3% but at M = 32, 7% less.)
//   Row tiles: more of them read X less often, and leave fewer workgroups. In us, W from memory, at K = 4096 (2000 for N = 5003), N = 4096 /
//   5003 / 14336 with 1, 2 and 4 row tiles: M = 16 4.9 5.8 7.2 / 5.5 5.0 6.2 / 14.4 10.9 10.1, M = 32 6.0 7.1 9.9 / 7.3 6.3 7.7 /
//   20.3 14.9 12.9, M = 64 9.6 10.1 13.7 / 14.8 9.4 11.9 / 35.9 23.6 17.9. So four where that leaves 192 workgroups or
//   more, else two where that leaves 144.
//   Slices: past 16 rows X's bytes, read once per row tile, are what a long K costs, so where four row tiles leave few
//   workgroups, K is cut among them as long as every wave of eight keeps three tiles: M = 64, N = 4096, K = 14336 takes 22.5 us
//   in four slices, 30.9 with one row tile per workgroup and none; M = 32 16.9 and 19.6. (At K = 4096 12.8 and 9.6.)
struct W4Plan {
    int rt;
    uint32_t slices;
};

W4Plan w4_plan(int64_t M, int64_t N, int64_t K, bool up)
{
    const int64_t T = tiles16(N), mb = (M + 63) / 64;
    const int64_t four = (T * (up ? 2 : 1) + 3) / 4 * mb, two = (T * (up ? 2 : 1) + 1) / 2 * mb;
    if (four >= 192) return {4, 1};
    if (M > 16 && four <= 128) {
        int64_t s = 256 / four, most = tiles128(K) / 24;
        s = s < most ? s : most;
        if (s > 1) return {4, static_cast<uint32_t>(s < 8 ? s : 8)};
    }
    return {two >= 144 ? 2 : 1, 1};
}

// Bytes of the slices' partial sums.
size_t w4_part_bytes(int64_t M, int64_t N, bool up, uint32_t slices)
{
    return slices > 1 ? static_cast<size_t>(slices) * (up ? 2 : 1) * M * N * sizeof(float) : 0;
}

template <int XR, int U, bool UP>
hipError_t launch_planned(const W4Args& a, int rt, int32_t group, hipStream_t s)
{
    // (of each of two planes with UP, where two row tiles of one plane are the least)
    if (rt == 4) return launch_skinny<XR, UP ? 2 : 4, U, 8, UP>(a, group, s);
    if (!UP && rt == 2) return launch_skinny<XR, UP ? 1 : 2, U, 8, UP>(a, group, s);
    return launch_skinny<XR, 1, U, 8, UP>(a, group, s);
}

template <bool UP>
uw_status run_product(W4Args a, int32_t group, void* d_ws, size_t ws_bytes, hipStream_t s)
{
    hipError_t e;
    if (tiles16(a.N) * ((a.M + 15) / 16) > kThreadsMost / 1024) return fail(UW_EUNSUPPORTED, "M x N too large for one launch");
    if (a.M <= 4) {
        // One row tile per workgroup; with few of those the CU is filled with waves instead. In us, W from memory, with 8 and 16 waves: M = 1,
        // 4096 x 14336 (N x K) 9.7 and 8.5, 14336 x 4096 8.5 and 9.4, gate and up of that 13.6 and 17.2.
        const bool wide = tiles16(a.N) < 512;
        if (a.M == 1)
            e = wide ? launch_skinny<1, 1, 2, 16, UP>(a, group, s) : launch_skinny<1, 1, 2, 8, UP>(a, group, s);
        else
            e = wide ? launch_skinny<4, 1, 2, 16, UP>(a, group, s) : launch_skinny<4, 1, 2, 8, UP>(a, group, s);
    } else {
        const W4Plan p = w4_plan(a.M, a.N, a.K, UP);
        int rt = p.rt;
        a.slices = p.slices;
        while (a.slices > 1 && (!d_ws || w4_part_bytes(a.M, a.N, UP, a.slices) > ws_bytes)) a.slices--;
        if (p.slices > 1 && a.slices == 1) rt = 1;
        a.part = a.slices > 1 ? static_cast<float*>(d_ws) : nullptr;
        if (a.M <= 16)
            e = launch_planned<16, 2, UP>(a, rt, group, s);
        else if (a.M <= 32)
            e = launch_planned<32, 1, UP>(a, rt, group, s);
        else
            e = launch_planned<64, 1, UP>(a, rt, group, s);
        if (e == hipSuccess && a.slices > 1) {
            hipLaunchKernelGGL(w4_join<UP>, dim3(static_cast<uint32_t>((a.M * a.N + 255) / 256)), dim3(256), 0, s, a);
            e = hipGetLastError();
        }
    }
    return e == hipSuccess ? UW_OK : fail(UW_EHIP, "4-bit product launch failed: %s", hipGetErrorString(e));
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

template <class T, int GROUP, bool ZEROS>
void launch_quantize(const PlaneArgs& a, hipStream_t s)
{
    const int64_t T16 = tiles16(a.N);
    if (T16 * a.J >= 8192)
        hipLaunchKernelGGL((w4_quantize_kernel<T, GROUP, ZEROS, 4>), dim3(static_cast<uint32_t>(T16 * ((a.J + 3) / 4))), dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((w4_quantize_kernel<T, GROUP, ZEROS, 1>), dim3(static_cast<uint32_t>(T16 * a.J)), dim3(256), 0, s, a);
}
template <class T, int GROUP>
void launch_quantize(const PlaneArgs& a, bool zeros, hipStream_t s)
{
    zeros ? launch_quantize<T, GROUP, true>(a, s) : launch_quantize<T, GROUP, false>(a, s);
}
template <class T>
void launch_quantize(const PlaneArgs& a, int32_t group, bool zeros, hipStream_t s)
{
    group == 128 ? launch_quantize<T, 128>(a, zeros, s) : group == 64 ? launch_quantize<T, 64>(a, zeros, s) : launch_quantize<T, 32>(a, zeros, s);
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
    if (p->ldx > kMostLd) return fail(UW_EUNSUPPORTED, "ldx over 2^25");
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
    a.slices = 1;
    hipStream_t s = static_cast<hipStream_t>(stream);
    return up ? run_product<true>(a, p->group, p->d_ws, p->ws_bytes, s) : run_product<false>(a, p->group, p->d_ws, p->ws_bytes, s);
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
    if (M < 5 || M > INT32_MAX || check_plane(N, K, 128) != UW_OK) return 0;
    return w4_part_bytes(M, N, false, w4_plan(M, N, K, false).slices);
}
