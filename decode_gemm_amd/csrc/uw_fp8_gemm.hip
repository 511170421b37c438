// The 8-bit block-scaled GEMM: Y[M][N] = X[M][K] W[N][K]^T from e4m3 codes, X with one fp32
// scale per row and 128 values of K, W with one per 128 x 128 block.
//
// Mathematics. A scale group is 128 values of K. Its sum comes out of the matrix unit and is
// then added into the fp32 accumulator times sx * sw, four fmas per lane and 16 x 16 tile. W is
// the A operand (D's four registers run along n, inside one 128 block, where the scale is one
// number) and X the B operand (D's column, the lane's low four bits, is the row m): the
// product of scales is one number per lane and tile column, shared by all W tiles of a wave.
// Within an MFMA the assignment of k to (lane group, slot) only has to agree between A and B:
// lane group g takes the 16-byte chunks g and 4 + g of each operand row's 128 bytes.
//
// The group sum is taken in one of two ways. v_mfma_f32_16x16x128_f8f6f4 reads the codes as they
// are, at twice the bf16 rate, but lines its products up to the largest and drops the low bits
// of the others: measured against 64 bits, group sums of Gaussian operands are off by 1.3e-5 of
// their norm, and by up to 2^-11.4 of the group's largest product with codes of all sizes.
// That is below the 2^-9 of a bf16 output, and far above fp32's 2^-24. So fp32 outputs convert
// the codes to bf16 (exact, in registers, two to an instruction) for v_mfma_f32_16x16x32_bf16, whose sums of
// the same operands are off by 1.4e-8.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "uw_internal.h"
#include "uw_recon.h"
#include "uw_tiles.h"

namespace uw {

namespace {

typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef int intx8 __attribute__((ext_vector_type(8)));

constexpr int kG = UW_FP8_GROUP;

struct F8Args {
    const uint8_t* x;
    const float* sx;
    const uint8_t* w;
    const float* sw;
    void* y;
    int64_t M, N, K, ldx, ldsx, ldw, ldsw, ldy;
    int32_t bf16;     // Y is bf16
    float* part;      // K slices: partial sums [slice][M][N4], N4 = N rounded up to 4
    int64_t N4;
    uint32_t slice;   // groups per K slice
};

// 32 bytes of an operand row (the lane's chunks of one group).
struct F8 {
    u32x4 a, b;
};

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// The same as bf16, in the four operand pieces of a 16x16x32 MFMA each.
struct B16 {
    u32x4 p[4];
};

__device__ __forceinline__ uint32_t two_bf16(uint32_t codes, bool high)
{
    const bf16x2 v = high ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, 1.0f, true)
                          : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, 1.0f, false);
    return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ B16 to_bf16(const F8& f)
{
    B16 o;
#pragma unroll
    for (int h = 0; h < 4; h++) {
        const uint32_t c0 = h < 2 ? f.a[2 * h] : f.b[2 * h - 4], c1 = h < 2 ? f.a[2 * h + 1] : f.b[2 * h - 3];
        o.p[h] = u32x4{two_bf16(c0, false), two_bf16(c0, true), two_bf16(c1, false), two_bf16(c1, true)};
    }
    return o;
}

__device__ __forceinline__ floatx4 group_sum(const B16& a, const B16& b)
{
    floatx4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int h = 0; h < 4; h++)
        d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a.p[h]), __builtin_bit_cast(bf16x8, b.p[h]), d, 0, 0, 0);
    return d;
}

__device__ __forceinline__ floatx4 group_sum(const F8& a, const F8& b)
{
    const intx8 av = {(int)a.a.x, (int)a.a.y, (int)a.a.z, (int)a.a.w, (int)a.b.x, (int)a.b.y, (int)a.b.z, (int)a.b.w};
    const intx8 bv = {(int)b.a.x, (int)b.a.y, (int)b.a.z, (int)b.a.w, (int)b.b.x, (int)b.b.y, (int)b.b.z, (int)b.b.w};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, floatx4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}

template <bool EXACT>
struct Operand {
    typedef F8 type;
};
template <>
struct Operand<true> {
    typedef B16 type;
};
template <bool EXACT>
__device__ __forceinline__ typename Operand<EXACT>::type operand(const F8& f)
{
    if constexpr (EXACT)
        return to_bf16(f);
    else
        return f;
}

// A 16-byte chunk of which the first `left` bytes belong to the row: the others become 0.
__device__ __forceinline__ u32x4 cut(u32x4 v, int left)
{
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int keep = left < 4 * i ? 0 : left > 4 * i + 4 ? 4 : left - 4 * i;
        v[i] &= static_cast<uint32_t>((uint64_t{1} << (8 * keep)) - 1);
    }
    return v;
}

// The same of the chunk at p; one with nothing of the row is not read.
__device__ __forceinline__ u32x4 chunk_cut(const uint8_t* p, int left)
{
    if (left <= 0) return u32x4{0, 0, 0, 0};
    return cut(*reinterpret_cast<const u32x4*>(p), left);
}

// Y[m][n .. n+3] (those inside), or the K slice's partial sums.
__device__ __forceinline__ void store4(const F8Args& a, int64_t m, int64_t n, const floatx4& v)
{
    if (m >= a.M || n >= a.N) return;
    if (a.part) {
        *reinterpret_cast<floatx4*>(a.part + (static_cast<int64_t>(blockIdx.z) * a.M + m) * a.N4 + n) = v;
        return;
    }
    const bool vec = n + 3 < a.N && (a.ldy & 3) == 0;
    if (a.bf16) {
        uint16_t* y = static_cast<uint16_t*>(a.y) + m * a.ldy + n;
        uint32_t o[4];
#pragma unroll
        for (int q = 0; q < 4; q++) o[q] = f32_to_bf16_rne(v[q]);
        if (vec) {
            *reinterpret_cast<uint2*>(y) = make_uint2(o[0] | (o[1] << 16), o[2] | (o[3] << 16));
        } else {
            for (int q = 0; q < 4; q++)
                if (n + q < a.N) y[q] = static_cast<uint16_t>(o[q]);
        }
    } else {
        float* y = static_cast<float*>(a.y) + m * a.ldy + n;
        if (vec) {
            *reinterpret_cast<floatx4*>(y) = v;
        } else {
            for (int q = 0; q < 4; q++)
                if (n + q < a.N) y[q] = v[q];
        }
    }
}

// ------------------------------------------------------------------------- skinny
// Few rows of X: 16 RT rows of W x 16 CT rows of X per workgroup, whose NW waves take the
// groups j = wave (mod NW) of the K slice and meet in LDS. Each wave keeps U groups of both
// operands in flight in registers. Bound by HBM (W once), so it takes the exact sums always.
template <int CT, int RT, int U, int NW>
__global__ void __launch_bounds__(64 * NW) fp8_skinny(F8Args a)
{
    __shared__ floatx4 red[NW][RT * CT][64];
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t tiles_n = static_cast<uint32_t>((a.N + 16 * RT - 1) / (16 * RT));
    const int64_t n0 = static_cast<int64_t>(blockIdx.x % tiles_n) * (16 * RT);
    const int64_t m0 = static_cast<int64_t>(blockIdx.x / tiles_n) * (16 * CT);
    const uint32_t full = static_cast<uint32_t>(a.K / kG), G = static_cast<uint32_t>((a.K + kG - 1) / kG);
    const uint32_t j0 = blockIdx.z * a.slice, j1 = j0 + a.slice < G ? j0 + a.slice : G;
    const uint32_t f1 = j1 < full ? j1 : full;  // whole groups of this slice end here

    const uint8_t* wp[RT];
    const uint8_t* xp[CT];
    const float* sxp[CT];
#pragma unroll
    for (int i = 0; i < RT; i++) {
        const int64_t n = n0 + 16 * i + r;
        wp[i] = a.w + (n < a.N ? n : a.N - 1) * a.ldw + 16 * g;
    }
#pragma unroll
    for (int c = 0; c < CT; c++) {
        const int64_t m = m0 + 16 * c + r, mm = m < a.M ? m : a.M - 1;
        xp[c] = a.x + mm * a.ldx + 16 * g;
        sxp[c] = a.sx + mm;
    }
    const float* swp = a.sw + n0 / kG * a.ldsw;

    floatx4 acc[RT][CT];
#pragma unroll
    for (int i = 0; i < RT; i++)
#pragma unroll
        for (int c = 0; c < CT; c++) acc[i][c] = floatx4{0.f, 0.f, 0.f, 0.f};

    F8 wv[U][RT], xv[U][CT];
    float sv[U][CT], tv[U];
    auto load = [&](int u, uint32_t j) {
        const int64_t o = static_cast<int64_t>(j) * kG;
#pragma unroll
        for (int i = 0; i < RT; i++) {
            wv[u][i].a = *reinterpret_cast<const u32x4*>(wp[i] + o);
            wv[u][i].b = *reinterpret_cast<const u32x4*>(wp[i] + o + 64);
        }
#pragma unroll
        for (int c = 0; c < CT; c++) {
            xv[u][c].a = *reinterpret_cast<const u32x4*>(xp[c] + o);
            xv[u][c].b = *reinterpret_cast<const u32x4*>(xp[c] + o + 64);
            sv[u][c] = sxp[c][j * a.ldsx];
        }
        tv[u] = swp[j];
    };
    auto multiply = [&](int u) {
        B16 wb[RT];
#pragma unroll
        for (int i = 0; i < RT; i++) wb[i] = to_bf16(wv[u][i]);
#pragma unroll
        for (int c = 0; c < CT; c++) {
            const float s = sv[u][c] * tv[u];
            const B16 xb = to_bf16(xv[u][c]);
#pragma unroll
            for (int i = 0; i < RT; i++) {
                const floatx4 d = group_sum(wb[i], xb);
#pragma unroll
                for (int q = 0; q < 4; q++) acc[i][c][q] = __builtin_fmaf(d[q], s, acc[i][c][q]);
            }
        }
    };
    if (j0 + wave < f1) {
        const uint32_t last = f1 - 1;
#pragma unroll
        for (int u = 0; u < U; u++) {
            const uint32_t j = j0 + wave + u * NW;
            load(u, j < last ? j : last);
        }
        for (uint32_t j = j0 + wave; j < f1; j += U * NW)
#pragma unroll
            for (int u = 0; u < U; u++) {
                if (j + u * NW < f1) multiply(u);
                const uint32_t next = j + (u + U) * NW;
                load(u, next < last ? next : last);
            }
    }
    if (j1 > full && j0 <= full && wave == static_cast<int>((full - j0) % NW)) {  // the group that K ends inside
        const int rest = static_cast<int>(a.K % kG);
        const int64_t o = static_cast<int64_t>(full) * kG;
#pragma unroll
        for (int i = 0; i < RT; i++) {
            wv[0][i].a = chunk_cut(wp[i] + o, rest - 16 * g);
            wv[0][i].b = chunk_cut(wp[i] + o + 64, rest - 16 * g - 64);
        }
#pragma unroll
        for (int c = 0; c < CT; c++) {
            xv[0][c].a = chunk_cut(xp[c] + o, rest - 16 * g);
            xv[0][c].b = chunk_cut(xp[c] + o + 64, rest - 16 * g - 64);
            sv[0][c] = sxp[c][full * a.ldsx];
        }
        tv[0] = swp[full];
        multiply(0);
    }
#pragma unroll
    for (int i = 0; i < RT; i++)
#pragma unroll
        for (int c = 0; c < CT; c++) red[wave][i * CT + c][lane] = acc[i][c];
    __syncthreads();
    for (int e = threadIdx.x; e < RT * CT * 64; e += 64 * NW) {
        const int t = e >> 6, l = e & 63;
        floatx4 s = red[0][t][l];
#pragma unroll
        for (int v = 1; v < NW; v++) s += red[v][t][l];
        store4(a, m0 + 16 * (t % CT) + (l & 15), n0 + 16 * (t / CT) + 4 * (l >> 4), s);
    }
}

// -------------------------------------------------------------------------- tiles
// A BN x BM output tile per workgroup of WN x WM waves, K in steps of one scale group, both
// operands and the scales sent from global memory straight into LDS (DMA) through NST stages.
//
// LDS layout of an operand in a stage: row rho at 128 rho, its 16-byte chunk c at slot
// c ^ ((rho >> 1) & 7). A transfer covers 1 KB, lane l landing at 16 l: row 8 i + l / 8, slot
// l mod 8, so it fetches chunk (l mod 8) ^ ((rho >> 1) & 7); the eight lanes of a row read its
// whole 128-byte segment. A fragment read (lane 16 g + r: row 16 t + r, chunks g and 4 + g) hits
// 16 distinct 16-byte bank groups in every 16 lanes.
//
// One barrier per step: behind it the step's transfers have landed (each wave waits for its own
// before it) and every wave is done with the step before, whose stage takes the step NST - 1 ahead.
__device__ __forceinline__ void dma4(const void* base, uint32_t voff, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dword %1, %2" ::"s"(__builtin_amdgcn_readfirstlane(lds)), "v"(voff), "s"(base)
                 : "memory");
}

template <int BN, int BM>
constexpr int stage_bytes()
{
    return (BN + BM) * 128 + (BM < 64 ? 64 : BM) * 4 + BN / 128 * 256;
}

template <int BN, int BM, int WN, int WM, int NST, bool EXACT>
__global__ void __launch_bounds__(64 * WN * WM) fp8_tile(F8Args a)
{
    constexpr int NW = WN * WM, TN = BN / 16 / WN, TM = BM / 16 / WM;
    constexpr int OPW = BN * 128, OPX = BM * 128, SEG = BM < 64 ? 1 : BM / 64;
    constexpr int STAGE = stage_bytes<BN, BM>();
    constexpr int NLW = BN / 8 / NW, NLX = BM / 8 / NW;
    constexpr int NL = NLW + NLX + 2;  // transfers per wave and step
    static_assert(BN % 128 == 0 && 16 * TN <= 128 && 128 % (16 * TN) == 0 && NLX >= 1 && SEG <= NW, "tile shape");
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];

    const uint32_t tiles_n = static_cast<uint32_t>((a.N + BN - 1) / BN), tiles_m = static_cast<uint32_t>((a.M + BM - 1) / BM);
    uint32_t tn, tm;
    tile_of_block(blockIdx.x, gridDim.x, tiles_n, tiles_m, tn, tm);
    const int64_t n0 = static_cast<int64_t>(tn) * BN, m0 = static_cast<int64_t>(tm) * BM;
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wn = wave / WM, wm = wave % WM;
    const uint32_t G = static_cast<uint32_t>((a.K + kG - 1) / kG);
    const uint32_t j0 = blockIdx.z * a.slice, j1 = j0 + a.slice < G ? j0 + a.slice : G;
    const int rest = static_cast<int>(a.K % kG);  // the last group's values, 0 = all

    // per-lane byte offsets of this wave's transfers from the tile's first row (rows past N or M
    // read the last row; 256 rows of less than 2^24 bytes stay below 2^32)
    uint32_t woff[NLW], xoff[NLX], soff;
    const int slot = lane & 7;
#pragma unroll
    for (int q = 0; q < NLW; q++) {
        const int rho = 8 * (NLW * wave + q) + (lane >> 3);
        const int64_t n = n0 + rho < a.N ? rho : a.N - 1 - n0;
        woff[q] = static_cast<uint32_t>(n * a.ldw) + 16 * (slot ^ ((rho >> 1) & 7));
    }
#pragma unroll
    for (int q = 0; q < NLX; q++) {
        const int rho = 8 * (NLX * wave + q) + (lane >> 3);
        const int64_t m = m0 + rho < a.M ? rho : a.M - 1 - m0;
        xoff[q] = static_cast<uint32_t>(m * a.ldx) + 16 * (slot ^ ((rho >> 1) & 7));
    }
    {
        const int m = 64 * (wave % SEG) + lane;
        soff = 4 * static_cast<uint32_t>(m0 + m < a.M ? m : a.M - 1 - m0);
    }
    const uint32_t lds0 = lds_offset(lds);
    const uint8_t* const wbase = a.w + n0 * a.ldw;
    const uint8_t* const xbase = a.x + m0 * a.ldx;
    const float* const sxbase = a.sx + m0;
    const int nb = wn * (16 * TN) / 128;  // this wave's 128 block of the tile
    const int64_t nblk = n0 / 128 + nb;
    const float* const swbase = a.sw + (nblk < (a.N + 127) / 128 ? nblk : (a.N - 1) / 128) * a.ldsw;
    // A short last group is read as the 128 bytes that end at K rounded up to 16, so that nothing behind
    // a row is read (K >= 128); the bytes before its start and past K are cut to zero at use.
    const int64_t last = (a.K + 15) / 16 * 16 - kG;
    auto issue = [&](uint32_t j, int st) {
        const int64_t k = rest && j + 1 == G ? last : static_cast<int64_t>(j) * kG;
        const uint8_t* wb = wbase + k;
        const uint8_t* xb = xbase + k;
        const uint32_t dst = lds0 + st * STAGE;
#pragma unroll
        for (int q = 0; q < NLW; q++) dma16(wb, woff[q], dst + 1024 * (NLW * wave + q));
#pragma unroll
        for (int q = 0; q < NLX; q++) dma16(xb, xoff[q], dst + OPW + 1024 * (NLX * wave + q));
        dma4(sxbase + static_cast<int64_t>(j) * a.ldsx, soff, dst + OPW + OPX + 256 * (wave % SEG));
        dma4(swbase + j, 0, dst + OPW + OPX + 256 * (SEG + nb));
    };

    const int fo0 = 128 * r + 16 * (g ^ ((r >> 1) & 7)), fo1 = 128 * r + 16 * ((4 + g) ^ ((r >> 1) & 7));
    auto frag = [&](const uint8_t* p, bool tail) {
        F8 f;
        f.a = *reinterpret_cast<const u32x4*>(p + fo0);
        f.b = *reinterpret_cast<const u32x4*>(p + fo1);
        if (tail) {
            const int from = kG - (rest + 15) / 16 * 16, to = from + rest;  // the group's bytes of the 128
            f.a = cut(f.a, 16 * g < from ? 0 : to - 16 * g);
            f.b = cut(f.b, 16 * g + 64 < from ? 0 : to - 16 * g - 64);
        }
        return f;
    };

    floatx4 acc[TN][TM];
#pragma unroll
    for (int i = 0; i < TN; i++)
#pragma unroll
        for (int c = 0; c < TM; c++) acc[i][c] = floatx4{0.f, 0.f, 0.f, 0.f};

    auto step = [&](const uint8_t* S, auto tail) {
        using Op = typename Operand<EXACT>::type;
        const uint8_t* const W = S + 2048 * TN * wn;
        const uint8_t* const X = S + OPW + 2048 * TM * wm;
        const float* const sx = reinterpret_cast<const float*>(S + OPW + OPX) + 16 * TM * wm + r;
        const float sw = *reinterpret_cast<const float*>(S + OPW + OPX + 256 * (SEG + nb));
        Op bf[TM];
        float s[TM];
#pragma unroll
        for (int c = 0; c < TM; c++) {
            bf[c] = operand<EXACT>(frag(X + 2048 * c, tail));
            s[c] = sx[16 * c] * sw;
        }
        F8 an = frag(W, tail);
#pragma unroll
        for (int i = 0; i < TN; i++) {
            const Op ac = operand<EXACT>(an);
            if (i + 1 < TN) an = frag(W + 2048 * (i + 1), tail);
#pragma unroll
            for (int c = 0; c < TM; c++) {
                const floatx4 d = group_sum(ac, bf[c]);
#pragma unroll
                for (int q = 0; q < 4; q++) acc[i][c][q] = __builtin_fmaf(d[q], s[c], acc[i][c][q]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };

#pragma unroll
    for (int p = 0; p < NST - 1; p++)
        if (j0 + p < j1) issue(j0 + p, p);
    int st = 0, sn = NST - 1;  // stages of this step and of the one NST - 1 ahead
    auto arrive = [&](uint32_t j) {
        // this wave's transfers of step j have landed when only those of the NST - 2 younger steps
        // may be left
        if (NST > 2 && j + NST - 2 < j1) {
            constexpr int younger = (NST > 2 ? NST - 2 : 0) * NL;
            static_assert(younger < 64, "wait counter");
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"(younger) : "memory");
        } else {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        }
        __syncthreads();
    };
    const bool tail = rest && j1 == G;
    const uint32_t jf = tail ? j1 - 1 : j1;
    for (uint32_t j = j0; j < jf; j++) {
        arrive(j);
        if (j + NST - 1 < j1) issue(j + NST - 1, sn);
        step(lds + st * STAGE, std::false_type{});
        st = st + 1 < NST ? st + 1 : 0;
        sn = sn + 1 < NST ? sn + 1 : 0;
    }
    if (tail) {
        arrive(jf);
        step(lds + st * STAGE, std::true_type{});
    }
#pragma unroll
    for (int i = 0; i < TN; i++)
#pragma unroll
        for (int c = 0; c < TM; c++)
            store4(a, m0 + 16 * (TM * wm + c) + r, n0 + 16 * (TN * wn + i) + 4 * g, acc[i][c]);
}

// Sum of the K slices' partial results, in slice order.
__global__ void __launch_bounds__(256) fp8_join(F8Args a, const float* part, uint32_t slices)
{
    const int64_t q = a.N4 / 4, e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (e >= a.M * q) return;
    const float* p = part + 4 * e;
    floatx4 s = *reinterpret_cast<const floatx4*>(p);
    for (uint32_t z = 1; z < slices; z++) s += *reinterpret_cast<const floatx4*>(p + z * a.M * a.N4);
    store4(a, e / q, 4 * (e % q), s);
}

template <int CT, int RT, int U, int NW>
hipError_t launch_skinny(const F8Args& a, uint32_t slices, hipStream_t s)
{
    const dim3 grid(static_cast<uint32_t>(((a.N + 16 * RT - 1) / (16 * RT)) * ((a.M + 16 * CT - 1) / (16 * CT))), 1, slices);
    hipLaunchKernelGGL((fp8_skinny<CT, RT, U, NW>), grid, dim3(64 * NW), 0, s, a);
    return hipGetLastError();
}

template <int BN, int BM, int WN, int WM, int NST, bool EXACT>
hipError_t launch_tile(const F8Args& a, uint32_t slices, hipStream_t s)
{
    constexpr size_t lds = NST * stage_bytes<BN, BM>();
    static_assert(lds <= 160 * 1024, "LDS");
    static uint64_t attr_done = 0;  // devices the LDS limit was raised on
    const void* fn = reinterpret_cast<const void*>(&fp8_tile<BN, BM, WN, WM, NST, EXACT>);
    hipError_t e = allow_lds(fn, lds, attr_done);
    if (e != hipSuccess) return e;
    const dim3 grid(static_cast<uint32_t>(((a.N + BN - 1) / BN) * ((a.M + BM - 1) / BM)), 1, slices);
    hipLaunchKernelGGL((fp8_tile<BN, BM, WN, WM, NST, EXACT>), grid, dim3(64 * WN * WM), lds, s, a);
    return hipGetLastError();
}

uw_status check_gemm(const uw_fp8_gemm_args* p)
{
    if (!p) return fail(UW_EINVAL, "NULL argument");
    if (p->M < 0 || p->N < 1 || p->K < 1)
        return fail(UW_ESHAPE, "bad shape M=%lld N=%lld K=%lld", (long long)p->M, (long long)p->N, (long long)p->K);
    if (p->M > INT32_MAX || p->N > INT32_MAX || p->K > INT32_MAX) return fail(UW_EUNSUPPORTED, "M, N or K too large");
    if (p->y_type != UW_F32 && p->y_type != UW_BF16) return fail(UW_EINVAL, "bad y_type %d", p->y_type);
    if (p->M == 0) return UW_OK;
    if (!p->d_x || !p->d_sx || !p->d_w || !p->d_sw || !p->d_y) return fail(UW_EINVAL, "NULL device pointer");
    if (!aligned(p->d_x, 16) || !aligned(p->d_w, 16) || !aligned(p->d_y, 16))
        return fail(UW_EINVAL, "codes and Y must be 16-byte aligned");
    if (!aligned(p->d_sx, 4) || !aligned(p->d_sw, 4)) return fail(UW_EINVAL, "scales must be 4-byte aligned");
    if (p->ldx < p->K || p->ldx % 16 || p->ldw < p->K || p->ldw % 16)
        return fail(UW_EINVAL, "ldx and ldw must be >= K and multiples of 16");
    if (p->ldx >= (1 << 24) || p->ldw >= (1 << 24)) return fail(UW_EUNSUPPORTED, "ldx or ldw >= 2^24");
    if (p->ldsx < p->M || p->ldsw < (p->K + kG - 1) / kG) return fail(UW_EINVAL, "ldsx must be >= M, ldsw >= ceil(K / 128)");
    if (p->ldy < p->N) return fail(UW_EINVAL, "ldy must be >= N");
    if (p->d_ws && !aligned(p->d_ws, 16)) return fail(UW_EINVAL, "d_ws must be 16-byte aligned");
    return UW_OK;
}

}  // namespace

}  // namespace uw

using namespace uw;

size_t uw_fp8_gemm_workspace(int64_t M, int64_t N, int64_t K)
{
    (void)M;
    (void)N;
    (void)K;
    return 0;
}

uw_status uw_fp8_gemm(const uw_fp8_gemm_args* p, void* stream)
{
    clear_error();
    uw_status st = check_gemm(p);
    if (st != UW_OK || p->M == 0) return st;
    F8Args a{};
    a.x = p->d_x;
    a.sx = p->d_sx;
    a.w = p->d_w;
    a.sw = p->d_sw;
    a.y = p->d_y;
    a.M = p->M;
    a.N = p->N;
    a.K = p->K;
    a.ldx = p->ldx;
    a.ldsx = p->ldsx;
    a.ldw = p->ldw;
    a.ldsw = p->ldsw;
    a.ldy = p->ldy;
    a.bf16 = p->y_type == UW_BF16;
    a.slice = static_cast<uint32_t>((p->K + kG - 1) / kG);
    // the smallest tiles are 16 x 16
    if ((a.M + 15) / 16 * ((a.N + 15) / 16) > INT32_MAX) return fail(UW_EUNSUPPORTED, "more than 2^31 - 1 tiles");
    hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t e;
    if (a.M <= 16)
        e = launch_skinny<1, 1, 4, 4>(a, 1, s);
    else if (a.M <= 32)
        e = launch_skinny<2, 2, 2, 4>(a, 1, s);
    else if (a.M <= 64 || a.K < kG)  // the tiles read whole groups of K
        e = launch_skinny<4, 4, 2, 4>(a, 1, s);
    else if (a.bf16)
        e = launch_tile<256, 256, 2, 4, 2, false>(a, 1, s);
    else
        e = launch_tile<256, 256, 2, 4, 2, true>(a, 1, s);
    return e == hipSuccess ? UW_OK : fail(UW_EHIP, "GEMM launch failed: %s", hipGetErrorString(e));
}
