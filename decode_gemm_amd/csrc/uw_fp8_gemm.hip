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
    uint32_t slices;  // K slices: slice z takes the groups z, z + slices, ... (so that the slices that run
                      // together read neighbouring bytes of a row)
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

// Y[m][n .. n+3] (those inside), or the K slice's partial sums. Four values are one store also where
// ldy is odd: global stores need no alignment. (One by one they took 2.0 us more for a bf16 Y of 333
// rows with ldy 5003, 3.1 us more in fp32.)
__device__ __forceinline__ void store4(const F8Args& a, int64_t m, int64_t n, const floatx4& v)
{
    if (m >= a.M || n >= a.N) return;
    if (a.part) {
        *reinterpret_cast<floatx4*>(a.part + (static_cast<int64_t>(blockIdx.z) * a.M + m) * a.N4 + n) = v;
        return;
    }
    const bool all = n + 3 < a.N;
    if (a.bf16) {
        uint16_t* y = static_cast<uint16_t*>(a.y) + m * a.ldy + n;
        uint32_t o[4];
#pragma unroll
        for (int q = 0; q < 4; q++) o[q] = f32_to_bf16_rne(v[q]);
        if (all) {
            const uint2 w = make_uint2(o[0] | (o[1] << 16), o[2] | (o[3] << 16));
            __builtin_memcpy(y, &w, sizeof w);
        } else {
            for (int q = 0; q < 4; q++)
                if (n + q < a.N) y[q] = static_cast<uint16_t>(o[q]);
        }
    } else {
        float* y = static_cast<float*>(a.y) + m * a.ldy + n;
        if (all) {
            __builtin_memcpy(y, &v, sizeof v);
        } else {
            for (int q = 0; q < 4; q++)
                if (n + q < a.N) y[q] = v[q];
        }
    }
}

// ------------------------------------------------------------------------- skinny
// Few rows of X: 16 RT rows of W x 16 CT rows of X per workgroup, whose NW waves take the
// groups in turn and meet in LDS. Each wave keeps U groups of both operands in flight in registers; many
// small workgroups serve better than deep queues per wave, as W streams past once and the rest is the
// launch and the last loads' latency. Bound by the stream of W, so it takes the exact sums always: M = 1,
// N = 14336, K = 4096 (59 MB) takes 14.8 us with W from memory (24 such matrices in turn, 1.4 GB: 4.0 TB/s, where
// a large copy reaches 5.2 and takes 11.4 us for as much), 14.0 when W stays in the 256 MB cache.
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
    // groups first, first + stride, ...: the waves of all slices take neighbouring ones
    const uint32_t stride = NW * a.slices, first = blockIdx.z * NW + wave;
    if (first < full) {
        const uint32_t last = full - 1;
#pragma unroll
        for (int u = 0; u < U; u++) {
            const uint32_t j = first + u * stride;
            load(u, j < last ? j : last);
        }
        for (uint32_t j = first; j < full; j += U * stride)
#pragma unroll
            for (int u = 0; u < U; u++) {
                if (j + u * stride < full) multiply(u);
                const uint32_t next = j + (u + U) * stride;
                load(u, next < last ? next : last);
            }
    }
    if (G > full && full % stride == first) {  // the group that K ends inside
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

// What a workgroup of either tile kernel reads, and its place in the output.
template <int BN, int BM, int WN, int WM>
struct Tile {
    static constexpr int NW = WN * WM, TN = BN / 16 / WN, TM = BM / 16 / WM;
    static constexpr int OPW = BN * 128, OPX = BM * 128, SEG = BM < 64 ? 1 : BM / 64;
    static constexpr int STAGE = stage_bytes<BN, BM>();
    static constexpr int NLW = BN / 8 / NW, NLX = BM / 8 / NW;
    static constexpr int NL = NLW + NLX + 2;  // transfers per wave and step
    static_assert(BN % 128 == 0 && 16 * TN <= 128 && 128 % (16 * TN) == 0 && NLX >= 1 && SEG <= NW, "tile shape");

    int64_t n0, m0;
    int lane, r, g, wave, wn, wm, nb;
    uint32_t G, steps;  // groups of K, and of this slice: blockIdx.z + i * slices, i < steps
    uint32_t slices;
    int rest;  // the last group's values, 0 = all
    uint32_t woff[NLW], xoff[NLX], soff;
    const uint8_t *wbase, *xbase;
    const float *sxbase, *swbase;
    int64_t last, ldsx;
    int fo0, fo1;

    __device__ __forceinline__ explicit Tile(const F8Args& a)
    {
        const uint32_t tiles_n = static_cast<uint32_t>((a.N + BN - 1) / BN), tiles_m = static_cast<uint32_t>((a.M + BM - 1) / BM);
        uint32_t tn, tm;
        tile_of_block(blockIdx.x, gridDim.x, tiles_n, tiles_m, tn, tm);
        n0 = static_cast<int64_t>(tn) * BN;
        m0 = static_cast<int64_t>(tm) * BM;
        lane = threadIdx.x & 63;
        r = lane & 15;
        g = lane >> 4;
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        wn = wave / WM;
        wm = wave % WM;
        G = static_cast<uint32_t>((a.K + kG - 1) / kG);
        slices = a.slices;
        steps = (G - blockIdx.z + slices - 1) / slices;
        rest = static_cast<int>(a.K % kG);
        // per-lane byte offsets of this wave's transfers from the tile's first row (rows past N or M
        // read the last row; 256 rows of less than 2^24 bytes stay below 2^32)
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
        const int m = 64 * (wave % SEG) + lane;
        soff = 4 * static_cast<uint32_t>(m0 + m < a.M ? m : a.M - 1 - m0);
        wbase = a.w + n0 * a.ldw;
        xbase = a.x + m0 * a.ldx;
        sxbase = a.sx + m0;
        nb = wn * (16 * TN) / 128;  // this wave's 128 block of the tile
        const int64_t nblk = n0 / 128 + nb, blocks = (a.N + 127) / 128;
        swbase = a.sw + (nblk < blocks ? nblk : blocks - 1) * a.ldsw;
        // A short last group is read as the 128 bytes that end at K rounded up to 16, so that nothing
        // behind a row is read (K >= 128); the bytes before its start and past K are cut at use.
        last = (a.K + 15) / 16 * 16 - kG;
        ldsx = a.ldsx;
        fo0 = 128 * r + 16 * (g ^ ((r >> 1) & 7));
        fo1 = 128 * r + 16 * ((4 + g) ^ ((r >> 1) & 7));
    }

    // Whether the slice ends with a short group.
    __device__ __forceinline__ bool short_end() const { return rest && blockIdx.z + (steps - 1) * slices + 1 == G; }

    // Send the slice's i-th group to the stage at LDS offset dst.
    __device__ __forceinline__ void issue(uint32_t i, uint32_t dst) const
    {
        const uint32_t j = blockIdx.z + i * slices;
        const int64_t k = rest && j + 1 == G ? last : static_cast<int64_t>(j) * kG;
        const uint8_t* wb = wbase + k;
        const uint8_t* xb = xbase + k;
#pragma unroll
        for (int q = 0; q < NLW; q++) dma16(wb, woff[q], dst + 1024 * (NLW * wave + q));
#pragma unroll
        for (int q = 0; q < NLX; q++) dma16(xb, xoff[q], dst + OPW + 1024 * (NLX * wave + q));
        dma4(sxbase + static_cast<int64_t>(j) * ldsx, soff, dst + OPW + OPX + 256 * (wave % SEG));
        dma4(swbase + j, 0, dst + OPW + OPX + 256 * (SEG + nb));
    }

    __device__ __forceinline__ F8 frag(const uint8_t* p) const
    {
        F8 f;
        f.a = *reinterpret_cast<const u32x4*>(p + fo0);
        f.b = *reinterpret_cast<const u32x4*>(p + fo1);
        return f;
    }
    __device__ __forceinline__ F8 wfrag(const uint8_t* S, int i) const { return frag(S + 2048 * (TN * wn + i)); }
    __device__ __forceinline__ F8 xfrag(const uint8_t* S, int c) const { return frag(S + OPW + 2048 * (TM * wm + c)); }
    // scale of X for tile column c, and of this wave's W block
    __device__ __forceinline__ float sx(const uint8_t* S, int c) const
    {
        return reinterpret_cast<const float*>(S + OPW + OPX)[16 * (TM * wm + c) + r];
    }
    __device__ __forceinline__ float sw(const uint8_t* S) const
    {
        return *reinterpret_cast<const float*>(S + OPW + OPX + 256 * (SEG + nb));
    }

    // The bytes of the short last group among the 128 read.
    __device__ __forceinline__ F8 cut_tail(F8 f) const
    {
        const int from = kG - (rest + 15) / 16 * 16, to = from + rest;
        f.a = cut(f.a, 16 * g < from ? 0 : to - 16 * g);
        f.b = cut(f.b, 16 * g + 64 < from ? 0 : to - 16 * g - 64);
        return f;
    }

    // A row's stores follow one another, so that whole lines leave the L2 (4096 x 14336 bf16: 117 MB
    // written; 177 MB with the rows inside).
    __device__ __forceinline__ void store(const F8Args& a, const floatx4 (&acc)[TN][TM]) const
    {
#pragma unroll
        for (int c = 0; c < TM; c++)
#pragma unroll
            for (int i = 0; i < TN; i++) store4(a, m0 + 16 * (TM * wm + c) + r, n0 + 16 * (TN * wn + i) + 4 * g, acc[i][c]);
    }
};

// Wait until this wave's transfers of a step have landed, `younger` later steps of NL transfers
// each being allowed to be on the way.
template <int N>
__device__ __forceinline__ void wait_transfers()
{
    static_assert(N >= 0 && N < 64, "wait counter");
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// M = 4096, N = 14336, K = 4096 into bf16: 244 to 258 us, 1.87 to 1.97 PFLOP/s with 256 x 256 tiles (278
// with 256 x 128, 310 with 128 x 128). The matrix cores are busy 96 us of it. No one thing accounts for the rest:
// the same launch takes 230 us on operands that are all zero (power), and as timing copies 225 us without
// transfers, 246 without the fmas, 184 without matrix products. Into fp32 446 to 453 us (1.07 PFLOP/s, a
// large bf16 product's rate being 1.37: it takes that matrix instruction, and every wave converts the codes of
// its operands beside it). Small products are bound by the launch, the pipeline's first loads and the joining
// of K slices: M = 64, N = 4096, K = 14336 into fp32 19.3 us with 128 x 64 tiles and eight slices, about 5 of
// them joining (30 without slices); 23.3 with W from memory.
//
// One barrier per step, placed where every fragment of the
// step is in registers: behind it the stage takes the step NST ahead, and the next step's
// fragments of X replace this step's as the last MFMAs let go of them, so the matrix cores do not
// wait for LDS at the start of a step. The wave's W tiles go through registers one ahead of their
// MFMAs; the last P of them are held (ar) and multiplied behind the barrier, column by column. A
// group sum is added one W tile (or column) after its MFMA, so no MFMA is waited for.
// EXACT: the codes become bf16 behind the LDS reads.
template <int BN, int BM, int WN, int WM, int NST, int P, bool EXACT>
__global__ void __launch_bounds__(64 * WN * WM) fp8_tile(F8Args a)
{
    using T = Tile<BN, BM, WN, WM>;
    constexpr int TN = T::TN, TM = T::TM, F = TN - P, NL = T::NL;
    static_assert(P >= 1 && F >= P && NST >= 2, "W tiles before and behind the barrier");
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const T t(a);
    const uint32_t steps = t.steps, lds0 = lds_offset(lds);

    floatx4 acc[TN][TM];
#pragma unroll
    for (int i = 0; i < TN; i++)
#pragma unroll
        for (int c = 0; c < TM; c++) acc[i][c] = floatx4{0.f, 0.f, 0.f, 0.f};
    using Op = typename Operand<EXACT>::type;
    F8 an, ar[P];
    Op bf[TM];
    float s[TM];
    auto add = [&](int i, int c, const floatx4& d) {
#pragma unroll
        for (int q = 0; q < 4; q++) acc[i][c][q] = __builtin_fmaf(d[q], s[c], acc[i][c][q]);
    };

#pragma unroll
    for (int p = 0; p < NST; p++)
        if (p < steps) t.issue(p, lds0 + p * T::STAGE);
    if (NST - 1 < steps)
        wait_transfers<(NST - 1) * NL>();
    else
        wait_transfers<0>();
    __syncthreads();
    {
        const float sw = t.sw(lds);
        an = t.wfrag(lds, 0);
#pragma unroll
        for (int c = 0; c < TM; c++) {
            bf[c] = operand<EXACT>(t.xfrag(lds, c));
            s[c] = t.sx(lds, c) * sw;
        }
    }
    int st = 0;
    const bool tail = t.short_end();
    const uint32_t whole = tail ? steps - 1 : steps;
    for (uint32_t j = 0; j < whole; j++) {
        const int sn = st + 1 < NST ? st + 1 : 0;
        const uint8_t *S = lds + st * T::STAGE, *Sn = lds + sn * T::STAGE;
        floatx4 d[TM];
#pragma unroll
        for (int i = 0; i < F; i++) {
            const Op ac = operand<EXACT>(an);
            if (i + 1 < F) an = t.wfrag(S, i + 1);
            if (i >= F - P) ar[i - (F - P)] = t.wfrag(S, F + i - (F - P));
#pragma unroll
            for (int c = 0; c < TM; c++) {
                const floatx4 e = group_sum(ac, bf[c]);
                if (i > 0) {
                    add(i - 1, c, d[c]);
                    // held here: the compiler would sink the sums past the branch below, and the MFMA
                    // results with them into 100 registers that are not there
                    asm volatile("" : "+v"(acc[i - 1][c]));
                }
                d[c] = e;
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if (NST > 2 && j + NST - 1 < steps)
            wait_transfers<(NST > 2 ? NST - 2 : 0) * NL>();
        else
            wait_transfers<0>();
        __syncthreads();
        if (j + NST < steps) t.issue(j + NST, lds0 + st * T::STAGE);
        // (past the last step these reads find an older step's bytes, and nothing uses them)
        float sx[TM];
        const float sw = t.sw(Sn);
#pragma unroll
        for (int c = 0; c < TM; c++) sx[c] = t.sx(Sn, c);
        an = t.wfrag(Sn, 0);
        Op aw[P];
        floatx4 h[P];
#pragma unroll
        for (int i = 0; i < P; i++) aw[i] = operand<EXACT>(ar[i]);
#pragma unroll
        for (int c = 0; c < TM; c++) {
            floatx4 e[P];
#pragma unroll
            for (int i = 0; i < P; i++) e[i] = group_sum(aw[i], bf[c]);
            bf[c] = operand<EXACT>(t.xfrag(Sn, c));
            add(F - 1, c, d[c]);
            if (c > 0) {
#pragma unroll
                for (int i = 0; i < P; i++) add(F + i, c - 1, h[i]);
                s[c - 1] = sx[c - 1] * sw;
            }
#pragma unroll
            for (int i = 0; i < P; i++) h[i] = e[i];
        }
#pragma unroll
        for (int i = 0; i < P; i++) add(F + i, TM - 1, h[i]);
        s[TM - 1] = sx[TM - 1] * sw;
        __builtin_amdgcn_sched_barrier(0);
        st = sn;
    }
    if (tail) {
        const uint8_t* S = lds + st * T::STAGE;
#pragma unroll
        for (int c = 0; c < TM; c++) bf[c] = operand<EXACT>(t.cut_tail(t.xfrag(S, c)));
#pragma unroll
        for (int i = 0; i < TN; i++) {
            const Op ac = operand<EXACT>(t.cut_tail(t.wfrag(S, i)));
#pragma unroll
            for (int c = 0; c < TM; c++) add(i, c, group_sum(ac, bf[c]));
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    t.store(a, acc);
}

// Sum of the K slices' partial results, in slice order.
__global__ void __launch_bounds__(256) fp8_join(F8Args a, const float* part, uint32_t slices)
{
    const int64_t q = a.N4 / 4, e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (e >= a.M * q) return;
    const float* p = part + 4 * e;
    floatx4 s = {0.f, 0.f, 0.f, 0.f};
    for (uint32_t z = 0; z < slices; z += 4) {  // four loads on the way at a time
        floatx4 v[4];
#pragma unroll
        for (uint32_t i = 0; i < 4; i++) v[i] = *reinterpret_cast<const floatx4*>(p + (z + i < slices ? z + i : z) * a.M * a.N4);
#pragma unroll
        for (uint32_t i = 0; i < 4; i++)
            if (z + i < slices) s += v[i];
    }
    store4(a, e / q, 4 * (e % q), s);
}

template <int CT, int RT, int U, int NW>
hipError_t launch_skinny(const F8Args& a, hipStream_t s)
{
    const dim3 grid(static_cast<uint32_t>(((a.N + 16 * RT - 1) / (16 * RT)) * ((a.M + 16 * CT - 1) / (16 * CT))), 1, a.slices);
    hipLaunchKernelGGL((fp8_skinny<CT, RT, U, NW>), grid, dim3(64 * NW), 0, s, a);
    return hipGetLastError();
}

template <int BN, int BM, int WN, int WM, int NST, int P, bool EXACT>
hipError_t launch_tile(const F8Args& a, hipStream_t s)
{
    constexpr size_t lds = NST * stage_bytes<BN, BM>();
    static_assert(lds <= 160 * 1024, "LDS");
    static uint64_t attr_done = 0;  // devices the LDS limit was raised on
    const auto fn = fp8_tile<BN, BM, WN, WM, NST, P, EXACT>;
    hipError_t e = allow_lds(reinterpret_cast<const void*>(fn), lds, attr_done);
    if (e != hipSuccess) return e;
    const dim3 grid(static_cast<uint32_t>(((a.N + BN - 1) / BN) * ((a.M + BM - 1) / BM)), 1, a.slices);
    hipLaunchKernelGGL(fn, grid, dim3(64 * WN * WM), lds, s, a);
    return hipGetLastError();
}

// ------------------------------------------------------------------------- choice
// Kernel shapes and what a launch of them takes. The time of a launch is modelled as
//   fixed + max(rounds of workgroups, bytes from HBM, bytes into the CUs) [+ joining K slices]
// with constants fitted to 22600 launches measured on MI355X (M 1 to 4096, 15 pairs of N and K from
// 64 to 28672, K slices 1 to 16): over those sizes the shape that the model picks takes 1.6% longer
// than the fastest one on average, and 8% longer or more for one size in twenty. The launches took
// their operands in rotation from 180 MB at most, so W came from the 256 MB cache and `hbm` is the rate from
// there (17 TB/s where it decided nothing); with W from memory the choice has not been measured. The whole
// device is meant: on a stream of fewer CUs the choice is the same.
struct Shape {
    int bn, bm, waves_k;  // rows of W and X per workgroup; waves that share a group out (tiles: 1)
    int per_cu;           // workgroups that fit a CU
    hipError_t (*launch)(const F8Args&, hipStream_t);
    float fixed;       // us: launch, first loads, last stores
    float extra;       // steps: filling and draining the pipeline
    float step1, stepn;  // us per step with one and with per_cu workgroups on a CU
    float hbm, cu;     // TB/s from memory, into the CUs
    float again;       // share of W read again for every further tile along M
};
constexpr float kJoinFixed = 3.4f, kJoinRate = 2.7f;  // us; TB/s of partial sums written and read

const Shape kSums[] = {
    {256, 256, 1, 1, launch_tile<256, 256, 2, 4, 2, 2, false>, 3.81f, 1.55f, 1.38f, 1.38f, 4.34f, 9.27f, 0.862f},
    {256, 128, 1, 1, launch_tile<256, 128, 4, 2, 3, 2, false>, 2.72f, 2.71f, 0.829f, 0.829f, 6.07f, 10.4f, 0.325f},
    {128, 128, 1, 2, launch_tile<128, 128, 4, 2, 2, 1, false>, 3.57f, 0.391f, 0.582f, 0.994f, 6.09f, 14.0f, 0.759f},
    {128, 64, 1, 2, launch_tile<128, 64, 4, 2, 3, 1, false>, 3.66f, 0.0f, 0.37f, 0.743f, 7.06f, 30.8f, 0.505f},
    {128, 32, 1, 2, launch_tile<128, 32, 4, 1, 3, 1, false>, 2.95f, 0.618f, 0.354f, 0.531f, 6.81f, 19.5f, 0.33f},
    {16, 16, 8, 8, launch_skinny<1, 1, 1, 8>, 2.27f, 0.419f, 0.704f, 4.15f, 5.78f, 9.93f, 0.3f},
    {32, 16, 16, 2, launch_skinny<1, 2, 1, 16>, 2.34f, 0.346f, 2.26f, 4.62f, 4.99f, 8.56f, 0.3f},
    {32, 32, 16, 1, launch_skinny<2, 2, 1, 16>, 2.56f, 0.274f, 3.11f, 3.11f, 3.64f, 8.01f, 0.301f},
    {32, 64, 8, 2, launch_skinny<4, 2, 1, 8>, 2.74f, 0.256f, 2.24f, 4.11f, 2.96f, 8.85f, 0.59f},
};
const Shape kExact[] = {
    {256, 128, 1, 1, launch_tile<256, 128, 4, 2, 3, 1, true>, 2.91f, 1.26f, 1.66f, 1.66f, 3.6f, 6.49f, 0.734f},
    {128, 128, 1, 2, launch_tile<128, 128, 4, 2, 2, 1, true>, 3.11f, 0.947f, 1.02f, 2.06f, 3.3f, 7.33f, 0.777f},
    {128, 64, 1, 2, launch_tile<128, 64, 4, 2, 3, 1, true>, 3.7f, 0.0f, 0.671f, 1.15f, 5.17f, 10.7f, 0.594f},
    {128, 32, 1, 2, launch_tile<128, 32, 4, 1, 3, 1, true>, 3.06f, 0.431f, 0.513f, 0.754f, 6.03f, 17.7f, 0.402f},
    {16, 16, 8, 8, launch_skinny<1, 1, 1, 8>, 2.22f, 0.424f, 0.703f, 4.14f, 17.1f, 9.95f, 0.3f},
    {32, 16, 16, 2, launch_skinny<1, 2, 1, 16>, 2.29f, 0.347f, 2.26f, 4.62f, 5.0f, 8.56f, 0.337f},
    {32, 32, 16, 1, launch_skinny<2, 2, 1, 16>, 2.51f, 0.275f, 3.11f, 3.11f, 3.65f, 7.98f, 0.301f},
    {32, 64, 8, 2, launch_skinny<4, 2, 1, 8>, 2.69f, 0.248f, 2.24f, 4.17f, 2.98f, 8.89f, 0.64f},
};
constexpr uint32_t kSlices[] = {1, 2, 3, 4, 6, 8, 12, 16};

struct Plan {
    const Shape* shape;
    uint32_t slices;
    double us;
};

size_t part_bytes(int64_t M, int64_t N, uint32_t slices)
{
    return slices > 1 ? static_cast<size_t>(slices) * M * ((N + 3) / 4 * 4) * sizeof(float) : 0;
}

double model_us(const Shape& h, int64_t M, int64_t N, int64_t K, bool bf16, uint32_t slices, uint32_t cus)
{
    const int64_t G = (K + kG - 1) / kG, tn = (N + h.bn - 1) / h.bn, tm = (M + h.bm - 1) / h.bm;
    const int64_t groups = tn * tm * slices, round = static_cast<int64_t>(cus) * h.per_cu;
    const int64_t last = (groups % round + cus - 1) / cus;
    auto step = [&](int64_t k) {
        return k == 0 ? 0.0 : h.per_cu == 1 ? h.step1 : h.step1 + (h.stepn - h.step1) * static_cast<double>(k - 1) / (h.per_cu - 1);
    };
    const double steps = static_cast<double>((G + slices - 1) / slices) / h.waves_k + h.extra;
    const double run = (static_cast<double>(groups / round) * step(h.per_cu) + step(last)) * steps;
    const double nk = static_cast<double>(N) * K, mk = static_cast<double>(M) * K, mn = static_cast<double>(M) * N;
    const double hbm = (mk + nk * (1 + h.again * static_cast<double>((tm < 4 ? tm : 4) - 1)) + mn * (bf16 ? 2 : 4)) / (h.hbm * 1e6);
    const double cu = static_cast<double>(tn) * tm * G * (h.bn + h.bm) * kG / (h.cu * 1e6);
    const double join = slices > 1 ? kJoinFixed + static_cast<double>(part_bytes(M, N, slices)) / (kJoinRate * 1e6) : 0.0;
    return h.fixed + (run > hbm ? (run > cu ? run : cu) : (hbm > cu ? hbm : cu)) + join;
}

// The fastest shape and slice count by the model, for a workspace of ws bytes; no shape where none can
// be launched.
Plan make_plan(int64_t M, int64_t N, int64_t K, bool bf16, size_t ws, uint32_t cus)
{
    const Shape* shapes = bf16 ? kSums : kExact;
    const int n = bf16 ? sizeof kSums / sizeof(Shape) : sizeof kExact / sizeof(Shape);
    const int64_t G = (K + kG - 1) / kG;
    Plan best = {nullptr, 1, 0};
    for (int i = 0; i < n; i++) {
        if (shapes[i].waves_k == 1 && K < kG) continue;  // the tiles read whole groups of K
        const int64_t groups = ((M + shapes[i].bm - 1) / shapes[i].bm) * ((N + shapes[i].bn - 1) / shapes[i].bn);
        if (groups * (shapes[i].waves_k > 1 ? 64 * shapes[i].waves_k : 512) > kThreadsMost) continue;
        for (uint32_t s : kSlices) {
            if (s > 1 && (G < 2 * s || part_bytes(M, N, s) > ws)) break;
            const double us = model_us(shapes[i], M, N, K, bf16, s, cus);
            if (!best.shape || us < best.us) best = {&shapes[i], s, us};
        }
    }
    return best;
}

// The plan of a call, kept per thread by the sizes it follows from (the model takes about 2 us).
Plan plan_for(int64_t M, int64_t N, int64_t K, bool bf16, size_t ws)
{
    struct Entry {
        int64_t M, N, K;
        size_t ws;
        uint32_t cus;
        bool bf16;
        Plan plan;
    };
    static thread_local Entry kept[64] = {};
    const uint32_t cus = cu_count();
    const uint64_t hash = static_cast<uint64_t>(M) * 0x9E3779B97F4A7C15u ^ static_cast<uint64_t>(N) * 0xC2B2AE3D27D4EB4Fu ^
                          static_cast<uint64_t>(K) * 0x165667B19E3779F9u ^ (bf16 ? 0x27D4EB2F165667C5u : 0);
    Entry& e = kept[hash >> 58];
    if (!e.plan.shape || e.M != M || e.N != N || e.K != K || e.ws != ws || e.cus != cus || e.bf16 != bf16)
        e = {M, N, K, ws, cus, bf16, make_plan(M, N, K, bf16, ws, cus)};
    return e.plan;
}

hipError_t run_plan(F8Args& a, const Plan& p, void* d_ws, hipStream_t s)
{
    if (p.slices == 1) return p.shape->launch(a, s);
    a.slices = p.slices;
    a.N4 = (a.N + 3) / 4 * 4;
    a.part = static_cast<float*>(d_ws);
    const hipError_t e = p.shape->launch(a, s);
    if (e != hipSuccess) return e;
    a.part = nullptr;
    const int64_t quads = a.M * (a.N4 / 4);
    hipLaunchKernelGGL(fp8_join, dim3(static_cast<uint32_t>((quads + 255) / 256)), dim3(256), 0, s, a,
                       static_cast<const float*>(d_ws), p.slices);
    return hipGetLastError();
}

constexpr size_t kWorkspaceMost = size_t{256} << 20;  // K slices that need more are not planned

bool gemm_sizes_ok(int64_t M, int64_t N, int64_t K)
{
    return M >= 0 && N >= 1 && K >= 1 && M <= INT32_MAX && N <= INT32_MAX && K <= INT32_MAX &&
           (M + 15) / 16 * ((N + 15) / 16) <= INT32_MAX;  // the smallest tiles are 16 x 16
}

uw_status check_sizes(int64_t M, int64_t N, int64_t K, int32_t y_type)
{
    if (M < 0 || N < 1 || K < 1) return fail(UW_ESHAPE, "bad shape M=%lld N=%lld K=%lld", (long long)M, (long long)N, (long long)K);
    if (!gemm_sizes_ok(M, N, K)) return fail(UW_EUNSUPPORTED, "M, N or K too large");
    if (y_type != UW_F32 && y_type != UW_BF16) return fail(UW_EINVAL, "bad y_type %d", y_type);
    return UW_OK;
}

size_t usable_workspace(size_t bytes) { return bytes < kWorkspaceMost ? bytes : kWorkspaceMost; }

uw_status check_gemm(const uw_fp8_gemm_args* p)
{
    if (!p) return fail(UW_EINVAL, "NULL argument");
    const uw_status st = check_sizes(p->M, p->N, p->K, p->y_type);
    if (st != UW_OK || p->M == 0) return st;
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
    if (!gemm_sizes_ok(M, N, K) || M == 0) return 0;
    size_t most = 0;
    for (int bf16 = 0; bf16 < 2; bf16++) {
        const Plan p = plan_for(M, N, K, bf16, kWorkspaceMost);
        const size_t need = p.shape ? part_bytes(M, N, p.slices) : 0;
        most = need > most ? need : most;
    }
    return most;
}

uw_status uw_fp8_gemm_plan(int64_t M, int64_t N, int64_t K, int32_t y_type, size_t ws_bytes, uw_fp8_plan* out)
{
    clear_error();
    if (!out) return fail(UW_EINVAL, "NULL argument");
    *out = {};
    const uw_status st = check_sizes(M, N, K, y_type);
    if (st != UW_OK || M == 0) return st;
    const Plan p = plan_for(M, N, K, y_type == UW_BF16, usable_workspace(ws_bytes));
    if (!p.shape) return fail(UW_EUNSUPPORTED, "M x N too large for one launch");
    *out = {p.shape->bn, p.shape->bm, static_cast<int32_t>(p.slices), y_type == UW_F32 || p.shape->waves_k > 1};
    return UW_OK;
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
    a.slices = 1;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const Plan plan = plan_for(a.M, a.N, a.K, a.bf16, p->d_ws ? usable_workspace(p->ws_bytes) : 0);
    if (!plan.shape) return fail(UW_EUNSUPPORTED, "M x N too large for one launch");
    const hipError_t e = run_plan(a, plan, p->d_ws, s);
    return e == hipSuccess ? UW_OK : fail(UW_EHIP, "GEMM launch failed: %s", hipGetErrorString(e));
}
