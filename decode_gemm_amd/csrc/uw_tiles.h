// Device and launch helpers shared by the GEMM kernels: LDS DMA, the mapping of workgroups to
// output tiles, and the LDS limit of a launch.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace uw {

// LDS byte offset of a pointer into the workgroup's LDS.
__device__ __forceinline__ uint32_t lds_offset(const void* p)
{
    return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const void*)p));
}

// One LDS DMA of 16 bytes per lane: lane l's bytes at base + voff go to LDS at lds + 16 l.
// Issued from asm so that the compiler's wait counting does not make every later LDS read
// wait for the newest transfer; the compiler then undercounts outstanding loads, which
// only ever makes its own waits stricter. Callers order the reads of the target
// themselves (a wait for a load issued after the transfer).
__device__ __forceinline__ void dma16(const uint8_t* base, uint32_t voff, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(__builtin_amdgcn_readfirstlane(lds)), "v"(voff), "s"(base)
                 : "memory");
}

// blockIdx -> (n tile, m tile): consecutive hardware workgroups are dealt round-robin to
// the 8 XCDs, so first regroup them so each XCD gets a contiguous run of logical tiles,
// then walk the tiles in groups of 8 n-tiles so that concurrently resident workgroups
// share W slices (same n tile) and X slices (same m tile) in that XCD's L2.
__device__ __forceinline__ void tile_of_block(uint32_t bid, uint32_t nblocks, uint32_t tiles_n, uint32_t tiles_m,
                                              uint32_t& tn, uint32_t& tm)
{
    constexpr uint32_t XCD = 8, GROUP = 8;
    uint32_t pid = bid;
    const uint32_t full = nblocks / XCD * XCD;
    if (bid < full) pid = (bid % XCD) * (nblocks / XCD) + bid / XCD;
    const uint32_t per_group = GROUP * tiles_m;
    const uint32_t group = pid / per_group;
    const uint32_t first_n = group * GROUP;
    const uint32_t gsize = (tiles_n - first_n) < GROUP ? (tiles_n - first_n) : GROUP;
    const uint32_t in_group = pid % per_group;
    tn = first_n + in_group % gsize;
    tm = in_group / gsize;
}

// Raise a kernel's dynamic LDS limit past the 64 KB default (gfx950 has 160 KB per CU),
// once per device (bit d of `done`; a lost update between racing threads only repeats the
// call).
inline hipError_t allow_lds(const void* fn, size_t bytes, uint64_t& done)
{
    if (bytes <= 64 * 1024) return hipSuccess;
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) dev = 0;
    if ((done >> dev) & 1u) return hipSuccess;
    hipError_t e = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
    if (e == hipSuccess) done |= uint64_t{1} << dev;
    return e;
}

}  // namespace uw
