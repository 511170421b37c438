// Device helpers of the kernels that order the tokens of a row of logits.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace uw {

namespace {

typedef unsigned long long u64;

__device__ __forceinline__ float value(const float* x, int i) { return x[i]; }
__device__ __forceinline__ float value(const uint16_t* x, int i) { return __uint_as_float(static_cast<uint32_t>(x[i]) << 16); }

// Sort key of (logit, index): ascending keys are the order. -0 and +0 are equal logits.
__device__ __forceinline__ uint32_t order_bits(float l)
{
    const uint32_t b = __float_as_uint(l + 0.0f);
    return (b & 0x80000000u) ? b : ~(b | 0x80000000u);  // larger logits get smaller bits
}
__device__ __forceinline__ float order_value(uint32_t o) { return __uint_as_float((o & 0x80000000u) ? o : ~o & 0x7FFFFFFFu); }
__device__ __forceinline__ u64 key_of(float l, int i) { return (static_cast<u64>(order_bits(l)) << 32) | static_cast<uint32_t>(i); }
__device__ __forceinline__ float key_value(u64 key) { return order_value(static_cast<uint32_t>(key >> 32)); }

}  // namespace

}  // namespace uw
