// ckpt_format.cuh -- values of an 8-bit activation checkpoint: code * 2^(E - 133).
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

namespace muon {

// bf16 bits of 2^(E - 133): subnormal below E = 7, NaN at 255
__device__ __forceinline__ uint32_t unit_bf16(uint32_t e) {
    return e == 255u ? 0x7FC0u : e >= 7u ? (e - 6u) << 7 : 1u << e;
}

// Two codes (the low bytes of the halves of x) times the unit pair.  128 + (c & 127) and
// 128, or 256 for negative c, are bf16 bit patterns away from the code, and their difference
// is c.
__device__ __forceinline__ uint32_t codes_to_bf16(uint32_t x, __nv_bfloat162 unit) {
    const uint32_t a = (x & 0x007F007Fu) | 0x43004300u, b = (x & 0x00800080u) | 0x43004300u;
    const __nv_bfloat162 v =
        __hmul2(__hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b)), unit);
    return *reinterpret_cast<const uint32_t*>(&v);
}

}  // namespace muon
