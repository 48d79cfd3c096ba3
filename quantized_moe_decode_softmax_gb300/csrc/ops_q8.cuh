// ops_q8.cuh -- 8-bit codes as f16, for the products of moe_linear_q8 and
// moe_grouped_linear_q8.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

namespace moe {
namespace ops {

// Four int8 as f16, exact, in order. q + 128 is a byte without sign; with 0x64 above it
// it is the f16 1024 + 128 + q, whose last place is 1.
__device__ __forceinline__ uint2 codes_to_f16(uint32_t q) {
    const uint32_t u = q ^ 0x80808080u;
    const uint32_t lo = __byte_perm(u, 0x64646464u, 0x4140), hi = __byte_perm(u, 0x64646464u, 0x4342);
    const uint32_t bias = 0x64806480u;  // 1152, twice
    const __half2 b = *reinterpret_cast<const __half2 *>(&bias);
    const __half2 l = __hsub2(*reinterpret_cast<const __half2 *>(&lo), b);
    const __half2 h = __hsub2(*reinterpret_cast<const __half2 *>(&hi), b);
    return make_uint2(*reinterpret_cast<const uint32_t *>(&l), *reinterpret_cast<const uint32_t *>(&h));
}

// A sum of products of codes, scaled. The sum is 0 or between 1 and 2^30 (K <= 65536), so that its product
// with a weight's scale loses nothing to underflow, and stays finite up to scales of 2^97. In the
// other order a row's scale (up to 2^121 from bf16 values) could make it infinite before a weight's
// brings it back.
__device__ __forceinline__ float scaled(float sum, float w_scale, float x_scale) { return sum * w_scale * x_scale; }

__device__ __forceinline__ uint32_t word(const uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

}  // namespace ops
}  // namespace moe
