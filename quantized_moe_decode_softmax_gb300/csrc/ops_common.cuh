// ops_common.cuh -- 16-bit types and the epilogue of the products of moe_ops.h.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ops_internal.h"

namespace moe {
namespace ops {

template <typename T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> __device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ __nv_bfloat16 from_f32(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f32(float v) { return __float2half_rn(v); }

// two values rounded to T, the first in the low half
template <typename T> __device__ __forceinline__ uint32_t pack2(float a, float b);
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
template <> __device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

template <typename T> __device__ __forceinline__ float2 unpack2(uint32_t v);
template <> __device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}
template <> __device__ __forceinline__ float2 unpack2<__half>(uint32_t v) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&v));
}

// 2^v and 1 / v to about 2^-22 relative (one instruction each; subnormals are zeros)
__device__ __forceinline__ float exp2_fast(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float rcp_fast(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// act(z), to about 2^-20 relative (the results are rounded to 16 bits). SiLU and the
// tanh form of GELU are both z / (1 + exp(-a)): a = z, or twice the tanh's argument,
// which also avoids the cancellation of 1 + tanh for negative z. With the bare
// instructions this is 6 (9) operations; exp and the division cost the epilogue of
// a gated product a third more time. The exact GELU is z erfc(-z / sqrt 2) / 2 with
// erfc(x) = t (a1 + t (a2 + ...)) exp(-x^2), t = 1 / (1 + p x), x >= 0 (Abramowitz and
// Stegun, formula 7.1.26: off by at most 1.5e-7): 15 operations; erff takes about 40.
__device__ __forceinline__ float unary_act(int act, float z) {
    if (act == MOE_EPI_NONE) return z;
    constexpr float kLog2e = 1.4426950408889634f;
    if (act == MOE_EPI_GELU) {
        const float x = fabsf(z) * 0.70710678118654752f, t = rcp_fast(1.0f + 0.3275911f * x);
        const float poly = t * (0.254829592f + t * (-0.284496736f + t * (1.421413741f + t * (-1.453152027f + t * 1.061405429f))));
        const float c = 0.5f * poly * exp2_fast(-kLog2e * x * x);  // erfc(x) / 2
        return z * (z > 0.f ? 1.0f - c : c);
    }
    constexpr float kTwoC = 1.5957691216057308f;  // 2 sqrt(2 / pi)
    const float t = act == MOE_EPI_SILU ? -kLog2e * z
                                        : z * (-kLog2e * kTwoC - kLog2e * kTwoC * 0.044715f * (z * z));
    return z * rcp_fast(1.0f + exp2_fast(t));
}

// the same on 16 values, branching once
__device__ __forceinline__ void unary_act_all(int act, float (&v)[16]) {
    if (act == MOE_EPI_SILU) {
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = unary_act(MOE_EPI_SILU, v[j]);
    } else if (act == MOE_EPI_GELU) {
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = unary_act(MOE_EPI_GELU, v[j]);
    } else if (act == MOE_EPI_GELU_TANH) {
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = unary_act(MOE_EPI_GELU_TANH, v[j]);
    }
}

// a NaN stays a NaN (fminf and fmaxf would drop it)
__device__ __forceinline__ float clamp_hi(float v, float hi) { return v > hi ? hi : v; }
__device__ __forceinline__ float clamp_lo(float v, float lo) { return v < lo ? lo : v; }

// act(g) * u with the clamp of a gated product (limit > 0)
__device__ __forceinline__ float gated_act(int act, float limit, float g, float u) {
    if (limit > 0.f) {
        g = clamp_hi(g, limit);
        u = clamp_lo(clamp_hi(u, limit), -limit);
    }
    return unary_act(act, g) * u;
}

// rows [lo, hi) of group e, inside 0..rows whatever the offsets hold
__device__ __forceinline__ void group_rows(const Product &p, int e, int &lo, int &hi) {
    if (!p.offsets) {
        lo = 0;
        hi = p.rows;
        return;
    }
    lo = min(max(p.offsets[e], 0), p.rows);
    hi = min(max(p.offsets[e + 1], lo), p.rows);
}

// the row of x that feeds row r, inside 0..x_rows-1 whatever row_token holds
__device__ __forceinline__ int input_row(const Product &p, int r) {
    r = min(max(r, 0), p.rows - 1);
    return min(p.row_token ? max(p.row_token[r], 0) : r, p.x_rows - 1);
}

}  // namespace ops
}  // namespace moe
