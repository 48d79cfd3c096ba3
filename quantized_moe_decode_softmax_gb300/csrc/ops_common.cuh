// ops_common.cuh -- 16-bit types and the epilogue of the products of moe_ops.h.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

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

// act(z), with a bounded relative error over every z whose result a 16-bit type holds:
//   SiLU       2^-19 + |z| 2^-23
//   tanh GELU  2^-19 + |t| 2^-22, t = log2(e) times twice the tanh's argument
//   GELU       2^-18 + z^2 2^-23
// (the second terms are the rounding of the exponent; half a step of f16 is 2^-11).
// SiLU and the tanh form of GELU are both z / (1 + 2^t), which also avoids the
// cancellation of 1 + tanh for negative z. It is computed as z (k / (k + k 2^t)) with
// k = 2^-16: the reciprocal of 1 + 2^t by itself would be flushed to zero from t = 126
// on, where z 2^-t is still a normal bf16 number (SiLU below -87.3); with k that comes
// after the smallest subnormal of bf16. The exact GELU is z Phi(z), with
// Phi(-x) = exp(-x^2 / 2) t (a1 + t (a2 + ...)), t = 1 / (1 + p x), x >= 0: a minimax fit
// of the relative error (1e-6) of exp(x^2 / 2) Phi(-x) over 0 <= x <= 14.5, so that the
// tail keeps its digits; the exponential is the square of half its exponent's, again
// for numbers below 2^-126. 6 (8, 17) operations; exp and the division cost the epilogue
// of a gated product a third more time than the bare instructions, erff takes about 40.
__device__ __forceinline__ float unary_act(int act, float z) {
    if (act == MOE_EPI_NONE) return z;
    constexpr float kLog2e = 1.4426950408889634f;
    if (act == MOE_EPI_GELU) {
        const float x = fabsf(z), t = rcp_fast(1.0f + 0.36f * x);
        const float poly =
            t * (0.14370854f + t * (0.14183695f + t * (0.1393632f + t * (0.027526388f + t * (0.17953743f +
            t * (-0.17872778f + t * 0.04675479f))))));
        const float h = exp2_fast((-0.25f * kLog2e) * x * x), c = poly * h * h;  // Phi(-x)
        return z * (z > 0.f ? 1.0f - c : c);
    }
    constexpr float kTwoC = 1.5957691216057308f;  // 2 sqrt(2 / pi)
    const float t = act == MOE_EPI_SILU ? fmaf(-kLog2e, z, -16.0f)
                                        : fmaf(z, fmaf(-kLog2e * kTwoC * 0.044715f, z * z, -kLog2e * kTwoC), -16.0f);
    constexpr float k = 0x1p-16f;
    return z * (rcp_fast(k + exp2_fast(t)) * k);
}

// the same on N values, branching once
template <int N> __device__ __forceinline__ void unary_act_all(int act, float (&v)[N]) {
    if (act == MOE_EPI_SILU) {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = unary_act(MOE_EPI_SILU, v[j]);
    } else if (act == MOE_EPI_GELU) {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = unary_act(MOE_EPI_GELU, v[j]);
    } else if (act == MOE_EPI_GELU_TANH) {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = unary_act(MOE_EPI_GELU_TANH, v[j]);
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

// the g-th group that holds rows, or -1 (one warp; E <= 1024)
__device__ __forceinline__ int nth_group(const Product &p, int g) {
    const int lane = threadIdx.x & 31;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
        int lo = 0, hi = 0;
        if (e0 + lane < p.E) group_rows(p, e0 + lane, lo, hi);
        const unsigned m = __ballot_sync(0xffffffffu, hi > lo);
        const int c = __popc(m);
        if (g < c) return e0 + __fns(m, 0, g + 1);
        g -= c;
    }
    return -1;
}

// SMs of the current device, looked up once per device
inline cudaError_t sm_count(int &sms) {
    static std::atomic<int> known[64];
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    sms = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
    if (sms > 0) return cudaSuccess;
    if ((err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return err;
    if (dev < 64) known[dev].store(sms, std::memory_order_relaxed);
    return cudaSuccess;
}

}  // namespace ops
}  // namespace moe
