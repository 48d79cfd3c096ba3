// ops_quantize.cu -- rows of 16-bit values as 8-bit codes with a scale (moe_quantize_rows).
//
//   scale[r] = max_k |x[r, k]| / 127      code[r, k] = round(127 x[r, k] / max_k |x[r, k]|)
//
// Bound: 3 bytes per value, each moved once. A row stays in registers between its
// maximum and its codes: T threads share it, V loads of 16 bytes each, all in flight
// before the first is used; V is as large as that allows (8), so that few threads
// have to meet. Rows of more than 512 x 8 loads go through the same loop twice.
//
// Codes are those of the exact quotient, halves to even. 127 x is exact in f32 (18
// bits), and a quotient of two 16-bit values that is not a half is at least 1e-6 of
// itself away from one, so that one product with 127 / max (error 2^-22) decides all
// but the values within 1e-4 of a half; those are divided. The row is scaled by a power
// of two first where 127 x or 127 / max would leave the range of f32.
#include "ops_common.cuh"
#include "ptx.cuh"

namespace moe {
namespace ops {
namespace {

constexpr float kMagic = 12582912.0f;  // 1.5 x 2^23: adding it rounds to a whole number
constexpr int kVec = 8;                // values of a 16-byte load

// |x| as bits: finite values order like numbers, NaN comes above infinity
template <typename T> __device__ __forceinline__ uint32_t largest(uint32_t m, uint32_t two) {
    const uint32_t lo = two & 0x7fffu, hi = (two >> 16) & 0x7fffu;
    return max(m, max(lo, hi));
}

template <typename T> __device__ __forceinline__ float from_bits(uint32_t b) { return unpack2<T>(b).x; }

// The codes of one row: how its values become whole numbers.
struct Scaling {
    float up;    // a power of two
    float most;  // max|x| up
    float rcp;   // 127 / most
};

// scale of a row from the bits of its max|x|, and what its codes need
template <typename T> __device__ __forceinline__ float scaling(uint32_t bits, Scaling &s) {
    const float most = from_bits<T>(bits);
    if (!(most > 0.f && most < INFINITY)) {  // zeros; or an infinity or NaN, which the scale passes on
        s.up = s.most = s.rcp = 0.f;
        return most == 0.f ? 0.f : most;
    }
    s.up = most > 0x1p100f ? 0x1p-64f : most < 0x1p-60f ? 0x1p64f : 1.f;
    s.most = most * s.up;
    s.rcp = __fdiv_rn(127.f, s.most);
    return __fdiv_rn(most, 127.f);
}

__device__ __noinline__ float divided(float x, const Scaling &s) { return rintf(__fdiv_rn(127.f * x, s.most)); }

// 4 codes, the first in the low byte
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, const Scaling &s) {
    float v[4] = {a, b, c, d}, q[4], off = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] *= s.up;
        q[i] = fmaf(v[i], s.rcp, kMagic);
        off = fmaxf(off, fabsf(fmaf(v[i], s.rcp, kMagic - q[i])));
    }
    if (off > 0.4999f) {
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = kMagic + divided(v[i], s);
    }
    const uint32_t lo = __byte_perm(__float_as_uint(q[0]), __float_as_uint(q[1]), 0x0040);
    const uint32_t hi = __byte_perm(__float_as_uint(q[2]), __float_as_uint(q[3]), 0x0040);
    return __byte_perm(lo, hi, 0x5410);
}

template <typename T> __device__ __forceinline__ uint2 codes8(const uint4 &w, const Scaling &s) {
    if (s.up == 0.f) return make_uint2(0u, 0u);
    const float2 a = unpack2<T>(w.x), b = unpack2<T>(w.y), c = unpack2<T>(w.z), d = unpack2<T>(w.w);
    return make_uint2(codes4(a.x, a.y, b.x, b.y, s), codes4(c.x, c.y, d.x, d.y, s));
}

// the largest over the T threads of a row; ROWS rows per block (T >= 32)
template <int T> __device__ __forceinline__ uint32_t row_max(uint32_t m, uint32_t *part) {
    m = __reduce_max_sync(0xffffffffu, m);
    if constexpr (T > 32) {
        const int warp = threadIdx.x >> 5, first = warp / (T / 32) * (T / 32);
        if ((threadIdx.x & 31) == 0) part[warp] = m;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < T / 32; ++i) m = max(m, part[first + i]);
    }
    return m;
}

// T threads a row, V loads each; a block of B threads takes B / T rows. VECTOR: rows of x and
// codes at multiples of 16 and 8 bytes, K a multiple of 8.
template <typename T_, int T, int V, int B>
__global__ void __launch_bounds__(B) quantize_kernel(const char *x, long long ldx, int n, int K, char *codes,
                                                     long long ldc, float *scale) {
    __shared__ uint32_t part[B / 32];
    ptx::griddep_wait();
    const int t = threadIdx.x % T;
    const long long row = (long long)blockIdx.x * (B / T) + threadIdx.x / T;
    const bool live = row < n;
    const uint4 *src = reinterpret_cast<const uint4 *>(x + 2 * row * ldx);
    const int pieces = K / kVec;
    uint4 v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = live && t + i * T < pieces ? src[t + i * T] : make_uint4(0u, 0u, 0u, 0u);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        m = largest<T_>(m, v[i].x);
        m = largest<T_>(m, v[i].y);
        m = largest<T_>(m, v[i].z);
        m = largest<T_>(m, v[i].w);
    }
    m = row_max<T>(m, part);
    if (!live) return;
    Scaling s;
    const float sc = scaling<T_>(m, s);
    if (t == 0) scale[row] = sc;
    uint2 *dst = reinterpret_cast<uint2 *>(codes + row * ldc);
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (t + i * T < pieces) dst[t + i * T] = codes8<T_>(v[i], s);
}

// any row: one block each, value by value, x read twice
template <typename T_>
__global__ void __launch_bounds__(256) quantize_any_kernel(const char *x, long long ldx, int n, int K, char *codes,
                                                           long long ldc, float *scale) {
    __shared__ uint32_t part[8];
    ptx::griddep_wait();
    const long long row = blockIdx.x;
    const uint16_t *src = reinterpret_cast<const uint16_t *>(x + 2 * row * ldx);
    uint32_t m = 0;
    for (int k = threadIdx.x; k < K; k += 256) m = max(m, src[k] & 0x7fffu);
    m = row_max<256>(m, part);
    Scaling s;
    const float sc = scaling<T_>(m, s);
    if (threadIdx.x == 0) scale[row] = sc;
    char *dst = codes + row * ldc;
    for (int k = threadIdx.x; k < K; k += 256)
        dst[k] = s.up == 0.f ? (char)0 : (char)(int)divided(from_bits<T_>(src[k]) * s.up, s);
}

template <typename T_>
cudaError_t launch(const void *xv, long long ldx, int n, int K, int8_t *codes, long long ldc, float *scale,
                   cudaStream_t st) {
    const char *x = static_cast<const char *>(xv);
    char *c = reinterpret_cast<char *>(codes);
    const int pieces = K / kVec;
    const bool vector = K % kVec == 0 && ldx % kVec == 0 && ldc % kVec == 0 && ((uintptr_t)x & 15u) == 0 &&
                        ((uintptr_t)c & 7u) == 0;
    if (!vector || pieces > 512 * 8)
        return launch_overlapped(quantize_any_kernel<T_>, dim3((unsigned)n), 256, 0, 1, st, x, ldx, n, K, c, ldc, scale);
    auto go = [&](auto kernel, int rows, int threads) {
        return launch_overlapped(kernel, dim3((unsigned)((n + rows - 1) / rows)), threads, 0, 1, st, x, ldx, n, K, c, ldc,
                                 scale);
    };
    if (pieces <= 32) return go(quantize_kernel<T_, 32, 1, 128>, 4, 128);
    if (pieces <= 64) return go(quantize_kernel<T_, 32, 2, 128>, 4, 128);
    if (pieces <= 128) return go(quantize_kernel<T_, 32, 4, 128>, 4, 128);
    if (pieces <= 256) return go(quantize_kernel<T_, 64, 4, 128>, 2, 128);
    if (pieces <= 512) return go(quantize_kernel<T_, 128, 4, 128>, 1, 128);
    if (pieces <= 1024) return go(quantize_kernel<T_, 256, 4, 256>, 1, 256);
    if (pieces <= 2048) return go(quantize_kernel<T_, 512, 4, 512>, 1, 512);
    return go(quantize_kernel<T_, 512, 8, 512>, 1, 512);
}

}  // namespace

cudaError_t launch_quantize_rows(int dtype, const void *x, long long ldx, int n, int K, int8_t *codes, long long ldc,
                                 float *scale, cudaStream_t st) {
    return dtype == MOE_DTYPE_BF16 ? launch<__nv_bfloat16>(x, ldx, n, K, codes, ldc, scale, st)
                                   : launch<__half>(x, ldx, n, K, codes, ldc, scale, st);
}

}  // namespace ops
}  // namespace moe
