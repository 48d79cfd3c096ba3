// ops_quantize.cu -- rows of 16-bit values as 8-bit codes with a scale (moe_quantize_rows).
//
//   scale[r] = max_k |x[r, k]| / 127      code[r, k] = round(127 x[r, k] / max_k |x[r, k]|)
//
// Bound: 3 bytes per value, each moved once. A row stays in registers between its
// maximum and its codes: T threads share it, V loads of 16 bytes each, all in flight
// before the first is used (8192 x 4096: 15.2 us, 6.6 TB/s). Rows of more than 512 x 8 loads
// are read twice.
//
// Codes are those of the exact quotient, halves to even, for one product and one rounding
// each: round(x r) with r = 127 / max rounded up. Why that is exact: let x be a times its
// last place and max be b times that, a < 2^11. The quotient 127 a / b is j + 1/2 + d, and
// d is 0 or at least 1 / (254 a) of the quotient, since 254 a - (2 j + 1) b is a whole number:
// 1.9e-6, sixteen times the error of r, 2^-23. And d = 0 takes (2 j + 1) b = 254 a, so that 127
// divides one of them. If it is 2 j + 1, the quotient is 63.5 (x is half of max): r above
// 127 / max makes it 64, the even one. If it is b, then max is 127 c and r = 1 / c is exact for
// c a power of two, as it always is in bf16; the other rows (7 of 1024 in f16), and those of
// a max so small that r would be infinite, are divided value by value.
#include "ops_common.cuh"
#include "ptx.cuh"

namespace moe {
namespace ops {
namespace {

constexpr float kMagic = 12582912.0f;  // 1.5 x 2^23: adding it rounds to a whole number
constexpr int kVec = 8;                // values of a 16-byte load

// the larger |x| of two pairs, as bits: finite values order like numbers, NaN comes above infinity
__device__ __forceinline__ uint32_t larger(uint32_t m, uint32_t two) { return __vmaxu2(m, two & 0x7fff7fffu); }

template <typename T> struct Mantissa;  // its bits
template <> struct Mantissa<__nv_bfloat16> { static constexpr int bits = 7; };
template <> struct Mantissa<__half> { static constexpr int bits = 10; };

template <typename T> __device__ __forceinline__ float from_bits(uint32_t b) { return unpack2<T>(b).x; }

// How the values of one row become codes.
struct Scaling {
    enum { zeros, product, division } way;
    float rcp;   // product: 127 / max|x|, rounded up
    float up;    // division: a power of two
    float most;  //           max|x| up
};

// scale of a row from the bits of its max|x|, and what its codes need
template <typename T> __device__ __forceinline__ float scaling(uint32_t bits, Scaling &s) {
    const float most = from_bits<T>(bits);
    s.way = Scaling::zeros;
    s.rcp = s.up = s.most = 0.f;
    if (!(most > 0.f && most < INFINITY)) return most;  // zeros; or an infinity or NaN, which the scale passes on
    const uint32_t exponent = bits >> Mantissa<T>::bits, low = bits & ((1u << Mantissa<T>::bits) - 1u);
    const uint32_t mantissa = exponent ? low | (1u << Mantissa<T>::bits) : low, c = mantissa / 127u;
    s.way = most < 0x1p-60f || (c * 127u == mantissa && (c & (c - 1u))) ? Scaling::division : Scaling::product;
    s.rcp = __fdiv_ru(127.f, most);
    s.up = most < 0x1p-60f ? 0x1p64f : 1.f;
    s.most = most * s.up;
    return __fdiv_rn(most, 127.f);
}

// a whole number near kMagic: the code in its low byte
__device__ __noinline__ float divided(float x, const Scaling &s) { return kMagic + rintf(__fdiv_rn(127.f * (x * s.up), s.most)); }

// 4 codes, the first in the low byte
__device__ __forceinline__ uint32_t bytes4(float a, float b, float c, float d) {
    const uint32_t lo = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x0040);
    const uint32_t hi = __byte_perm(__float_as_uint(c), __float_as_uint(d), 0x0040);
    return __byte_perm(lo, hi, 0x5410);
}

template <typename T> __device__ __forceinline__ uint2 codes8(const uint4 &w, const Scaling &s) {
    const float2 a = unpack2<T>(w.x), b = unpack2<T>(w.y), c = unpack2<T>(w.z), d = unpack2<T>(w.w);
    if (s.way == Scaling::product)
        return make_uint2(bytes4(fmaf(a.x, s.rcp, kMagic), fmaf(a.y, s.rcp, kMagic), fmaf(b.x, s.rcp, kMagic),
                                 fmaf(b.y, s.rcp, kMagic)),
                          bytes4(fmaf(c.x, s.rcp, kMagic), fmaf(c.y, s.rcp, kMagic), fmaf(d.x, s.rcp, kMagic),
                                 fmaf(d.y, s.rcp, kMagic)));
    if (s.way == Scaling::zeros) return make_uint2(0u, 0u);
    return make_uint2(bytes4(divided(a.x, s), divided(a.y, s), divided(b.x, s), divided(b.y, s)),
                      bytes4(divided(c.x, s), divided(c.y, s), divided(d.x, s), divided(d.y, s)));
}

// the largest over the T threads of a row; ROWS rows per block (T >= 32)
template <int T> __device__ __forceinline__ uint32_t row_max(uint32_t m, uint32_t *part) {
    m = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
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
        m = larger(m, v[i].x);
        m = larger(m, v[i].y);
        m = larger(m, v[i].z);
        m = larger(m, v[i].w);
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
    for (int k = threadIdx.x; k < K; k += 256) m = max(m, (uint32_t)src[k] & 0x7fffu);
    m = row_max<256>(m, part);
    Scaling s;
    const float sc = scaling<T_>(m, s);
    if (threadIdx.x == 0) scale[row] = sc;
    char *dst = codes + row * ldc;
    for (int k = threadIdx.x; k < K; k += 256) {
        const float v = from_bits<T_>(src[k]);
        const float q = s.way == Scaling::product ? fmaf(v, s.rcp, kMagic) : divided(v, s);
        dst[k] = s.way == Scaling::zeros ? (char)0 : (char)__float_as_uint(q);
    }
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
