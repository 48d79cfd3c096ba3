// ops_rows_q8.cu -- products of 8-bit codes over some rows, 5 to 64 mostly (moe_linear_q8,
// moe_grouped_linear_q8).
//
//   out[r, c] = act(sx[r] sw[c] sum_k x[r, k] w[c, k] + bias[c]) (* the up product) (+ residual[r, c])
//
// Bound: the weights' bytes, half of what 16 bits take, and for more than 8 rows the conversions.
// The plan is that of the 16-bit products (ops_rows.cu): a CTA owns 16 output columns of one
// expert, its 8 warps split K in interleaved slices, and mma.sync takes the weights as A and 8
// rows of x as B straight from 16-byte loads, in any order of k that both operands share. On this
// GPU the integer mma.sync is slow (s8: 8.3 ns per 16x8x32 and SM; its 512 bytes of weights
// arrive in 11.5) and the f16 one is not (1.06 ns per 16x8x16), so that codes become f16
// on the way: two per byte permute and one subtraction, 5 instructions for 4 codes. Whole
// numbers to 2048 are exact in f16 and so is their product in f32; a sum is exact to
// 2^24 (any of 1024 inputs, most of tens of thousands), beyond it rounds as f32 does.
// 8192x4096, 8 rows 9.2 us (33.6 MB: 3.7 TB/s), 16 rows 12; 4096x4096, 32 rows 10.1.
#include "ops_common.cuh"
#include "ops_q8.cuh"
#include "ptx.cuh"

namespace moe {
namespace ops {
namespace {

constexpr int kCols = 16;    // output columns of a CTA
constexpr int kWarps = 8;

// 16 codes of a row from input k on, zeros from K on (K is a multiple of 16) or for an absent row
__device__ __forceinline__ uint4 load16(const void *row, int k, int K) {
    if (!row || k >= K) return make_uint4(0, 0, 0, 0);
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(static_cast<const char *>(row) + k));
    return v;
}

constexpr int min_ctas(int mats, int tb, bool ahead) { return ahead ? 2 : mats * tb <= 2 ? 4 : 2; }

// MATS 1 or 2 (gated) weight matrices, TB blocks of 8 rows at a time. AHEAD: as for 16 bits
template <typename T, int MATS, int TB, bool AHEAD>
__global__ void __launch_bounds__(32 * kWarps, min_ctas(MATS, TB, AHEAD)) product_rows_q8_kernel(const Product p) {
    __shared__ float part[kWarps][MATS][TB * 8][kCols + 1];
    __shared__ int s_e;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    int e = 0;
    ptx::griddep_wait();
    if (p.offsets) {
        if (warp == 0) {
            const int f = nth_group(p, blockIdx.y);
            if (lane == 0) s_e = f;
        }
        __syncthreads();
        e = s_e;
        if (e < 0) return;
    }
    int lo, hi;
    group_rows(p, e, lo, hi);
    const int c0 = blockIdx.x * kCols;
    const void *wrow[MATS][2];
#pragma unroll
    for (int m = 0; m < MATS; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c = c0 + g + 8 * h;
            const char *base = static_cast<const char *>(m ? p.w_up : p.w);
            wrow[m][h] = c < p.N ? base + (size_t)e * p.stride_e + (size_t)c * p.ldw : nullptr;
        }
    for (int r0 = lo; r0 < hi; r0 += 8 * TB) {
        const void *xrow[TB];
#pragma unroll
        for (int b = 0; b < TB; ++b) {
            const int r = r0 + 8 * b + g;
            xrow[b] = r < hi ? static_cast<const char *>(p.x) + (size_t)input_row(p, r) * p.ldx : nullptr;
        }
        float acc[MATS][TB][4];
#pragma unroll
        for (int m = 0; m < MATS; ++m)
#pragma unroll
            for (int b = 0; b < TB; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[m][b][i] = 0.f;
        constexpr int kSlice = AHEAD || MATS * TB > 1 ? 128 : 256;  // inputs of a warp's step
        // x is loaded with the weights: by itself it would be one more wait for L2 per 64 inputs
        // (4096x4096, 32 rows: 10.3 us, 12.3 with)
        uint4 wn[MATS][kSlice / 64][2], xn[TB][kSlice / 64];
        auto load = [&](int k0) {
#pragma unroll
            for (int m = 0; m < MATS; ++m)
#pragma unroll
                for (int s = 0; s < kSlice / 64; ++s)
#pragma unroll
                    for (int h = 0; h < 2; ++h) wn[m][s][h] = load16(wrow[m][h], k0 + 64 * s + 16 * t, p.K);
#pragma unroll
            for (int s = 0; s < kSlice / 64; ++s)
#pragma unroll
                for (int b = 0; b < TB; ++b) xn[b][s] = load16(xrow[b], k0 + 64 * s + 16 * t, p.K);
        };
        if (AHEAD) load(warp * kSlice);
        for (int k0 = warp * kSlice; k0 < p.K; k0 += kWarps * kSlice) {
            if (!AHEAD) load(k0);
            uint4 wv[MATS][kSlice / 64][2], xv[TB][kSlice / 64];
#pragma unroll
            for (int m = 0; m < MATS; ++m)
#pragma unroll
                for (int s = 0; s < kSlice / 64; ++s)
#pragma unroll
                    for (int h = 0; h < 2; ++h) wv[m][s][h] = wn[m][s][h];
#pragma unroll
            for (int b = 0; b < TB; ++b)
#pragma unroll
                for (int s = 0; s < kSlice / 64; ++s) xv[b][s] = xn[b][s];
            if (AHEAD) load(k0 + kWarps * kSlice);
#pragma unroll
            for (int s = 0; s < kSlice / 64; ++s) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {  // 4 codes of each row per MMA
                    uint2 a[MATS][2];
#pragma unroll
                    for (int m = 0; m < MATS; ++m)
#pragma unroll
                        for (int h = 0; h < 2; ++h) a[m][h] = codes_to_f16(word(wv[m][s][h], i));
#pragma unroll
                    for (int b = 0; b < TB; ++b) {
                        const uint2 x2 = codes_to_f16(word(xv[b][s], i));
#pragma unroll
                        for (int m = 0; m < MATS; ++m) {
                            const uint32_t av[4] = {a[m][0].x, a[m][1].x, a[m][0].y, a[m][1].y};
                            ptx::mma_f16_16816(acc[m][b], av, x2.x, x2.y);
                        }
                    }
                }
            }
        }
#pragma unroll
        for (int m = 0; m < MATS; ++m)
#pragma unroll
            for (int b = 0; b < TB; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i)  // weight row g (+ 8), x row 2 t (+ 1)
                    part[warp][m][8 * b + 2 * t + (i & 1)][g + 8 * (i >> 1)] = acc[m][b][i];
        __syncthreads();
        for (int i = tid; i < TB * 8 * kCols; i += 32 * kWarps) {
            const int r = r0 + i / kCols, c = c0 + i % kCols;
            if (r < hi && c < p.N) {
                const float sx = p.x_scale[input_row(p, r)];
                float v[MATS];
#pragma unroll
                for (int m = 0; m < MATS; ++m) {
                    v[m] = 0.f;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) v[m] += part[w][m][i / kCols][i % kCols];
                    v[m] = scaled(v[m], (m ? p.w_up_scale : p.w_scale)[(size_t)e * p.N + c], sx);
                    const T *bias = static_cast<const T *>(m ? p.bias_up : p.bias);
                    if (bias) v[m] += to_f32(bias[(size_t)e * p.N + c]);
                }
                float o = MATS == 2 ? gated_act(p.act, p.limit, v[0], v[MATS - 1]) : unary_act(p.act, v[0]);
                if (p.residual) o += to_f32(static_cast<const T *>(p.residual)[(size_t)r * p.ldr + c]);
                static_cast<T *>(p.out)[(size_t)r * p.ldo + c] = from_f32<T>(o);
            }
        }
        __syncthreads();
    }
}

template <typename T, int MATS, int TB>
cudaError_t launch(const Product &p, int sms, cudaStream_t st) {
    const dim3 grid((p.N + kCols - 1) / kCols, p.offsets ? min(p.E, p.rows) : 1);
    return launch_overlapped((long long)grid.x * grid.y <= 2 * sms ? product_rows_q8_kernel<T, MATS, TB, true>
                                                                   : product_rows_q8_kernel<T, MATS, TB, false>,
                             grid, 32 * kWarps, 0, 1, st, p);
}

template <typename T, int MATS>
cudaError_t pick(const Product &p, cudaStream_t st) {
    int sms = 0;
    const cudaError_t err = sm_count(sms);
    if (err != cudaSuccess) return err;
    // rows of a typical group
    const int groups = p.offsets ? min(p.E, p.rows) : 1;
    const int mean = (p.rows + groups - 1) / groups;
    if (mean <= 8) return launch<T, MATS, 1>(p, sms, st);
    if (mean <= 16) return launch<T, MATS, 2>(p, sms, st);
    return launch<T, MATS, 4>(p, sms, st);
}

}  // namespace

cudaError_t launch_product_rows_q8(const Product &p, cudaStream_t st) {
    if (p.dtype == MOE_DTYPE_BF16)
        return p.w_up ? pick<__nv_bfloat16, 2>(p, st) : pick<__nv_bfloat16, 1>(p, st);
    return p.w_up ? pick<__half, 2>(p, st) : pick<__half, 1>(p, st);
}

}  // namespace ops
}  // namespace moe
