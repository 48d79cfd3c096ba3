// ops_rows.cu -- products over few rows (moe_linear, moe_grouped_linear).
//
//   out[r, c] = act(sum_k x[r, k] w[c, k] + bias[c]) (* the up product) (+ residual[r, c])
//
// Bound: the weights' bytes. With 1..32 rows a weight is used at most 32 times,
// so the kernel is a stream over the weights and everything else has to stay
// out of its way. A CTA owns 16 output columns of one expert; its 8 warps split
// K in interleaved slices, so a small matrix still keeps every SM
// loading (N = 2048: 128 CTAs). mma.sync m16n8k16 does the products: its A
// operand is 16 weight rows and its B operand 8 rows of x, both straight from
// 16-byte global loads. That works without shuffles because a sum over k may
// take any order as long as both operands take the same: lane 4 g + t loads
// inputs 8 t .. 8 t + 7 of a 32-input step from weight rows g and g + 8 and from
// x row g, and feeds them to two MMAs four inputs at a time. The f32 partials of
// the 8 warps are summed in warp order.
//
// Measured (GB300, bf16, us back to back in a graph): 2048x2048, one row 2.8; 4096x4096
// 6.0 (5.6 TB/s); 4096x8192 13.6 (4.9 TB/s); 8 of 128 experts, gated 2048 -> 768, one
// row each 11.2 (4.5 TB/s). Up to about 10 MB the time is launch, one load latency per
// slice and the reduction; above, the weights' bytes.
#include "ops_common.cuh"
#include "ptx.cuh"

namespace moe {
namespace ops {
namespace {

constexpr int kCols = 16;    // output columns of a CTA
constexpr int kWarps = 8;

template <typename T>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma<__nv_bfloat16>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    ptx::mma_bf16_16816(d, a, b0, b1);
}
template <>
__device__ __forceinline__ void mma<__half>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    ptx::mma_f16_16816(d, a, b0, b1);
}

// 16 bytes of a row's inputs k.., zeros from K on or for an absent row. (volatile keeps
// the loads of a slice together, ahead of the MMAs.)
__device__ __forceinline__ uint4 load8(const void *row, int k, int K) {
    if (!row || k >= K) return make_uint4(0, 0, 0, 0);
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(static_cast<const char *>(row) + 2 * (size_t)k));
    return v;
}

// MATS 1 or 2 (gated) weight matrices, TB blocks of 8 rows at a time. AHEAD: the
// weights of the next slice are loaded while this one's are used, with registers
// for two CTAs per SM. That is the faster way while the grid fits the SMs at two
// CTAs each (4096x4096, one row: 5.8 against 9.0 us). A larger grid does better with
// fewer registers, more CTAs per SM and an even end (128 experts, 8 in use, gated
// 2048 -> 768: 12.0 against 14.5 us).
constexpr int min_ctas(int mats, int tb, bool ahead) {
    return ahead ? 2 : mats * tb == 1 ? 6 : mats * tb == 2 ? 4 : mats * tb == 4 ? 3 : 2;
}

template <typename T, int MATS, int TB, bool AHEAD>
__global__ void __launch_bounds__(32 * kWarps, min_ctas(MATS, TB, AHEAD)) product_rows_kernel(const Product p) {
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
    const size_t esz = 2;
    const void *wrow[MATS][2];
#pragma unroll
    for (int m = 0; m < MATS; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c = c0 + g + 8 * h;
            const char *base = static_cast<const char *>(m ? p.w_up : p.w);
            wrow[m][h] = c < p.N ? base + esz * ((size_t)e * p.stride_e + (size_t)c * p.ldw) : nullptr;
        }
    for (int r0 = lo; r0 < hi; r0 += 8 * TB) {
        const void *xrow[TB];
#pragma unroll
        for (int b = 0; b < TB; ++b) {
            const int r = r0 + 8 * b + g;
            xrow[b] = r < hi ? static_cast<const char *>(p.x) + esz * ((size_t)input_row(p, r) * p.ldx) : nullptr;
        }
        float acc[MATS][TB][4];
#pragma unroll
        for (int m = 0; m < MATS; ++m)
#pragma unroll
            for (int b = 0; b < TB; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[m][b][i] = 0.f;
        constexpr int kSlice = AHEAD ? 64 : 128;  // inputs of a warp's step
        uint4 wn[MATS][kSlice / 32][2];
        auto load_w = [&](int k0) {
#pragma unroll
            for (int m = 0; m < MATS; ++m)
#pragma unroll
                for (int s = 0; s < kSlice / 32; ++s)
#pragma unroll
                    for (int h = 0; h < 2; ++h) wn[m][s][h] = load8(wrow[m][h], k0 + 32 * s + 8 * t, p.K);
        };
        if (AHEAD) load_w(warp * kSlice);
        for (int k0 = warp * kSlice; k0 < p.K; k0 += kWarps * kSlice) {
            if (!AHEAD) load_w(k0);
            uint4 wv[MATS][kSlice / 32][2];
#pragma unroll
            for (int m = 0; m < MATS; ++m)
#pragma unroll
                for (int s = 0; s < kSlice / 32; ++s)
#pragma unroll
                    for (int h = 0; h < 2; ++h) wv[m][s][h] = wn[m][s][h];
            if (AHEAD) load_w(k0 + kWarps * kSlice);
#pragma unroll
            for (int s = 0; s < kSlice / 32; ++s) {
#pragma unroll
                for (int b = 0; b < TB; ++b) {
                    const uint4 xv = load8(xrow[b], k0 + 32 * s + 8 * t, p.K);
#pragma unroll
                    for (int m = 0; m < MATS; ++m) {
                        const uint4 v0 = wv[m][s][0], v1 = wv[m][s][1];
                        const uint32_t a0[4] = {v0.x, v1.x, v0.y, v1.y}, a1[4] = {v0.z, v1.z, v0.w, v1.w};
                        mma<T>(acc[m][b], a0, xv.x, xv.y);
                        mma<T>(acc[m][b], a1, xv.z, xv.w);
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
                float v[MATS];
#pragma unroll
                for (int m = 0; m < MATS; ++m) {
                    v[m] = 0.f;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) v[m] += part[w][m][i / kCols][i % kCols];
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
    return launch_overlapped((long long)grid.x * grid.y <= 2 * sms ? product_rows_kernel<T, MATS, TB, true>
                                                                   : product_rows_kernel<T, MATS, TB, false>,
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

cudaError_t launch_product_rows(const Product &p, cudaStream_t st) {
    if (p.dtype == MOE_DTYPE_BF16)
        return p.w_up ? pick<__nv_bfloat16, 2>(p, st) : pick<__nv_bfloat16, 1>(p, st);
    return p.w_up ? pick<__half, 2>(p, st) : pick<__half, 1>(p, st);
}

}  // namespace ops
}  // namespace moe
