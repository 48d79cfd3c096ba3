// ops_dot_q8.cu -- products of 8-bit codes over a handful of rows, or over more of them by few
// columns (moe_linear_q8, moe_grouped_linear_q8).
//
//   out[r, c] = act(sx[r] sw[c] sum_k x[r, k] w[c, k] + bias[c]) (* the up product) (+ residual[r, c])
//
// Bound: the weights' bytes. With up to 4 rows the byte dot product (dp4a) keeps up with
// them, and needs no conversion: per KB of weights 8 instructions a row, where the way
// over f16 (ops_rows_q8.cu) takes 67 for 1 to 8 rows and is bound by them (8 of 128
// experts, 2048 -> 2 x 768, one row each: 9.9 us). Sums are whole numbers, exact for every
// K (65536 x 128^2 is 2^30).
//
// A warp owns R weight rows (gated: R / 2 of each matrix) and walks K in steps of 512
// inputs, 16 bytes a lane: every load is 512 contiguous bytes of a row. D steps are in
// flight. Where there are few columns, 2 or 4 warps of a block share the rows and take the
// steps in turn. A block takes NX rows of x; more rows of a group are other blocks, which
// find the weights in L2. 2048x2048, one row 3.1 us, 8192x4096 7.4 (4.5 TB/s); 8 of 128 experts,
// gated 2048 -> 768, one row each 6.6 (25 MB); 64 rows of 512x4096 5.5.
#include "ops_common.cuh"
#include "ops_q8.cuh"
#include "ptx.cuh"

namespace moe {
namespace ops {
namespace {

constexpr int kWarps = 4;
constexpr int kStep = 512;  // inputs of a warp's step

// 16 codes, zeros where !in
__device__ __forceinline__ uint4 load16(const char *p, bool in) {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (in)
        asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "l"(p));
    return v;
}

__device__ __forceinline__ int dot16(const uint4 &a, const uint4 &b, int c) {
    c = __dp4a((int)a.x, (int)b.x, c);
    c = __dp4a((int)a.y, (int)b.y, c);
    c = __dp4a((int)a.z, (int)b.z, c);
    return __dp4a((int)a.w, (int)b.w, c);
}

// The g-th run of at most NX rows of a group, in the order of the groups: its group (-1: none) and
// rows lo .. hi - 1. By a warp; the offsets of 256 groups load together.
template <int NX> __device__ __forceinline__ int nth_run(const Product &p, int g, int &lo, int &hi) {
    const int lane = threadIdx.x & 31;
    for (int e0 = 0; e0 < p.E; e0 += 256) {
        int from[8], to[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int e = e0 + 32 * i + lane;
            from[i] = e < p.E ? p.offsets[e] : 0;
            to[i] = e < p.E ? p.offsets[e + 1] : 0;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int l = min(max(from[i], 0), p.rows), h = min(max(to[i], l), p.rows);  // as group_rows
            const int runs = (h - l + NX - 1) / NX, all = (int)__reduce_add_sync(0xffffffffu, (unsigned)runs);
            if (g < all) {
                int before = runs;  // inclusive sums
#pragma unroll
                for (int d = 1; d < 32; d *= 2) {
                    const int v = __shfl_up_sync(0xffffffffu, before, d);
                    if (lane >= d) before += v;
                }
                const int at = __popc(__ballot_sync(0xffffffffu, before <= g));  // lanes whose runs all come before
                lo = __shfl_sync(0xffffffffu, l + (g - before + runs) * NX, at);
                hi = min(lo + NX, __shfl_sync(0xffffffffu, h, at));
                return e0 + 32 * i + at;
            }
            g -= all;
        }
    }
    return -1;
}

// MATS 1 or 2 (gated) weight matrices; R weight rows of a warp; NX rows of x; D steps in
// flight; B blocks on an SM. share: warps of the block on the same weight rows (1, 2 or 4)
template <typename T, int MATS, int R, int NX, int D, int B>
__global__ void __launch_bounds__(32 * kWarps, B) product_dot_q8_kernel(const Product p, const int share) {
    constexpr int kCols = R / MATS;  // output columns of a warp
    __shared__ int part[kWarps][MATS][kCols * NX];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int e = 0, lo = blockIdx.y * NX, hi = min(lo + NX, p.rows);
    ptx::griddep_wait();
    if (p.offsets && (e = nth_run<NX>(p, blockIdx.y, lo, hi)) < 0) return;
    const int turn = warp % share, c0 = (blockIdx.x * (kWarps / share) + warp / share) * kCols;
    const char *wrow[R];
#pragma unroll
    for (int j = 0; j < R; ++j)  // (a row past the end repeats the last one, and is not stored)
        wrow[j] = static_cast<const char *>(j >= kCols ? p.w_up : p.w) + (size_t)e * p.stride_e +
                  (size_t)min(c0 + j % kCols, p.N - 1) * p.ldw + 16 * lane;
    const int k0 = kStep * turn, dk = kStep * share;
    const char *xrow[NX];
#pragma unroll
    for (int b = 0; b < NX; ++b)
        xrow[b] = static_cast<const char *>(p.x) + (size_t)input_row(p, min(lo + b, hi - 1)) * p.ldx + 16 * lane;
    int acc[R][NX];
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
        for (int b = 0; b < NX; ++b) acc[j][b] = 0;
    uint4 w[D][R], x[D][NX];
    auto load = [&](int d, int k) {
        const bool in = k + 16 * lane < p.K;
#pragma unroll
        for (int j = 0; j < R; ++j) w[d][j] = load16(wrow[j] + k, in);
#pragma unroll
        for (int b = 0; b < NX; ++b) x[d][b] = load16(xrow[b] + k, in);
    };
#pragma unroll
    for (int d = 0; d < D; ++d) load(d, k0 + d * dk);
    for (int k = k0; k < p.K; k += D * dk) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
#pragma unroll
            for (int j = 0; j < R; ++j)
#pragma unroll
                for (int b = 0; b < NX; ++b) acc[j][b] = dot16(w[d][j], x[d][b], acc[j][b]);
            load(d, k + (D + d) * dk);
        }
    }
    int sum[MATS];  // of all lanes: lane j NX + b has those of column j and row b
#pragma unroll
    for (int m = 0; m < MATS; ++m) {
        sum[m] = 0;
#pragma unroll
        for (int j = 0; j < kCols; ++j)
#pragma unroll
            for (int b = 0; b < NX; ++b) {
                const int s = __reduce_add_sync(0xffffffffu, acc[m * kCols + j][b]);
                if (lane == j * NX + b) sum[m] = s;
            }
    }
    if (share > 1) {
        if (lane < kCols * NX) {
#pragma unroll
            for (int m = 0; m < MATS; ++m) part[warp][m][lane] = sum[m];
        }
        __syncthreads();
        if (turn == 0 && lane < kCols * NX) {
            for (int i = 1; i < share; ++i)
#pragma unroll
                for (int m = 0; m < MATS; ++m) sum[m] += part[warp + i][m][lane];
        }
    }
    const int c = c0 + lane / NX, r = lo + lane % NX;
    if (turn == 0 && lane < kCols * NX && c < p.N && r < hi) {
        const float sx = p.x_scale[input_row(p, r)];
        float v[MATS];
#pragma unroll
        for (int m = 0; m < MATS; ++m) {
            v[m] = scaled((float)sum[m], (m ? p.w_up_scale : p.w_scale)[(size_t)e * p.N + c], sx);
            const T *bias = static_cast<const T *>(m ? p.bias_up : p.bias);
            if (bias) v[m] += to_f32(bias[(size_t)e * p.N + c]);
        }
        float o = MATS == 2 ? gated_act(p.act, p.limit, v[0], v[MATS - 1]) : unary_act(p.act, v[0]);
        if (p.residual) o += to_f32(static_cast<const T *>(p.residual)[(size_t)r * p.ldr + c]);
        static_cast<T *>(p.out)[(size_t)r * p.ldo + c] = from_f32<T>(o);
    }
}

template <typename T, int MATS, int R, int NX, int D, int B>
cudaError_t launch(const Product &p, int sms, cudaStream_t st) {
    constexpr int kCols = R / MATS;
    // runs, at most: a group's last one may be short
    const int runs = p.offsets ? min((p.rows + NX - 1) / NX + min(p.E, p.rows), p.rows) : (p.rows + NX - 1) / NX;
    const long long tiles = (long long)runs * ((p.N + kCols - 1) / kCols);
    // several warps on the same rows while the SMs hold them all at once, and each has a step
    int share = 1;
    while (share < kWarps && tiles * share * 2 <= 3LL * B * sms && p.K > kStep * share) share *= 2;
    const int cols = kCols * kWarps / share;
    const dim3 grid((p.N + cols - 1) / cols, runs);
    return launch_overlapped(product_dot_q8_kernel<T, MATS, R, NX, D, B>, grid, 32 * kWarps, 0, 1, st, p, share);
}

// R, D and B: more weight rows per warp amortise the start of a block (a group's is longer) and
// the loads of x; fewer keep more warps busy on one matrix; short rows need no depth. Measured
// (us, R = 4 and D = 4, B = 4 / R = 8 and D = 2, B = 4; short rows D = 1, B = 6):
//   8192x4096, one row                                     7.4 / 9.3
//   8 of 128 experts, gated 2048 -> 768, one row each      8.5 / 6.8
//   the same, 768 -> 2048                                 10.1 / 6.7
template <typename T, int MATS>
cudaError_t pick(const Product &p, cudaStream_t st) {
    int sms = 0;
    const cudaError_t err = sm_count(sms);
    if (err != cudaSuccess) return err;
    // rows of x of a block: a group may hold twice the mean
    const int groups = p.offsets ? min(p.E, p.rows) : 1;
    const int mean = (p.rows + groups - 1) / groups, most = p.offsets ? 2 * mean : mean;
    if (p.K <= 2 * kStep && most <= 2)
        return most <= 1 ? launch<T, MATS, 8, 1, 1, 6>(p, sms, st) : launch<T, MATS, 8, 2, 1, 6>(p, sms, st);
    if (p.offsets && most <= 2) return launch<T, MATS, 8, 2, 2, 4>(p, sms, st);
    return most <= 1 ? launch<T, MATS, 4, 1, 4, 4>(p, sms, st) : launch<T, MATS, 4, 4, 2, 4>(p, sms, st);
}

}  // namespace

cudaError_t launch_product_dot_q8(const Product &p, cudaStream_t st) {
    if (p.dtype == MOE_DTYPE_BF16)
        return p.w_up ? pick<__nv_bfloat16, 2>(p, st) : pick<__nv_bfloat16, 1>(p, st);
    return p.w_up ? pick<__half, 2>(p, st) : pick<__half, 1>(p, st);
}

}  // namespace ops
}  // namespace moe
