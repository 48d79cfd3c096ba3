// ops_internal.h -- arguments and launchers of the operators of moe_ops.h.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_ops.h"

namespace moe {
namespace ops {

// One product, as the kernels see it (device pointers). offsets == nullptr: one
// group of all `rows` rows (moe_linear).
struct Product {
    const void *x;
    const void *w, *w_up;        // w_up: nullptr = not gated
    const void *bias, *bias_up;  // may be nullptr
    const void *residual;        // may be nullptr
    void *out;
    const int *offsets, *row_token;
    long long ldx, ldw, stride_e, ldr, ldo;
    int x_rows, rows;
    int E, N, K;
    int dtype, act;
    float limit;                 // 0: no clamp
    // products of 8-bit codes: a scale per row of x and per row of each weight matrix
    // (x, w and w_up are then int8, and ldx, ldw and stride_e count bytes)
    const float *x_scale, *w_scale, *w_up_scale;
};

// One routing (moe_route), device pointers.
struct RouteArgs {
    const void *logits;
    const float *bias;           // may be nullptr
    int *topk_idx;
    float *topk_w;
    long long ldl;
    int n, E, k, dtype, score;
    int groups, top_groups;
    bool top2;                   // a group's score is the sum of its best two
    bool renormalize;
    bool vector;                 // rows of logits are aligned for wide loads
    int words;                   // of shared memory per warp, 4 bytes each
    float scale;
};

// A kernel launch that may begin before the stream's previous kernel has ended: the
// kernel calls griddep_wait before its first access to global memory, so only its
// start-up overlaps the other's end (about 1 us less between two small kernels).
// What the other wrote must not be read through the non-coherent cache, which may
// have been filled meanwhile: no __ldg and no __restrict__ inputs in these kernels.
template <typename... P, typename... A>
cudaError_t launch_overlapped(void (*kernel)(P...), dim3 grid, int threads, int smem, int cluster, cudaStream_t st,
                              A... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// few rows per expert: the weights are streamed once per 32 rows (ops_rows.cu)
cudaError_t launch_product_rows(const Product &p, cudaStream_t st);
// many rows per expert: tcgen05 (ops_gemm.cu); cudaErrorNotSupported, with nothing
// launched, where the driver declines a tensor map
cudaError_t launch_product_gemm(const Product &p, cudaStream_t st);
// the same for products of 8-bit codes: a handful of rows per expert (ops_dot_q8.cu), few
// (ops_rows_q8.cu), many (ops_gemm_q8.cu)
cudaError_t launch_product_dot_q8(const Product &p, cudaStream_t st);
cudaError_t launch_product_rows_q8(const Product &p, cudaStream_t st);
cudaError_t launch_product_gemm_q8(const Product &p, cudaStream_t st);
// the status words of the current device's kernels with waits: set when one gave up
unsigned *ops_status(cudaError_t *err);
unsigned *ops_status_q8(cudaError_t *err);

cudaError_t launch_route(const RouteArgs &a, cudaStream_t st);
cudaError_t launch_quantize_rows(int dtype, const void *x, long long ldx, int n, int K, int8_t *codes, long long ldc,
                                 float *scale, cudaStream_t st);
cudaError_t launch_group_slots(const int *topk_idx, int n, int top_k, int E, int e_lo, int e_hi, int *offsets,
                               int *slot_token, int *slot_k, int *slot_of, cudaStream_t st);
cudaError_t launch_combine_slots(int dtype, const void *y, long long ldy, int rows, const int *slot_of,
                                 const float *topk_w, int n, int top_k, int N, const void *residual,
                                 long long ldr, void *out, long long ldo, cudaStream_t st);

}  // namespace ops
}  // namespace moe
