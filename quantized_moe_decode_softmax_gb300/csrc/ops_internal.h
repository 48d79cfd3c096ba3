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
// the status word of the current device's operators, cleared if it was set
cudaError_t read_ops_status(unsigned *value, cudaStream_t st);

cudaError_t launch_group_slots(const int *topk_idx, int n, int top_k, int E, int e_lo, int e_hi, int *offsets,
                               int *slot_token, int *slot_k, int *slot_of, cudaStream_t st);
cudaError_t launch_combine_slots(int dtype, const void *y, long long ldy, int rows, const int *slot_of,
                                 const float *topk_w, int n, int top_k, int N, const void *residual,
                                 long long ldr, void *out, long long ldo, cudaStream_t st);

}  // namespace ops
}  // namespace moe
