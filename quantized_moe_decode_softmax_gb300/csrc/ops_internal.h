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
