// ops_api.cu -- the C entry points of moe_ops.h: argument checks and dispatch.
//
// As for the step (mlxcel issue #1616, Implementation Notes), shapes are
// validated before any dispatch and what the kernels do not cover is declined.
#include <cuda_runtime.h>

#include "ops_internal.h"

using namespace moe::ops;

namespace {

constexpr int kMaxE = 1024, kMaxK = 65536, kMaxN = 1 << 20, kMaxRows = 1 << 24, kMaxRanks = 64;

bool misaligned(const void *p, unsigned bytes) { return ((uintptr_t)p & (bytes - 1)) != 0; }

moe_status of(cudaError_t err) {
    if (err == cudaSuccess) return MOE_OK;
    cudaGetLastError();
    return MOE_ERR_CUDA;
}

moe_status check_product(const moe_product *p) {
    if (!p || !p->w) return MOE_ERR_INVALID_ARG;
    if (p->dtype == MOE_DTYPE_F32) return MOE_ERR_UNSUPPORTED;
    if (p->dtype != MOE_DTYPE_BF16 && p->dtype != MOE_DTYPE_F16) return MOE_ERR_INVALID_ARG;
    if (p->E < 1 || p->N < 1 || p->K < 1) return MOE_ERR_INVALID_ARG;
    if (p->E > kMaxE || p->N > kMaxN || p->K > kMaxK || p->K % 8) return MOE_ERR_UNSUPPORTED;
    if (p->ldw < p->K || p->ldw % 8 || p->ldw > (1LL << 32)) return MOE_ERR_INVALID_ARG;
    if (p->E > 1 && (p->stride_e < 0 || p->stride_e % 8 || p->stride_e > (1LL << 36))) return MOE_ERR_INVALID_ARG;
    if (misaligned(p->w, 16) || misaligned(p->w_up, 16) || misaligned(p->bias, 2) || misaligned(p->bias_up, 2))
        return MOE_ERR_INVALID_ARG;
    if (p->bias_up && !p->w_up) return MOE_ERR_INVALID_ARG;
    if (p->activation < MOE_EPI_NONE || p->activation > MOE_EPI_GELU_TANH) return MOE_ERR_INVALID_ARG;
    // finite and not negative (NaN fails); a clamp needs both products
    if (!(p->act_limit >= 0.0f && p->act_limit <= 3.0e38f) || (p->act_limit > 0.0f && !p->w_up))
        return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

// rows `ld` elements apart that hold `cols` elements each
bool bad_rows(int64_t ld, int64_t cols) { return ld < cols || ld > (1LL << 32); }

Product product_of(const moe_product *p) {
    Product a{};
    a.w = p->w;
    a.w_up = p->w_up;
    a.bias = p->bias;
    a.bias_up = p->bias_up;
    a.ldw = p->ldw;
    a.stride_e = p->E > 1 ? p->stride_e : 0;
    a.E = p->E;
    a.N = p->N;
    a.K = p->K;
    a.dtype = p->dtype;
    a.act = p->activation;
    a.limit = p->act_limit;
    return a;
}

// Which kernel. Streaming (ops_rows.cu) has the shorter way from launch to result,
// tcgen05 (ops_gemm.cu) the higher rate once a product is long enough to fill it. By
// the rows of a typical group and the bytes of weights read (us, streamed / tcgen05):
//   2048x2048             48 rows  7.5 / 7.6    64 rows  8.1 / 7.6
//   4096x4096             32 rows 11.0 / 13.7   48 rows 16.5 / 13.7
//   8192x4096             16 rows 14.6 / 17.6   24 rows 24.2 / 17.7
//   768x2048 gated        32 rows  6.6 / 10.3   48 rows 11.1 / 10.3
//   8 of 128 experts, 768x2048 gated, one row each  11.9 / 16.4 (50 MB)
//   6 of 256 experts, 2048x4096 gated, one row each 40.1 / 35.7 (201 MB)
// Groups besides stream only up to 64 rows in all, because only the device knows how
// they fall: 64 experts of 256x512, 64 rows 5.4 / 7.1 one on each and 11.5 / 6.8 all on
// one; 256 rows 5.6 / 7.0 and 41.0 / 9.1.
bool streams(const Product &a) {
    const int groups = a.offsets ? min(a.E, a.rows) : 1;
    const int mean = (a.rows + groups - 1) / groups;
    const double mb = 2e-6 * groups * a.N * (double)a.K * (a.w_up ? 2 : 1);
    const double work = mb * ((mean + 7) / 8);  // rows cost in blocks of 8
    if (a.offsets) return a.rows <= 64 && work <= 60.0;
    return mean <= 32 ? work <= 150.0 : mean <= 64 && !a.w_up && work <= 55.0;
}

moe_status run(const Product &a, cudaStream_t st) {
    if (!streams(a)) {
        const cudaError_t err = launch_product_gemm(a, st);
        if (err != cudaErrorNotSupported) return of(err);
    }
    return of(launch_product_rows(a, st));
}

}  // namespace

extern "C" {

moe_status moe_linear(const moe_product *p, const void *x, int64_t ldx, int n, const void *residual, int64_t ldr,
                      void *out, int64_t ldo, void *stream) {
    const moe_status bad = check_product(p);
    if (bad != MOE_OK) return bad;
    if (!x || !out || n < 0 || p->E != 1) return MOE_ERR_INVALID_ARG;
    if (n > kMaxRows) return MOE_ERR_UNSUPPORTED;
    if (bad_rows(ldx, p->K) || ldx % 8 || bad_rows(ldo, p->N) || (residual && bad_rows(ldr, p->N)))
        return MOE_ERR_INVALID_ARG;
    if (misaligned(x, 16) || misaligned(out, 2) || misaligned(residual, 2) || out == x) return MOE_ERR_INVALID_ARG;
    if (residual == out && ldr != ldo) return MOE_ERR_INVALID_ARG;
    if (n == 0) return MOE_OK;
    Product a = product_of(p);
    a.x = x;
    a.ldx = ldx;
    a.x_rows = a.rows = n;
    a.residual = residual;
    a.ldr = ldr;
    a.out = out;
    a.ldo = ldo;
    return run(a, static_cast<cudaStream_t>(stream));
}

moe_status moe_grouped_linear(const moe_product *p, const int32_t *offsets, const int32_t *row_token, const void *x,
                              int64_t ldx, int x_rows, int rows, void *out, int64_t ldo, void *stream) {
    const moe_status bad = check_product(p);
    if (bad != MOE_OK) return bad;
    if (!offsets || !x || !out || rows < 0 || x_rows < 0) return MOE_ERR_INVALID_ARG;
    if (rows > kMaxRows || x_rows > kMaxRows) return MOE_ERR_UNSUPPORTED;
    if (bad_rows(ldx, p->K) || ldx % 8 || bad_rows(ldo, p->N)) return MOE_ERR_INVALID_ARG;
    if (misaligned(x, 16) || misaligned(out, 2) || misaligned(offsets, 4) || misaligned(row_token, 4) || out == x)
        return MOE_ERR_INVALID_ARG;
    if (rows > 0 && (row_token ? x_rows == 0 : x_rows < rows)) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    Product a = product_of(p);
    a.x = x;
    a.ldx = ldx;
    a.x_rows = x_rows;
    a.rows = rows;
    a.offsets = offsets;
    a.row_token = row_token;
    a.out = out;
    a.ldo = ldo;
    return run(a, static_cast<cudaStream_t>(stream));
}

moe_status moe_group_slots(const int32_t *topk_idx, int n, int top_k, int E, int expert_begin, int expert_end,
                           int32_t *offsets, int32_t *slot_token, int32_t *slot_k, int32_t *slot_of, void *stream) {
    if (!topk_idx || !offsets || !slot_token || !slot_of || n < 0 || top_k < 1 || E < 1) return MOE_ERR_INVALID_ARG;
    if (expert_begin < 0 || expert_begin > expert_end || expert_end > E) return MOE_ERR_INVALID_ARG;
    if (misaligned(topk_idx, 4) || misaligned(offsets, 4) || misaligned(slot_token, 4) || misaligned(slot_k, 4) ||
        misaligned(slot_of, 4))
        return MOE_ERR_INVALID_ARG;
    if (E > kMaxE || top_k > kMaxRanks || (long long)n * top_k > kMaxRows) return MOE_ERR_UNSUPPORTED;
    return of(launch_group_slots(topk_idx, n, top_k, E, expert_begin, expert_end, offsets, slot_token, slot_k, slot_of,
                                 static_cast<cudaStream_t>(stream)));
}

moe_status moe_combine_slots(int dtype, const void *y, int64_t ldy, int rows, const int32_t *slot_of,
                             const float *topk_w, int n, int top_k, int N, const void *residual, int64_t ldr,
                             void *out, int64_t ldo, void *stream) {
    if ((!y && rows != 0) || !slot_of || !topk_w || !out || rows < 0 || n < 0 || top_k < 1 || N < 1)
        return MOE_ERR_INVALID_ARG;
    if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F16) return MOE_ERR_UNSUPPORTED;
    if (top_k > kMaxRanks || N > kMaxN || n > kMaxRows) return MOE_ERR_UNSUPPORTED;
    if (bad_rows(ldy, N) || bad_rows(ldo, N) || (residual && bad_rows(ldr, N))) return MOE_ERR_INVALID_ARG;
    if (misaligned(y, 2) || misaligned(out, 2) || misaligned(residual, 2) || misaligned(slot_of, 4) ||
        misaligned(topk_w, 4) || out == y || (residual == out && ldr != ldo))
        return MOE_ERR_INVALID_ARG;
    if (n == 0) return MOE_OK;
    return of(launch_combine_slots(dtype, y, ldy, rows, slot_of, topk_w, n, top_k, N, residual, ldr, out, ldo,
                                   static_cast<cudaStream_t>(stream)));
}

moe_status moe_ops_check(void *stream) {
    unsigned status = 0;
    const moe_status st = of(read_ops_status(&status, static_cast<cudaStream_t>(stream)));
    return st != MOE_OK ? st : status ? MOE_ERR_TIMEOUT : MOE_OK;
}

}  // extern "C"
