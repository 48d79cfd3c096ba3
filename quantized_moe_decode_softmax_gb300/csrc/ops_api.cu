// ops_api.cu -- the C entry points of moe_ops.h: argument checks and dispatch.
//
// As for the step (mlxcel issue #1616, Implementation Notes), shapes are
// validated before any dispatch and what the kernels do not cover is declined.
#include <cuda_runtime.h>

#include "ops_internal.h"

using namespace moe::ops;

namespace {

constexpr int kMaxE = 1024, kMaxK = 65536, kMaxN = 1 << 20, kMaxRows = 1 << 24, kMaxRanks = 64;
constexpr long long kMaxSlots = 1 << 24;  // as moe_group_slots takes

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

moe_status check_product_q8(const moe_product_q8 *p) {
    if (!p || !p->w || !p->scale || (p->w_up && !p->scale_up)) return MOE_ERR_INVALID_ARG;
    if (p->dtype == MOE_DTYPE_F32) return MOE_ERR_UNSUPPORTED;
    if (p->dtype != MOE_DTYPE_BF16 && p->dtype != MOE_DTYPE_F16) return MOE_ERR_INVALID_ARG;
    if (p->E < 1 || p->N < 1 || p->K < 1) return MOE_ERR_INVALID_ARG;
    if (p->E > kMaxE || p->N > kMaxN || p->K > kMaxK || p->K % 16) return MOE_ERR_UNSUPPORTED;
    if (p->ldw < p->K || p->ldw % 16 || p->ldw > (1LL << 32)) return MOE_ERR_INVALID_ARG;
    if (p->E > 1 && (p->stride_e < 0 || p->stride_e % 16 || p->stride_e > (1LL << 36))) return MOE_ERR_INVALID_ARG;
    if (misaligned(p->w, 16) || misaligned(p->w_up, 16) || misaligned(p->bias, 2) || misaligned(p->bias_up, 2) ||
        misaligned(p->scale, 4) || misaligned(p->scale_up, 4))
        return MOE_ERR_INVALID_ARG;
    if ((p->bias_up || p->scale_up) && !p->w_up) return MOE_ERR_INVALID_ARG;
    if (p->activation < MOE_EPI_NONE || p->activation > MOE_EPI_GELU_TANH) return MOE_ERR_INVALID_ARG;
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

Product product_of(const moe_product_q8 *p) {
    Product a{};
    a.w = p->w;
    a.w_up = p->w_up;
    a.w_scale = p->scale;
    a.w_up_scale = p->scale_up;
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

// The same for 8-bit codes, with a third way for few rows: dot products (ops_dot_q8.cu), f16 on
// mma.sync (ops_rows_q8.cu), f16 on tcgen05 (ops_gemm_q8.cu). Measured (us, dot / mma.sync /
// tcgen05):
//   2048x2048              1 row  3.1 / 3.5 / 9.5     8 rows  3.7 / 3.5 / 9.5    64 rows  10.6 / 8.7 / 9.6
//   8192x4096              1 row  7.5 / 9.3 / 14.7   16 rows  18 / 12 / 14.4     24 rows  24 / 19.2 / 14.5
//   4096x4096             32 rows  16 / 10.1 / 13.8  48 rows  22 / 17.1 / 14.3
//   512x4096              32 rows  4.8 / 7.0 / 13.4  64 rows  5.5 / 11.9 / 13.8
//   1024x2048             64 rows  6.6 / 8.1 / 9.2  128 rows  10.5 / 14.5 / 9.5
//   2048x4096 gated       16 rows  10.7 / 8.3 / 20.5 64 rows  28 / 19.7 / 20.9
//   512x4096 gated        32 rows  5.5 / 11.6 / 20.5
//   768x2048 gated, 128 experts, top 8   1 token 6.6 / 9.5 / 16    16 tokens 47 / 63 / 53   32 tokens 82 / 78 / 65
//   the same, all on the same experts                              16 tokens 24 / 17 / 16
//   512x1024 gated, 8 experts, top 2     8 tokens 4.1 / 4.4 / 10   32 tokens 7.0 / 6.2 / 10.6
// From 8 to 128 rows none of them is near the bytes of the codes, and some calls take as long as 16-bit
// weights do, or longer (the chosen kernel / the 16-bit product of twice the bytes): 2048x2048 32 rows 4.6 / 4.4,
// 64 rows 8.8 / 7.9; 2048x4096 gated 64 rows 20.1 / 19.2; but 8192x4096 8 rows 8.0 / 13.7. A block of ops_rows_q8.cu
// converts all rows of x for 16 columns, and the weights again for every 32 rows; ops_gemm_q8.cu has a pair of
// SMs for 256 columns, so that narrow products leave most idle.
// Of a linear product the three are weighed by their times (us) as fitted to such figures: dot by
// bytes, bytes times rows in fours, and outputs; mma.sync by its walk along K, for more than 16
// rows in passes of 32 and rounds of 304 blocks of 16 columns; tcgen05 by its walk along K or the
// bytes. Of 900 calls drawn at random (40..12288 columns, 128..8192 inputs, 1..256 rows) the choice
// was more than 10 % slower than the best in 24, at most 24 %.
enum class Q8 { dot, rows, gemm };
Q8 kernel_q8(const Product &a) {
    const int groups = a.offsets ? min(a.E, a.rows) : 1, mats = a.w_up ? 2 : 1;
    const int mean = (a.rows + groups - 1) / groups;
    const double mb = 1e-6 * groups * a.N * (double)a.K * mats;
    if (a.offsets) {
        const double work = mb * ((mean + 7) / 8);  // rows cost in blocks of 8
        return a.rows <= 128 && mean <= 2 ? Q8::dot : a.rows <= 64 && work <= 60.0 ? Q8::rows : Q8::gemm;
    }
    const int n = a.rows;
    if (n > 256) return Q8::gemm;
    const double k = a.K / 1024.0;
    const int fours = n == 1 ? 1 : (n + 3) / 4 * 4, blocks = (a.N + 15) / 16;
    const double dot = 1.8 + mb * (0.1 + 0.0215 * fours) + 3e-5 * a.N * mats * fours;
    const double per_k = n <= 8 ? (mats == 2 ? 1.05 : 0.48) : n <= 16 ? (mats == 2 ? 1.5 : 0.6)
                         : blocks <= 152 ? (mats == 2 ? 2.3 : 1.33) : (mats == 2 ? 2.9 : 1.9);
    const double rows = n <= 16 ? 1.4 + max(1.0, a.N / 2048.0) * ((mats == 2 ? 0.6 : 0.45) + k * per_k)
                                : 1.2 + (n + 31) / 32 * ((blocks + 303) / 304) * ((mats == 2 ? 2.2 : 1.3) + k * per_k);
    const double gemm = max(mats == 2 ? 5.6 + 3.7 * k : 4.4 + 2.15 * k, 4.0 + 0.25 * mb);
    if (dot < gemm && (n > 64 || dot < rows)) return Q8::dot;
    return n <= 64 && rows < gemm ? Q8::rows : Q8::gemm;
}

moe_status run_q8(const Product &a, cudaStream_t st) {
    const Q8 k = kernel_q8(a);
    if (k == Q8::dot) return of(launch_product_dot_q8(a, st));
    if (k == Q8::gemm) {
        const cudaError_t err = launch_product_gemm_q8(a, st);
        if (err != cudaErrorNotSupported) return of(err);
    }
    return of(launch_product_rows_q8(a, st));
}

// both status words of the current device, or'ed; cleared if one was set
cudaError_t read_status(unsigned *value, cudaStream_t st) {
    *value = 0;
    cudaError_t err;
    unsigned word[2] = {0, 0}, *at[2];
    at[0] = ops_status(&err);
    if (err == cudaSuccess) at[1] = ops_status_q8(&err);
    for (int i = 0; i < 2 && err == cudaSuccess; ++i) err = cudaMemcpyAsync(&word[i], at[i], 4, cudaMemcpyDeviceToHost, st);
    if (err == cudaSuccess) err = cudaStreamSynchronize(st);
    if (err != cudaSuccess) return err;
    *value = word[0] | word[1];
    if (*value == 0) return err;
    for (int i = 0; i < 2 && err == cudaSuccess; ++i) err = cudaMemsetAsync(at[i], 0, 4, st);
    return err == cudaSuccess ? cudaStreamSynchronize(st) : err;
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

moe_status moe_linear_q8(const moe_product_q8 *p, const int8_t *x, int64_t ldx, const float *x_scale, int n,
                         const void *residual, int64_t ldr, void *out, int64_t ldo, void *stream) {
    const moe_status bad = check_product_q8(p);
    if (bad != MOE_OK) return bad;
    if (!x || !x_scale || !out || n < 0 || p->E != 1) return MOE_ERR_INVALID_ARG;
    if (n > kMaxRows) return MOE_ERR_UNSUPPORTED;
    if (bad_rows(ldx, p->K) || ldx % 16 || bad_rows(ldo, p->N) || (residual && bad_rows(ldr, p->N)))
        return MOE_ERR_INVALID_ARG;
    if (misaligned(x, 16) || misaligned(x_scale, 4) || misaligned(out, 2) || misaligned(residual, 2) || out == x ||
        out == x_scale || (residual == out && ldr != ldo))
        return MOE_ERR_INVALID_ARG;
    if (n == 0) return MOE_OK;
    Product a = product_of(p);
    a.x = x;
    a.x_scale = x_scale;
    a.ldx = ldx;
    a.x_rows = a.rows = n;
    a.residual = residual;
    a.ldr = ldr;
    a.out = out;
    a.ldo = ldo;
    return run_q8(a, static_cast<cudaStream_t>(stream));
}

moe_status moe_grouped_linear_q8(const moe_product_q8 *p, const int32_t *offsets, const int32_t *row_token,
                                 const int8_t *x, int64_t ldx, const float *x_scale, int x_rows, int rows, void *out,
                                 int64_t ldo, void *stream) {
    const moe_status bad = check_product_q8(p);
    if (bad != MOE_OK) return bad;
    if (!offsets || !x || !x_scale || !out || rows < 0 || x_rows < 0) return MOE_ERR_INVALID_ARG;
    if (rows > kMaxRows || x_rows > kMaxRows) return MOE_ERR_UNSUPPORTED;
    if (bad_rows(ldx, p->K) || ldx % 16 || bad_rows(ldo, p->N)) return MOE_ERR_INVALID_ARG;
    if (misaligned(x, 16) || misaligned(x_scale, 4) || misaligned(out, 2) || misaligned(offsets, 4) ||
        misaligned(row_token, 4) || out == x || out == x_scale)
        return MOE_ERR_INVALID_ARG;
    if (rows > 0 && (row_token ? x_rows == 0 : x_rows < rows)) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    Product a = product_of(p);
    a.x = x;
    a.x_scale = x_scale;
    a.ldx = ldx;
    a.x_rows = x_rows;
    a.rows = rows;
    a.offsets = offsets;
    a.row_token = row_token;
    a.out = out;
    a.ldo = ldo;
    return run_q8(a, static_cast<cudaStream_t>(stream));
}

moe_status moe_quantize_rows(int dtype, const void *x, int64_t ldx, int n, int K, int8_t *codes, int64_t ldc,
                             float *scale, void *stream) {
    if (!x || !codes || !scale || n < 0 || K < 1) return MOE_ERR_INVALID_ARG;
    if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F16) return MOE_ERR_UNSUPPORTED;
    if (n > kMaxRows || K > kMaxN) return MOE_ERR_UNSUPPORTED;
    if (bad_rows(ldx, K) || bad_rows(ldc, K) || misaligned(x, 2) || misaligned(scale, 4) || x == codes ||
        x == (const void *)scale || (const void *)codes == (const void *)scale)
        return MOE_ERR_INVALID_ARG;
    if (n == 0) return MOE_OK;
    return of(launch_quantize_rows(dtype, x, ldx, n, K, codes, ldc, scale, static_cast<cudaStream_t>(stream)));
}

moe_status moe_route(const moe_router *r, int dtype, const void *logits, int64_t ldl, int n, int32_t *topk_idx,
                     float *topk_w, void *stream) {
    if (!r || !logits || !topk_idx || !topk_w || n < 0) return MOE_ERR_INVALID_ARG;
    if (r->E < 1 || r->top_k < 1 || r->groups < 1 || r->top_groups < 1 || r->top_groups > r->groups ||
        r->E % r->groups)
        return MOE_ERR_INVALID_ARG;
    if (r->score != MOE_SCORE_SOFTMAX && r->score != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
    if (r->group_best != 1 && r->group_best != 2) return MOE_ERR_INVALID_ARG;
    if (r->top_k > (long long)r->top_groups * (r->E / r->groups)) return MOE_ERR_INVALID_ARG;
    if (!(r->scale >= -3.0e38f && r->scale <= 3.0e38f)) return MOE_ERR_INVALID_ARG;
    if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F16 && dtype != MOE_DTYPE_F32) return MOE_ERR_INVALID_ARG;
    if (r->E > kMaxE || r->top_k > kMaxRanks || r->groups > 32 || n > kMaxRows || (long long)n * r->top_k > kMaxSlots)
        return MOE_ERR_UNSUPPORTED;
    const unsigned size = dtype == MOE_DTYPE_F32 ? 4 : 2;
    if (bad_rows(ldl, r->E) || misaligned(logits, size) || misaligned(r->bias, 4) || misaligned(topk_idx, 4) ||
        misaligned(topk_w, 4) || (const void *)topk_idx == (const void *)topk_w || logits == (const void *)topk_idx ||
        logits == (const void *)topk_w)
        return MOE_ERR_INVALID_ARG;
    if (n == 0) return MOE_OK;
    RouteArgs a{};
    a.logits = logits;
    a.bias = r->bias;
    a.topk_idx = topk_idx;
    a.topk_w = topk_w;
    a.ldl = ldl;
    a.n = n;
    a.E = r->E;
    a.k = r->top_k;
    a.dtype = dtype;
    a.score = r->score;
    a.groups = r->top_groups < r->groups ? r->groups : 1;  // all of them stay: no groups
    a.top_groups = r->top_groups;
    a.top2 = r->group_best == 2;
    a.renormalize = r->renormalize != 0;
    a.scale = r->scale;
    return of(launch_route(a, static_cast<cudaStream_t>(stream)));
}

moe_status moe_group_slots(const int32_t *topk_idx, int n, int top_k, int E, int expert_begin, int expert_end,
                           int32_t *offsets, int32_t *slot_token, int32_t *slot_k, int32_t *slot_of, void *stream) {
    if (!topk_idx || !offsets || !slot_token || !slot_of || n < 0 || top_k < 1 || E < 1) return MOE_ERR_INVALID_ARG;
    if (expert_begin < 0 || expert_begin > expert_end || expert_end > E) return MOE_ERR_INVALID_ARG;
    if (misaligned(topk_idx, 4) || misaligned(offsets, 4) || misaligned(slot_token, 4) || misaligned(slot_k, 4) ||
        misaligned(slot_of, 4))
        return MOE_ERR_INVALID_ARG;
    if (E > kMaxE || top_k > kMaxRanks || (long long)n * top_k > kMaxSlots) return MOE_ERR_UNSUPPORTED;
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
    const moe_status st = of(read_status(&status, static_cast<cudaStream_t>(stream)));
    return st != MOE_OK ? st : status ? MOE_ERR_TIMEOUT : MOE_OK;
}

}  // extern "C"
