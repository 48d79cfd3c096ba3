// ops_route.cu -- routing to experts (moe_route): scores, groups, top-k, weights.
//
//   s_e = softmax(l)_e or 1 / (1 + exp(-l_e)),  c_e = s_e + bias_e
//   the top_groups groups with the best sum of their best one or two c_e stay;
//   ids = the top_k experts by c_e in them, ties to the lower id;
//   w_j = s of the j-th, divided by the sum of all of them if asked, times scale.
//
// Bound: latency for a few rows, the issue of instructions for many (a row is E logits, a few
// hundred bytes). One warp takes a row: lane i holds the V experts V i .. V i + V - 1, which
// makes the lowest lane of a tie the lowest id. A key is its f32 as an unsigned number that
// sorts alike (0: not available). The keys lie in shared memory and each lane keeps the
// largest of its own, so that a rank is one redux over the lanes, and another over the V keys
// of the lane that had it, which V lanes read side by side: about 25 instructions whatever V
// is (50 for V = 8 and 160 for V = 32 with the keys in registers).
//
// The ids are those of exact scores. Without a bias the order of c is the order of the
// logits, and no score is computed for it. With a bias (or with sums of two per group)
// c is computed in f32, the ranks are taken to top_k + 1 places, and wherever two
// neighbours are nearer to each other than the f32 errors (below), the row is ranked
// again in f64, over the experts that can still be among the first. For trained
// routers that is one row in some thousands.
#include "ops_common.cuh"
#include "ptx.cuh"

namespace moe {
namespace ops {
namespace {

constexpr int kWarps = 4;
constexpr unsigned kAll = 0xffffffffu;

// Error of an f32 score of a key (at most 1). Sigmoid: the argument's rounding moves the result
// by at most |l| s (1 - s) 2^-24 < 2^-26, exp2 and the reciprocal are good to 2^-22, 1 + e rounds
// to 2^-24: together below 2^-21. A softmax also rounds l - max and its product with log2(e) (error times score at
// most 2^-24) and sums up to 32 terms in a lane and 5 across, 37 roundings of 2^-24.
constexpr float kSigmoidErr = 0x1p-21f, kSoftmaxErr = 0x1p-18f;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ uint32_t sortable(float v) {
    const uint32_t b = __float_as_uint(v);
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float unsortable(uint32_t k) {
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

__device__ __forceinline__ float logit(const RouteArgs &a, long long row, int e) {
    const long long i = row * a.ldl + e;
    if (a.dtype == MOE_DTYPE_F32) return static_cast<const float *>(a.logits)[i];
    if (a.dtype == MOE_DTYPE_BF16) return to_f32(static_cast<const __nv_bfloat16 *>(a.logits)[i]);
    return to_f32(static_cast<const __half *>(a.logits)[i]);
}

// an expert whose logit is -inf or NaN, or whose bias is, takes no part
__device__ __forceinline__ bool takes_part(float v) { return v > -INFINITY; }

// scores for keys, to the errors above
__device__ __forceinline__ float sigmoid_key(float l) { return rcp_fast(1.0f + exp2_fast(-kLog2e * l)); }
__device__ __forceinline__ float exp_key(float l, float m) { return l == m ? 1.f : exp2_fast(kLog2e * (l - m)); }

// 1 / (1 + exp(-l)), also where it is subnormal
__device__ __forceinline__ float sigmoid(float l) {
    const float t = expf(-fabsf(l));
    return (l >= 0.f ? 1.f : t) / (1.0f + t);
}
__device__ __forceinline__ double sigmoid(double l) {
    const double t = exp(-fabs(l));
    return (l >= 0.0 ? 1.0 : t) / (1.0 + t);
}

// l - m with m >= l, where infinities of both are equal
__device__ __forceinline__ float below(float l, float m) { return l == m ? 0.f : l - m; }

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, d));
    return v;
}
template <typename F> __device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
    return v;
}

// Which groups stay, as a mask of bits, by the keys of all experts in `key` (shared memory; f32
// as sortable numbers, or f64 with -inf for those not available). F: the precision. 32 / 2^ceil(log2 groups) lanes share a
// group. *gap: the distance of the worst group that stays from the best that does not
// (inf if there are not both). logits: the keys are logits, and a sum of two is one of
// their scores.
__device__ __forceinline__ float key_value(uint32_t k) { return k ? unsortable(k) : -INFINITY; }
__device__ __forceinline__ double key_value(double k) { return k; }

template <typename F, typename K>
__device__ unsigned best_groups(const RouteArgs &a, const K *key, float max_logit, bool logits, F *gap, F *worst) {
    const int lane = threadIdx.x & 31, size = a.E / a.groups;
    int per = 32;  // lanes per group
    while (32 / per < a.groups) per >>= 1;
    const int g = lane / per;
    const F none = -INFINITY;
    F m1 = none, m2 = none;
    if (g < a.groups)
        for (int i = lane % per; i < size; i += per) {
            const F v = key_value(key[g * size + i]);
            if (v > m1) {
                m2 = m1;
                m1 = v;
            } else if (v > m2) {
                m2 = v;
            }
        }
    for (int d = 1; d < per; d <<= 1) {
        const F o1 = __shfl_xor_sync(kAll, m1, d), o2 = __shfl_xor_sync(kAll, m2, d);
        const F lo = o1 < m1 ? o1 : m1;
        m1 = o1 > m1 ? o1 : m1;
        m2 = o2 > m2 ? o2 : m2;
        m2 = lo > m2 ? lo : m2;
    }
    F score = m1;
    if (a.top2) {
        if (logits && m1 > none) {
            // (of a softmax without its common divisor)
            auto s = [&](F v) -> F {
                if (v == none) return 0;
                if constexpr (sizeof(F) == 4)
                    return a.score == MOE_SCORE_SOFTMAX ? exp_key(v, max_logit) : sigmoid_key(v);
                else
                    return a.score == MOE_SCORE_SOFTMAX ? (v == (F)max_logit ? 1.0 : exp(v - (F)max_logit)) : sigmoid(v);
            };
            score = s(m1) + s(m2);
        } else if (m2 > none) {
            score = m1 + m2;
        }
    }
    int before = 0;
    for (int o = 0; o < a.groups; ++o) {
        const F s = __shfl_sync(kAll, score, o * per);
        before += s > score || (s == score && o < g);
    }
    const bool live = g < a.groups && m1 > none, stays = live && before < a.top_groups;
    F w = stays ? score : (F)INFINITY, b = live && !stays ? score : none;
    for (int d = 16; d; d >>= 1) {
        const F ow = __shfl_xor_sync(kAll, w, d), ob = __shfl_xor_sync(kAll, b, d);
        w = ow < w ? ow : w;
        b = ob > b ? ob : b;
    }
    *gap = w == (F)INFINITY || b == none ? (F)INFINITY : w - b;
    *worst = w;
    unsigned mask = 0;
    for (int o = 0; o < a.groups; ++o) mask |= ((__ballot_sync(kAll, stays) >> (o * per)) & 1u) << o;
    return mask;
}

// The row again in f64: the ids of ranks lane and 32 + lane (-1: none left). again: the
// groups too; otherwise only experts with a key (of those left in `list`) of at least
// `from`, and those of `ids`, can be among the first. key: E doubles of this warp; list: its
// sortable keys, which the ids in question replace.
__device__ __noinline__ int2 rank_exactly(const RouteArgs &a, long long row, bool again, unsigned groups, float from,
                                          float max_logit, int2 ids, int next, double *key, uint32_t *list) {
    const int lane = threadIdx.x & 31, size = a.E / a.groups;
    const double none = -INFINITY;
    __syncwarp();
    double sum = 1.0;
    if (a.score == MOE_SCORE_SOFTMAX && a.bias) {
        sum = 0.0;
        for (int e = lane; e < a.E; e += 32) {
            const float l = logit(a, row, e);
            if (takes_part(l)) sum += l == max_logit ? 1.0 : exp((double)l - (double)max_logit);
        }
        sum = warp_sum(sum);
    }
    // the experts in question are dealt to the lanes: an f64 exponential takes a warp as
    // long for one lane as for 32
    int found = 0;
    auto add = [&](bool take, int e) {
        const unsigned m = __ballot_sync(0xffffffffu, take);
        if (take) list[found + __popc(m & ((1u << lane) - 1u))] = (uint32_t)e;
        found += __popc(m);
    };
    for (int e0 = 0; e0 < a.E; e0 += 32) {
        const int e = e0 + lane;
        bool take = false;
        if (e < a.E) {
            if (again) take = takes_part(logit(a, row, e)) && (!a.bias || takes_part(a.bias[e]));
            else take = list[e] && unsortable(list[e]) >= from;
        }
        __syncwarp();
        add(take, e);  // (never beyond what has been read)
        __syncwarp();
    }
    if (!again) {  // the ranks so far, and the next one, have no keys any more
        add(ids.x >= 0, ids.x);
        add(ids.y >= 0, ids.y);
        add(lane == 0 && next >= 0, next);
    }
    __syncwarp();
    auto score = [&](int e) -> double {
        const float l = logit(a, row, e);
        if (!a.bias) return l;  // the order of the logits
        const double s = a.score == MOE_SCORE_SOFTMAX
                             ? (l == max_logit ? 1.0 : exp((double)l - (double)max_logit)) / sum
                             : sigmoid((double)l);
        return s + (double)a.bias[e];
    };
    int2 out = make_int2(-1, -1);
    if (!again && found <= 32 && a.k <= 32) {
        // one each: a rank is the number of lanes that come before
        const int e = lane < found ? (int)list[lane] : 0x7fffffff;
        const double c = lane < found ? score(e) : none;
        int rank = 0;
        for (int i = 0; i < found; ++i) {
            const double o = __shfl_sync(0xffffffffu, c, i);
            const int oe = __shfl_sync(0xffffffffu, e, i);
            rank += o > c || (o == c && oe < e);
        }
        __syncwarp();
        if (lane < found) list[rank] = (uint32_t)e;
        __syncwarp();
        if (lane < a.k && lane < found) out.x = (int)list[lane];
        return out;
    }
    if (again)
        for (int e = lane; e < a.E; e += 32) key[e] = none;
    __syncwarp();
    for (int i = lane; i < found; i += 32) key[list[i]] = score((int)list[i]);
    __syncwarp();
    if (again && a.groups > 1) {
        double gap, worst;
        groups = best_groups<double>(a, key, max_logit, !a.bias, &gap, &worst);
    }
    for (int j = 0; j < a.k; ++j) {
        double best = none;
        int at = 0x7fffffff;
        for (int i = lane; i < found; i += 32) {
            const int e = (int)list[i];
            const double c = key[e];
            if (((groups >> (e / size)) & 1u) && (c > best || (c == best && c > none && e < at))) {
                best = c;
                at = e;
            }
        }
        for (int d = 16; d; d >>= 1) {
            const double ob = __shfl_xor_sync(0xffffffffu, best, d);
            const int oa = __shfl_xor_sync(0xffffffffu, at, d);
            if (ob > best || (ob == best && oa < at)) {
                best = ob;
                at = oa;
            }
        }
        const bool none_left = !(best > none);
        if (lane == (j & 31)) (j < 32 ? out.x : out.y) = none_left ? -1 : at;
        if (!none_left && lane == 0) key[at] = none;
        __syncwarp();
    }
    return out;
}

template <int V>
__global__ void __launch_bounds__(32 * kWarps) route_kernel(const RouteArgs a) {
    extern __shared__ __align__(16) double scratch[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long row = (long long)blockIdx.x * kWarps + warp;
    ptx::griddep_wait();
    if (row >= a.n) return;
    double *mine = scratch + (size_t)warp * a.scratch;
    uint32_t *keys = reinterpret_cast<uint32_t *>(mine + (a.scratch - a.keys));
    const int e0 = lane * V;

    // the logits, and the largest of them that takes part
    float l[V];
    const size_t esz = a.dtype == MOE_DTYPE_F32 ? 4 : 2;
    const char *src = static_cast<const char *>(a.logits) + ((size_t)row * a.ldl + e0) * esz;
    if (a.vector && e0 + V <= a.E) {
        if (a.dtype == MOE_DTYPE_F32) {
            if constexpr (V >= 4) {
#pragma unroll
                for (int j = 0; j < V / 4; ++j) {
                    const float4 v = reinterpret_cast<const float4 *>(src)[j];
                    l[4 * j] = v.x;
                    l[4 * j + 1] = v.y;
                    l[4 * j + 2] = v.z;
                    l[4 * j + 3] = v.w;
                }
            }
        } else {
            uint32_t v[V / 2];
            if constexpr (V == 4) {
                const uint2 w = *reinterpret_cast<const uint2 *>(src);
                v[0] = w.x;
                v[1] = w.y;
            } else {
#pragma unroll
                for (int j = 0; j < V / 8; ++j) {
                    const uint4 w = reinterpret_cast<const uint4 *>(src)[j];
                    v[4 * j] = w.x;
                    v[4 * j + 1] = w.y;
                    v[4 * j + 2] = w.z;
                    v[4 * j + 3] = w.w;
                }
            }
#pragma unroll
            for (int j = 0; j < V / 2; ++j) {
                const float2 f = a.dtype == MOE_DTYPE_BF16 ? unpack2<__nv_bfloat16>(v[j]) : unpack2<__half>(v[j]);
                l[2 * j] = f.x;
                l[2 * j + 1] = f.y;
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) l[j] = e0 + j < a.E ? logit(a, row, e0 + j) : -INFINITY;
    }
    const bool softmax = a.score == MOE_SCORE_SOFTMAX;
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < V; ++j) m = fmaxf(m, l[j]);  // (a NaN is passed over)
    if (softmax) m = warp_max(m);

    // the divisor of a softmax, where its scores themselves are asked for
    float rcp_sum = 1.f;
    if (softmax && (a.bias || !a.renormalize)) {
        float t = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (takes_part(l[j])) t += expf(below(l[j], m));
        rcp_sum = 1.0f / warp_sum(t);
    }

    // sortable keys; 0: takes no part
    uint32_t key[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        float c = l[j];
        bool ok = takes_part(c);
        if (a.bias && ok) {
            const float b = a.bias[e0 + j];
            ok = takes_part(b);
            c = (softmax ? exp_key(c, m) * rcp_sum : sigmoid_key(c)) + b;
        }
        key[j] = ok ? sortable(c + 0.f) : 0u;  // (-0 ties with 0)
    }
    const float err = softmax ? kSoftmaxErr : kSigmoidErr;

    if (V % 4 == 0 && e0 + V <= a.E) {
#pragma unroll
        for (int j = 0; j < V / 4; ++j)
            reinterpret_cast<uint4 *>(keys + e0)[j] = make_uint4(key[4 * j], key[4 * j + 1], key[4 * j + 2], key[4 * j + 3]);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (e0 + j < a.E) keys[e0 + j] = key[j];
    }
    __syncwarp();

    unsigned groups = 1u;
    bool unsure = false, again = false;
    if (a.groups > 1) {
        float gap, worst;
        groups = best_groups<float>(a, keys, m, !a.bias, &gap, &worst);
        // errors of two sums of one or two keys
        if ((a.bias || a.top2) && !(gap > 2.f * (2.f * err + 0x1p-22f * fabsf(worst)))) unsure = again = true;
        const int size = a.E / a.groups;
        int g = e0 / size, left = size - (e0 - g * size);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (g >= 32 || !((groups >> g) & 1u)) {
                key[j] = 0u;
                if (e0 + j < a.E) keys[e0 + j] = 0u;
            }
            if (--left == 0) {
                ++g;
                left = size;
            }
        }
        __syncwarp();
    }

    int2 ids = make_int2(-1, -1);  // of ranks lane and 32 + lane
    if (!unsure) {
        uint32_t best = key[0];  // of this lane's
#pragma unroll
        for (int j = 1; j < V; ++j) best = max(best, key[j]);
        float last = 0.f, from = 0.f;
        int last_at = -1, next = -1;
        const int ranks = a.bias ? a.k + 1 : a.k;
        for (int r = 0; r < ranks; ++r) {
            const uint32_t top = __reduce_max_sync(kAll, best);
            if (top == 0u) break;
            const int owner = __ffs(__ballot_sync(kAll, best == top)) - 1, first = owner * V;
            // its keys, one to a lane
            const uint32_t k = lane < V && first + lane < a.E ? keys[first + lane] : 0u;
            const int at_lane = __ffs(__ballot_sync(kAll, k == top)) - 1, at = first + at_lane;
            const uint32_t rest = __reduce_max_sync(kAll, lane == at_lane ? 0u : k);
            if (lane == owner) best = rest;
            if (lane == at_lane) keys[at] = 0u;
            if (r == a.k) next = at;
            else if (lane == (r & 31)) (r < 32 ? ids.x : ids.y) = at;
            if (a.bias) {
                const float c = unsortable(top);
                const float near = 2.f * (err + 0x1p-23f * (fabsf(c) + fabsf(last)));
                // (the same logit and the same bias are an exact tie)
                if (r && !(last - c > near) &&
                    (logit(a, row, at) != logit(a, row, last_at) || a.bias[at] != a.bias[last_at]))
                    unsure = true;
                from = c == INFINITY ? 3.0e38f : c - 2.f * near;
                last = c;
                last_at = at;
            }
            __syncwarp();
        }
        if (unsure) ids = rank_exactly(a, row, false, groups, from, m, ids, next, mine, keys);
    } else {
        ids = rank_exactly(a, row, again, groups, 0.f, m, ids, -1, mine, keys);
    }

    // weights: lane j has ranks j and 32 + j
    const int id[2] = {ids.x, ids.y};
    float z[2], w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) z[h] = id[h] >= 0 ? logit(a, row, id[h]) : -INFINITY;
    float top = -INFINITY;
    if (a.renormalize) top = warp_max(fmaxf(z[0], z[1]));
    // relative to the largest chosen logit where that keeps small scores in range: they are
    // divided by their sum. (exp(l) is all of a sigmoid below -40.)
    const bool shifted = a.renormalize && (softmax || top < -40.f);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (id[h] < 0) w[h] = 0.f;
        else if (shifted) w[h] = expf(below(z[h], top));
        else w[h] = softmax ? expf(below(z[h], m)) * rcp_sum : sigmoid(z[h]);
    }
    float by = a.scale;
    if (a.renormalize) {
        const float sum = warp_sum(w[0] + w[1]);
        by = sum > 0.f ? a.scale / sum : 0.f;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = lane + 32 * h;
        if (r < a.k) {
            a.topk_idx[row * a.k + r] = id[h];
            a.topk_w[row * a.k + r] = w[h] * by;
        }
    }
}

template <int V>
cudaError_t launch(RouteArgs a, cudaStream_t st) {
    const int esz = a.dtype == MOE_DTYPE_F32 ? 4 : 2;
    const unsigned piece = min(16, V * esz);  // bytes of a load
    a.vector = ((uintptr_t)a.logits % piece) == 0 && (a.ldl * esz) % piece == 0;
    // E keys; and E in f64 where a row may have to be ranked again
    a.keys = (a.E + 3) / 4 * 2;
    a.scratch = a.keys + (a.bias || (a.groups > 1 && a.top2) ? (a.E + 1) / 2 * 2 : 0);  // (of 16 bytes' alignment)
    const int smem = kWarps * a.scratch * 8;  // at most 48 KB
    return launch_overlapped(route_kernel<V>, dim3((unsigned)((a.n + kWarps - 1) / kWarps)), 32 * kWarps, smem, 1, st, a);
}

}  // namespace

cudaError_t launch_route(const RouteArgs &a, cudaStream_t st) {
    if (a.E <= 128) return launch<4>(a, st);
    if (a.E <= 256) return launch<8>(a, st);
    if (a.E <= 512) return launch<16>(a, st);
    return launch<32>(a, st);
}

}  // namespace ops
}  // namespace moe
