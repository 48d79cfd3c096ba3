// ops_route.cu -- routing to experts (moe_route): scores, groups, top-k, weights.
//
//   s_e = softmax(l)_e or 1 / (1 + exp(-l_e)),  c_e = s_e + bias_e
//   the top_groups groups with the best sum of their best one or two c_e stay;
//   ids = the top_k experts by c_e in them, ties to the lower id;
//   w_j = s of the j-th, divided by the sum of all of them if asked, times scale.
//
// Bound: latency, of launch and one row for a few rows, of the chain of dependent reductions that a
// row's ranks are for many (8192 x 256: 13 warps an SM issue 1.3 instructions a cycle, the integer pipe is 27 %
// busy, 4 % of HBM). L lanes take a row: all 32 of a warp, so that a row is done soon, or 8 where
// there are rows enough to fill the SMs, so that an instruction serves four rows (8192 x 256,
// top 6: 5.5 us, with a bias 9.0; a warp each 9.1 and 14). Lane i holds the V experts V i ..
// V i + V - 1, which makes the lowest lane of a tie the lowest id. A key is its f32 as an
// unsigned number that sorts alike (0: not available). Each lane keeps the largest of its own, so
// that a rank is one maximum over the lanes, and another over the V keys of the lane that had it:
// by that lane in its registers, or, of many keys or rows, by all lanes side by side in shared
// memory. One row of 128: 2.7 us, of which 1.4 an empty kernel would take.
//
// The ids are those of exact scores. Without a bias the order of c is the order of the
// logits, and no score is computed for it. With a bias (or with sums of two per group)
// c is computed in f32, and the ranks are taken to top_k + 1 places. Neighbours among the
// first top_k that are farther apart than the f32 errors (below), or tie exactly, stand in
// their exact order, and so do all of these by the chain of them. At the cut there is no chain: an
// expert far down may be off by more than the next one. So where the first expert left out is
// within the errors of the last one chosen, all that are left out and as near are compared with it. A row
// with a pair that this does not settle is ranked again, over the experts that can still be among
// the first: in pairs of f32 or in f64. For trained routers that is one row in some thousands.
#include "ops_common.cuh"
#include "ptx.cuh"

namespace moe {
namespace ops {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kMaxK = 64;
constexpr int kManyRows = 4096;  // rows from which on eight lanes take one

// Error of an f32 score of a key (at most 1). Sigmoid: the argument's rounding moves the result
// by at most |l| s (1 - s) 2^-24 < 2^-26, exp2 and the reciprocal are good to 2^-22, 1 + e rounds
// to 2^-24: together below 2^-21. A softmax also rounds l - max and its product with log2(e)
// (error times score at most 2^-24) and sums up to 32 terms in a lane and 5 across, 37
// roundings of 2^-24. Of a score p that is less than 2^-18 p + 2^-23 p log(1 / p), and the second
// term below 2^-23 sqrt(p).
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

__device__ __forceinline__ float sqrt_fast(float v) {  // to 2^-22
    float r;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// Whether keys c1 >= c2 of experts with these logits and biases may be in the wrong order: they are
// nearer than the errors of both (`near`, at the most), and no exact tie, which goes to the lower id.
__device__ __forceinline__ bool may_swap(bool softmax, float c1, float l1, float b1, float c2, float l2, float b2, float near) {
    if (c1 - c2 > near || (l1 == l2 && b1 == b2)) return false;
    if (!softmax) return true;
    // by the errors of these two scores, which are c - bias (317 x 256: 5 us, 11 with kSoftmaxErr)
    const float rounding = 0x1p-22f * (fabsf(c1) + fabsf(c2)), p = fmaxf(c1 - b1, c2 - b2) + rounding;
    return !(c1 - c2 > 2.f * (kSoftmaxErr * p + 0x1p-23f * sqrt_fast(p)) + rounding);
}

// over the L lanes of a row
template <int L> __device__ __forceinline__ float row_max(float v) {
#pragma unroll
    for (int d = L / 2; d; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, d));
    return v;
}
template <int L> __device__ __forceinline__ uint32_t row_max(uint32_t v) {
    if constexpr (L == 32) {
        return __reduce_max_sync(kAll, v);
    } else {
#pragma unroll
        for (int d = L / 2; d; d >>= 1) v = max(v, __shfl_xor_sync(kAll, v, d));
        return v;
    }
}
template <int L, typename F> __device__ __forceinline__ F row_sum(F v) {
#pragma unroll
    for (int d = L / 2; d; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
    return v;
}
// the lanes of the own row where `p` holds, the row's first lane in bit 0
template <int L> __device__ __forceinline__ unsigned row_ballot(bool p) {
    const unsigned m = __ballot_sync(kAll, p);
    if constexpr (L == 32) return m;
    else return (m >> (threadIdx.x & 31 & ~(L - 1))) & ((1u << L) - 1u);
}

// The place of expert e among a row's keys: the V of a lane and 4 more, so that 16-byte accesses of
// eight lanes side by side meet different banks.
template <int V> struct Keys {
    uint32_t *at;
    __device__ __forceinline__ static int place(int e) { return e / V * (V + 4) + e % V; }
    __device__ __forceinline__ uint32_t &operator[](int e) const { return at[place(e)]; }
};

__device__ __forceinline__ float key_value(uint32_t k) { return k ? unsortable(k) : -INFINITY; }
__device__ __forceinline__ double key_value(double k) { return k; }

// Which groups stay, as a mask of bits, by the keys of all experts (f32 as sortable numbers, or
// f64 with -inf for those not available), by the L lanes of a row; at most L groups, L / 2^ceil(log2
// groups) lanes share one. F: the precision. *settled (f32): whether every group that stays is ahead of
// all that do not by more than their errors; err is a score's, and what rounds in a sum of two goes
// by the size of its terms, which may cancel. logits: the keys are logits, and a sum of
// two is one of their scores. cut, unless null: for each group the least key that its score has.
template <int L, typename F, typename K>
__device__ __forceinline__ unsigned best_groups(const RouteArgs &a, const K &key, float max_logit, bool logits, float err,
                                                bool *settled, float *cut) {
    const int lane = threadIdx.x & (L - 1), size = a.E / a.groups;
    int per = L;  // lanes per group
    while (L / per < a.groups) per >>= 1;
    const int g = lane / per;
    const F none = -INFINITY;
    F m1 = none, m2 = none;
    if (g < a.groups)
        for (int i = lane % per; i < size; i += per) {
            const F v = key_value(key[g * size + i]);
            m2 = v > m1 ? m1 : v > m2 ? v : m2;
            m1 = v > m1 ? v : m1;
        }
    for (int d = 1; d < per; d <<= 1) {
        const F o1 = __shfl_xor_sync(kAll, m1, d), o2 = __shfl_xor_sync(kAll, m2, d);
        const F lo = o1 < m1 ? o1 : m1;
        m1 = o1 > m1 ? o1 : m1;
        m2 = o2 > m2 ? o2 : m2;
        m2 = lo > m2 ? lo : m2;
    }
    if (cut && g < a.groups && lane % per == 0) cut[g] = (float)(a.top2 && m2 > none ? m2 : m1);
    F score = m1, size_of = m1 < 0 ? -m1 : m1;  // size_of: of the terms
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
            score = size_of = s(m1) + s(m2);
        } else if (m2 > none) {
            score = m1 + m2;
            size_of += m2 < 0 ? -m2 : m2;
        }
    }
    int before = 0;
    for (int o = 0; o < a.groups; ++o) {
        const F s = __shfl_sync(kAll, score, o * per, L);
        before += s > score || (s == score && o < g);
    }
    const bool live = g < a.groups && m1 > none, stays = live && before < a.top_groups;
    if constexpr (sizeof(F) == 4) {
        // (without a bias the best one is a logit, which is exact)
        if (a.bias || a.top2) {
            const float by = 2.f * err + 0x1p-22f * size_of;
            float w = !stays ? INFINITY : by < INFINITY ? score - by : -INFINITY;
            float b = !live || stays ? -INFINITY : by < INFINITY ? score + by : INFINITY;
#pragma unroll
            for (int d = L / 2; d; d >>= 1) {
                w = fminf(w, __shfl_xor_sync(kAll, w, d));
                b = fmaxf(b, __shfl_xor_sync(kAll, b, d));
            }
            *settled = w > b;
        }
    }
    // bit o: group o's lanes, the first of each
    const unsigned lanes = row_ballot<L>(stays);
    unsigned mask = 0;
    for (int o = 0; o < a.groups; ++o) mask |= ((lanes >> (o * per)) & 1u) << o;
    return mask;
}

// c_e of one expert in f64 (without a bias its logit, which has the same order). sum: the divisor of a
// softmax
__device__ __forceinline__ double exact_key(const RouteArgs &a, long long row, int e, float max_logit, double sum) {
    const float l = logit(a, row, e);
    if (!a.bias) return l;
    const double s = a.score == MOE_SCORE_SOFTMAX ? (l == max_logit ? 1.0 : exp((double)l - (double)max_logit)) / sum
                                                  : sigmoid((double)l);
    return s + (double)a.bias[e];
}

__device__ __forceinline__ double exact_sum(const RouteArgs &a, long long row, float max_logit) {
    if (a.score != MOE_SCORE_SOFTMAX || !a.bias) return 1.0;
    double sum = 0.0;
    for (int e = threadIdx.x & 31; e < a.E; e += 32) {
        const float l = logit(a, row, e);
        if (takes_part(l)) sum += l == max_logit ? 1.0 : exp((double)l - (double)max_logit);
    }
    return row_sum<32>(sum);
}

// The experts whose key, among the row's keys at `list`, is at least what `least` says for them:
// their ids replace the keys, in order; how many. By a whole warp. (The experts in question
// are then dealt to the lanes: an f64 exponential takes a warp as long for one lane as for 32.)
template <int V, typename F> __device__ __forceinline__ int pick_experts(const RouteArgs &a, uint32_t *list, F least) {
    const int lane = threadIdx.x & 31;
    int found = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
        const int e = e0 + lane;
        const uint32_t k = e < a.E ? list[Keys<V>::place(e)] : 0u;
        const bool take = k && unsortable(k) >= least(e);
        const unsigned m = __ballot_sync(kAll, take);
        if (take) list[found + __popc(m & ((1u << lane) - 1u))] = (uint32_t)e;  // (never beyond what has been read)
        found += __popc(m);
        __syncwarp();
    }
    return found;
}

// The groups of one row again in f64, by a whole warp: their mask. cut: best_groups'. key: E doubles;
// list: the row's keys, which are lost.
template <int V>
__device__ __noinline__ unsigned groups_exactly(const RouteArgs &a, long long row, float err, float max_logit,
                                                const float *cut, double *key, uint32_t *list) {
    const int lane = threadIdx.x & 31, size = a.E / a.groups;
    for (int e = lane; e < a.E; e += 32) key[e] = -INFINITY;
    const double sum = exact_sum(a, row, max_logit);
    const int found = pick_experts<V>(a, list, [&](int e) {
        const float c = cut[e / size];
        return !a.bias || c == INFINITY ? c : c - (4.f * err + 0x1p-21f * fabsf(c));
    });
    for (int i = lane; i < found; i += 32) key[list[i]] = exact_key(a, row, (int)list[i], max_logit, sum);
    __syncwarp();
    return best_groups<32, double>(a, key, max_logit, !a.bias, 0.f, nullptr, nullptr);
}

// A number as the sum of two f32, the second at most half a last place of the first
struct Two {
    float hi, lo;
};
__device__ __forceinline__ Two sum_of(float a, float b) {  // exact (Knuth)
    const float s = a + b, t = s - a;
    return {s, (a - (s - t)) + (b - t)};
}
__device__ __forceinline__ Two quick_sum_of(float a, float b) {  // exact for |a| >= |b| (Dekker)
    const float s = a + b;
    return {s, b - (s - a)};
}
// a b + c. (__fmul_rn: a product that is a term of a sum as well, and must not become part of an fma)
__device__ __forceinline__ Two times_plus(Two a, Two b, float c_hi, float c_lo) {
    const float p = __fmul_rn(a.hi, b.hi), e = fmaf(a.hi, b.hi, -p) + fmaf(a.hi, b.lo, a.lo * b.hi);
    const Two s = sum_of(c_hi, p);
    return quick_sum_of(s.hi, s.lo + (e + c_lo));
}
// 1 / (1 + exp(-l)) to 2^-45 (the largest of 2^28 errors: 2^-45.8). exp(-|l|) = 2^k exp(r): r is
// x - k ln 2, with ln 2 in three parts of which k times the first is exact, and exp(r) its
// Taylor series to r^11, from r^6 / 720 on (the last term first) in two parts.
__device__ __forceinline__ Two sigmoid_two(float l) {
    const float x = -fabsf(l);
    Two t = {0.f, 0.f};
    if (x > -87.f) {
        const float k = rintf(x * kLog2e);
        constexpr float ln2_1 = 0x1.62e4p-1f, ln2_2 = 0x1.7f7d1cp-20f, ln2_3 = 0x1.ef357ap-45f;
        const float a = fmaf(-k, ln2_1, x), p = __fmul_rn(k, ln2_2), e = fmaf(k, ln2_2, -p);
        Two r = sum_of(a, -p);
        r = quick_sum_of(r.hi, r.lo - fmaf(k, ln2_3, e));
        float q = 1.f / 39916800.f;
        q = fmaf(q, r.hi, 1.f / 3628800.f);
        q = fmaf(q, r.hi, 1.f / 362880.f);
        q = fmaf(q, r.hi, 1.f / 40320.f);
        q = fmaf(q, r.hi, 1.f / 5040.f);
        t = {q, 0.f};
        t = times_plus(t, r, 0x1.6c16c2p-10f, -0x1.27d27ep-35f);  // 1 / 720
        t = times_plus(t, r, 0x1.111112p-7f, -0x1.dddddep-32f);   // 1 / 120
        t = times_plus(t, r, 0x1.555556p-5f, -0x1.555556p-30f);   // 1 / 24
        t = times_plus(t, r, 0x1.555556p-3f, -0x1.555556p-28f);   // 1 / 6
        t = times_plus(t, r, 0.5f, 0.f);
        t = times_plus(t, r, 1.f, 0.f);
        t = times_plus(t, r, 1.f, 0.f);
        const float two_k = __int_as_float(((int)k + 127) << 23);
        t = {__fmul_rn(t.hi, two_k), t.lo * two_k};
    }
    const Two n = l >= 0.f ? Two{1.f, 0.f} : t;
    Two d = quick_sum_of(1.f, t.hi);
    d.lo += t.lo;
    const float q = n.hi / d.hi, p = __fmul_rn(q, d.hi);
    const float rest = ((n.hi - p) - fmaf(q, d.hi, -p)) + (n.lo - q * d.lo);
    return quick_sum_of(q, rest / d.hi);
}

// The ranks of one row again, exactly, by a whole warp. Only the experts that `ranks` has (`ranked` of
// them), and others that are left with a key of at least `from`, can be among the first. key: E
// doubles; list: the row's keys, which are lost.
template <int V>
__device__ __noinline__ void rank_exactly(const RouteArgs &a, long long row, float from, float max_logit, int *ranks,
                                          int ranked, double *key, uint32_t *list) {
    const int lane = threadIdx.x & 31;
    int found = pick_experts<V>(a, list, [&](int) { return from; });
    for (int r = lane; r < ranked; r += 32) list[found + r] = (uint32_t)ranks[r];  // (these have no key any more)
    found += ranked;
    __syncwarp();
    if (found <= 32 && a.score == MOE_SCORE_SIGMOID) {
        // One each: a rank is the number of lanes that come before. In pairs of f32, which are enough
        // for all but one row in millions: c is off by less than 2^-45 + 2^-48 |c|. (8192 x 256: 9.8 us,
        // 10.5 with the f64 exponential and division, which all other rows wait for.)
        const int e = lane < found ? (int)list[lane] : 0x7fffffff;
        const float l = lane < found ? logit(a, row, e) : 0.f, b = lane < found ? a.bias[e] : 0.f;
        Two c = sigmoid_two(l);
        const Two s = sum_of(c.hi, b);
        c = {s.hi, s.lo + c.lo};
        int rank = 0;
        bool open = false;
        for (int i = 0; i < found; ++i) {
            const float by = (__shfl_sync(kAll, c.hi, i) - c.hi) + (__shfl_sync(kAll, c.lo, i) - c.lo);
            const float ol = __shfl_sync(kAll, l, i), ob = __shfl_sync(kAll, b, i);
            const int oe = __shfl_sync(kAll, e, i);
            const bool same = ol == l && ob == b;  // an exact tie
            open |= lane < found && !same && !(fabsf(by) > 0x1p-42f * (1.f + fabsf(c.hi)));
            rank += same ? oe < e : by > 0.f;
        }
        if (!__any_sync(kAll, open)) {
            if (lane < found) ranks[rank] = e;
            __syncwarp();
            return;
        }
    }
    const double none = -INFINITY, sum = exact_sum(a, row, max_logit);
    if (found <= 32) {
        const int e = lane < found ? (int)list[lane] : 0x7fffffff;
        const double c = lane < found ? exact_key(a, row, e, max_logit, sum) : none;
        int rank = 0;
        for (int i = 0; i < found; ++i) {
            const double o = __shfl_sync(kAll, c, i);
            const int oe = __shfl_sync(kAll, e, i);
            rank += o > c || (o == c && oe < e);
        }
        if (lane < found) ranks[rank] = e;
        __syncwarp();
        return;
    }
    for (int i = lane; i < found; i += 32) key[list[i]] = exact_key(a, row, (int)list[i], max_logit, sum);
    __syncwarp();
    for (int j = 0; j < a.k; ++j) {
        double best = none;
        int at = 0x7fffffff;
        for (int i = lane; i < found; i += 32) {
            const int e = (int)list[i];
            const double c = key[e];
            if (c > best || (c == best && c > none && e < at)) {
                best = c;
                at = e;
            }
        }
        for (int d = 16; d; d >>= 1) {
            const double ob = __shfl_xor_sync(kAll, best, d);
            const int oa = __shfl_xor_sync(kAll, at, d);
            if (ob > best || (ob == best && oa < at)) {
                best = ob;
                at = oa;
            }
        }
        const bool none_left = !(best > none);
        if (lane == 0) {
            ranks[j] = none_left ? -1 : at;
            if (!none_left) key[at] = none;
        }
        __syncwarp();
    }
}

// shared memory of a warp in 4-byte words: its rows' keys, ranks and weights, of one place more than a row
// has (the first that is left out) in multiples of 16 bytes; E doubles
constexpr int kPlaces = kMaxK + 4;
__host__ __device__ constexpr int row_words(int L, int V) { return L * (V + 4) + 2 * kPlaces; }
__host__ __device__ constexpr int warp_words(int L, int V, int E, bool f64) {
    return 32 / L * row_words(L, V) + (f64 ? (2 * E + 3) / 4 * 4 : 0);
}

// REGS: the lanes find the ranks in their registers, instead of by way of shared memory
template <int L, int V, bool REGS>
__global__ void __launch_bounds__(128) route_kernel(const RouteArgs a) {
    extern __shared__ __align__(16) uint32_t words[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane & (L - 1);
    const long long first_row = ((long long)blockIdx.x * (blockDim.x >> 5) + warp) * (32 / L);
    const long long row = first_row + lane / L;
    const bool live = row < a.n;
    ptx::griddep_wait();
    constexpr bool kShared = L < 32;  // the biases by way of shared memory (see the launch)
    float *biases = reinterpret_cast<float *>(words);
    uint32_t *own = words + (kShared && a.bias ? L * (V + 4) : 0) + (size_t)warp * a.words;
    uint32_t *mine = own + lane / L * row_words(L, V);
    const Keys<V> keys{mine};
    int *ranks = reinterpret_cast<int *>(mine + L * (V + 4));
    float *weights = reinterpret_cast<float *>(mine + L * (V + 4) + kPlaces);
    const int e0 = sub * V;

    // the logits, and the largest of them that takes part
    float l[V];
    const size_t esz = a.dtype == MOE_DTYPE_F32 ? 4 : 2;
    const char *src = static_cast<const char *>(a.logits) + ((size_t)row * a.ldl + e0) * esz;
    if (live && a.vector && e0 + V <= a.E) {
        if (a.dtype == MOE_DTYPE_F32) {
#pragma unroll
            for (int j = 0; j < V / 4; ++j) {
                const float4 v = reinterpret_cast<const float4 *>(src)[j];
                l[4 * j] = v.x;
                l[4 * j + 1] = v.y;
                l[4 * j + 2] = v.z;
                l[4 * j + 3] = v.w;
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
            if (a.dtype == MOE_DTYPE_BF16) {
#pragma unroll
                for (int j = 0; j < V / 2; ++j) {
                    const float2 f = unpack2<__nv_bfloat16>(v[j]);
                    l[2 * j] = f.x;
                    l[2 * j + 1] = f.y;
                }
            } else {
#pragma unroll
                for (int j = 0; j < V / 2; ++j) {
                    const float2 f = unpack2<__half>(v[j]);
                    l[2 * j] = f.x;
                    l[2 * j + 1] = f.y;
                }
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) l[j] = live && e0 + j < a.E ? logit(a, row, e0 + j) : -INFINITY;
    }
    if (kShared && a.bias) {
        for (int e = threadIdx.x; e < L * V; e += blockDim.x) biases[Keys<V>::place(e)] = e < a.E ? a.bias[e] : -INFINITY;
        __syncthreads();
    }
    if (first_row >= a.n) return;
    const bool softmax = a.score == MOE_SCORE_SOFTMAX;
    float m = -INFINITY;
    if (softmax) {
#pragma unroll
        for (int j = 0; j < V; ++j) m = fmaxf(m, l[j]);  // (a NaN is passed over)
        m = row_max<L>(m);
    }

    // the divisor of a softmax, where its scores themselves are asked for
    float rcp_sum = 1.f;
    if (softmax && (a.bias || !a.renormalize)) {
        float t = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (takes_part(l[j])) t += expf(below(l[j], m));
        rcp_sum = 1.0f / row_sum<L>(t);
    }

    // sortable keys; 0: takes no part
    uint32_t key[V], best = 0u;
    if (!a.bias) {
#pragma unroll
        for (int j = 0; j < V; ++j) key[j] = takes_part(l[j]) ? sortable(l[j] + 0.f) : 0u;  // (-0 ties with 0)
    } else {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            float b[4];
            if constexpr (kShared) {
                const float4 v = *reinterpret_cast<const float4 *>(biases + sub * (V + 4) + i);
                b[0] = v.x;
                b[1] = v.y;
                b[2] = v.z;
                b[3] = v.w;
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) b[j] = e0 + i + j < a.E ? a.bias[e0 + i + j] : -INFINITY;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float z = l[i + j], c = (softmax ? exp_key(z, m) * rcp_sum : sigmoid_key(z)) + b[j];
                key[i + j] = takes_part(z) && takes_part(b[j]) ? sortable(c + 0.f) : 0u;
            }
        }
    }
    const float err = softmax ? kSoftmaxErr : kSigmoidErr;
    static_assert(!REGS || L == 32, "a rank's owner is one lane of the warp");
    auto store_keys = [&] {
#pragma unroll
        for (int j = 0; j < V / 4; ++j)
            *reinterpret_cast<uint4 *>(mine + sub * (V + 4) + 4 * j) =
                make_uint4(key[4 * j], key[4 * j + 1], key[4 * j + 2], key[4 * j + 3]);
        __syncwarp();
    };
    if (!REGS || a.groups > 1) store_keys();

    double *const f64 = reinterpret_cast<double *>(own + 32 / L * row_words(L, V));
    if (a.groups > 1) {
        bool settled = true;
        unsigned groups = best_groups<L, float>(a, keys, m, !a.bias, err, &settled, weights);
        const bool unsure = live && !settled;
        __syncwarp();
        for (unsigned flagged = __ballot_sync(kAll, sub == 0 && unsure); flagged; flagged &= flagged - 1) {
            const int at = __ffs(flagged) - 1;
            uint32_t *words_of = own + at / L * row_words(L, V);
            const unsigned g = groups_exactly<V>(a, first_row + at / L, err, __shfl_sync(kAll, m, at),
                                                 reinterpret_cast<float *>(words_of + L * (V + 4) + kPlaces), f64, words_of);
            if (lane / L == at / L) groups = g;
        }
        const int size = a.E / a.groups;
        int g = e0 / size, left = size - (e0 - g * size);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (g >= 32 || !((groups >> g) & 1u)) key[j] = 0u;
            if (--left == 0) {
                ++g;
                left = size;
            }
        }
        __syncwarp();
        if (!REGS) store_keys();
    }
#pragma unroll
    for (int j = 0; j < V; ++j) best = max(best, key[j]);

    // The ranks. By way of shared memory: P keys of the owner to a lane
    constexpr int P = V > L ? V / L : 1;
    const int places = a.bias ? a.k + 1 : a.k;  // (with a bias one more: the first that is left out)
    bool unsure = false;
    uint32_t chosen = 0u, left_out = 0u;  // of the row: the keys of the last two places
    float last = 0.f, from = INFINITY;  // of the row: the key of the last rank; the least of them, less the errors
    int ranked = 0;
    for (int r0 = 0; r0 < places; r0 += L) {
        uint32_t held = 0u;  // the key of rank r0 + sub
        const int here = min(L, places - r0);
        if constexpr (REGS) {
            for (int i = 0; i < here; ++i) {
                const uint32_t top = row_max<L>(best);
                chosen = left_out;
                left_out = top;
                if (lane == __ffs(__ballot_sync(kAll, best == top)) - 1) {
                    int at = V - 1;
                    float z = l[V - 1];
#pragma unroll
                    for (int j = V - 2; j >= 0; --j)
                        if (key[j] == top) {
                            at = j;
                            z = l[j];
                        }
                    best = 0u;
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        key[j] = j == at ? 0u : key[j];
                        best = max(best, key[j]);
                    }
                    ranks[r0 + i] = top ? e0 + at : -1;  // (-1: none left)
                    weights[r0 + i] = top ? z : -INFINITY;
                }
                if (lane == i) held = top;
                __syncwarp();
            }
        } else {
            for (int i = 0; i < here; ++i) {
                const uint32_t top = row_max<L>(best);
                chosen = left_out;
                left_out = top;
                const int owner = __ffs(row_ballot<L>(best == top)) - 1;
                uint32_t *theirs = mine + owner * (V + 4) + sub * P;
                uint32_t k[P];
#pragma unroll
                for (int q = 0; q < P; ++q) k[q] = 0u;
                if (P > 1 || sub < V) {
                    if constexpr (P == 4) {
                        const uint4 w = *reinterpret_cast<const uint4 *>(theirs);
                        k[0] = w.x;
                        k[1] = w.y;
                        k[2] = w.z;
                        k[3] = w.w;
                    } else if constexpr (P == 2) {
                        const uint2 w = *reinterpret_cast<const uint2 *>(theirs);
                        k[0] = w.x;
                        k[1] = w.y;
                    } else {
                        k[0] = theirs[0];
                    }
                }
                int at = P;
#pragma unroll
                for (int q = P - 1; q >= 0; --q)
                    if (k[q] == top) at = q;
                const int first = __ffs(row_ballot<L>(at < P && top)) - 1;  // (-1: none left)
                if (sub == first) {
#pragma unroll
                    for (int q = 0; q < P; ++q)
                        if (q == at) k[q] = 0u;
                    theirs[at] = 0u;
                    ranks[r0 + i] = owner * V + sub * P + at;
                }
                if (first < 0 && sub == 0) ranks[r0 + i] = -1;
                uint32_t rest = k[0];
#pragma unroll
                for (int q = 1; q < P; ++q) rest = max(rest, k[q]);
                rest = row_max<L>(rest);
                if (sub == owner) best = rest;
                if (sub == i) held = top;
                __syncwarp();
            }
        }
        if (a.bias) {
            const bool has = held != 0u;
            const float c = has ? unsortable(held) : 0.f, up = __shfl_up_sync(kAll, c, 1, L), before = sub ? up : last;
            const float near = 2.f * (err + 0x1p-23f * (fabsf(c) + (r0 + sub ? fabsf(before) : 0.f)));
            bool close = has && r0 + sub > 0 && !(before - c > near);
            if (close) {
                const int i = ranks[r0 + sub], j = ranks[r0 + sub - 1];
                close = may_swap(softmax, before, logit(a, row, j), a.bias[j], c, logit(a, row, i), a.bias[i], near);
            }
            unsure |= row_ballot<L>(close) != 0u;  // (every lane votes, whatever its row has found)
            from = fminf(from, has ? (c == INFINITY ? 3.0e38f : c - 2.f * near) : INFINITY);
            last = __shfl_sync(kAll, c, L - 1, L);
            ranked += __popc(row_ballot<L>(has));
        }
    }
    // the cut: the others that are left out (the first of them, by key, has been compared)
    if (a.bias) {
        const float in = key_value(chosen);
        float near = 2.f * (err + 0x1p-23f * (fabsf(in) + fabsf(key_value(left_out))));
        bool others = best && !unsure && !(in - unsortable(best) > near);  // (best: of the lane's keys)
        if (softmax && __any_sync(kAll, others)) {
            // a score next to `in` is at most `in` less the least bias (of a row with one large score all others
            // are near otherwise: 15 us for 8192 x 256, 10.8 so)
            float least = INFINITY;
#pragma unroll 4
            for (int e = sub; e < a.E; e += L) least = fminf(least, takes_part(a.bias[e]) ? a.bias[e] : INFINITY);
            const float rounding = 0x1p-21f * (fabsf(in) + near), p = in + row_max<L>(-least) + rounding;
            near = fminf(near, 2.f * (kSoftmaxErr * p + 0x1p-23f * sqrt_fast(p)) + rounding);
            others = others && !(in - unsortable(best) > near);
        }
        bool close = false;
        if (REGS && __any_sync(kAll, others)) store_keys();
        if (others) {
            const int id = ranks[a.k - 1];
            const float li = logit(a, row, id), bi = a.bias[id];
#pragma unroll 1
            for (int j = 0; j < V; j += 4) {
                const uint32_t *at = mine + sub * (V + 4) + j;
                const uint4 k = *reinterpret_cast<const uint4 *>(at);
                auto is_near = [&](uint32_t v) { return (unsigned)(v && !(in - unsortable(v) > near)); };
#pragma unroll 1
                for (unsigned m = is_near(k.x) | is_near(k.y) << 1 | is_near(k.z) << 2 | is_near(k.w) << 3; m; m &= m - 1) {
                    const int i = __ffs(m) - 1, e = e0 + j + i;
                    close |= may_swap(softmax, in, li, bi, unsortable(at[i]), logit(a, row, e), a.bias[e], near);
                }
            }
        }
        unsure |= row_ballot<L>(close) != 0u;
    }
    // rows to be ranked again, one after another by the whole warp
    if (REGS && unsure) store_keys();
    for (unsigned flagged = __ballot_sync(kAll, sub == 0 && unsure); flagged; flagged &= flagged - 1) {
        const int at = __ffs(flagged) - 1;
        const float f = -row_max<L>(-from);  // the lanes of the row have theirs
        uint32_t *words_of = own + at / L * row_words(L, V);
        rank_exactly<V>(a, first_row + at / L, __shfl_sync(kAll, f, at), __shfl_sync(kAll, m, at),
                        reinterpret_cast<int *>(words_of + L * (V + 4)), __shfl_sync(kAll, ranked, at), f64, words_of);
    }
    __syncwarp();

    // weights, of L ranks at a time
    float top = -INFINITY;
    for (int r = sub; r < a.k; r += L) {
        const int id = ranks[r];
        const float z = REGS && !unsure ? weights[r] : live && id >= 0 ? logit(a, row, id) : -INFINITY;
        weights[r] = z;
        top = fmaxf(top, z);
    }
    if (a.renormalize) top = row_max<L>(top);
    // relative to the largest chosen logit where that keeps small scores in range: they are
    // divided by their sum. (exp(l) is all of a sigmoid below -40.)
    const bool shifted = a.renormalize && (softmax || top < -40.f);
    float by = a.scale, sum = 0.f;
    for (int r = sub; r < a.k; r += L) {
        const float z = weights[r];
        float w = 0.f;
        if (z > -INFINITY) w = shifted ? expf(below(z, top)) : softmax ? expf(below(z, m)) * rcp_sum : sigmoid(z);
        weights[r] = w;
        sum += w;
    }
    if (a.renormalize) {
        sum = row_sum<L>(sum);
        by = sum > 0.f ? a.scale / sum : 0.f;
        if (fabsf(by) == INFINITY) {  // (a scale near the largest f32: a weight alone is no larger than it)
            for (int r = sub; r < a.k; r += L) weights[r] /= sum;
            by = a.scale;
        }
    }
    if (!live) return;
    for (int r = sub; r < a.k; r += L) {
        a.topk_idx[row * a.k + r] = ranks[r];
        a.topk_w[row * a.k + r] = weights[r] * by;
    }
}

template <int L, int V, bool REGS = false>
cudaError_t launch(RouteArgs a, cudaStream_t st) {
    const int esz = a.dtype == MOE_DTYPE_F32 ? 4 : 2;
    const unsigned piece = min(16, V * esz);  // bytes of a load
    a.vector = ((uintptr_t)a.logits % piece) == 0 && (a.ldl * esz) % piece == 0;
    a.words = warp_words(L, V, a.E, a.bias || (a.groups > 1 && a.top2));
    // eight lanes read the biases from a copy of the block's: from where they lie it would be V loads a
    // lane, of 8 sectors each (8192 x 256: 8.9 us, 9.8 from there)
    const int shared = L < 32 && a.bias ? L * (V + 4) : 0;
    const int warps = min(4, (12 * 1024 - shared) / a.words), rows = warps * (32 / L);
    return launch_overlapped(route_kernel<L, V, REGS>, dim3((unsigned)((a.n + rows - 1) / rows)), 32 * warps,
                             4 * (shared + warps * a.words), 1, st, a);
}

}  // namespace

cudaError_t launch_route(const RouteArgs &a, cudaStream_t st) {
    if (a.n >= kManyRows && a.E <= 256 && a.groups <= 8) {
        if (a.E <= 64) return launch<8, 8>(a, st);
        if (a.E <= 128) return launch<8, 16>(a, st);
        return launch<8, 32>(a, st);
    }
    // in registers a rank is found sooner, and takes more instructions the more keys a lane has (us,
    // registers / shared memory: 64 rows of 128 2.8 / 3.2, 4095 5.7 / 5.9; of 256 3.0 / 3.2 and 7.4 / 5.7,
    // 600 rows 3.2 / 3.4, 1200 3.8 / 3.7)
    if (a.E <= 128) return launch<32, 4, true>(a, st);
    if (a.E <= 256) return a.n <= 800 ? launch<32, 8, true>(a, st) : launch<32, 8>(a, st);
    if (a.E <= 512) return launch<32, 16>(a, st);
    return launch<32, 32>(a, st);
}

}  // namespace ops
}  // namespace moe
