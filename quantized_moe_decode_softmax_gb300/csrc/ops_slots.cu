// ops_slots.cu -- the slot bookkeeping of moe_ops.h: grouping (moe_group_slots)
// and the weighted combine (moe_combine_slots).
//
// Grouping is a stable counting sort of n * top_k expert ids with at most 1024
// keys, in one launch of one cluster of up to 8 CTAs and without a workspace.
// Slots are cut into contiguous runs, one per warp, in slot order.
//   1. Each warp counts its run per expert. __match_any_sync groups the lanes of
//      one round by id, the lowest lane of a group adds its size to the warp's
//      own counter, so the counters need no atomics.
//   2. Counters are summed: over the warps of a CTA into a prefix per (warp,
//      expert), over the CTAs through distributed shared memory, over the
//      experts by a block scan (the offsets).
//   3. Each warp walks its run again: a slot's row is its warp's counter plus
//      the number of lower lanes with the same id, and the leader moves the
//      counter on. The order (expert, token, rank) needs no atomics either, so
//      the result does not depend on timing.
// Bound: latency. 64 slots take one CTA and a few dependent steps, 2.9 us; 49152 slots
// read and write 0.8 MB on 8 SMs in 8.4 us, about the time of the steps around it.
// The combine reaches 6.3 TB/s on 8192 tokens of 8 ranks (53 us).
#include <cooperative_groups.h>

#include <atomic>

#include "ops_common.cuh"
#include "ptx.cuh"

namespace moe {
namespace ops {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kCombineThreads = 128;

constexpr int kAhead = 8;  // rounds whose ids are loaded together

__global__ void __launch_bounds__(kThreads)
    group_slots_kernel(const int *topk_idx, long long S, int top_k, int E, int e_lo, int e_hi,
                       int *offsets, int *slot_token, int *slot_k,
                       int *slot_of) {
    extern __shared__ int sm[];
    int *cnt = sm;                 // [kWarps][E] counters, then the rows of the earlier warps per expert
    int *total = sm + kWarps * E;  // [E] this CTA's counts (read by the cluster), then its first rows
    __shared__ int warp_sum[kWarps];
    cg::cluster_group cluster = cg::this_cluster();
    const int ctas = cluster.num_blocks(), cta = cluster.block_rank();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const long long rounds = (S + 32LL * ctas * kWarps - 1) / (32LL * ctas * kWarps);
    // slots [first, last) are this warp's; later warps than `used` of a CTA have none
    const long long first = min((long long)(cta * kWarps + warp) * rounds * 32, S), last = min(first + rounds * 32, S);
    const int used = rounds ? (int)min((S + 32 * rounds - 1) / (32 * rounds), (long long)kWarps) : 0;
    for (int i = tid; i < used * E; i += kThreads) cnt[i] = 0;
    ptx::griddep_wait();
    __syncthreads();
    int *mine = cnt + warp * E;
    // the ids of kAhead rounds; -1 outside the experts and the run
    int ids[kAhead];
    auto load = [&](long long i) {
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
            const long long at = i + 32 * a + lane;
            const int id = at < last ? topk_idx[at] : -1;
            ids[a] = id >= e_lo && id < e_hi ? id : -1;
        }
    };
    for (long long i = first; i < last; i += 32 * kAhead) {
        load(i);
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
            if (i + 32 * a >= last) break;
            const int id = ids[a];
            const unsigned same = __match_any_sync(0xffffffffu, id);
            if (id >= 0 && (same & ((1u << lane) - 1)) == 0) mine[id] += __popc(same);
            __syncwarp();
        }
    }
    __syncthreads();
    // thread e: prefix over the CTA's warps (E <= kThreads)
    int sum = 0;
    if (tid < E) {
#pragma unroll 8
        for (int w = 0; w < used; ++w) {
            const int c = cnt[w * E + tid];
            cnt[w * E + tid] = sum;
            sum += c;
        }
        total[tid] = sum;
    }
    if (ctas > 1) cluster.sync();
    // counts of the earlier CTAs and of all
    int before = 0, all = sum;
    if (ctas > 1 && tid < E) {
        all = 0;
        for (int c = 0; c < ctas; ++c) {
            const int v = cluster.map_shared_rank(total, c)[tid];
            if (c < cta) before += v;
            all += v;
        }
    }
    if (ctas > 1) cluster.sync();  // no CTA leaves, or reuses its counts, while another reads them
    // exclusive scan of the counts over the experts
    int scan = all;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int v = __shfl_up_sync(0xffffffffu, scan, d);
        if (lane >= d) scan += v;
    }
    if (lane == 31) warp_sum[warp] = scan;
    __syncthreads();
    if (warp == 0) {
        int v = warp_sum[lane];
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int u = __shfl_up_sync(0xffffffffu, v, d);
            if (lane >= d) v += u;
        }
        warp_sum[lane] = v;
    }
    __syncthreads();
    const int base = scan - all + (warp ? warp_sum[warp - 1] : 0);
    const int rows = warp_sum[kWarps - 1];
    if (tid < E) {
        if (cta == 0) {
            offsets[tid] = base;
            if (tid == E - 1) offsets[E] = rows;
        }
        total[tid] = base + before;
    }
    __syncthreads();
    for (long long i = first; i < last; i += 32 * kAhead) {
        if (rounds > kAhead) load(i);  // a shorter run's ids are still there
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
            if (i + 32 * a >= last) break;
            const int id = ids[a];
            const unsigned same = __match_any_sync(0xffffffffu, id);
            const unsigned lower = same & ((1u << lane) - 1);
            const int at = id >= 0 ? total[id] + mine[id] + __popc(lower) : -1;
            __syncwarp();
            if (id >= 0 && lower == 0) mine[id] += __popc(same);
            __syncwarp();
            const long long slot = i + 32 * a + lane;
            if (slot < last) slot_of[slot] = at;
            if (id >= 0) {
                const int t = (int)slot / top_k;
                slot_token[at] = t;
                if (slot_k) slot_k[at] = (int)slot - t * top_k;
            }
        }
    }
    // rows that no slot takes
    for (long long i = (long long)rows + cta * kThreads + tid; i < S; i += (long long)ctas * kThreads) {
        slot_token[i] = -1;
        if (slot_k) slot_k[i] = -1;
    }
}

// A thread owns 8 columns of a token (one where rows are not on 16-byte
// boundaries), blockIdx.y the token. Bound: the bytes of y. Eight ranks at a time
// their rows are looked up, then all their loads are issued before the first is used
// (8 x 16 bytes in flight per thread); the sum keeps the order of the ranks.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kCombineThreads)
    combine_slots_kernel(const T *y, long long ldy, int rows, const int *slot_of,
                         const float *topk_w, int n, int top_k, int N, const T *residual,
                         long long ldr, T *out, long long ldo) {
    constexpr int V = VEC ? 8 : 1, R = 8;
    const int c = (blockIdx.x * kCombineThreads + threadIdx.x) * V;
    ptx::griddep_wait();
    if (c >= N) return;
    for (int t = blockIdx.y; t < n; t += gridDim.y) {
        float acc[V];
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = 0.f;
        for (int j0 = 0; j0 < top_k; j0 += R) {
            int s[R];
            float w[R];
#pragma unroll
            for (int j = 0; j < R; ++j) {
                const bool in = j0 + j < top_k;
                s[j] = in ? slot_of[(size_t)t * top_k + j0 + j] : -1;
                w[j] = in ? topk_w[(size_t)t * top_k + j0 + j] : 0.f;
            }
            if constexpr (VEC) {
                uint4 v[R];
#pragma unroll
                for (int j = 0; j < R; ++j)
                    if (s[j] >= 0 && s[j] < rows) v[j] = __ldcs(reinterpret_cast<const uint4 *>(y + (size_t)s[j] * ldy + c));
#pragma unroll
                for (int j = 0; j < R; ++j) {
                    if (s[j] < 0 || s[j] >= rows) continue;
                    const uint32_t u[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 f = unpack2<T>(u[i]);
                        acc[2 * i] += w[j] * f.x;
                        acc[2 * i + 1] += w[j] * f.y;
                    }
                }
            } else {
#pragma unroll
                for (int j = 0; j < R; ++j)
                    if (s[j] >= 0 && s[j] < rows) acc[0] += w[j] * to_f32(y[(size_t)s[j] * ldy + c]);
            }
        }
        T *o = out + (size_t)t * ldo + c;
        const T *r = residual ? residual + (size_t)t * ldr + c : nullptr;
        if constexpr (VEC) {
            if (r) {
                const uint4 v = *reinterpret_cast<const uint4 *>(r);
                const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = unpack2<T>(u[i]);
                    acc[2 * i] += f.x;
                    acc[2 * i + 1] += f.y;
                }
            }
            *reinterpret_cast<uint4 *>(o) = make_uint4(pack2<T>(acc[0], acc[1]), pack2<T>(acc[2], acc[3]),
                                                       pack2<T>(acc[4], acc[5]), pack2<T>(acc[6], acc[7]));
        } else {
            if (r) acc[0] += to_f32(*r);
            *o = from_f32<T>(acc[0]);
        }
    }
}

// whether rows of 16-bit elements start on 16-byte boundaries
bool rows16(const void *p, long long ld) { return ((uintptr_t)p & 15u) == 0 && ld % 8 == 0; }

template <typename T>
cudaError_t combine(const void *y, long long ldy, int rows, const int *slot_of, const float *topk_w, int n, int top_k,
                    int N, const void *residual, long long ldr, void *out, long long ldo, cudaStream_t st) {
    const bool vec = N % 8 == 0 && rows16(y, ldy) && rows16(out, ldo) && (!residual || rows16(residual, ldr));
    const int cols = vec ? N / 8 : N;
    const dim3 grid((cols + kCombineThreads - 1) / kCombineThreads, min(n, 65535));
    auto k = vec ? combine_slots_kernel<T, true> : combine_slots_kernel<T, false>;
    return launch_overlapped(k, grid, kCombineThreads, 0, 1, st, static_cast<const T *>(y), ldy, rows, slot_of, topk_w,
                             n, top_k, N, static_cast<const T *>(residual), ldr, static_cast<T *>(out), ldo);
}

}  // namespace

cudaError_t launch_group_slots(const int *topk_idx, int n, int top_k, int E, int e_lo, int e_hi, int *offsets,
                               int *slot_token, int *slot_k, int *slot_of, cudaStream_t st) {
    const long long S = (long long)n * top_k;
    const int ctas = S <= 4 * kThreads ? 1 : 8;
    const int smem = (kWarps + 1) * E * 4;
    if (smem > 32 << 10) {  // above what a kernel may ask for by itself: raise the limit, once per device
        static std::atomic<unsigned long long> raised{0};
        int dev = 0;
        cudaError_t err = cudaGetDevice(&dev);
        if (err != cudaSuccess) return err;
        const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
        if (!(raised.load(std::memory_order_acquire) & bit) || !bit) {
            err = cudaFuncSetAttribute(group_slots_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (kWarps + 1) * kThreads * 4);
            if (err != cudaSuccess) return err;
            raised.fetch_or(bit, std::memory_order_release);
        }
    }
    return launch_overlapped(group_slots_kernel, dim3(ctas), kThreads, smem, ctas, st, topk_idx, S, top_k, E, e_lo,
                             e_hi, offsets, slot_token, slot_k, slot_of);
}

cudaError_t launch_combine_slots(int dtype, const void *y, long long ldy, int rows, const int *slot_of,
                                 const float *topk_w, int n, int top_k, int N, const void *residual,
                                 long long ldr, void *out, long long ldo, cudaStream_t st) {
    if (dtype == MOE_DTYPE_BF16)
        return combine<__nv_bfloat16>(y, ldy, rows, slot_of, topk_w, n, top_k, N, residual, ldr, out, ldo, st);
    return combine<__half>(y, ldy, rows, slot_of, topk_w, n, top_k, N, residual, ldr, out, ldo, st);
}

}  // namespace ops
}  // namespace moe
