// ops_pair.cuh -- what the products on CTA pairs share (ops_gemm.cu, ops_gemm_q8.cu): the
// constants of a tile, barriers with bounded waits, TMA loads, MMAs and tensor memory of a
// pair, the walk over the work items, and the epilogue.
#pragma once

#include <cudaTypedefs.h>

#include <atomic>

#include "ops_common.cuh"
#include "ptx.cuh"
#include "tcgen05.cuh"

namespace moe {
namespace ops {
namespace {

constexpr int kM = 128;            // output columns per CTA
constexpr int kPair = 2;           // CTAs per tile
constexpr int kK = 64;             // inputs per stage: one 128-byte row of a swizzled tile
constexpr int kBoxRows = 64;       // rows of x per TMA box, or half as many for the last one
constexpr int kStepRows = 32;      // rows per tile come in multiples of this
constexpr int kBand = 8;           // row tiles that share their pass over the weights: 65536 x 4096 x 4096 takes
                                   // 1146 us in bands of 8, 1421 us without (x is then read once per block)
constexpr int kEpilogue = 8;       // epilogue warps, two per quadrant of the tensor-memory lanes
constexpr int kTmemCols = 512;
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);  // see tc::smem_desc_sw128
constexpr unsigned long long kWaitNs = 1000000000ull;

// [0]: set when a wait gave up, until moe_ops_check reads it
__device__ unsigned g_ops_status[4];

// what the two kinds of tiles have in common; a kernel adds its own
struct Tiles {
    int tcap;       // rows per tile, at most: a multiple of kStepRows
    int mblocks;    // blocks of kPair * kM output columns
    int bufs;       // accumulator sets in tensor memory, 1 or 2
    bool paired;    // columns of out (and residual) come in aligned pairs
};

__device__ __forceinline__ unsigned long long globaltimer() {
    unsigned long long t;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
    return t;
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
    cluster_arrive();
    cluster_wait();
}

// the cluster address of this CTA's barrier `bar` in the pair's first CTA
__device__ __forceinline__ uint32_t in_first(uint32_t bar) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(bar));
    return a;
}

// Barriers and ring stages are held as shared-memory addresses: the loops below
// are bound by their instruction count.
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// wait for an mbarrier phase that a first try did not find complete; false once any
// role of the CTA gave up
__device__ __noinline__ bool wait_more(uint32_t bar, uint32_t parity, volatile int *abort_flag) {
    const unsigned long long t0 = globaltimer();
    for (;;) {
        if (try_wait(bar, parity)) return true;
        if (*abort_flag) return false;
        if (globaltimer() - t0 > kWaitNs) {
            *abort_flag = 1;
            atomicOr(&g_ops_status[0], 1u);
            return false;
        }
    }
}

__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile int *abort_flag) {
    return try_wait(bar, parity) || wait_more(bar, parity, abort_flag);
}

// the same at the end of a role: up to time t0 + kWaitNs, no flag, no report
__device__ __noinline__ void settle(uint32_t bar, uint32_t parity, unsigned long long t0) {
    while (!try_wait(bar, parity) && globaltimer() - t0 < kWaitNs) {
    }
}

// the position of a role in the ring of stages
struct Ring {
    uint32_t stage, empty, full;  // addresses of the current stage and its barriers
    uint32_t s, phase;
    __device__ __forceinline__ void next(uint32_t stages, uint32_t stage_bytes) {
        stage += stage_bytes;
        empty += 8;
        full += 8;
        if (++s == stages) {
            stage -= stages * stage_bytes;
            empty -= stages * 8;
            full -= stages * 8;
            s = 0;
            phase ^= 1;
        }
    }
};

__device__ __forceinline__ void expect_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}

// Relaxed: what it orders is tensor-memory reads that have completed (wait::ld). A
// release at cluster scope would first wait for the warp's stores to reach L2: about a
// microsecond per tile, in which a tile with one accumulator set cannot begin.
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// TMA loads into this CTA's shared memory, counted by a barrier of the pair's
// first CTA (a cluster address)
__device__ __forceinline__ void tma_2d(uint32_t dst, const void *map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, "
        "%3}], [%4];" ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_3d(uint32_t dst, const void *map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, "
        "%3, %4}], [%5];" ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
// four rows of a map whose box is one row high
__device__ __forceinline__ void tma_gather4(uint32_t dst, const void *map, int x, const int (&r)[4], uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes.cta_group::2 [%0], "
        "[%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst), "l"(map), "r"(x), "r"(r[0]), "r"(r[1]),
        "r"(r[2]), "r"(r[3]), "r"(bar)
        : "memory");
}

// D[tmem of both CTAs] (+)= A * B^T: each CTA's shared memory holds its 128 rows of A and
// half of B's rows; issued by one thread of the first CTA
// a and b are the low words of their descriptors, whose high words are all alike
// (128-byte swizzle, 8-row atoms of 1024 bytes)
__device__ __forceinline__ void mma_pair(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 ad, bd;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 ad, {%1, %5};\n\t"
        "mov.b64 bd, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], ad, bd, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescHigh)
        : "memory");
}
__device__ __forceinline__ uint32_t desc_low(uint32_t addr) { return ((addr >> 4) & 0x3FFFu) | (1u << 16); }
// arrive on both CTAs' barriers once the MMAs issued before have completed
__device__ __forceinline__ void commit_pair(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t *slot, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc::smem_u32(slot)),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t addr, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}

// 16 consecutive f32 columns of this thread's lane, complete after tmem_wait_ld
__device__ __forceinline__ void tmem_ld16(uint32_t addr, float (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
          "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
        : "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// rows that the boxes of `half` rows of x cover
__host__ __device__ __forceinline__ int box_rows(int half) {
    return (half + kBoxRows / 2 - 1) / (kBoxRows / 2) * (kBoxRows / 2);
}

// A group of c rows in equal tiles of at most tcap rows: rows per tile
__host__ __device__ __forceinline__ int tile_rows(int c, int tcap) {
    const int nt = (c + tcap - 1) / tcap;
    return ((c + nt - 1) / nt + kStepRows - 1) / kStepRows * kStepRows;
}

// One work item.
struct Item {
    int e;          // expert
    int r0, rows;   // first row and number of rows to store
    int T;          // rows of the tile's MMAs
    int m;          // block of output columns
};

// The items of all groups, numbered group by group: first[e] is the first of
// group e (shared memory; null: one group).
struct Walk {
    const Product &p;
    const Tiles &g;
    const int *first;
    int total;

    __device__ __forceinline__ bool get(int i, Item &it) const {
        if (i >= total) return false;
        int e = 0;
        if (first) {  // the last group that starts at or before item i
            int hi = p.E;
            while (hi - e > 1) {
                const int mid = (e + hi) >> 1;
                if (first[mid] <= i) e = mid;
                else hi = mid;
            }
            i -= first[e];
        }
        int lo, hi;
        group_rows(p, e, lo, hi);
        // (offsets that do not ascend number the items wrongly: the bounds below keep
        // such an item's tile in shape and its rows in range)
        const int c = max(hi - lo, 1), T = tile_rows(c, g.tcap), nt = (c + T - 1) / T;
        // bands of kBand row tiles: the tiles of a band run side by side on one
        // weight block, then on the next
        const int per_band = kBand * g.mblocks, band = i / per_band, r = i - band * per_band;
        const int bh = max(min(kBand, nt - band * kBand), 1);
        it.e = e;
        it.m = r / bh;
        it.T = T;
        it.r0 = lo + (band * kBand + r % bh) * T;
        it.rows = min(T, hi - it.r0);
        return true;
    }
};

// The items of one pair, each role walking for itself.
struct OwnWalk {
    const Walk &walk;
    int i, step;
    __device__ __forceinline__ bool next(Item &it) {
        const bool more = walk.get(i, it);
        i += step;
        return more;
    }
};

// The first item of each group (`first`, shared memory) and the number of all items, by a
// block of THREADS threads; without groups no table. warp_sum: THREADS / 32 numbers.
template <int THREADS>
__device__ __forceinline__ int number_items(const Product &p, const Tiles &g, int *first, int *warp_sum) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (!p.offsets) {
        const int t = tile_rows(p.rows, g.tcap);
        return (p.rows + t - 1) / t * g.mblocks;
    }
    // items per group and their exclusive prefix, THREADS groups at a time
    int base = 0;
    for (int e0 = 0; e0 < p.E; e0 += THREADS) {
        const int e = e0 + tid;
        int items = 0;
        if (e < p.E) {
            int lo, hi;
            group_rows(p, e, lo, hi);
            if (hi > lo) {
                const int t = tile_rows(hi - lo, g.tcap);
                items = (hi - lo + t - 1) / t * g.mblocks;
            }
        }
        int scan = items;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int v = __shfl_up_sync(0xffffffffu, scan, d);
            if (lane >= d) scan += v;
        }
        if (lane == 31) warp_sum[warp] = scan;
        __syncthreads();
        int before = base, sum = 0;
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w) {
            if (w < warp) before += warp_sum[w];
            sum += warp_sum[w];
        }
        if (e < p.E) first[e] = before + scan - items;
        base += sum;
        __syncthreads();
    }
    return base;
}

// The epilogue of a pair's tiles, by warp w of kEpilogue (and lane quadrant w % 4 of tensor
// memory). SCALED: sums of 8-bit codes, to be multiplied by the scale of their row (row_scale:
// 128 floats of shared memory of this warp) and of their column. items: next(it) gives the
// pair's items in turn.
template <typename T, int MATS, bool SCALED, typename Items>
__device__ __forceinline__ void store_tiles(const Product &p, const Tiles &g, Items items, int rank, uint32_t tmem, int w,
                                            uint32_t acc_full_addr, uint32_t acc_empty_addr, volatile int *abort_flag,
                                            float *row_scale) {
    const int lane = threadIdx.x & 31;
    const int q = w & 3;      // the lanes this warp can read
    const int part = w >> 2;  // its half of the tile's pieces of 16 rows
    constexpr int W = 16;     // rows of a chunk
    const uint32_t tlane = tmem + ((uint32_t)(32 * q) << 16);
    int n = 0;
    Item it;
    for (; items.next(it); ++n) {
        const int c = (it.m * kPair + rank) * kM + 32 * q + lane;
        const bool mine = c < p.N;
        float b0 = 0.f, b1 = 0.f;
        if (mine && p.bias) b0 = to_f32(static_cast<const T *>(p.bias)[(size_t)it.e * p.N + c]);
        if (MATS == 2 && mine && p.bias_up) b1 = to_f32(static_cast<const T *>(p.bias_up)[(size_t)it.e * p.N + c]);
        float s0 = 1.f, s1 = 1.f;
        if constexpr (SCALED) {
            if (mine) s0 = p.w_scale[(size_t)it.e * p.N + c];
            if (MATS == 2 && mine) s1 = p.w_up_scale[(size_t)it.e * p.N + c];
            // the rows of this warp's chunks, 16 of every 32
            __syncwarp();
#pragma unroll
            for (int j = lane; j < 128; j += 32) {
                const int r = 16 * part + 32 * (j >> 4) + (j & 15);
                if (r < it.rows) row_scale[j] = p.x_scale[input_row(p, it.r0 + r)];
            }
            __syncwarp();
        }
        const int rows = mine ? it.rows : 0;  // rows this thread stores
        // Two lanes that own neighbouring columns trade rows, so that each moves two
        // columns of every other row in one 4-byte access: an access takes the same
        // time whatever its width. g.paired: columns and addresses allow it.
        const int odd = lane & 1;
        const uint32_t trade = odd ? 0x3276u : 0x5410u;  // (theirs.hi, mine.hi) or (mine.lo, theirs.lo)
        const size_t rstep = (g.paired ? 4 : 2) * p.ldr, ostep = (g.paired ? 4 : 2) * p.ldo;  // bytes
        const char *res = static_cast<const char *>(p.residual);
        char *out = static_cast<char *>(p.out);
        const long long c_first = g.paired ? c - odd : c, r_first = it.r0 + (g.paired ? odd : 0);
        if (res) res += 2 * (r_first * p.ldr + c_first);
        out += 2 * (r_first * p.ldo + c_first);
        // a residual is read two chunks ahead, the first two before the tile is done (SCALED,
        // where more warps share the registers: one); the values stay as loaded until they
        // are used, so that nothing waits for them earlier
        constexpr int kHeld = SCALED && MATS == 2 ? W / 2 : W;  // (half: unpaired values are read when they are used)
        uint32_t ra[kHeld], rb[SCALED ? 1 : W];
        auto load_res = [&](uint32_t (&d)[kHeld], int t0) {
            const char *s = res + 2 * (size_t)t0 * p.ldr;
            if (g.paired) {
#pragma unroll
                for (int j = 0; j < W / 2; ++j, s += rstep)
                    if (t0 + 2 * j + odd < rows) d[j] = *reinterpret_cast<const uint32_t *>(s);
            } else if constexpr (kHeld == W) {
#pragma unroll
                for (int j = 0; j < W; ++j, s += rstep)
                    if (t0 + j < rows) d[j] = *reinterpret_cast<const uint16_t *>(s);
            }
        };
        if (res) {
            load_res(ra, 16 * part);
            if constexpr (!SCALED) load_res(rb, 16 * part + 32);
        }
        const int buf = g.bufs == 2 ? n & 1 : 0, use = g.bufs == 2 ? n >> 1 : n;
        if (!__all_sync(0xffffffffu, wait(acc_full_addr + 8 * buf, (uint32_t)(use & 1), abort_flag))) break;
        tc::fence_after_sync();
        const uint32_t acc = tlane + (uint32_t)(buf * MATS * g.tcap);
        // the next tile's MMAs may overwrite this accumulator set
        auto done_reading = [&] {
            tc::fence_before_sync();
            if (lane == 0) arrive_cluster(in_first(acc_empty_addr + 8 * buf));
        };
        auto chunk = [&](int t0, uint32_t (&r)[kHeld]) {
            float v[W], u[MATS == 2 ? W : 1];
            tmem_ld16(acc + t0, v);
            if constexpr (MATS == 2) tmem_ld16(acc + g.tcap + t0, u);
            tmem_wait_ld();
            if (t0 + 32 >= it.rows) done_reading();
            if constexpr (SCALED) {
                // the column's scale first, as in scaled() of ops_q8.cuh
                const float4 *s = reinterpret_cast<const float4 *>(row_scale + ((t0 - 16 * part) >> 1));
#pragma unroll
                for (int j = 0; j < W / 4; ++j) {
                    const float4 f = s[j];
                    const float by[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        v[4 * j + i] = fmaf(v[4 * j + i] * s0, by[i], b0);
                        if constexpr (MATS == 2) u[4 * j + i] = fmaf(u[4 * j + i] * s1, by[i], b1);
                    }
                }
            } else {
#pragma unroll
                for (int j = 0; j < W; ++j) v[j] += b0;
            }
            if constexpr (MATS == 2) {
                if constexpr (!SCALED) {
#pragma unroll
                    for (int j = 0; j < W; ++j) u[j] += b1;
                }
                if (p.limit > 0.f) {
#pragma unroll
                    for (int j = 0; j < W; ++j) {
                        v[j] = clamp_hi(v[j], p.limit);
                        u[j] = clamp_lo(clamp_hi(u[j], p.limit), -p.limit);
                    }
                }
            }
            if (p.act != MOE_EPI_NONE) unary_act_all(p.act, v);
            if constexpr (MATS == 2) {
#pragma unroll
                for (int j = 0; j < W; ++j) v[j] *= u[j];
            }
            if (res) {  // (unset past the end of the tile, where nothing is stored)
#pragma unroll
                for (int j = 0; j < W / 2; ++j) {
                    uint32_t two;
                    if (g.paired) {
                        two = __byte_perm(r[j], __shfl_xor_sync(0xffffffffu, r[j], 1), trade);
                    } else if constexpr (kHeld < W) {
                        const char *s = res + (size_t)(t0 + 2 * j) * rstep;
                        const uint32_t lo = t0 + 2 * j < rows ? *reinterpret_cast<const uint16_t *>(s) : 0u;
                        const uint32_t hi = t0 + 2 * j + 1 < rows ? *reinterpret_cast<const uint16_t *>(s + rstep) : 0u;
                        two = lo | hi << 16;
                    } else {
                        two = __byte_perm(r[2 * j], r[2 * j + 1], 0x5410u);
                    }
                    const float2 f = unpack2<T>(two);
                    v[2 * j] += f.x;
                    v[2 * j + 1] += f.y;
                }
                load_res(r, t0 + (SCALED ? 32 : 64));
            }
            char *o = out + 2 * (size_t)t0 * p.ldo;
            if (g.paired) {
#pragma unroll
                for (int j = 0; j < W / 2; ++j, o += ostep) {
                    const uint32_t w = pack2<T>(v[2 * j], v[2 * j + 1]);
                    const uint32_t x = __byte_perm(w, __shfl_xor_sync(0xffffffffu, w, 1), trade);
                    if (t0 + 2 * j + odd < rows) *reinterpret_cast<uint32_t *>(o) = x;
                }
            } else {
#pragma unroll
                for (int j = 0; j < W; ++j, o += ostep)
                    if (t0 + j < rows) *reinterpret_cast<T *>(o) = from_f32<T>(v[j]);
            }
        };
        if constexpr (SCALED && MATS == 1) {  // (one copy of the code: it is fetched anew for each tile)
#pragma unroll 1
            for (int t0 = 16 * part; t0 < it.rows; t0 += 32) chunk(t0, ra);
        } else {
#pragma unroll 1
            for (int t0 = 16 * part; t0 < it.rows; t0 += 64) {
                chunk(t0, ra);
                if constexpr (SCALED) {
                    if (t0 + 32 < it.rows) chunk(t0 + 32, ra);
                } else {
                    if (t0 + 32 < it.rows) chunk(t0 + 32, rb);
                }
            }
        }
        if (16 * part >= it.rows) done_reading();  // a tile of at most 16 rows has no chunk for the other half
    }
}

// the driver's tensor-map encoder, resolved once; null if there is none
inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        PFN_cuTensorMapEncodeTiled_v12000 r = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            r = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
        cudaGetLastError();
        return r;
    }();
    return fn;
}

}  // namespace
}  // namespace ops
}  // namespace moe
