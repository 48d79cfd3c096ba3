// ops_gemm.cu -- products over many rows (moe_linear, moe_grouped_linear) on the
// 5th-generation tensor cores.
//
//   out[r, c] = act(sum_k x[r, k] w[c, k] + bias[c]) (* the up product) (+ residual[r, c])
//
// A pair of CTAs (one cluster, cta_group::2 MMAs) shares a tile. The tile is
// transposed: the weights are the M operand (256 output columns, 128 per CTA, one
// per tensor-memory lane) and the rows of x are the N operand, up to 256 of them.
//   - N is any multiple of 32, so a ragged group wastes at most 31 rows of its
//     tiles, where a 128-row M tile would waste up to 127: the groups of a prompt
//     hold a few hundred rows each. A group is cut into equal tiles.
//   - A thread of the epilogue owns one output column: its bias is a register,
//     and odd sizes need no other path. A gated product finds gate and up of an output
//     in the same lane.
//   - Each CTA of the pair loads its own weights and half of the rows; the MMA
//     reads both halves. Per step of 64 inputs at 256 rows a CTA fetches 32 KB from L2
//     for 512 tensor-core cycles (gated: 48 KB for 1024). The way from L2 into an SM
//     takes about 64 bytes a cycle: a CTA by itself would need 48 KB for 512 cycles.
//   - Two accumulator sets fit tensor memory up to 256 rows (gated: 128), and the
//     epilogue of a tile then runs beside the MMAs of the next. A gated product may
//     still take tiles of 256 rows and one set: it gives the overlap away and halves
//     the weights' traffic.
//
// Persistent pairs walk the work items (group, block of output columns, tile of
// rows) in a fixed order. Warps 0..3 load, per step of 64 inputs, the weight
// boxes and the rows of x (boxes, or tile::gather4 through row_token) by TMA
// with the 128-byte swizzle into a ring of stages (where four such stages fit, a step
// has 128 inputs: fewer rounds of waiting, 9.6 to 7.6 us at 96 x 2048 x 2048). One warp of the first CTA issues
// the MMAs for both. Eight warps run the epilogue. Inputs past K read as zeros in
// both operands; rows past the group's end are computed and not stored, and since
// the rows of a product do not mix, what they hold (even NaN) does not matter.
//
// Bound: the tensor cores for long products, the weights' bytes for groups of few
// rows. Measured (GB300, bf16, clocks as they come, 2.0 GHz at best):
//   65536 x 4096 x 4096                          1146 us  1918 TFLOP/s
//   8192 x 4096 x 4096                            145 us  1900 TFLOP/s (library 138)
//   8192 x 4096 x 2 x 2048 gated, SiLU        146..171 us  1880..1610 TFLOP/s
//   8192 tokens x 8 of 128 experts, 2048 -> 2 x 768, gathered  277..325 us  1490..1270 TFLOP/s
//   64 tokens x 8 of 128 experts, 768 -> 2048     65.3 us  6.1 TB/s
// (The ranges are the clock under the power limit: short runs and long ones, several boards.)
// Dealing each pair one contiguous run of rows, for an even end, was slower on the
// grouped product (455 against 300 us): pairs then no longer share a weight block
// while it is in L2.
//
// Every wait is bounded (1 s, reported through moe_ops_check); after one gives
// up, all roles stop and the pair waits for its copies in flight before it ends.
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
constexpr int kTileA = kM * kK * 2;
constexpr int kBoxRows = 64;       // rows of x per TMA box, or half as many for the last one
constexpr int kStepRows = 32;      // rows per tile come in multiples of this
constexpr int kMaxStages = 8;
constexpr int kBand = 8;           // row tiles that share their pass over the weights: 65536 x 4096 x 4096 takes
                                   // 1146 us in bands of 8, 1421 us without (x is then read once per block)
constexpr int kLoaders = 4;        // load warps
constexpr int kEpilogue = 8;       // epilogue warps, two per quadrant of the tensor-memory lanes
constexpr int kMmaWarp = kLoaders + kEpilogue;
constexpr int kThreads = 32 * (kMmaWarp + 1);
constexpr int kTmemCols = 512;
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);  // see tc::smem_desc_sw128
constexpr unsigned long long kWaitNs = 1000000000ull;

// [0]: set when a wait gave up, until moe_ops_check reads it
__device__ unsigned g_ops_status[4];

struct Tiling {
    int tcap;       // rows per tile, at most: a multiple of kStepRows
    int stages;
    int stage_bytes;
    int mblocks;    // blocks of kPair * kM output columns
    int bufs;       // accumulator sets in tensor memory, 1 or 2
    bool wide;      // a stage holds 128 inputs: tiles w, w, x, x of 64 each (MATS = 1, no row_token)
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

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
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
    const Tiling &g;
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

template <typename T, int MATS>
__global__ void __launch_bounds__(kThreads, 1)
    product_gemm_kernel(const __grid_constant__ Product p, const __grid_constant__ Tiling g,
                        const __grid_constant__ CUtensorMap tmx, const __grid_constant__ CUtensorMap tmx_half,
                        const __grid_constant__ CUtensorMap tmw, const __grid_constant__ CUtensorMap tmu) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    // full and acc_empty are used in the first CTA only, for both
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], drain;
    __shared__ uint32_t tslot;
    __shared__ int abort_word, warp_sum[kThreads / 32];
    volatile int *abort_flag = &abort_word;
    unsigned char *ring = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
    int *first = reinterpret_cast<int *>(ring + g.stages * g.stage_bytes);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = (int)cluster_rank();
    const int item0 = blockIdx.x / kPair, item_step = gridDim.x / kPair;

    if (tid == 0) {
        abort_word = 0;
        for (int i = 0; i < g.stages; ++i) {
            ptx::mbar_init(&full[i], 1);
            ptx::mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&acc_full[i], 1);
            ptx::mbar_init(&acc_empty[i], kEpilogue * kPair);  // the epilogues' warps
        }
        ptx::mbar_init(&drain, 1);
        ptx::mbar_fence_init();
        ptx::prefetch_tensormap(&tmx);
        ptx::prefetch_tensormap(&tmx_half);
        ptx::prefetch_tensormap(&tmw);
        if (MATS == 2) ptx::prefetch_tensormap(&tmu);
    }
    if (warp == kMmaWarp) tmem_alloc_pair(&tslot, kTmemCols);
    ptx::griddep_wait();
    int total;
    if (p.offsets) {
        // items per group and their exclusive prefix, kThreads groups at a time
        int base = 0;
        for (int e0 = 0; e0 < p.E; e0 += kThreads) {
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
            for (int w = 0; w < kThreads / 32; ++w) {
                if (w < warp) before += warp_sum[w];
                sum += warp_sum[w];
            }
            if (e < p.E) first[e] = before + scan - items;
            base += sum;
            __syncthreads();
        }
        total = base;
    } else {
        const int t = tile_rows(p.rows, g.tcap);
        total = (p.rows + t - 1) / t * g.mblocks;
        first = nullptr;
    }
    tc::fence_before_sync();
    __syncthreads();
    cluster_sync();  // the peer's barriers are ready
    tc::fence_after_sync();
    const uint32_t tmem = tslot;
    const uint32_t ring_addr = tc::smem_u32(ring), full_addr = tc::smem_u32(full), empty_addr = tc::smem_u32(empty);
    const uint32_t acc_full_addr = tc::smem_u32(acc_full), acc_empty_addr = tc::smem_u32(acc_empty);
    const Walk walk{p, g, first, total};
    // steps of a tile; a wide one reaches past K with its second half if need be (zeros)
    const bool wide = MATS == 1 && g.wide;
    const int step_k = wide ? 2 * kK : kK, nk = (p.K + step_k - 1) / step_k;
    const uint32_t x_at = wide ? 2 * kTileA : MATS * kTileA, x_half = (g.stage_bytes - x_at) / 2;

    if (warp < kLoaders) {
        // ---- loads ------------------------------------------------------------
        const bool gather = p.row_token != nullptr;
        // A step of a load loop is a chain of about 450 cycles (wait, elect, copy),
        // whatever it copies, so the steps are dealt to two pairs of warps: warps 0 and 1
        // take the even ones, 2 and 3 the odd ones; 0 and 2 load the weights, 1 and 3 the
        // rows of x. With row_token every warp takes part in every step, with every
        // fourth copy of four rows; warps 0 and 2 load the weights beside it.
        // (A warp that skips steps stays less than two laps of the ring ahead of the
        // MMAs all the same, by the waits of the steps that it takes, so that parities
        // tell the phases of a barrier apart.)
        Ring at{ring_addr, empty_addr, in_first(full_addr), 0, 1};  // a fresh barrier passes the wait for phase 1
        const uint32_t stages = g.stages, stage_bytes = g.stage_bytes;
        const bool odd = warp >= 2;
        bool skip = odd && !gather;  // the next step belongs to the other pair
        Item it;
        bool ok = true;
        for (int i = item0; ok && walk.get(i, it); i += item_step) {
            const int half = it.T / kPair;  // rows of x that this CTA loads
            const int r0 = it.r0 + rank * half;
            const uint32_t bytes = (wide ? 2 : 1) * kPair * (MATS * kTileA + (gather ? half : box_rows(half)) * 128);
            const int col = (it.m * kPair + rank) * kM, plane = p.stride_e ? it.e : 0;
            const int k_end = nk * step_k;
            if (gather) {
                // lane j's rows are the warp's j-th copy; rows past the end repeat the last one
                const int fours = (half / 4 - warp + kLoaders - 1) / kLoaders;
                int rows[4] = {};
                if (lane < fours) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        rows[j] = input_row(p, min(r0 + 4 * (warp + kLoaders * lane) + j, it.r0 + it.rows - 1));
                }
                const uint32_t dst = MATS * kTileA + (warp + kLoaders * lane) * 512;
                const CUtensorMap *map = warp == 0 ? &tmw : &tmu;
                const bool loads_w = warp == 0 || (MATS == 2 && warp == 2), counts = warp == 0 && rank == 0;
#pragma unroll 1
                for (int k = 0; k < k_end; k += kK) {
                    if (!(ok = __all_sync(0xffffffffu, wait(at.empty, at.phase, abort_flag)))) break;
                    if (loads_w && tc::elect_one()) {
                        if (counts) expect_tx(full_addr + 8 * at.s, bytes);
                        tma_3d(at.stage + (warp == 0 ? 0 : kTileA), map, k, col, plane, at.full);
                    }
                    if (lane < fours) tma_gather4(at.stage + dst, &tmx, k, rows, at.full);
                    at.next(stages, stage_bytes);
                }
            } else if (warp & 1) {
                // two boxes of x at most: the last one is half as high if that is enough
                const int n1 = half > kBoxRows ? (half - kBoxRows > kBoxRows / 2 ? 2 : 1) : 0;
                const CUtensorMap *map0 = half > kBoxRows / 2 ? &tmx : &tmx_half, *map1 = n1 == 2 ? &tmx : &tmx_half;
#pragma unroll 1
                for (int k = 0; k < k_end; k += step_k) {
                    if (!skip) {
                        if (!(ok = __all_sync(0xffffffffu, wait(at.empty, at.phase, abort_flag)))) break;
                        if (tc::elect_one()) {
                            tma_2d(at.stage + x_at, map0, k, r0, at.full);
                            if (n1) tma_2d(at.stage + x_at + kBoxRows * 128, map1, k, r0 + kBoxRows, at.full);
                            if (wide) {
                                tma_2d(at.stage + x_at + x_half, map0, k + kK, r0, at.full);
                                if (n1)
                                    tma_2d(at.stage + x_at + x_half + kBoxRows * 128, map1, k + kK, r0 + kBoxRows, at.full);
                            }
                        }
                    }
                    skip = !skip;
                    at.next(stages, stage_bytes);
                }
            } else {
#pragma unroll 1
                for (int k = 0; k < k_end; k += step_k) {
                    if (!skip) {
                        if (!(ok = __all_sync(0xffffffffu, wait(at.empty, at.phase, abort_flag)))) break;
                        if (tc::elect_one()) {
                            if (rank == 0) expect_tx(full_addr + 8 * at.s, bytes);
                            tma_3d(at.stage, &tmw, k, col, plane, at.full);
                            if (wide) tma_3d(at.stage + kTileA, &tmw, k + kK, col, plane, at.full);
                            if (MATS == 2) tma_3d(at.stage + kTileA, &tmu, k, col, plane, at.full);
                        }
                    }
                    skip = !skip;
                    at.next(stages, stage_bytes);
                }
            }
        }
        // Before the pair may end, every copy has landed and every stage has been handed
        // back (both have, or are about to, unless a wait gave up). The stages before
        // `at` were last filled in its lap, the others in the one before; a fresh
        // barrier passes.
        if (warp == 0) {
            const unsigned long long t0 = globaltimer();
            for (uint32_t i = 0; i < stages; ++i) {
                const uint32_t next = i < at.s ? at.phase ^ 1 : at.phase;  // the parity that its next fill would wait for
                if (rank == 0) settle(full_addr + 8 * i, next, t0);
                settle(empty_addr + 8 * i, next, t0);
            }
        }
        __syncwarp();
    } else if (warp == kMmaWarp && rank == 0) {
        // ---- MMAs --------------------------------------------------------------
        if (tc::elect_one()) {
            Ring at{ring_addr, empty_addr, full_addr, 0, 0};
            const uint32_t stages = g.stages, stage_bytes = g.stage_bytes;
            int n = 0;
            Item it;
            bool ok = true;
            const uint32_t base = p.dtype == MOE_DTYPE_BF16 ? tc::idesc_bf16_f32(kPair * kM, 0)
                                                            : tc::idesc_f16_f32(kPair * kM, 0);
            for (int i = item0; ok && walk.get(i, it); i += item_step, ++n) {
                const uint32_t idesc = base | ((uint32_t)(it.T >> 3) << 17);
                const int buf = g.bufs == 2 ? n & 1 : 0, use = g.bufs == 2 ? n >> 1 : n;
                const uint32_t acc = tmem + (uint32_t)(buf * MATS * g.tcap), acc_up = acc + g.tcap;
                // the epilogues have read what this accumulator set held
                if (!(ok = wait(acc_empty_addr + 8 * buf, (uint32_t)((use & 1) ^ 1), abort_flag))) break;
                tc::fence_after_sync();
#pragma unroll 1
                for (int k = 0; k < nk; ++k) {
                    if (!(ok = wait(at.full, at.phase, abort_flag))) break;
                    tc::fence_after_sync();
                    const uint32_t a = desc_low(at.stage), b = a + (x_at >> 4);
                    // the first MMA of a tile overwrites
                    mma_pair(acc, a, b, idesc, k);
                    if (MATS == 2) mma_pair(acc_up, a + (kTileA >> 4), b, idesc, k);
#pragma unroll
                    for (int q = 1; q < kK / 16; ++q) {
                        mma_pair(acc, a + 2 * q, b + 2 * q, idesc, 1);
                        if (MATS == 2) mma_pair(acc_up, a + (kTileA >> 4) + 2 * q, b + 2 * q, idesc, 1);
                    }
                    if (wide) {
#pragma unroll
                        for (int q = 0; q < kK / 16; ++q)
                            mma_pair(acc, a + (kTileA >> 4) + 2 * q, b + (x_half >> 4) + 2 * q, idesc, 1);
                    }
                    commit_pair(at.empty);
                    at.next(stages, stage_bytes);
                }
                if (ok) commit_pair(acc_full_addr + 8 * buf);
            }
            if (!ok) {  // let the MMAs in flight end before the tensor memory is freed
                commit_pair(tc::smem_u32(&drain));
                settle(tc::smem_u32(&drain), 0, globaltimer());
            }
        }
        __syncwarp();
    } else if (warp >= kLoaders && warp < kMmaWarp) {
        // ---- epilogue ----------------------------------------------------------
        const int q = warp & 3;                  // the lanes this warp can read
        const int part = (warp - kLoaders) >> 2; // its half of the tile's chunks of 16 rows
        const uint32_t tlane = tmem + ((uint32_t)(32 * q) << 16);
        int n = 0;
        Item it;
        for (int i = item0; walk.get(i, it); i += item_step, ++n) {
            const int c = (it.m * kPair + rank) * kM + 32 * q + lane;
            const bool mine = c < p.N;
            float b0 = 0.f, b1 = 0.f;
            if (mine && p.bias) b0 = to_f32(static_cast<const T *>(p.bias)[(size_t)it.e * p.N + c]);
            if (MATS == 2 && mine && p.bias_up) b1 = to_f32(static_cast<const T *>(p.bias_up)[(size_t)it.e * p.N + c]);
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
            // a residual is read two chunks ahead, the first two before the tile is done;
            // the values stay as loaded until they are used, so that nothing waits for
            // them earlier
            uint32_t ra[16], rb[16];
            auto load_res = [&](uint32_t (&d)[16], int t0) {
                const char *s = res + 2 * (size_t)t0 * p.ldr;
                if (g.paired) {
#pragma unroll
                    for (int j = 0; j < 8; ++j, s += rstep)
                        if (t0 + 2 * j + odd < rows) d[j] = *reinterpret_cast<const uint32_t *>(s);
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j, s += rstep)
                        if (t0 + j < rows) d[j] = *reinterpret_cast<const uint16_t *>(s);
                }
            };
            if (res) {
                load_res(ra, 16 * part);
                load_res(rb, 16 * part + 32);
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
            auto chunk = [&](int t0, uint32_t (&r)[16]) {
                float v[16], u[MATS == 2 ? 16 : 1];
                tmem_ld16(acc + t0, v);
                if constexpr (MATS == 2) tmem_ld16(acc + g.tcap + t0, u);
                tmem_wait_ld();
                if (t0 + 32 >= it.rows) done_reading();
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] += b0;
                if constexpr (MATS == 2) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) u[j] += b1;
                    if (p.limit > 0.f) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            v[j] = clamp_hi(v[j], p.limit);
                            u[j] = clamp_lo(clamp_hi(u[j], p.limit), -p.limit);
                        }
                    }
                }
                if (p.act != MOE_EPI_NONE) unary_act_all(p.act, v);
                if constexpr (MATS == 2) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] *= u[j];
                }
                if (res) {  // (unset past the end of the tile, where nothing is stored)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint32_t w = g.paired ? __byte_perm(r[j], __shfl_xor_sync(0xffffffffu, r[j], 1), trade)
                                                    : __byte_perm(r[2 * j], r[2 * j + 1], 0x5410u);
                        const float2 f = unpack2<T>(w);
                        v[2 * j] += f.x;
                        v[2 * j + 1] += f.y;
                    }
                    load_res(r, t0 + 64);
                }
                char *o = out + 2 * (size_t)t0 * p.ldo;
                if (g.paired) {
#pragma unroll
                    for (int j = 0; j < 8; ++j, o += ostep) {
                        const uint32_t w = pack2<T>(v[2 * j], v[2 * j + 1]);
                        const uint32_t x = __byte_perm(w, __shfl_xor_sync(0xffffffffu, w, 1), trade);
                        if (t0 + 2 * j + odd < rows) *reinterpret_cast<uint32_t *>(o) = x;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j, o += ostep)
                        if (t0 + j < rows) *reinterpret_cast<T *>(o) = from_f32<T>(v[j]);
                }
            };
#pragma unroll 1
            for (int t0 = 16 * part; t0 < it.rows; t0 += 64) {
                chunk(t0, ra);
                if (t0 + 32 < it.rows) chunk(t0 + 32, rb);
            }
            if (16 * part >= it.rows) done_reading();  // a tile of at most 16 rows has no chunk for the other half
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    cluster_sync();  // neither CTA ends while the other may still use its memory
    tc::fence_after_sync();
    if (warp == kMmaWarp) tmem_dealloc_pair(tmem, kTmemCols);
}

// the driver's tensor-map encoder, resolved once; null if there is none
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
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

// 16-bit rows of `cols` elements `ld` apart, `planes` of them (rank 3) or one
// (rank 2), boxes of 64 columns x box_rows rows; what lies outside reads as zeros
bool encode(CUtensorMap *m, int dtype, const void *base, long long cols, long long rows, long long ld, int planes,
            long long stride, int box_rows) {
    PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn();
    if (!fn) return false;
    const int rank = planes ? 3 : 2;
    cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)(planes ? planes : 1)};
    cuuint64_t strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)stride * 2};
    cuuint32_t box[3] = {(cuuint32_t)kK, (cuuint32_t)box_rows, 1};
    cuuint32_t es[3] = {1, 1, 1};
    return fn(m, dtype == MOE_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rank,
              const_cast<void *>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// what a launch needs to know of a device, looked up once
struct Device {
    std::atomic<int> pairs{0};       // CTA pairs that run at once
    std::atomic<int> smem{0};        // dynamic shared memory a CTA may ask for
    std::atomic<unsigned> ready{0};  // kernels whose shared-memory limit is raised
};
constexpr int kMaxDevices = 64;
Device g_devices[kMaxDevices];

// Rows per tile: the least time of a simple model, in cycles. Waves of tiles on the
// pairs, each nk steps of the longest of the MMAs (2 per row and matrix and 64
// inputs), the loads (64 bytes a cycle from L2 into an SM) and the issue of a step
// (350); then the epilogue of the last tile, and a third of it for every tile where
// it cannot run beside the next tile's MMAs (one accumulator set: 256 gated rows
// measured 316 us on 8192 tokens, 128 experts, K = 2048, and 128 rows 382 us).
int pick_rows(const Product &p, int mblocks, int groups, int mean, int nk, int pairs) {
    const int mats = p.w_up ? 2 : 1;
    const int per_row = 20 + 15 * (mats - 1) + (p.act != MOE_EPI_NONE ? 15 : 0) + (p.residual ? 15 : 0);
    int best = kStepRows;
    long long least = -1;
    for (int cap = 256; cap >= kStepRows; cap -= kStepRows) {
        const int t = tile_rows(mean, cap);
        const long long items = (long long)groups * mblocks * ((mean + t - 1) / t);
        const long long waves = (items + pairs - 1) / pairs;
        const int mma = 2 * mats * t, loads = (mats * kTileA + box_rows(t / kPair) * 128) / 64;
        const long long step = max(350, max(mma, loads));
        const long long cost = waves * nk * step + per_row * t + (2 * mats * cap > kTmemCols ? waves * per_row * t / 3 : 0);
        if (least < 0 || cost < least) {
            least = cost;
            best = cap;
        }
    }
    return best;
}

cudaError_t look_up(int dev, Device &d) {
    int smem = 0, sms = 0, pairs = 0;
    cudaFuncAttributes fa;
    cudaError_t err;
    auto k = product_gemm_kernel<__half, 2>;
    if ((err = cudaDeviceGetAttribute(&smem, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev)) != cudaSuccess ||
        (err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess ||
        (err = cudaFuncGetAttributes(&fa, k)) != cudaSuccess)
        return err;
    smem -= (int)((fa.sharedSizeBytes + 127) / 128 * 128);
    if ((err = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return err;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(sms / kPair * kPair);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kPair;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if ((err = cudaOccupancyMaxActiveClusters(&pairs, k, &cfg)) != cudaSuccess) return err;
    if (pairs < 1) return cudaErrorNotSupported;
    d.smem.store(smem, std::memory_order_relaxed);
    d.pairs.store(min(pairs, sms / kPair), std::memory_order_release);
    return cudaSuccess;
}

template <typename T, int MATS>
cudaError_t launch(const Product &p, const Tiling &g, int pairs, int smem, Device &d, const CUtensorMap &tmx,
                   const CUtensorMap &tmx_half, const CUtensorMap &tmw, const CUtensorMap &tmu, cudaStream_t st) {
    auto k = product_gemm_kernel<T, MATS>;
    const unsigned bit = 1u << (MATS - 1 + (p.dtype == MOE_DTYPE_BF16 ? 2 : 0));
    if (!(d.ready.load(std::memory_order_acquire) & bit)) {
        const cudaError_t err = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                     d.smem.load(std::memory_order_relaxed));
        if (err != cudaSuccess) return err;
        d.ready.fetch_or(bit, std::memory_order_release);
    }
    return launch_overlapped(k, dim3(kPair * pairs), kThreads, smem, kPair, st, p, g, tmx, tmx_half, tmw, tmu);
}

}  // namespace

cudaError_t launch_product_gemm(const Product &p, cudaStream_t st) {
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    Device &d = g_devices[dev];
    if (d.pairs.load(std::memory_order_acquire) == 0 && (err = look_up(dev, d)) != cudaSuccess) return err;
    const int all = d.pairs.load(std::memory_order_acquire);
    const int mats = p.w_up ? 2 : 1;
    const int mblocks = (p.N + kPair * kM - 1) / (kPair * kM);
    const int groups = p.offsets ? min(p.E, p.rows) : 1;
    Tiling g;
    g.tcap = pick_rows(p, mblocks, groups, (p.rows + groups - 1) / groups, (p.K + kK - 1) / kK, all);
    g.stage_bytes = mats * kTileA + box_rows(g.tcap / kPair) * 128;
    g.wide = mats == 1 && !p.row_token && p.K > 2 * kK && 4 * 2 * g.stage_bytes <= d.smem.load(std::memory_order_relaxed) - 8192;
    if (g.wide) g.stage_bytes *= 2;
    g.bufs = 2 * mats * g.tcap <= kTmemCols ? 2 : 1;
    g.mblocks = mblocks;
    auto pairs_up = [](const void *q, long long ld) { return ((uintptr_t)q & 3u) == 0 && ld % 2 == 0; };
    g.paired = p.N % 2 == 0 && pairs_up(p.out, p.ldo) && (!p.residual || pairs_up(p.residual, p.ldr));
    const int table = p.offsets ? p.E * 4 : 0;
    const int budget = d.smem.load(std::memory_order_relaxed) - 1024 - table;
    g.stages = min(kMaxStages, budget / g.stage_bytes);
    if (g.stages < 2) return cudaErrorNotSupported;
    const int smem = 1024 + g.stages * g.stage_bytes + table;
    const long long most = ((p.rows + kStepRows - 1) / kStepRows + groups) * (long long)mblocks;  // >= the items
    // items are numbered in 32 bits, also where offsets that do not ascend give every
    // expert all rows
    if ((p.offsets ? p.E : 1) * ((p.rows + g.tcap - 1) / g.tcap) * (long long)mblocks > 0x7fff0000LL)
        return cudaErrorNotSupported;
    const int planes = p.stride_e ? p.E : 1;  // experts may share one matrix
    alignas(64) CUtensorMap tmx, tmx_half, tmw, tmu;
    if (!encode(&tmx, p.dtype, p.x, p.K, p.x_rows, p.ldx, 0, 0, p.row_token ? 1 : kBoxRows) ||
        !encode(&tmx_half, p.dtype, p.x, p.K, p.x_rows, p.ldx, 0, 0, kBoxRows / 2) ||
        !encode(&tmw, p.dtype, p.w, p.K, p.N, p.ldw, planes, p.stride_e ? p.stride_e : p.ldw, kM))
        return cudaErrorNotSupported;
    tmu = tmw;
    if (mats == 2 && !encode(&tmu, p.dtype, p.w_up, p.K, p.N, p.ldw, planes, p.stride_e ? p.stride_e : p.ldw, kM))
        return cudaErrorNotSupported;
    const int n = (int)min(most, (long long)all);
    if (p.dtype == MOE_DTYPE_BF16)
        return mats == 2 ? launch<__nv_bfloat16, 2>(p, g, n, smem, d, tmx, tmx_half, tmw, tmu, st)
                         : launch<__nv_bfloat16, 1>(p, g, n, smem, d, tmx, tmx_half, tmw, tmu, st);
    return mats == 2 ? launch<__half, 2>(p, g, n, smem, d, tmx, tmx_half, tmw, tmu, st)
                     : launch<__half, 1>(p, g, n, smem, d, tmx, tmx_half, tmw, tmu, st);
}

cudaError_t read_ops_status(unsigned *value, cudaStream_t st) {
    *value = 0;
    cudaError_t err = cudaMemcpyFromSymbolAsync(value, g_ops_status, 4, 0, cudaMemcpyDeviceToHost, st);
    if (err == cudaSuccess) err = cudaStreamSynchronize(st);
    if (err != cudaSuccess || *value == 0) return err;
    const unsigned zero = 0;
    err = cudaMemcpyToSymbolAsync(g_ops_status, &zero, 4, 0, cudaMemcpyHostToDevice, st);
    return err == cudaSuccess ? cudaStreamSynchronize(st) : err;
}

}  // namespace ops
}  // namespace moe
