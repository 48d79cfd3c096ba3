// ops_gemm_q8.cu -- products of 8-bit codes over many rows (moe_linear_q8,
// moe_grouped_linear_q8) on the 5th-generation tensor cores.
//
//   out[r, c] = act(sx[r] sw[c] sum_k x[r, k] w[c, k] + bias[c]) (* the up product) (+ residual[r, c])
//
// The tensor cores of this GPU take no 8-bit integers (tcgen05 kind::i8 is not there,
// mma.sync reaches 150 TOPS), and no pair of 8-bit floats holds one. They take f16 at
// full rate, where whole numbers to 2048 are exact, so the codes become f16 between
// shared memory and the MMA. The sums in f32 are exact to 2^24.
//
// Tiles, work items and epilogue are those of the 16-bit products (ops_gemm.cu, ops_pair.cuh): a
// pair of CTAs, 128 weight rows per CTA as the M operand, up to 256 rows of x (gated: 128) as N.
// New is what lies between the loads and the MMAs:
//   - a load stage holds 128 inputs as codes: 16 KB of weights (per matrix) and half of
//     the tile's rows of x, 128 bytes each, by TMA with the 128-byte swizzle. A warp loads the
//     weights, one or two the rows of x, and another finds the work items for all;
//   - three groups of four warps convert, a unit each in turn: a half stage, or a whole one of
//     short tiles. The weights go to tensor memory (thread = weight row = lane; the MMA takes A
//     from there), the rows of x to a second ring in shared memory, in the swizzled layout of a
//     16-bit tile;
//   - A in tensor memory is what makes the rates meet: per 64 inputs at 256 rows a CTA's MMAs
//     take 512 cycles, in which its shared memory moves 64 KB: 16 in by TMA, 16 read by the
//     converters, 16 written by them (x) and 16 read by the MMAs (x). With A there too it
//     would be 96. Tensor memory then has room for one accumulator set at 256 rows (two up
//     to 192; gated: one at 128 and two up to 64).
//
// 24 warps at 80 registers: what does not fit in those spills into the conversion loop or the
// epilogue and costs at once (gated 8192x4096x2048, 20 bytes spilled: 165 us, without 155). So does
// every instruction of the conversion loop: a sixth for 4 codes makes it 179, and the 8 selects a
// piece that kept neighbouring pieces of x on different banks made it 152 of 149.
//
// Bound. Long products: the tensor cores, but for the epilogue of a single accumulator set, in
// which they stand still (8192x4096x4096 146 us, 1880 TFLOP/s; gated 8192x4096x2048 149 us,
// 1850; the tensor pipe is busy 80 % of the second's cycles). Short tiles: the converters,
// whose 5 operations for 4 codes share the integer pipe (62 % busy), and their waits for each other:
// about 650 cycles per 128 inputs. A few hundred rows: 2.5 us before the first MMA, and the epilogue
// (317x2032x4104 with GELU and a residual 12.8 us: 5 of them steps, 2.7 the epilogue). Few rows
// per expert: HBM (64 tokens, 768 -> 2048, 128 experts: 38 us, 5.3 TB/s).
//
// Every wait is bounded (1 s, reported through moe_ops_check); after one gives
// up, all roles stop and the pair waits for its copies in flight before it ends.
#include "ops_pair.cuh"
#include "ops_q8.cuh"

namespace moe {
namespace ops {
namespace {

constexpr int kIn = 128;                 // inputs of a load stage: one 128-byte row of a swizzled tile
constexpr int kTileW = kM * kIn;         // bytes of a weight tile
constexpr int kMaxStages = 12;           // load stages
constexpr int kUnits = 4;                // hand-overs to the MMAs in flight: half stages, or stages
constexpr int kItems = 4;                // work items that the loads may be ahead
constexpr int kGroups = 3;               // groups of four converter warps, one per quadrant of the tensor-memory lanes
constexpr int kConvert = 4 * kGroups;
constexpr int kLoadW = kConvert + kEpilogue, kLoadX = kLoadW + 1, kWalker = kLoadX + 1, kMmaWarp = kWalker + 1;
constexpr int kThreads = 32 * (kMmaWarp + 1);

struct Tiling : Tiles {
    int stages;
    int stage_bytes;
    int half_bytes;   // shared memory of a half stage as f16: the rows of x
    int a_col;        // tensor memory: first column of the weights as f16
};

// TMA loads into this CTA's shared memory, counted by its own barrier
__device__ __forceinline__ void load_2d(uint32_t dst, const void *map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void load_3d(uint32_t dst, const void *map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void load_gather4(uint32_t dst, const void *map, int x, const int (&r)[4], uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(map), "r"(x), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(bar)
        : "memory");
}

__device__ __forceinline__ uint4 lds(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void sts(uint32_t addr, uint2 a, uint2 b) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a.x), "r"(a.y), "r"(b.x), "r"(b.y) : "memory");
}

__device__ __forceinline__ void arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// On a barrier of the pair's first CTA. What it orders is in this SM and has completed: stores
// to tensor memory (wait::st) and to shared memory (the proxy fence); the MMA reads both in
// this SM. A release at cluster scope would wait for a round trip to L2 in each half stage.
__device__ __forceinline__ void arrive_in_first(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// D[tmem of both CTAs] (+)= A * B^T: each CTA's tensor memory holds its 128 rows of A, its
// shared memory half of B's rows; issued by one thread of the first CTA
__device__ __forceinline__ void mma_pair_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 bd;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 bd, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], bd, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescHigh)
        : "memory");
}

// The groups in shared memory: their first item, first row, rows, and tiles x 32 + rows of a tile
// / 16.
struct Group {
    int first, lo, rows, tiles;
};

// Fill the table, by the block; the number of all items. warp_sum: kThreads / 32 numbers.
__device__ __forceinline__ int number_groups(const Product &p, const Tiles &g, Group *table, int *warp_sum) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int base = 0;
    for (int e0 = 0; e0 < p.E; e0 += kThreads) {
        const int e = e0 + tid;
        int items = 0, lo = 0, hi = 0, t = kStepRows, nt = 0;
        if (e < p.E) {
            group_rows(p, e, lo, hi);
            if (hi > lo) {
                t = tile_rows(hi - lo, g.tcap);
                nt = (hi - lo + t - 1) / t;
                items = nt * g.mblocks;
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
        if (e < p.E) table[e] = Group{before + scan - items, lo, hi - lo, nt * 32 + t / 16};
        base += sum;
        __syncthreads();
    }
    return base;
}

// Item i of all (i < total), by a whole warp: two rounds of 32 comparisons find its group. one:
// the only group, without offsets.
__device__ __forceinline__ Item find_item(const Product &p, const Group *table, const Group &one, int mblocks, int i) {
    const int lane = threadIdx.x & 31;
    int e = 0;
    Group g = one;
    if (p.offsets) {
        const int step = (p.E + 31) >> 5;  // <= 32
        const int c = lane * step;
        e = (__popc(__ballot_sync(0xffffffffu, c < p.E && table[c].first <= i)) - 1) * step;
        const int f = e + lane;
        e += __popc(__ballot_sync(0xffffffffu, lane < step && f < p.E && table[f].first <= i)) - 1;
        g = table[e];
    }
    const int nt = max(g.tiles >> 5, 1), T = (g.tiles & 31) * 16;
    i -= g.first;
    // bands of kBand row tiles: the tiles of a band run side by side on one weight block, then
    // on the next
    int band = 0, bh = nt;
    if (nt > kBand) {
        band = i / (kBand * mblocks);
        i -= band * kBand * mblocks;
        bh = max(min(kBand, nt - band * kBand), 1);
    }
    Item it;
    it.m = bh == 1 ? i : i / bh;
    it.e = e;
    const int first = (band * kBand + i - it.m * bh) * T;
    it.r0 = g.lo + first;
    it.rows = min(T, g.rows - first);
    it.T = tile_rows(it.rows, T);  // (a group's last tile may be shorter)
    return it;
}

// The pair's items, as one warp has found them. (To find one takes longer than a short
// tile's conversions.)
struct RingItems {
    const Item *ring;
    uint32_t full, empty;
    volatile int *abort_flag;
    uint32_t n;
    __device__ __forceinline__ bool next(Item &it) {
        const uint32_t s = n % kItems;
        if (!__all_sync(0xffffffffu, wait(full + 8 * s, (n / kItems) & 1, abort_flag))) return false;
        it = ring[s];
        __syncwarp();
        if ((threadIdx.x & 31) == 0) arrive(empty + 8 * s);
        ++n;
        return it.T != 0;
    }
};

template <typename T, int MATS, bool WIDE>
__global__ void __launch_bounds__(kThreads, 1)
    product_gemm_q8_kernel(const __grid_constant__ Product p, const __grid_constant__ Tiling g,
                           const __grid_constant__ CUtensorMap tmx, const __grid_constant__ CUtensorMap tmx_half,
                           const __grid_constant__ CUtensorMap tmw, const __grid_constant__ CUtensorMap tmu) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    // full, empty: load stages of this CTA. u_full (the first CTA's counts for both), u_empty: units.
    // acc_empty: the first CTA's counts for both
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages], u_full[kUnits], u_empty[kUnits];
    __shared__ uint64_t acc_full[2], acc_empty[2], item_full[kItems], item_empty[kItems], drain;
    __shared__ Item item_ring[kItems];
    __shared__ uint32_t tslot;
    __shared__ int abort_word, warp_sum[kThreads / 32];
    __shared__ __align__(16) float row_scale[kEpilogue][128];
    constexpr uint32_t kHalves = WIDE ? 2 : 1;  // half stages of a unit
    volatile int *abort_flag = &abort_word;
    unsigned char *ring = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
    unsigned char *f16_ring = ring + g.stages * g.stage_bytes;
    Group *table = reinterpret_cast<Group *>(f16_ring + kUnits * kHalves * g.half_bytes);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = (int)cluster_rank();
    const int item0 = blockIdx.x / kPair, item_step = gridDim.x / kPair;

    if (tid == 0) {
        abort_word = 0;
        for (int i = 0; i < g.stages; ++i) {
            ptx::mbar_init(&full[i], 1);
            ptx::mbar_init(&empty[i], 8 / kHalves);  // the warps that convert it
        }
        for (int i = 0; i < kUnits; ++i) {
            ptx::mbar_init(&u_full[i], 4 * kPair);
            ptx::mbar_init(&u_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&acc_full[i], 1);
            ptx::mbar_init(&acc_empty[i], kEpilogue * kPair);  // the epilogues' warps
        }
        for (int i = 0; i < kItems; ++i) {
            ptx::mbar_init(&item_full[i], 1);
            ptx::mbar_init(&item_empty[i], kConvert + kEpilogue + 2 + (rank == 0 ? 1 : 0));  // all but the walker
        }
        ptx::mbar_init(&drain, 1);
        ptx::mbar_fence_init();
        ptx::prefetch_tensormap(&tmx);
        ptx::prefetch_tensormap(&tmx_half);
        ptx::prefetch_tensormap(&tmw);
        if (MATS == 2) ptx::prefetch_tensormap(&tmu);
    }
    if (warp == kMmaWarp) tmem_alloc_pair(&tslot, kTmemCols);
    tc::fence_before_sync();
    __syncwarp();
    cluster_arrive();
    Group one{0, 0, p.rows, 0};
    int total = 0;
    if (!p.offsets) {
        const int t = tile_rows(p.rows, g.tcap), nt = (p.rows + t - 1) / t;
        one.tiles = nt * 32 + t / 16;
        total = nt * g.mblocks;
    }
    ptx::griddep_wait();
    if (p.offsets) total = number_groups(p, g, table, warp_sum);
    cluster_wait();  // both CTAs' barriers are ready
    tc::fence_after_sync();
    const uint32_t tmem = tslot;
    const uint32_t ring_addr = tc::smem_u32(ring), full_addr = tc::smem_u32(full), empty_addr = tc::smem_u32(empty);
    const uint32_t f16_addr = tc::smem_u32(f16_ring), u_full_addr = tc::smem_u32(u_full), u_empty_addr = tc::smem_u32(u_empty);
    const uint32_t acc_full_addr = tc::smem_u32(acc_full), acc_empty_addr = tc::smem_u32(acc_empty);
    const int nk = (p.K + kIn - 1) / kIn, nh = 2 * nk;  // load stages and half stages of a tile (past K: zeros)
    RingItems items{item_ring, tc::smem_u32(item_full), tc::smem_u32(item_empty), abort_flag, 0};
    const uint32_t stages = g.stages, stage_bytes = g.stage_bytes;

    if (warp == kLoadW) {
        // ---- weights ------------------------------------------------------------
        Ring at{ring_addr, empty_addr, full_addr, 0, 1};  // a fresh barrier passes the wait for phase 1
        Item it;
        bool ok = true;
        while (ok && items.next(it)) {
            const int half = it.T / kPair;  // rows of x that this CTA loads
            const uint32_t bytes = MATS * kTileW + (p.row_token ? half : box_rows(half)) * kIn;
            const int col = (it.m * kPair + rank) * kM, plane = p.stride_e ? it.e : 0;
#pragma unroll 1
            for (int k = 0; k < nk; ++k) {
                if (!(ok = __all_sync(0xffffffffu, wait(at.empty, at.phase, abort_flag)))) break;
                if (tc::elect_one()) {
                    expect_tx(at.full, bytes);
                    load_3d(at.stage, &tmw, k * kIn, col, plane, at.full);
                    if (MATS == 2) load_3d(at.stage + kTileW, &tmu, k * kIn, col, plane, at.full);
                }
                at.next(stages, stage_bytes);
            }
        }
        // Before the CTA may end, every copy has landed and every stage has been handed back, as
        // in ops_gemm.cu.
        const unsigned long long t0 = globaltimer();
        for (uint32_t i = 0; i < stages; ++i) {
            const uint32_t next = i < at.s ? at.phase ^ 1 : at.phase;
            settle(full_addr + 8 * i, next, t0);
            settle(empty_addr + 8 * i, next, t0);
        }
        __syncwarp();
    } else if (warp == kLoadX || warp == kWalker) {
        // ---- rows of x; the walk over the items -----------------------------------------
        // Boxes are loaded by the first warp, gathered rows by both (every second copy of four
        // rows: a warp issues them one after another) unless tiles are the shortest.
        // (A warp that loads takes part in every stage: they are handed back out of order, and
        // one that skips some could take the phase of the lap before the last for the last.)
        Ring at{ring_addr + MATS * kTileW, empty_addr, full_addr, 0, 1};
        const int w = warp - kLoadX;
        Item it;
        bool ok = true;
        uint32_t n = 0;
        for (int i = item0; ok; i += item_step, ++n) {
            if (w) {
                const bool more = i < total;
                if (more) it = find_item(p, table, one, g.mblocks, i);
                const uint32_t slot = n % kItems;
                if (!(ok = __all_sync(0xffffffffu, wait(items.empty + 8 * slot, ((n / kItems) & 1) ^ 1, abort_flag)))) break;
                if (lane == 0) {
                    if (!more) it.T = 0;  // the end
                    item_ring[slot] = it;
                    arrive(items.full + 8 * slot);
                }
                __syncwarp();
                if (!more) break;
            } else if (!items.next(it)) {
                break;
            }
            const int half = it.T / kPair, r0 = it.r0 + rank * half;
            if (p.row_token) {
                // lane j's rows are the warp's j-th copy; rows past the end repeat the last one
                const int warps = g.tcap > kStepRows ? 2 : 1, copies = (half / 4 - w + warps - 1) / warps;
                if (w >= warps) continue;
                const int first_row = 4 * (w + warps * lane);
                int rows[4] = {};
                if (lane < copies) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) rows[j] = input_row(p, min(r0 + first_row + j, it.r0 + it.rows - 1));
                }
#pragma unroll 1
                for (int k = 0; k < nk; ++k) {
                    if (!(ok = __all_sync(0xffffffffu, wait(at.empty, at.phase, abort_flag)))) break;
                    if (lane < copies) load_gather4(at.stage + first_row * kIn, &tmx, k * kIn, rows, at.full);
                    at.next(stages, stage_bytes);
                }
            } else if (w == 0) {
                // two boxes of x at most: the last one is half as high if that is enough
                const int n1 = half > kBoxRows ? (half - kBoxRows > kBoxRows / 2 ? 2 : 1) : 0;
                const CUtensorMap *map0 = half > kBoxRows / 2 ? &tmx : &tmx_half, *map1 = n1 == 2 ? &tmx : &tmx_half;
#pragma unroll 1
                for (int k = 0; k < nk; ++k) {
                    if (!(ok = __all_sync(0xffffffffu, wait(at.empty, at.phase, abort_flag)))) break;
                    if (tc::elect_one()) {
                        load_2d(at.stage, map0, k * kIn, r0, at.full);
                        if (n1) load_2d(at.stage + kBoxRows * kIn, map1, k * kIn, r0 + kBoxRows, at.full);
                    }
                    at.next(stages, stage_bytes);
                }
            }
        }
        __syncwarp();
    } else if (warp == kMmaWarp && rank == 0) {
        // ---- MMAs --------------------------------------------------------------
        uint32_t c = 0;  // units so far
        Item it;
        bool ok = true;
        const uint32_t base = tc::idesc_f16_f32(kPair * kM, 0);
        const int units = nh / kHalves;  // of a tile
        int n = 0;
        for (; ok && items.next(it); ++n) {
            if (tc::elect_one()) {
                const uint32_t idesc = base | ((uint32_t)(it.T >> 3) << 17);
                const int buf = g.bufs == 2 ? n & 1 : 0, use = g.bufs == 2 ? n >> 1 : n;
                const uint32_t acc = tmem + (uint32_t)(buf * MATS * g.tcap), acc_up = acc + g.tcap;
                // the epilogues have read what this accumulator set held
                ok = wait(acc_empty_addr + 8 * buf, (uint32_t)((use & 1) ^ 1), abort_flag);
                tc::fence_after_sync();
#pragma unroll 1
                for (int k = 0; ok && k < units; ++k) {
                    const uint32_t u = (c + k) % kUnits;
                    if (!(ok = wait(u_full_addr + 8 * u, ((c + k) / kUnits) & 1, abort_flag))) break;
                    tc::fence_after_sync();
                    uint32_t a = tmem + g.a_col + u * kHalves * (MATS * kK / 2);
                    uint32_t b = desc_low(f16_addr + u * kHalves * g.half_bytes);
                    // the first MMA of a tile overwrites
#pragma unroll
                    for (int q = 0; q < kK / 16; ++q) {
                        mma_pair_ts(acc, a + 8 * q, b + 2 * q, idesc, q ? 1 : k);
                        if (MATS == 2) mma_pair_ts(acc_up, a + kK / 2 + 8 * q, b + 2 * q, idesc, q ? 1 : k);
                    }
                    if (WIDE) {
                        a += kK / 2;
                        b += g.half_bytes >> 4;
#pragma unroll
                        for (int q = 0; q < kK / 16; ++q) mma_pair_ts(acc, a + 8 * q, b + 2 * q, idesc, 1);
                    }
                    commit_pair(u_empty_addr + 8 * u);
                }
                if (ok) commit_pair(acc_full_addr + 8 * buf);
            }
            ok = __all_sync(0xffffffffu, ok);
            c += units;
        }
        // after an abort, let the MMAs in flight end before the tensor memory is freed
        if (__any_sync(0xffffffffu, *abort_flag) && tc::elect_one()) {
            commit_pair(tc::smem_u32(&drain));
            settle(tc::smem_u32(&drain), 0, globaltimer());
        }
        // the other CTA's arrivals on the accumulator sets are here before this one may end
        const unsigned long long t0 = globaltimer();
        for (int b = 0; b < g.bufs; ++b) {
            const int uses = (n + g.bufs - 1 - b) / g.bufs;
            if (uses > 0) settle(acc_empty_addr + 8 * b, (uint32_t)(uses - 1) & 1, t0);
        }
        __syncwarp();
    } else if (warp < kConvert) {
        // ---- codes to f16 --------------------------------------------------------
        // The units of all tiles are dealt to the groups in turn. (A wait takes a barrier two
        // phases behind for one that is done. None is: this group's last unit, v - 3, began once
        // the MMAs of unit v - 7 had ended. That is after the last use but one of the unit's
        // place, and after the last fill of the stage if there are at least 4 stages (wide: 7).)
        const int q = warp & 3;  // quadrant of the lanes
        const uint32_t peer_full = in_first(u_full_addr);
        // This thread's weight row, its first 16 codes; the j-th of the four pieces of a half stage
        // lies at that address ^ 16 j, and the second half at ^ 64.
        const int wr = 32 * q + lane;
        const uint32_t w_src = ring_addr + wr * 128 + ((wr & 7) << 4);
        // This thread's pieces of x: row and 16 codes of an atom of 8 rows. The lanes of a quarter
        // warp take rows r and r ^ 5, which lie on different banks in the reads (bit 2) and in the
        // writes (bit 0).
        const int l = lane & 7, xr = (lane >> 3) ^ (l & 4 ? 5 : 0);
        const uint32_t x_src = ring_addr + MATS * kTileW + q * 1024 + xr * 128 + (((l & 3) ^ xr) << 4);
        const uint32_t x_dst = f16_addr + q * 1024 + xr * 128 + (((2 * (l & 3)) ^ xr) << 4);
        const uint32_t a_at = tmem + ((uint32_t)(32 * q) << 16) + g.a_col;
        uint32_t v = warp >> 2;             // this group's unit
        uint32_t slot = v * kHalves / 2, phase = 0;  // its load stage in the ring, and the lap
        uint32_t end = 0;                   // units of the tiles so far
        int atoms = 0;                      // this warp's of the tile: every fourth
        bool ok = true;
        Item it;
        while ((ok = items.next(it))) {
            end += nh / kHalves;
            atoms = it.T / (kPair * 8) - q;
#pragma unroll 1
            for (; v < end; v += kGroups) {
                const uint32_t u = v % kUnits, stage = slot * stage_bytes;
                if (!(ok = __all_sync(0xffffffffu, wait(full_addr + 8 * slot, phase, abort_flag)))) break;
                constexpr int kX = MATS == 2 || WIDE ? 2 : 4;  // atoms of a warp, at most
                uint4 w[MATS][4], x[kX];
                auto load = [&](uint32_t turn) {
                    const uint32_t w_at = (w_src ^ turn) + stage, x_at = (x_src ^ turn) + stage;
#pragma unroll
                    for (int m = 0; m < MATS; ++m)
#pragma unroll
                        for (int j = 0; j < 4; ++j) w[m][j] = lds((w_at ^ (16 * j)) + m * kTileW);
#pragma unroll
                    for (int j = 0; j < kX; ++j)
                        if (4 * j < atoms) x[j] = lds(x_at + j * 4096);
                };
                auto store = [&](uint32_t place) {
                    const uint32_t a = a_at + place * (MATS * kK / 2), dst = x_dst + place * g.half_bytes;
#pragma unroll
                    for (int m = 0; m < MATS; ++m)
#pragma unroll
                        for (int j = 0; j < 4; j += 2) {
                            uint32_t f16[16];
#pragma unroll
                            for (int b = 0; b < 8; ++b) {
                                const uint2 f = codes_to_f16(word(w[m][j + (b >> 2)], b & 3));
                                f16[2 * b] = f.x;
                                f16[2 * b + 1] = f.y;
                            }
                            tc::st_32x32b_x16_async(a + m * (kK / 2) + 8 * j, f16);
                        }
#pragma unroll
                    for (int j = 0; j < kX; ++j) {
                        if (4 * j >= atoms) break;
                        sts(dst + j * 4096, codes_to_f16(x[j].x), codes_to_f16(x[j].y));
                        sts((dst ^ 16) + j * 4096, codes_to_f16(x[j].z), codes_to_f16(x[j].w));
                    }
                };
                load(WIDE ? 0u : (v & 1) << 6);
                // the MMAs have read what this unit held
                if (!(ok = __all_sync(0xffffffffu, wait(u_empty_addr + 8 * u, ((v / kUnits) & 1) ^ 1, abort_flag)))) break;
                tc::fence_after_sync();
                store(u * kHalves);
                if (WIDE) {
                    load(64u);
                    store(u * kHalves + 1);
                }
                tc::wait_st();
                tc::fence_async_shared();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    arrive_in_first(peer_full + 8 * u);
                    arrive(empty_addr + 8 * slot);
                }
                slot += WIDE ? kGroups : ((v + kGroups) >> 1) - (v >> 1);
                if (slot >= stages) {
                    slot -= stages;
                    phase ^= 1;
                }
            }
            if (!ok) break;
        }
        // the commits on the units have arrived before the CTA may end
        if (warp == 0) {
            const unsigned long long t0 = globaltimer();
            for (uint32_t u = 0; u < kUnits; ++u)
                if (end > u) settle(u_empty_addr + 8 * u, ((end - u - 1) / kUnits) & 1, t0);
        }
        __syncwarp();
    } else if (warp >= kConvert && warp < kConvert + kEpilogue) {
        // ---- epilogue ----------------------------------------------------------
        store_tiles<T, MATS, true>(p, g, items, rank, tmem, warp - kConvert, acc_full_addr, acc_empty_addr, abort_flag,
                                   row_scale[warp - kConvert]);
    }
    // Neither CTA ends while the other may still use its memory. (Relaxed: all arrivals that cross
    // have been waited for, unless a wait gave up. A release would wait for the last stores to reach
    // L2.)
    tc::fence_before_sync();
    if (*abort_flag) asm volatile("fence.acq_rel.cluster;" ::: "memory");
    __syncwarp();
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    cluster_wait();
    tc::fence_after_sync();
    if (warp == kMmaWarp) tmem_dealloc_pair(tmem, kTmemCols);
}

// rows of `cols` codes `ld` apart, `planes` of them (rank 3) or one (rank 2), boxes of
// 128 columns x box_rows rows; what lies outside reads as zeros
bool encode(CUtensorMap *m, const void *base, long long cols, long long rows, long long ld, int planes, long long stride,
            int box_rows) {
    PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn();
    if (!fn) return false;
    const int rank = planes ? 3 : 2;
    cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)(planes ? planes : 1)};
    cuuint64_t strides[2] = {(cuuint64_t)ld, (cuuint64_t)stride};
    cuuint32_t box[3] = {(cuuint32_t)kIn, (cuuint32_t)box_rows, 1};
    cuuint32_t es[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, rank, const_cast<void *>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
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

// A unit is a whole load stage of tiles of up to 96 rows (half as many hand-overs: 64 tokens down
// 49 to 39 us) where enough stages fit beside them and the table of the groups (of 1024 groups: up
// to 64 rows; 256 tokens, 8 of 1024 experts, 768 -> 2048: 210 us, 268 with 96 rows and half stages),
// otherwise half of one (long ones: 8192x4096x4096 152 us, 169 with whole stages). room: shared
// memory for all of that.
// Tensor memory beside the accumulator sets holds the kUnits units of weights as f16.
constexpr int half_cols(int mats) { return mats * kK / 2; }
constexpr int max_rows(int mats) { return mats == 2 ? 128 : 256; }
static_assert(max_rows(1) + kUnits * half_cols(1) <= kTmemCols && 2 * max_rows(2) + kUnits * half_cols(2) <= kTmemCols,
              "they fit");
int stage_bytes(int mats, int rows) { return mats * kTileW + box_rows(rows / kPair) * kIn; }
int half_bytes(int rows) { return rows / kPair * kK * 2; }
int stages_of(int mats, int rows, bool wide, int room) {
    return min(kMaxStages, (room - kUnits * (wide ? 2 : 1) * half_bytes(rows)) / stage_bytes(mats, rows));
}
int least_stages(bool wide) { return wide ? 7 : 4; }  // (see the converters)
bool wide_units(int mats, int rows, int room) {
    return mats == 1 && rows <= 96 && stages_of(mats, rows, true, room) >= least_stages(true);
}
int sets_of(int mats, int rows, bool wide) {
    return 2 * mats * rows + kUnits * (wide ? 2 : 1) * half_cols(mats) <= kTmemCols ? 2 : 1;
}

// Rows per tile: the least time of a simple model, in cycles, as in ops_gemm.cu. Waves of tiles
// on the pairs, each nk steps of 128 inputs: the longest of the MMAs (4 per row and matrix) and
// the converters (fitted to 64..256 rows of 8192x4096x4096 and of the gated 8192x4096x2048;
// short tiles hand over half stages less often); 500 for the tile itself; the epilogue of the
// last tile, and two thirds of it for every tile with one accumulator set. Among groups, of
// which some are larger than the mean, a larger cap may cost 8 % more (1024 tokens, 6 of
// 256 skewed experts, gated 4096 -> 2048: 340 us with 64 rows, 297 with 128).
int pick_rows(const Product &p, int mblocks, int groups, int mean, int nk, int pairs, int room) {
    const int mats = p.w_up ? 2 : 1;
    const int per_row = 20 + 15 * (mats - 1) + (p.act != MOE_EPI_NONE ? 15 : 0) + (p.residual ? 15 : 0);
    long long cost[256 / kStepRows + 1], least = -1;
    for (int cap = max_rows(mats); cap >= kStepRows; cap -= kStepRows) {
        const int t = tile_rows(mean, cap);
        const long long items = (long long)groups * mblocks * ((mean + t - 1) / t);
        const long long waves = (items + pairs - 1) / pairs;
        const int convert = mats == 2 ? 850 + 3 * t : 600 + 9 * t / 4;
        const bool wide = wide_units(mats, cap, room);
        const long long step = max(4 * mats * t, wide ? convert : max(convert, 850));
        const long long one_set = sets_of(mats, cap, wide) == 1 ? waves * per_row * t * 2 / 3 : 0;
        const long long c = cost[cap / kStepRows] = waves * (nk * step + 500) + per_row * t + one_set;
        if (least < 0 || c < least) least = c;
    }
    int cap = max_rows(mats);
    while (cost[cap / kStepRows] > (p.offsets ? least + least * 8 / 100 : least)) cap -= kStepRows;
    return cap;
}

cudaError_t look_up(int dev, Device &d) {
    int smem = 0, sms = 0, pairs = 0;
    cudaFuncAttributes fa;
    cudaError_t err;
    auto k = product_gemm_q8_kernel<__half, 2, false>;
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

template <typename T, int MATS, bool WIDE>
cudaError_t launch(const Product &p, const Tiling &g, int pairs, int smem, Device &d, const CUtensorMap &tmx,
                   const CUtensorMap &tmx_half, const CUtensorMap &tmw, const CUtensorMap &tmu, cudaStream_t st) {
    auto k = product_gemm_q8_kernel<T, MATS, WIDE>;
    const unsigned bit = 1u << (MATS - 1 + (WIDE ? 2 : 0) + (p.dtype == MOE_DTYPE_BF16 ? 4 : 0));
    if (!(d.ready.load(std::memory_order_acquire) & bit)) {
        const cudaError_t err = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                     d.smem.load(std::memory_order_relaxed));
        if (err != cudaSuccess) return err;
        d.ready.fetch_or(bit, std::memory_order_release);
    }
    return launch_overlapped(k, dim3(kPair * pairs), kThreads, smem, kPair, st, p, g, tmx, tmx_half, tmw, tmu);
}

}  // namespace

cudaError_t launch_product_gemm_q8(const Product &p, cudaStream_t st) {
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
    const int table = p.offsets ? p.E * (int)sizeof(Group) : 0;
    const int room = d.smem.load(std::memory_order_relaxed) - 1024 - table;
    Tiling g;
    g.tcap = pick_rows(p, mblocks, groups, (p.rows + groups - 1) / groups, (p.K + kIn - 1) / kIn, all, room);
    const bool wide = wide_units(mats, g.tcap, room);
    const int halves = wide ? 2 * kUnits : kUnits;
    g.a_col = kTmemCols - halves * half_cols(mats);
    g.bufs = sets_of(mats, g.tcap, wide);
    g.stages = stages_of(mats, g.tcap, wide, room);
    if (g.stages < least_stages(wide)) return cudaErrorNotSupported;
    g.stage_bytes = stage_bytes(mats, g.tcap);
    g.half_bytes = half_bytes(g.tcap);
    const int smem = 1024 + g.stages * g.stage_bytes + halves * g.half_bytes + table;
    g.mblocks = mblocks;
    auto pairs_up = [](const void *q, long long ld) { return ((uintptr_t)q & 3u) == 0 && ld % 2 == 0; };
    g.paired = p.N % 2 == 0 && pairs_up(p.out, p.ldo) && (!p.residual || pairs_up(p.residual, p.ldr));
    const long long most = ((p.rows + kStepRows - 1) / kStepRows + groups) * (long long)mblocks;  // >= the items
    // items are numbered in 32 bits, also where offsets that do not ascend give every
    // expert all rows
    if ((p.offsets ? p.E : 1) * ((p.rows + g.tcap - 1) / g.tcap) * (long long)mblocks > 0x7fff0000LL)
        return cudaErrorNotSupported;
    const int planes = p.stride_e ? p.E : 1;  // experts may share one matrix
    alignas(64) CUtensorMap tmx, tmx_half, tmw, tmu;
    if (!encode(&tmx, p.x, p.K, p.x_rows, p.ldx, 0, 0, p.row_token ? 1 : kBoxRows) ||
        !encode(&tmx_half, p.x, p.K, p.x_rows, p.ldx, 0, 0, kBoxRows / 2) ||
        !encode(&tmw, p.w, p.K, p.N, p.ldw, planes, p.stride_e ? p.stride_e : p.ldw, kM))
        return cudaErrorNotSupported;
    tmu = tmw;
    if (mats == 2 && !encode(&tmu, p.w_up, p.K, p.N, p.ldw, planes, p.stride_e ? p.stride_e : p.ldw, kM))
        return cudaErrorNotSupported;
    const int n = (int)min(most, (long long)all);
    auto go = [&](auto type) {
        using T = decltype(type);
        return mats == 2 ? launch<T, 2, false>(p, g, n, smem, d, tmx, tmx_half, tmw, tmu, st)
               : wide    ? launch<T, 1, true>(p, g, n, smem, d, tmx, tmx_half, tmw, tmu, st)
                         : launch<T, 1, false>(p, g, n, smem, d, tmx, tmx_half, tmw, tmu, st);
    };
    return p.dtype == MOE_DTYPE_BF16 ? go(__nv_bfloat16()) : go(__half());
}

unsigned *ops_status_q8(cudaError_t *err) {
    void *at = nullptr;
    *err = cudaGetSymbolAddress(&at, g_ops_status);
    return static_cast<unsigned *>(at);
}

}  // namespace ops
}  // namespace moe
