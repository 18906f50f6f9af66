// Products grouped by expert on the 5th-generation tensor cores (tcgen05 + TMEM): the
// product itself (16-bit and int8) and both gradients, one kernel.
//
// The accumulator D [M][N] holds the output transposed: its M rows (TMEM lanes) are the
// output's contiguous columns, its N columns are output rows. The ragged side, the rows of
// a group, is then the MMA's N, which takes any multiple of 16 (an expert with 20 rows
// costs 32 columns, not a 128-row tile), and a warp stores 32 neighbouring outputs of a
// row at a time. Operands, c the summed index:
//   product  A = w[e] (rows j, K-major),   B = x rows (K-major),    c = k
//   dx       A = w[e]^T (M-major: j runs along w's rows), B = dy rows (K-major), c = n
//   dw       A = x^T (M-major), B = dy^T (N-major), c = the rows of the group
// All of them are boxes of 128 bytes x rows in the 128-byte swizzle, by TMA from the
// tensors as they are; zero fill past n and k, so that neither needs to be a multiple of
// anything. Rows past a group's end are the next group's: in the product and in dx they
// give columns of D that nobody reads, in dw they are the sum's tail, and one warp zeroes
// them in shared memory (both operands: they may hold NaN) before the MMA sees them.
//
// A CTA, or a pair of CTAs as one cta_group::2 (then M = 256, each CTA holding 128 rows
// of A and half of B's columns: half the shared-memory traffic per MMA), walks its tiles
// in a fixed stride over all groups' tiles, which every CTA lists for itself from the
// offsets at its start: no host read-back, no workspace, no second launch. Where a few
// tiles have long sums, the CTAs of a cluster take a part of each and join them through
// each other's shared memory. The sums' order does not depend on timing.
#include <algorithm>
#include <cstring>
#include <mutex>

#include "products.cuh"
#include "tensor_map.cuh"

namespace nvmoe {
namespace {

constexpr int kEpiWarps = 8;            // two for each quarter of the TMEM lanes
constexpr int kTmaWarp = kEpiWarps, kMmaWarp = kEpiWarps + 1, kTailWarp = kEpiWarps + 2, kTileWarp = kEpiWarps + 3;
constexpr int kThreads = 32 * (kEpiWarps + 4);
constexpr int kScanThreads = 256;       // of the CTA's, list the groups
constexpr int kAccCols = 256;           // two accumulators of up to 256 columns
constexpr int kTmemCols = 2 * kAccCols;
constexpr int kLine = 128;              // bytes of a stage's K (or M, N) extent: one swizzle row
constexpr int kABytes = 128 * kLine;    // A: 128 rows (K-major) or 2 x 64 columns x 64 rows
constexpr int kTilesAhead = 4;          // tiles that the tile warp lists ahead
constexpr int kMaxStages = 10;
constexpr int kBand = 8;                // row tiles of a band (Tiles::at)
constexpr size_t kSmemLimit = 227 * 1024;
// Bounds of the waits: for what takes a stage's time, and on top of it for what takes a tile's
// whole sum, which may be long (2^30 rows of one group: 2^24 stages, over 3 s of one CTA; a stage
// takes some 0.2 to 0.4 us).
constexpr uint64_t kWaitNs = 2000000000ull, kStageNs = 4000ull;
constexpr uint64_t kDrainNs = 200000000ull;
constexpr uint64_t kSettleNs = 1000000ull;   // lets in-flight copies land after an abort

// Latched code and detail of a wait that gave up, per device.
__device__ int32_t g_status[kStatusWords];

struct MmaParams {
    Product p;
    uint32_t idesc;        // instruction descriptor without its N
    int32_t out_type;
    int32_t bn, bn_log2;   // most rows of a tile (N): 64, 128 or 256
    int32_t box;           // rows of the larger K-major B box
    int32_t stages;
    int32_t split;         // one-CTA tiles: CTAs of a cluster that share a tile's sum (1: none)
    int32_t staged;        // whole batches of outputs leave as boxes (map_o is set); rows are 16-byte aligned
    int32_t stall;         // test hook: the first CTA makes no copies
    uint64_t sum_ns;       // bound of a wait for a tile's sum
    int32_t a_whole, b_whole;   // M- or N-major operands: all of a stage's 64-column boxes as one
};

constexpr int kBoxSmall = 32;           // rows of the smaller K-major B box
constexpr int kOutBytes = 4 * 1024;     // a warp's staged outputs: 64 rows x 32 columns of 16 bits, 32 rows of 32 bits

struct __align__(16) Bars {
    uint64_t full[kMaxStages];    // leader: an arrival for each CTA of the group, and all their bytes
    uint64_t empty[kMaxStages];   // each CTA: the MMAs' commit
    uint64_t tail[kMaxStages];    // dw, each CTA: its own bytes of a stage with rows to zero
    uint64_t acc_full[2];         // each CTA: the MMAs' commit
    uint64_t acc_empty[2];        // leader: the epilogue warps of each CTA
    uint64_t tile_full[kTilesAhead];    // the tile warp's entry
    uint64_t tile_empty[kTilesAhead];   // the warps that have read it
    uint64_t drain;
    uint32_t tmem_slot;
    int abort;
};

struct __align__(16) OutTile {
    int32_t e;       // group, or -1 past the last tile
    int32_t m0;      // first output column
    int32_t row0;    // first output row: of all rows (product, dx), of the group's matrix (dw)
    int32_t nrow;    // output rows of the tile (1..bn)
    int32_t c0, c;   // the summed index: first and count (dw: among all rows), of this CTA's part
    int32_t pad[2];
};

// Shared memory behind the barriers: the tiles listed ahead, the groups' rows and the number
// of row tiles before each. As long as there are groups, for every KB counts: with up to
// about 180 of them (dw: 128) a sixth stage of a pair's tiles fits.
struct Groups {
    OutTile *ahead;                    // [kTilesAhead]
    int32_t *warp_sum, *warp_max;      // [kThreads / 32]
    int32_t *lo;                       // [groups + 1]: first row, and the last group's end
    int32_t *before;                   // [groups + 1]; dw: the groups by falling rows [the next power of two]
    __device__ Groups(void *p, int groups)
        : ahead(static_cast<OutTile *>(p)), warp_sum(reinterpret_cast<int32_t *>(ahead + kTilesAhead)),
          warp_max(warp_sum + kThreads / 32), lo(warp_max + kThreads / 32), before(lo + groups + 1) {}
};
inline size_t groups_bytes(int groups) {
    int all = 1;
    while (all < groups) all *= 2;
    return kTilesAhead * sizeof(OutTile) + 4 * (2 * kThreads / 32 + (groups + 1) + std::max(groups + 1, all));
}

inline size_t stage_bytes(int bn, int cg) { return kABytes + (size_t)bn / cg * kLine; }
inline size_t smem_bytes(int bn, int cg, int stages, int groups) {
    return 1024 + stages * stage_bytes(bn, cg) + kEpiWarps * kOutBytes + sizeof(Bars) + groups_bytes(groups);
}

template <int CG>
__device__ inline void tma_3d(void *dst, const CUtensorMap *map, uint64_t *bar, uint32_t bar_leader, int x, int y, int z) {
    if (CG == 1)
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
                smem_u32(dst)),
            "l"((uint64_t)map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
            "l"((uint64_t)map), "r"(bar_leader), "r"(x), "r"(y), "r"(z)
            : "memory");
}

// The same from a map whose columns are split into [blocks][64]: one copy for all of a
// stage's 64-column boxes.
template <int CG>
__device__ inline void tma_4d(void *dst, const CUtensorMap *map, uint64_t *bar, uint32_t bar_leader, int block, int y, int z) {
    if (CG == 1)
        asm volatile(
            "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(
                smem_u32(dst)),
            "l"((uint64_t)map), "r"(smem_u32(bar)), "r"(0), "r"(y), "r"(block), "r"(z)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
            "l"((uint64_t)map), "r"(bar_leader), "r"(0), "r"(y), "r"(block), "r"(z)
            : "memory");
}

// Bulk tensor store of an output box, a group of its own.
__device__ inline void tma_store_2d(const CUtensorMap *map, const void *src, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];\n cp.async.bulk.commit_group;" ::"l"(map),
                 "r"(smem_u32(src)), "r"(x), "r"(y)
                 : "memory");
}
// What this warp staged before has been read.
__device__ inline void left_stage(int lane) {
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncwarp();
}

// One column: this thread gets its lane's.
__device__ inline void tmem_ld1(uint32_t taddr, uint32_t &r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr));
}

// 16 lanes x 32 columns as fragments: registers 4i..4i+3 hold, of columns 8i + 2 (lane % 4)
// and the one after it, lane row lane / 4 and then row lane / 4 + 8.
__device__ inline void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// Four 8 x 8 matrices of 16 bits, transposed on the way: lane l gives the address of row
// l % 8 (16 bytes) of matrix l / 8.
__device__ inline void stmatrix_trans(void *row, const uint32_t (&w)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(smem_u32(row)), "r"(w[0]), "r"(w[1]),
                 "r"(w[2]), "r"(w[3])
                 : "memory");
}

__device__ inline uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ inline uint32_t pack_f16(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

template <int CG, bool kI8>
__device__ inline void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    if (CG == 1 && !kI8)
        asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
                     " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
                     "l"(a), "l"(b), "r"(idesc), "r"(acc));
    else if (CG == 2 && !kI8)
        tc_mma_f16_pair(d, a, b, idesc, acc);
    else if (CG == 1)
        asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
                     " tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n}" ::"r"(d),
                     "l"(a), "l"(b), "r"(idesc), "r"(acc));
    else
        asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
                     " tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n}" ::"r"(d),
                     "l"(a), "l"(b), "r"(idesc), "r"(acc));
}

// Arrives on `bar` (in every CTA of the group) once the MMAs issued so far are done.
template <int CG>
__device__ inline void commit(uint64_t *bar) {
    if (CG == 1)
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                     : "memory");
    else
        tc_commit_pair_mc(bar, 0x3);
}

template <int CG>
__device__ inline void tmem_alloc(uint32_t *slot) {
    if (CG == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(kTmemCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    } else {
        tmem_alloc_pair(slot, kTmemCols);
        tmem_relinquish_pair();
    }
}
template <int CG>
__device__ inline void tmem_dealloc(uint32_t t) {
    if (CG == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(t), "r"(kTmemCols));
    else
        tmem_dealloc_pair(t, kTmemCols);
}

// Arrival on a barrier of the leader CTA. The default release is this CTA's: what the
// arrival announces (accumulator columns read, rows of this CTA's own shared memory zeroed
// and fenced for the async proxy) has been done where it counts when the arrival leaves. A
// cluster-scope release cost about 1400 cycles each time (dw of 64 experts 141 us instead
// of 125).
template <int CG>
__device__ inline void arrive_leader(uint64_t *bar, int rank) {
    if (CG == 1 || rank == 0)
        mbar_arrive(bar);
    else
        mbar_arrive_cluster(mapa_shared(bar, 0));
}

// Shared-memory descriptor of an M-major (N-major) operand in the 128-byte swizzle: 64
// columns to a 128-byte row, 8 rows of c to a 1024-byte group (stride byte offset), the
// next 64 columns after the 64 rows of this box (leading byte offset).
__device__ inline uint64_t desc_mn(uint32_t saddr) {
    return (uint64_t)((saddr >> 4) & 0x3FFF) | (uint64_t)(64 * kLine >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// Has the phase with this parity completed? Does not wait.
template <bool kCluster>
__device__ inline bool mbar_test(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    if (kCluster)
        asm volatile("{\n .reg .pred p;\n mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
                     : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
    else
        asm volatile("{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
                     : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
    return ok != 0;
}

__device__ inline bool elect_one() {
    uint32_t r;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(r));
    return r != 0;
}
// A value that every lane has, as the compiler can see it.
__device__ inline int uni(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// A bounded wait by a whole warp, with one answer for all its lanes.
template <bool kCluster>
__device__ inline bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort, int where, uint64_t limit_ns = kWaitNs) {
    if (__all_sync(0xffffffffu, mbar_try_wait<kCluster>(bar, parity))) return true;
    return __all_sync(0xffffffffu, mbar_wait<kCluster>(bar, parity, abort, g_status, where, limit_ns));
}

template <int MODE, int CG>
struct Tiles {
    const MmaParams &q;
    const Groups &g;
    int mt, rt, nt, total;   // column tiles, row tiles (dw: of all groups, and of each), all tiles
    __device__ Tiles(const MmaParams &q_, const Groups &g_) : q(q_), g(g_) {
        mt = ((MODE == kFwd ? q.p.n : q.p.k) + 128 * CG - 1) / (128 * CG);
        nt = (q.p.n + q.bn - 1) >> q.bn_log2;
        rt = MODE == kDw ? q.p.groups * nt : g.before[q.p.groups];
        total = mt * rt;
    }
    // Tile i, by a whole warp. Tiles run down kBand row tiles before they step to the next
    // columns, so that those in flight at a time share both operands in L2: with whole
    // rows of tiles instead, 8192 x 8192 x 4096 read its operands seven times from memory.
    __device__ OutTile at(int i) const {
        OutTile t;
        const int lane = threadIdx.x & 31;
        const int band = i / (kBand * mt), j = i - band * kBand * mt, high = rt - band * kBand;
        const int m = high >= kBand ? j / kBand : j / high;
        const int r = band * kBand + j - m * min(kBand, high);
        t.m0 = m * 128 * CG;
        if (MODE == kDw) {
            const int at = r / nt;
            t.e = g.before[at] & 1023;
            t.row0 = (r - at * nt) * q.bn;
            t.nrow = min(q.bn, q.p.n - t.row0);
            t.c0 = g.lo[t.e];
            t.c = g.lo[t.e + 1] - t.c0;
        } else {
            // the last group with before[e] <= r: first among every 32nd, then among 32
            const int E = q.p.groups;
            const int hi = __popc(__ballot_sync(0xffffffffu, 32 * lane < E && g.before[32 * lane] <= r)) - 1;
            const int c = 32 * hi + lane;
            t.e = 32 * hi + __popc(__ballot_sync(0xffffffffu, c < E && g.before[min(c, E)] <= r)) - 1;
            // the group's rows in equal tiles, whole multiples of 16 per CTA
            const int n = g.before[t.e + 1] - g.before[t.e], cnt = g.lo[t.e + 1] - g.lo[t.e];
            const int each = ((n == 1 ? cnt : cdiv(cnt, n)) + 16 * CG - 1) / (16 * CG) * (16 * CG), first = (r - g.before[t.e]) * each;
            t.row0 = g.lo[t.e] + first;
            t.nrow = max(0, min(each, cnt - first));
            t.c0 = 0;
            t.c = MODE == kFwd ? q.p.k : q.p.n;
        }
        return t;
    }
};

template <int MODE, bool kI8, int CG, bool kF32, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
    product_mma_kernel(const __grid_constant__ MmaParams q, const __grid_constant__ CUtensorMap map_a,
                       const __grid_constant__ CUtensorMap map_b, const __grid_constant__ CUtensorMap map_b_small,
                       const __grid_constant__ CUtensorMap map_o) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t b_bytes = (uint32_t)q.bn / CG * kLine, stage_size = kABytes + b_bytes;
    uint8_t *out_stage = smem + q.stages * stage_size;
    Bars *bars = reinterpret_cast<Bars *>(out_stage + kEpiWarps * kOutBytes);
    const Groups groups(bars + 1, q.p.groups);
    volatile int *abort = &bars->abort;

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int rank = CG == 1 ? 0 : (int)cluster_ctarank();
    const int part = kSplit ? (int)cluster_ctarank() : 0;   // of a tile's sum
    const int share = kSplit ? q.split : CG, cid = (int)blockIdx.x / share, ncl = (int)gridDim.x / share;
    const int S = q.stages;
    constexpr int kStep = kI8 ? 128 : 64;   // the summed index's extent of a stage

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; s++) {
            mbar_init(&bars->full[s], CG);
            mbar_init(&bars->empty[s], 1);
            mbar_init(&bars->tail[s], 1);
        }
        for (int b = 0; b < 2; b++) {
            mbar_init(&bars->acc_full[b], 1);
            mbar_init(&bars->acc_empty[b], kEpiWarps * CG);
        }
        // read by the TMA warp, the leader's MMA warp, dw's tail warp and the epilogue
        for (int a = 0; a < kTilesAhead; a++) {
            mbar_init(&bars->tile_full[a], 1);
            mbar_init(&bars->tile_empty[a], 1 + (rank == 0) + (MODE == kDw) + kEpiWarps);
        }
        mbar_init(&bars->drain, 1);
        bars->abort = 0;
        fence_barrier_init();
    }
    if (warp == kTailWarp) tmem_alloc<CG>(&bars->tmem_slot);
    if (warp == kTmaWarp && lane == 0) {
        tma_prefetch_desc(&map_a);
        tma_prefetch_desc(&map_b);
    }
    // Barriers, TMEM and descriptors are ready; offsets may come from the kernel before.
    // Without them the wait for it comes later, when the first tiles are being listed.
    grid_dep_launch();
    if (q.p.offsets) grid_dep_wait();
    if (!q.p.offsets) {   // one group of all rows
        if (threadIdx.x == 0) {
            groups.lo[0] = groups.before[0] = 0;
            groups.lo[1] = q.p.rows;
            groups.before[1] = (q.p.rows + q.bn - 1) >> q.bn_log2;
        }
    } else {
        // The groups' rows and row tiles, four groups a thread: offsets clamped into the
        // rows and to no less than those before them (a running maximum), then summed.
        constexpr int kPer = NVFP4_MOE_MAX_GROUPS / kScanThreads;
        const int E = q.p.groups, e0 = kPer * threadIdx.x;
        int off[kPer + 1], top = 0;
#pragma unroll
        for (int i = 0; i <= kPer; i++) {
            off[i] = e0 + i > E ? 0 : min(max(q.p.offsets[e0 + i], 0), q.p.rows);
            top = max(top, off[i]);
        }
#pragma unroll
        for (int d = 1; d < 32; d *= 2) top = max(top, __shfl_up_sync(0xffffffffu, top, d));   // (itself below d)
        if (lane == 31) groups.warp_max[warp] = top;
        __syncthreads();
        int run = __shfl_up_sync(0xffffffffu, top, 1);
        if (lane == 0) run = 0;
        run = max(run, __reduce_max_sync(0xffffffffu, lane < warp ? groups.warp_max[lane] : 0));
        int tiles[kPer], sum = 0;
#pragma unroll
        for (int i = 0; i < kPer; i++) {
            run = max(run, off[i]);
            const int count = max(off[i + 1] - run, 0);
            if (e0 + i <= E) groups.lo[e0 + i] = run;
            tiles[i] = e0 + i < E ? (count + q.bn - 1) >> q.bn_log2 : 0;
            sum += tiles[i];
        }
        int upto = sum;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int o = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += o;
        }
        if (lane == 31) groups.warp_sum[warp] = upto;
        __syncthreads();
        upto += __reduce_add_sync(0xffffffffu, lane < warp ? groups.warp_sum[lane] : 0) - sum;
#pragma unroll
        for (int i = 0; i < kPer; i++) {
            if (MODE != kDw && e0 + i <= E) groups.before[e0 + i] = upto;
            upto += tiles[i];
        }
        if (MODE == kDw) {
            // The groups by falling rows (a bitonic sort of count | group), so that the tiles,
            // dealt out back and forth, come to about the same work for every CTA: 64 experts
            // of uneven popularity took 139 us in their own order and 109 us evenly filled.
            int all = 1;
            while (all < E) all *= 2;
            uint32_t *key = reinterpret_cast<uint32_t *>(groups.before);
            for (int e = threadIdx.x; e < all; e += kThreads)
                key[e] = e < E ? (uint32_t)min(groups.lo[e + 1] - groups.lo[e], (1 << 21) - 1) << 10 | e : 0u;
            for (int size = 2; size <= all; size *= 2)
                for (int d = size / 2; d > 0; d /= 2) {
                    __syncthreads();
                    for (int x = threadIdx.x; x < all / 2; x += kThreads) {
                        const int i = 2 * x - (x & (d - 1)), j = i + d;
                        const uint32_t u = key[i], v = key[j];
                        if ((u < v) == ((i & size) == 0)) {
                            key[i] = v;
                            key[j] = u;
                        }
                    }
                }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (CG == 2) cluster_sync_all();   // both CTAs' barriers initialised and TMEM allocated
    tc_fence_after();
    const uint32_t tmem_base = bars->tmem_slot;
    // Dense calls wait for the kernel before here, all warps but the tile warp, which lists the
    // first tiles meanwhile: before any wait of a bounded time, whose clock would else run while
    // that kernel does (one with more than two seconds left, or one that gives up itself, would
    // take this call with it).
    if (!q.p.offsets && warp != kTileWarp) grid_dep_wait();
    // The next tile, listed by the tile warp (finding it takes a few integer divisions: about
    // a thousand cycles that no other warp should spend between two tiles). e is -1 past
    // the last one, and after a wait that gave up.
    int slot = 0;
    uint32_t slot_phase = 0;
    auto next_tile = [&]() {
        OutTile t;
        t.e = -1;
        if (warp_wait<false>(&bars->tile_full[slot], slot_phase, abort, 7, q.sum_ns)) {
            t = groups.ahead[slot];
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->tile_empty[slot]);
            if (++slot == kTilesAhead) { slot = 0; slot_phase ^= 1; }
        }
        return t;
    };
    OutTile mine;        // split sums: the epilogue warps' tile and its accumulator
    int mine_buf = -1;
    mine.e = -1;
    int stage = 0;
    uint32_t phase = 0;
    auto next = [&]() {
        if (++stage == S) { stage = 0; phase ^= 1; }
    };

    // The TMA and the MMA warp run their loops converged, with warp-uniform values (uni), and
    // one elected lane issues: the copies and MMAs take their descriptors and coordinates
    // from uniform registers, which a loop inside `if (lane == 0)` has to fill one by one
    // before each of them.
    if (warp == kTmaWarp) {
        // ------------------------------------------------------------ TMA
        uint32_t issued = 0, issued_phase = 0;   // stages loaded, and the parity of their last use
        bool ok = !(q.stall && blockIdx.x == 0);
        const bool elected = elect_one();
        while (ok) {
            const OutTile t = next_tile();
            const int e = uni(t.e), tc = uni(t.c), c0 = uni(t.c0), half = uni(cdiv(t.nrow, 16 * CG) * 16);   // B columns of this CTA
            if (e < 0) break;
            const int brow = uni(t.row0) + rank * half, acol = uni(t.m0) + rank * 128;
            // A copy costs the TMA unit much the same whatever its rows: few and large ones
            // (one box of 128 rows instead of four of 32: 435 -> 373 us for 8192 x 8192 x
            // 4096), small ones where the tile has few rows.
            const bool few = half <= 2 * kBoxSmall;
            const int box = MODE == kDw ? 64 : few ? kBoxSmall : q.box;
            const int nbox = MODE == kDw ? q.b_whole ? q.bn / CG / 64 : cdiv(half, 64) : few ? cdiv(half, kBoxSmall) : half > q.box ? 2 : 1;
            const CUtensorMap *mb = MODE != kDw && few ? &map_b_small : &map_b;
            const uint32_t bytes = kABytes + nbox * box * kLine;
            const int z = MODE == kDw ? 0 : e;
            for (int c = 0; c < tc; c += kStep) {
                if (!warp_wait<CG == 2>(&bars->empty[stage], phase ^ 1, abort, 1)) { ok = false; break; }
                uint8_t *a = smem + stage * stage_size, *b = a + kABytes;
                // A stage whose last rows have to be zeroed is counted by each CTA for
                // itself first; every other one by the leader, for both.
                const bool tail = MODE == kDw && tc - c < kStep && ((tc - c) & 15);
                uint64_t *bar = tail ? &bars->tail[stage] : &bars->full[stage];
                const uint32_t leader = CG == 1 ? 0 : mapa_shared(bar, tail ? rank : 0);
                issued |= 1u << stage;
                issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
                if (elected) {
                    if (tail)
                        mbar_arrive_expect_tx(bar, bytes);
                    else if (rank == 0) {
                        mbar_arrive_expect_tx(bar, CG * bytes);
                        if (CG == 2) mbar_arrive(bar);   // the other CTA's arrival, which would take its time
                    }
                    if (MODE == kFwd)
                        tma_3d<CG>(a, &map_a, bar, leader, c0 + c, acol, z);
                    else if (q.a_whole)
                        tma_4d<CG>(a, &map_a, bar, leader, acol / 64, c0 + c, z);
                    else
                        for (int h = 0; h < 2; h++)
                            tma_3d<CG>(a + h * 64 * kLine, &map_a, bar, leader, acol + 64 * h, c0 + c, z);
                    if (MODE == kDw && q.b_whole)
                        tma_4d<CG>(b, &map_b, bar, leader, brow / 64, c0 + c, 0);
                    else if (MODE == kDw)
                        for (int j = 0; j < nbox; j++) tma_3d<CG>(b + j * 64 * kLine, mb, bar, leader, brow + 64 * j, c0 + c, 0);
                    else {
                        tma_3d<CG>(b, mb, bar, leader, c0 + c, brow, 0);
                        if (nbox > 1) tma_3d<CG>(b + box * kLine, mb, bar, leader, c0 + c, brow + box, 0);
                    }
                }
                __syncwarp();
                next();
            }
        }
        // The last load of every stage has landed before the CTA ends (after a give-up
        // nobody else has waited for them).
        if (rank == 0 && lane == 0)
            for (int s = 0; s < S; s++)
                if (issued & (1u << s)) mbar_wait_drain(&bars->full[s], (issued_phase >> s) & 1, kDrainNs);
        __syncwarp();
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------ MMA (leader)
        if (rank == 0) {
            uint32_t acc_phase = 0, it = 0;
            bool ok = true, ready = false;   // ready: the current stage has already been seen full
            const bool elected = elect_one();
            const uint32_t d0 = uni(tmem_base);
            const uint64_t a0 = MODE == kFwd ? smem_desc_sw128(smem_u32(smem)) : desc_mn(smem_u32(smem));
            const uint64_t b0 = MODE == kDw ? desc_mn(smem_u32(smem + kABytes)) : smem_desc_sw128(smem_u32(smem + kABytes));
            while (ok) {
                const OutTile t = next_tile();
                const int e = uni(t.e), tc = uni(t.c);
                const uint32_t idesc = q.idesc | (uint32_t)(uni(cdiv(t.nrow, 16 * CG)) * 2 * CG) << 17;
                if (e < 0) break;
                if ((MODE == kDw || kSplit) && tc == 0) continue;
                const int buf = it++ & 1;
                const uint32_t d = d0 + buf * kAccCols;
                ok = warp_wait<CG == 2>(&bars->acc_empty[buf], ((acc_phase >> buf) & 1) ^ 1, abort, 2);
                acc_phase ^= 1u << buf;
                tc_fence_after();
                for (int c = 0; ok && c < tc; c += kStep) {
                    if (!ready && !warp_wait<CG == 2>(&bars->full[stage], phase, abort, 3)) { ok = false; break; }
                    tc_fence_after();
                    // the address fields of both descriptors, in units of 16 bytes
                    const uint64_t ad = a0 + (uint32_t)stage * (stage_size >> 4), bd = b0 + (uint32_t)stage * (stage_size >> 4);
                    uint64_t *empty = &bars->empty[stage];
                    // the next stage is looked at while this one's MMAs go out
                    next();
                    // 32 bytes of K a step, or 16 rows of 128 bytes
                    constexpr int kA = MODE == kFwd ? 2 : 16 * kLine >> 4, kB = MODE == kDw ? 16 * kLine >> 4 : 2;
                    const int steps = MODE == kDw ? min(4, cdiv(tc - c, 16)) : 4;
                    if (elected) {
#pragma unroll
                        for (int s = 0; s < 4; s++)
                            if (s < steps) mma<CG, kI8>(d, ad + s * kA, bd + s * kB, idesc, s ? 1u : (uint32_t)c);
                        commit<CG>(empty);
                    }
                    __syncwarp();
                    ready = __all_sync(0xffffffffu, mbar_test<CG == 2>(&bars->full[stage], phase));
                }
                if (ok && elected) commit<CG>(&bars->acc_full[buf]);
                __syncwarp();
            }
            // every MMA that was issued completes before TMEM is freed
            if (elected) {
                if (CG == 1)
                    commit<1>(&bars->drain);
                else
                    tc_commit_pair(&bars->drain);
                mbar_wait_drain(&bars->drain, 0, kDrainNs);
            }
            __syncwarp();
        }
    } else if (warp == kTailWarp) {
        // --------------------------------------- dw: zeroes a group's last rows
        if (MODE == kDw) {
            uint32_t tail_phase = 0;
            while (true) {
                const OutTile t = next_tile();
                if (t.e < 0) break;
                const int half = cdiv(t.nrow, 16 * CG) * 16;
                const int steps = cdiv(t.c, kStep);
                const int left = t.c - (steps - 1) * kStep;   // rows of the last stage
                if (t.c && (left & 15)) {
                    const int last = (stage + steps - 1) % S;
                    const uint32_t parity = (tail_phase >> last) & 1;
                    if (!warp_wait<false>(&bars->tail[last], parity, abort, 4, q.sum_ns)) break;
                    tail_phase ^= 1u << last;
                    uint8_t *a = smem + last * stage_size, *b = a + kABytes;
                    const int pad = 16 - (left & 15), nb = cdiv(half, 64);   // rows to zero, in each 64-column box
                    for (int box = lane >> 3; box < 2 + nb; box += 4) {
                        uint8_t *to = (box < 2 ? a + box * 64 * kLine : b + (box - 2) * 64 * kLine) + left * kLine + (lane & 7) * 16;
#pragma unroll 4
                        for (int r = 0; r < pad; r++) *reinterpret_cast<uint4 *>(to + r * kLine) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) arrive_leader<CG>(&bars->full[last], rank);
                }
                stage = (stage + steps) % S;
            }
        }
    } else if (warp == kTileWarp) {
        // ---------------------------------------------------- lists the tiles
        const Tiles<MODE, CG> tiles(q, groups);
        for (int round = 0; ; round++) {
            OutTile t;
            t.e = -1;
            const int i = round * ncl + (MODE == kDw && (round & 1) ? ncl - 1 - cid : cid);
            if (i < tiles.total) t = tiles.at(i);
            if (kSplit && t.e >= 0) {
                const int steps = cdiv(t.c, kStep), per = cdiv(steps, q.split), from = min(part * per, steps) * kStep;
                t.c0 += from;
                t.c = max(0, min(t.c - from, per * kStep));
            }
            // (the first kTilesAhead slots are free: no wait on the clock)
            if (!q.p.offsets && round == kTilesAhead) grid_dep_wait();
            if (!warp_wait<false>(&bars->tile_empty[slot], slot_phase ^ 1, abort, 8, q.sum_ns)) break;
            if (lane == 0) {
                groups.ahead[slot] = t;
                mbar_arrive(&bars->tile_full[slot]);
            }
            __syncwarp();
            if (++slot == kTilesAhead) { slot = 0; slot_phase ^= 1; }
            if (t.e < 0) break;
        }
    } else if (warp < kEpiWarps) {
        // -------------------------------------------------------- epilogue
        // The eight warps are two halves of four, one warp of each to a quarter of the TMEM
        // lanes (32 output columns); the halves take batches of kBatch output rows in turn.
        // Shared memory is what the MMAs run on (each stage's bytes pass it twice in the time
        // of its MMAs) and a short sum leaves little time between two tiles, so what counts is
        // how few passes and waits a batch takes: each warp stages and stores for itself,
        // without a barrier (with four warps to a buffer and its stores 13615 x 2560 x 128 int8
        // took 21.7 us instead of 18.9, dw of 512 experts of 256 x 256 to FP32 38.6 instead of
        // 32.6; but 805 MB of FP32 185 instead of 201).
        constexpr int kBatch = kF32 ? 32 : 64, kBatches = kAccCols / (2 * kBatch);
        uint32_t acc_phase = 0, it = 0;
        const int cols = MODE == kFwd ? q.p.n : q.p.k;
        const int quarter = warp & 3, half = warp >> 2;
        uint8_t *os = out_stage + warp * kOutBytes;   // [row][32 columns]
        while (true) {
            const OutTile t = next_tile();
            // zeros: an expert without rows, or a part of a short sum
            const bool none = (MODE == kDw || kSplit) && t.e >= 0 && t.c == 0;
            const int col0 = t.m0 + rank * 128 + 32 * quarter, col = col0 + lane;   // of the warp, of this lane
            const int64_t orow = (MODE == kDw ? (int64_t)t.e * q.p.n : 0) + t.row0;
            // Scales of int8 products come in while the sums are still being formed: of the
            // columns and rows that a fragment gives this lane, or of its column and row.
            float cs[4], rs[kBatches][kF32 ? 1 : 16];
            float check[1 + kAccCols / 64];   // every scale of the warp's columns and rows, a lane each
            if (kI8 && !kSplit && t.e >= 0) {
                const float *ws = q.p.w_scale + (int64_t)t.e * q.p.n, *xs = q.p.x_scale + t.row0;
#pragma unroll
                for (int j = 0; j < 4; j++) cs[j] = ws[min(kF32 ? col : col0 + 8 * j + (lane >> 2), cols - 1)];
#pragma unroll
                for (int h = 0; h < kBatches; h++)
#pragma unroll
                    for (int j = 0; j < (kF32 ? 1 : 16); j++)
                        rs[h][j] = xs[min(kBatch * (2 * h + half) + (kF32 ? lane : 8 * (j >> 1) + 2 * (lane & 3) + (j & 1)), t.nrow - 1)];
                check[0] = ws[min(col, cols - 1)];
#pragma unroll
                for (int j = 0; j < kAccCols / 64; j++)
                    check[1 + j] = xs[min(kBatch * (2 * (j * 32 / kBatch) + half) + j * 32 % kBatch + lane, t.nrow - 1)];
            }
            const int buf = it & 1;
            if (t.e < 0 || (!none && !warp_wait<CG == 2>(&bars->acc_full[buf], (acc_phase >> buf) & 1, abort, 5, q.sum_ns))) break;
            if (none && q.p.out_add && !kSplit) continue;
            if (!none) {
                it++;
                acc_phase ^= 1u << buf;
                tc_fence_after();
            }
            if (kSplit) {   // its only tile: joined below
                mine = t;
                mine_buf = none ? -1 : buf;
                break;
            }
            // this warp has read what it needs of the accumulator
            auto release = [&]() {
                if (none) return;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_leader<CG>(&bars->acc_empty[buf], rank);
            };
            const uint32_t tbase = tmem_base + buf * kAccCols + ((uint32_t)(quarter * 32) << 16);
            // int8: are any scales of the warp's part of the tile not of usual size? Then the tile, a rare
            // one, is written here, a row at a time. Asked once a tile, and only when its first sums have
            // been read and the scales have had time to come in (pair by pair in the loops below, 64
            // experts, 20011 rows took 61 us instead of 49).
            auto unusual_scales = [&]() {
                bool usual = true;
#pragma unroll
                for (int j = 0; j < 1 + kAccCols / 64; j++) usual &= usual_scale(check[j]);
                if (__all_sync(0xffffffffu, usual)) return false;
                const float c = q.p.w_scale[(int64_t)t.e * q.p.n + min(col, cols - 1)];
#pragma unroll 1
                for (int r = kBatch * half; r < t.nrow; r += (r + 1) % kBatch ? 1 : kBatch + 1) {
                    uint32_t u;
                    __syncwarp();
                    tmem_ld1(tbase + r, u);
                    tmem_ld_wait();
                    if (col >= cols) continue;
                    const float v = scaled((int32_t)u, q.p.x_scale[t.row0 + r], c);
                    const int64_t at = (orow + r) * q.p.out_ld + col;
                    if constexpr (kF32) {
                        float *o = static_cast<float *>(q.p.out) + at;
                        *o = q.p.out_add ? *o + v : v;
                    } else
                        static_cast<uint16_t *>(q.p.out)[at] =
                            (uint16_t)(q.out_type == NVFP4_MOE_TYPE_BF16 ? pack_bf16(v, 0.0f) : pack_f16(v, 0.0f));
                }
                release();
                return true;
            };
            if (kBatch * half >= t.nrow) release();
#pragma unroll
            for (int h = 0; h < kBatches; h++) {
                const int r = kBatch * (2 * h + half);
                if (r >= t.nrow) break;
                const int n = min(kBatch, t.nrow - r);
                const bool last = r + 2 * kBatch >= t.nrow;
                if constexpr (!kF32) {
                    // Fragments of 16 lanes x 8 columns hold two rows' values of a column to a
                    // thread, which is what a transposing matrix store takes.
                    uint32_t f[2][2][16];
                    __syncwarp();
                    if (!none) {
#pragma unroll
                        for (int s = 0; s < 2; s++)
#pragma unroll
                            for (int b = 0; b < 2; b++) tmem_ld_frag(tbase + ((uint32_t)(16 * b) << 16) + r + 32 * s, f[s][b]);
                        tmem_ld_wait();
                    }
                    if (kI8 && h == 0 && unusual_scales()) break;
                    if (last) release();
                    uint32_t w[8][4];   // [8 rows][8 columns], two rows to a word
#pragma unroll
                    for (int i = 0; i < 8; i++)
#pragma unroll
                        for (int j = 0; j < 4; j++) {
                            const uint32_t *u = &f[i >> 2][j >> 1][4 * (i & 3) + 2 * (j & 1)];
                            float v0 = __uint_as_float(u[0]), v1 = __uint_as_float(u[1]);
                            if (kI8) {
                                v0 = scaled_usual((int32_t)u[0], rs[h][2 * i], cs[j]);
                                v1 = scaled_usual((int32_t)u[1], rs[h][2 * i + 1], cs[j]);
                            }
                            w[i][j] = none ? 0u : q.out_type == NVFP4_MOE_TYPE_BF16 ? pack_bf16(v0, v1) : pack_f16(v0, v1);
                        }
                    left_stage(lane);
                    // 64 bytes a row, in the 64-byte swizzle
                    const int k = lane & 7;
                    uint8_t *to = os + k * 64 + (((lane >> 3) ^ (k >> 1)) << 4);
#pragma unroll
                    for (int i = 0; i < 8; i++) stmatrix_trans(to + i * 8 * 64, w[i]);
                    if (q.staged && n == kBatch) {   // a whole box
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0 && col0 < cols) tma_store_2d(&map_o, os, col0, (int)(orow + r));
                    } else {   // a group's end, or rows that a box cannot have: 16 bytes at a time
                        __syncwarp();
                        for (int i = lane; i < n * 4; i += 32) {
                            const int row = i >> 2, pc = i & 3, c0 = col0 + 8 * pc;
                            const uint4 v = *reinterpret_cast<const uint4 *>(os + row * 64 + ((pc ^ ((row >> 1) & 3)) << 4));
                            uint16_t *o = static_cast<uint16_t *>(q.p.out) + (orow + r + row) * q.p.out_ld + c0;
                            if (q.staged && c0 + 8 <= cols)
                                *reinterpret_cast<uint4 *>(o) = v;
                            else {
                                const uint32_t e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                                for (int c = 0; c < 8; c++)
                                    if (c0 + c < cols) o[c] = (uint16_t)(e[c >> 1] >> (16 * (c & 1)));
                            }
                        }
                    }
                } else {
                    float v[32];
                    uint32_t u[32];
                    __syncwarp();
                    if (!none) {
                        tmem_ld32(tbase + r, u);
                        tmem_ld_wait();
                    }
                    if (kI8 && h == 0 && unusual_scales()) break;
                    if (last) release();
#pragma unroll
                    for (int j = 0; j < 32; j++)
                        v[j] = none ? 0.0f
                               : kI8 ? scaled_usual((int32_t)u[j], __shfl_sync(0xffffffffu, rs[h][0], j), cs[0])
                                     : __uint_as_float(u[j]);
                    if (q.staged && n == kBatch) {
                        left_stage(lane);
                        float *to = reinterpret_cast<float *>(os) + lane;
#pragma unroll
                        for (int j = 0; j < 32; j++) to[32 * j] = v[j];
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0 && col0 < cols) tma_store_2d(&map_o, os, col0, (int)(orow + r));
                    } else if (col < cols) {   // a warp has 128 bytes of a row as it is
                        float *o = static_cast<float *>(q.p.out) + (orow + r) * q.p.out_ld + col;
                        if (q.p.out_add) {
                            float b[32];
#pragma unroll
                            for (int j = 0; j < 32; j++) b[j] = j < n ? o[j * q.p.out_ld] : 0.0f;
#pragma unroll
                            for (int j = 0; j < 32; j++) v[j] += b[j];
                        }
#pragma unroll
                        for (int j = 0; j < 32; j++)
                            if (j < n) o[j * q.p.out_ld] = v[j];
                    }
                }
            }
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }

    if constexpr (kSplit) {
        // Every CTA leaves its sums in its own shared memory (its copies have all been
        // consumed), [row][128 columns] of 32 bits; then each adds up an equal share of the
        // rows, the parts in order, and writes it.
        const int quarter = warp & 3, half = warp >> 2;
        const bool some = warp < kEpiWarps && mine.e >= 0;
        uint32_t *sums = reinterpret_cast<uint32_t *>(smem) + 32 * quarter + lane;
        if (some)
            for (int r = 32 * half; r < mine.nrow; r += 64) {
                uint32_t u[32];
                __syncwarp();
                if (mine_buf >= 0) {
                    tmem_ld32(tmem_base + mine_buf * kAccCols + ((uint32_t)(quarter * 32) << 16) + r, u);
                    tmem_ld_wait();
                } else {
#pragma unroll
                    for (int j = 0; j < 32; j++) u[j] = 0;
                }
#pragma unroll
                for (int j = 0; j < 32; j++) sums[(r + j) * 128] = u[j];
            }
        __syncwarp();
        cluster_sync_all();
        const int cols = MODE == kFwd ? q.p.n : q.p.k, col = mine.m0 + 32 * quarter + lane;
        if (some && col < cols) {
            const int rows = cdiv(mine.nrow, q.split), end = min(mine.nrow, (part + 1) * rows);
            const float cs = kI8 ? q.p.w_scale[(int64_t)mine.e * q.p.n + col] : 1.0f;
            for (int r = part * rows + half; r < end; r += 8) {
                uint32_t w[4][8];   // four rows (every second one), all parts
#pragma unroll
                for (int o = 0; o < 8; o++) {
                    if (o >= q.split) break;
                    const uint32_t from = mapa_shared(sums + r * 128, o);
#pragma unroll
                    for (int j = 0; j < 4; j++)
                        if (r + 2 * j < end)
                            asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(w[j][o]) : "r"(from + j * 1024) : "memory");
                }
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const int row = r + 2 * j;
                    if (row >= end) break;
                    uint32_t u = w[j][0];
#pragma unroll
                    for (int o = 1; o < 8; o++)
                        if (o < q.split) u = kI8 ? u + w[j][o] : __float_as_uint(__uint_as_float(u) + __uint_as_float(w[j][o]));
                    float v = __uint_as_float(u);
                    if (kI8) v = scaled((int32_t)u, q.p.x_scale[mine.row0 + row], cs);
                    const int64_t at = ((MODE == kDw ? (int64_t)mine.e * q.p.n : 0) + mine.row0 + row) * q.p.out_ld + col;
                    if constexpr (kF32) {
                        float *out = static_cast<float *>(q.p.out) + at;
                        *out = q.p.out_add ? *out + v : v;
                    } else if (q.out_type == NVFP4_MOE_TYPE_BF16)
                        static_cast<__nv_bfloat16 *>(q.p.out)[at] = __float2bfloat16_rn(v);
                    else
                        static_cast<__half *>(q.p.out)[at] = __float2half_rn(v);
                }
            }
        }
        __syncwarp();
        cluster_sync_all();   // the sums have been read
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && *abort) {
        // after a give-up, copies that were started may still be landing
        const uint64_t t0 = globaltimer();
        while (globaltimer() - t0 < kSettleNs) __nanosleep(1000);
    }
    __syncthreads();
    if (CG == 2) cluster_sync_all();   // no MMA, copy or arrival of the pair touches either CTA past here
    if (warp == kTailWarp) {
        tc_fence_after();
        tmem_dealloc<CG>(tmem_base);
    }
}

// ------------------------------------------------------------------- host

struct Operand {
    const void *base;
    int64_t cols, rows, matrices, ld;   // [matrices][rows][cols], row stride in elements
};

CUtensorMapDataType map_type(nvfp4_moe_type t) {
    return t == NVFP4_MOE_TYPE_INT8  ? CU_TENSOR_MAP_DATA_TYPE_UINT8
           : t == NVFP4_MOE_TYPE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                     : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
}

// Boxes of 128 bytes x `rows` rows in the 128-byte swizzle, zeros outside. blocks > 0: the
// columns as [blocks of 64][64], that many of them to a box (cols a multiple of 64: past
// the last block there is nothing, within it no column is out of range).
bool map_operand(CUtensorMap *m, const Operand &o, nvfp4_moe_type type, int rows, int blocks) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const int es = type == NVFP4_MOE_TYPE_INT8 ? 1 : 2;
    const cuuint64_t row = (cuuint64_t)(o.ld * es), matrix = (cuuint64_t)(o.ld * es * (o.matrices > 1 ? o.rows : 1));
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    if (blocks) {
        const cuuint64_t dims[4] = {64, (cuuint64_t)o.rows, (cuuint64_t)(o.cols / 64), (cuuint64_t)o.matrices};
        const cuuint64_t strides[3] = {row, kLine, matrix};
        const cuuint32_t box[4] = {64, (cuuint32_t)rows, (cuuint32_t)blocks, 1};
        return fn(m, map_type(type), 4, const_cast<void *>(o.base), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
               CUDA_SUCCESS;
    }
    const cuuint64_t dims[3] = {(cuuint64_t)o.cols, (cuuint64_t)o.rows, (cuuint64_t)o.matrices};
    const cuuint64_t strides[2] = {row, matrix};
    const cuuint32_t box[3] = {(cuuint32_t)(kLine / es), (cuuint32_t)rows, 1};
    return fn(m, map_type(type), 3, const_cast<void *>(o.base), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

// Output rows as a store target: 16 bits in boxes of 32 columns x 64 rows in the 64-byte
// swizzle, 32 bits in plain boxes of 32 columns x 32 rows.
bool map_output(CUtensorMap *m, void *base, nvfp4_moe_type type, int64_t rows, int64_t cols, int64_t ld) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const bool f32 = type == NVFP4_MOE_TYPE_F32;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)(ld * (f32 ? 4 : 2))};
    const cuuint32_t box[2] = {32, f32 ? 32u : 64u}, ones[2] = {1, 1};
    return fn(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : map_type(type), 2, base, dims, strides, box, ones,
              CU_TENSOR_MAP_INTERLEAVE_NONE, f32 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

typedef void (*MmaKernel)(const MmaParams, const CUtensorMap, const CUtensorMap, const CUtensorMap, const CUtensorMap);

template <int CG, bool kF32, bool kSplit>
MmaKernel kernel_of(int mode, bool i8) {
    if (i8) return product_mma_kernel<kFwd, true, CG, kF32, kSplit>;
    return mode == kFwd  ? product_mma_kernel<kFwd, false, CG, kF32, kSplit>
           : mode == kDx ? product_mma_kernel<kDx, false, CG, kF32, kSplit>
                         : product_mma_kernel<kDw, false, CG, kF32, kSplit>;
}
MmaKernel kernel_of(int mode, bool i8, int cg, bool f32, bool split) {
    if (cg == 2) return f32 ? kernel_of<2, true, false>(mode, i8) : kernel_of<2, false, false>(mode, i8);
    if (split) return f32 ? kernel_of<1, true, true>(mode, i8) : kernel_of<1, false, true>(mode, i8);
    return f32 ? kernel_of<1, true, false>(mode, i8) : kernel_of<1, false, false>(mode, i8);
}

// attr: two of them.
cudaLaunchConfig_t config(int grid, int cluster, size_t smem, cudaStream_t s, cudaLaunchAttribute *attr) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    set_programmatic(&attr[0]);
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cfg;
}

// Per device, once: the kernels' shared memory, and how many CTAs and pairs are resident.
struct Resident {
    bool done;
    int ctas, pairs;
    int split[9];   // clusters of 2, 4 and 8 one-CTA tiles
};
std::mutex g_mu;
Resident g_resident[64];

cudaError_t resident(Resident *out) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(g_mu);
    Resident &r = g_resident[dev];
    if (!r.done) {
        for (int i = 0; i < 24; i++) {   // product, dx, dw and int8; one CTA, a pair, a split sum; 16 bits and 32
            const int kind = i % 4, form = i / 4 % 3;
            e = cudaFuncSetAttribute(kernel_of(kind % 3, kind == 3, form == 1 ? 2 : 1, i >= 12, form == 2),
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemLimit);
            if (e != cudaSuccess) return e;
        }
        e = cudaDeviceGetAttribute(&r.ctas, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        cudaLaunchAttribute attr[2];
        const cudaLaunchConfig_t cfg = config(2, 2, kSmemLimit, 0, attr);
        e = cudaOccupancyMaxActiveClusters(&r.pairs, kernel_of(kFwd, false, 2, false, false), &cfg);
        if (e != cudaSuccess) return e;
        if (r.pairs < 1) return cudaErrorInvalidConfiguration;
        for (int n = 2; n <= 8; n *= 2) {
            const cudaLaunchConfig_t c = config(n, n, kSmemLimit, 0, attr);
            e = cudaOccupancyMaxActiveClusters(&r.split[n], kernel_of(kFwd, false, 1, false, true), &c);
            if (e != cudaSuccess) return e;
        }
        r.done = true;
    }
    *out = r;
    return cudaSuccess;
}

int32_t g_stall = 0;   // test hook: launches to come that stall

// The tile shape: CTAs to a tile, its most rows, and CTAs that share its sum.
struct Shape {
    int cg, bn, split;
};

// The most tiles that there can be.
int64_t most_tiles(int mode, const Product &p, int cols, const Shape &s) {
    return (int64_t)cdiv(cols, 128 * s.cg) *
           (mode == kDw ? (int64_t)p.groups * cdiv(p.n, s.bn) : (int64_t)p.rows / s.bn + std::min(p.groups, p.rows));
}

// By an estimate of the time, in cycles of a CTA (or pair), for groups of average size:
// waves of tiles, each as long as the longer of its sum and its epilogue. A stage of a tile
// with N columns takes about max(380, 3.7 N) cycles in one CTA and max(400, 2.75 N) in a pair
// (all SMs busy, operands in L2), 32 columns of an epilogue 420 (16 bits); a tile costs 1200
// besides, a pair 2000 once. Small tiles fill the GPU where there are few rows (201 rows x
// 2048 x 768 int8, before launches overlapped: 6.4 us in tiles of 64, 9.7 in pairs of 256), pairs of 256 move the fewest
// bytes an MMA (4096 x 2560 x 2560 BF16: 44 us, 69 in tiles of 64; 64 experts, 16384 pairs,
// dx: 121 us, 131 in tiles of 64). Few tiles of long sums are split over clusters, whose
// join costs about 4500 cycles (dw of one group, 10000 rows, 200 x 304: 43 us whole, 12 in eight
// parts; 16384 rows, 512 x 512: 65 and 22 in four; 128 rows, 256 x 256: 6.0 and 6.9).
Shape choose(int mode, const Product &p, bool i8, int cols, const Resident &r) {
    static const Shape shapes[] = {{1, 64, 1},  {1, 128, 1}, {2, 128, 1}, {2, 256, 1}, {1, 64, 2},
                                   {1, 128, 2}, {1, 64, 4},  {1, 128, 4}, {1, 64, 8},  {1, 128, 8}};
    const int active = std::min(p.groups, p.rows), avg = cdiv(p.rows, active), step = i8 ? 128 : 64;
    Shape best = shapes[0];
    int64_t least = INT64_MAX;
    for (const Shape &s : shapes) {
        if (s.split > 1 && most_tiles(mode, p, cols, s) > r.split[s.split]) continue;   // one tile to a cluster
        const int total = mode == kDw ? p.n : avg, nt = cdiv(total, s.bn), n = cdiv(total, nt);
        const int64_t tiles = (int64_t)cdiv(cols, 128 * s.cg) * nt * active;
        const int stages = cdiv(cdiv(mode == kFwd ? p.k : mode == kDx ? p.n : avg, step), s.split);
        const int64_t sum = (int64_t)stages * (s.cg == 1 ? std::max(380, n * 37 / 10) : std::max(400, n * 11 / 4));
        const int64_t units = s.split > 1 ? r.split[s.split] : s.cg == 1 ? r.ctas : r.pairs;
        const int64_t cost = (tiles + units - 1) / units * (std::max<int64_t>(sum, n * 13) + 1200) + (s.cg == 2 ? 2000 : 0) +
                             (s.split > 1 ? 4500 : 0);
        if (s.split > 1 ? cost < least : cost <= least) {   // of equals the larger: groups are seldom all of a size
            least = cost;
            best = s;
        }
    }
    return best;
}

}  // namespace

cudaError_t launch_product_mma(int mode, const Product &p, nvfp4_moe_type type, nvfp4_moe_type out, cudaStream_t s) {
    if (p.rows == 0) {   // dw: zeros, or nothing added
        const size_t es = out == NVFP4_MOE_TYPE_F32 ? 4 : 2;
        if (p.out_add) return cudaSuccess;
        return cudaMemset2DAsync(p.out, p.out_ld * es, 0, p.k * es, (size_t)p.groups * p.n, s);
    }
    Resident r;
    cudaError_t err = resident(&r);
    if (err != cudaSuccess) return err;
    const bool i8 = type == NVFP4_MOE_TYPE_INT8;
    const int cols = mode == kFwd ? p.n : p.k;
    MmaParams q{};
    q.p = p;
    q.out_type = out;
    const Shape shape = choose(mode, p, i8, cols, r);
    const int cg = shape.cg;
    q.bn = shape.bn;
    q.bn_log2 = q.bn == 64 ? 6 : q.bn == 128 ? 7 : 8;
    q.box = std::min(128, q.bn / cg);
    q.stages = (int)std::min<size_t>(kMaxStages, (kSmemLimit - smem_bytes(q.bn, cg, 0, p.groups)) / stage_bytes(q.bn, cg));
    // D F32 (or S32), A and B F16, BF16 or S8, their majors, M
    q.idesc = i8 ? (2u << 4) | (1u << 7) | (1u << 10) : (1u << 4) | (type == NVFP4_MOE_TYPE_BF16 ? (1u << 7) | (1u << 10) : 0u);
    if (mode != kFwd) q.idesc |= 1u << 15;
    if (mode == kDw) q.idesc |= 1u << 16;
    q.idesc |= (uint32_t)(128 * cg >> 4) << 24;
    const Operand w{p.w, p.k, p.n, p.groups, p.w_ld}, x{p.x, p.k, p.rows, 1, p.x_ld}, dy{p.dy, p.n, p.rows, 1, p.dy_ld};
    const Operand &oa = mode == kDw ? x : w, &ob = mode == kFwd ? x : dy;
    q.a_whole = mode != kFwd && oa.cols % 64 == 0;
    q.b_whole = mode == kDw && ob.cols % 64 == 0 && p.n % (64 * cg) == 0;
    const int64_t out_rows = mode == kDw ? (int64_t)p.groups * p.n : p.rows;
    q.staged = (reinterpret_cast<uintptr_t>(p.out) & 15) == 0 && p.out_ld % (out == NVFP4_MOE_TYPE_F32 ? 4 : 8) == 0 &&
               p.out_ld < (int64_t(1) << 37) && !p.out_add;   // (a tensor map's strides end at 2^40 bytes)
    CUtensorMap a, b, b_small, o;
    bool ok = map_operand(&a, oa, type, mode == kFwd ? 128 : 64, q.a_whole ? 2 : 0);
    b = b_small = o = a;   // where they are not used
    if (ok && (mode == kDw || q.bn / cg > 2 * kBoxSmall))
        ok = map_operand(&b, ob, type, mode == kDw ? 64 : q.box, q.b_whole ? q.bn / cg / 64 : 0);
    if (ok && mode != kDw) ok = map_operand(&b_small, ob, type, kBoxSmall, 0);
    if (ok && q.staged) ok = map_output(&o, p.out, out, out_rows, cols, p.out_ld);
    if (!ok) return cudaErrorInvalidValue;
    q.split = shape.split;
    q.sum_ns = kWaitNs + kStageNs * cdiv(cdiv(mode == kFwd ? p.k : mode == kDx ? p.n : p.rows, i8 ? 128 : 64), q.split);
    if (g_stall > 0) {
        g_stall--;
        q.stall = 1;
    }
    // no more CTAs than there can be tiles
    const int64_t most = std::max<int64_t>(most_tiles(mode, p, cols, shape), 1);
    const int units = (int)std::min<int64_t>(q.split > 1 ? r.split[q.split] : cg == 2 ? r.pairs : r.ctas, most);
    cudaLaunchAttribute attr[2];
    const int cluster = cg * q.split;
    const cudaLaunchConfig_t cfg = config(units * cluster, cluster, smem_bytes(q.bn, cg, q.stages, p.groups), s, attr);
    return cudaLaunchKernelEx(&cfg, kernel_of(mode, i8, cg, out == NVFP4_MOE_TYPE_F32, q.split > 1), q, a, b, b_small, o);
}

void test_product_stall(int n) { g_stall = std::max(n, 0); }

int product_status(cudaStream_t s) {
    int32_t st[kStatusWords];
    if (cudaStreamSynchronize(s) != cudaSuccess || cudaMemcpyFromSymbol(st, g_status, sizeof(st)) != cudaSuccess)
        return NVFP4_MOE_ERR_CUDA;
    if (st[kStatusCode] != 0) {
        memset(st + 1, 0, sizeof(st) - sizeof(st[0]));
        const int32_t code = st[kStatusCode];
        st[kStatusCode] = 0;
        if (cudaMemcpyToSymbol(g_status, st, sizeof(st)) != cudaSuccess) return NVFP4_MOE_ERR_CUDA;
        return code;
    }
    return NVFP4_MOE_OK;
}

}  // namespace nvmoe
