// mx_product.cu -- y = alpha * X W^T of two microscaled 4-bit matrices, dense
// or grouped by expert, on the block-scaled tensor cores (tcgen05, fp32
// accumulators in tensor memory).
//
// Work unit ("tile"): up to NT rows of x of one group ("rows") against 128
// rows of the group's w ("features"), in steps of one 256-column tile of both.
// The MMA computes D[128 features x rows] = W[128 x 64] X[rows x 64]^T four
// times a step: with the features on M, a tile with few rows costs a small N
// rather than an idle M.
//
// Both operands are stored as the tensor core wants them in shared memory, so
// a step is plain bulk copies: one for a whole w tile (codes and scales), two
// per x row tile (its used rows' codes, its scales).  The MMA reads the scales
// from tensor memory: row r of a 128 x 4 scale atom in lane r % 32, column
// r / 32, the same in all four lane quarters.  Four warps put them there, an
// atom being one 16-byte shared load and four columns per lane; tcgen05.cp can
// do it too, but at about 50 cycles an atom in the MMA's own queue: 12 atoms
// against 512 cycles of MMA in the largest step.
//
// Warp roles of a persistent CTA (one per SM):
//   warps 0, 14, 15  one thread each issues the copies of w, of x's codes and of
//               x's scales, kStages steps ahead: a copy costs its thread about
//               80 cycles, so one thread for a step's five would take 440 of
//               the step's 600
//   warp 1      one thread issues MMAs and commits
//   warps 2-5   scales: shared memory -> tensor memory, lane quarter w % 4
//   warps 6-13  epilogue: tensor memory -> registers -> y; lane quarter w % 4,
//               two warps per quarter take the halves of the columns
// Where the tiles are too few for the SMs, a cluster shares one tile: each CTA
// takes a run of its steps, and at the end every CTA adds up a part of the
// results from all of the cluster's shared memories, in CTA order.
// The loops of the issuing warps are chains of dependent instructions, and a
// step with few rows lasts about as long as one of them (400 cycles); so they
// run warp-wide (uniform registers) and keep running counters instead of
// divisions, and the MMA warp learns a tile's rows from the copies' warp.
// The accumulator region holds 256 columns as two slots of 128: a tile of at
// most 128 rows takes one slot, a larger one both.  A slot is free again as
// soon as it has been read into registers.
// Measured (random codes, bf16 y):
//   7937 x 8192 x 8192   160 to 165 us, 6.6 PFLOP/s (147 in a CUDA graph of 21 calls);
//               without copies and stores an earlier build of the pair took 138:
//               a step is about 590 cycles of MMA against 512 at the nominal
//               rate, probably because shared memory moves 68 KB in it; long
//               runs are probably held by the power limit as well
//   40960 rows of 206 experts of mixed sizes x 1024 x 2048 (E4M3)   73 us for
//               374 MB: 634 MB from L2 to the SMs at low reuse (without MMAs and
//               stores 60 in an earlier build that took 78), and a large tile's
//               eight steps are followed by 1000 cycles in which its
//               accumulators are read
//   64 rows of 58 experts x 1024 x 2048 (E8M0)   15 us for 65 MB: 4 us to begin
//               and end, the rest at 6.1 TB/s
// Every wait is bounded; where one runs out, the CTA counts that in mapped host
// memory, drains its MMAs and copies, and frees its tensor memory.
#include <mutex>

#include "gemm_common.cuh"
#include "mx.h"

namespace moe {
namespace {

using namespace umma;
using namespace gemmc;

constexpr unsigned kAll = 0xffffffffu;
constexpr int kEpiWarp0 = 6, kEpiWarps = 8;
constexpr int kXWarp = kEpiWarp0 + kEpiWarps, kCopyWarps = 3;  // warps 0, kXWarp, kXWarp + 1
constexpr int kThreads = 32 * (kXWarp + 2);
constexpr int kPer = (1024 + kThreads - 1) / kThreads;  // groups per thread
constexpr int kTileRing = 16;  // rows of the tiles between the copies and the MMAs: more than kStages
constexpr int kTmemCols = 512;
constexpr int kScaleCol = 256;   // first scale column, behind the accumulators
constexpr unsigned long long kTimeoutNs = 1000000000ull;

struct ProductArgs {
    const uint8_t* x;
    const uint8_t* w;
    const int32_t* offsets;  // NULL: one group of x_rows rows
    const float* alpha;
    void* y;
    int64_t y_ld, x_rows, w_rows;
    int groups, steps, w_tiles, w_units;  // steps: column tiles; w_tiles: row tiles of one group of w; w_units: tiles or pairs
    unsigned long long* timeouts;  // mapped host memory: CTAs that gave up
    unsigned long long limit_ns;   // of a wait
    int fault;                     // tests: the second stage's scales never count as complete
};

// NT, the most rows of a tile: 256 a pair of CTAs (M = 256), 128 and 64 one CTA
template <int FMT, int NT>
struct Cfg {
    static constexpr bool kPair = NT == 256;
    static constexpr int kAtoms = FMT == MOE_MX_E8M0 ? 2 : 4;  // scale atoms of a 128 x 256 tile
    static constexpr int kScaleBytes = kAtoms * kMxAtomBytes;
    static constexpr int kTile = kMxCodeBytes + kScaleBytes;
    static constexpr int kXTiles = (NT + 127) / 128;
    // stage: w tile (codes, scales), x codes (half of the rows in each CTA of a pair), x scales; 1024-byte aligned parts
    static constexpr int kOffX = (kTile + 1023) / 1024 * 1024;
    static constexpr int kOffXs = kOffX + (kPair ? NT / 2 : NT) * 128;
    static constexpr int kStage = (kOffXs + kXTiles * kScaleBytes + 1023) / 1024 * 1024;
    static constexpr int kStages = (220 * 1024 / kStage) < 7 ? (220 * 1024 / kStage) : 7;
    // scale columns of a step: kAtoms x 4 for w, then kAtoms x (4 per 128 rows) for x
    static constexpr int kWCols = kAtoms * 4, kXCols = kAtoms * 4 * kXTiles;
    static constexpr int kStepCols = kWCols + kXCols;
    static_assert(kScaleCol + kStages * kStepCols <= kTmemCols, "tensor memory");
};

// ---------------------------------------------------------------------------
// forms for one CTA and for a pair
// ---------------------------------------------------------------------------
template <bool PAIR>
__device__ __forceinline__ void alloc_columns(uint32_t* dst, uint32_t ncols) {
    if constexpr (PAIR) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(ncols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
        tmem_alloc(dst, ncols);
    }
}
template <bool PAIR>
__device__ __forceinline__ void free_columns(uint32_t taddr, uint32_t ncols) {
    if constexpr (PAIR)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
    else
        tmem_dealloc(taddr, ncols);
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(r));
    return r;
}
// four floats at a shared-memory offset of CTA `rank` of the cluster
__device__ __forceinline__ float4 load_remote(uint32_t saddr, uint32_t rank) {
    float4 v;
    asm volatile(
        "{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %4, %5;\n ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n}"
        : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
        : "r"(saddr), "r"(rank)
        : "memory");
    return v;
}
// the same shared-memory offset in CTA 0 of the pair
__device__ __forceinline__ uint32_t leader_addr(uint32_t saddr) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(saddr));
    return r;
}

// 16 or 8 consecutive columns of the warp's lane quarter
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
template <int N>
__device__ __forceinline__ void store_columns(uint32_t taddr, const uint32_t (&v)[N]) {
    if constexpr (N == 8) {
        tmem_st(taddr, v);
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 16) {
            uint32_t u[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) u[j] = v[i + j];
            tmem_st(taddr + i, u);
        }
    }
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// instruction descriptor of the block-scaled kinds: e2m1 A and B, fp32 D, both
// K-major; scale type e8m0 or e4m3; `id`: first scale byte used of a column
template <int FMT>
__device__ __forceinline__ uint32_t idesc_mx(int M, int N, uint32_t id) {
    return (id << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((FMT == MOE_MX_E8M0 ? 1u : 0u) << 23) |
           ((uint32_t)(M >> 7) << 27) | (id << 29);
}
// The issuing instructions below take effect in the one thread whose `on` is
// set.  They are predicated rather than branched around: the warp stays
// converged, so their operands are uniform registers computed once for all.

// D (+)= A * B^T, the descriptors given as low words and one high word
template <int FMT, bool PAIR>
__device__ __forceinline__ void mma_mx(uint32_t on, uint32_t d, uint32_t alo, uint32_t blo, uint32_t dhi, uint32_t idesc,
                                       uint32_t sa, uint32_t sb, uint32_t accumulate) {
    if constexpr (PAIR && FMT == MOE_MX_E8M0)
        asm volatile(
            "{\n .reg .pred p, q;\n .reg .b64 ad, bd;\n mov.b64 ad, {%1, %3};\n mov.b64 bd, {%2, %3};\n"
            " setp.ne.b32 p, %7, 0;\n setp.ne.b32 q, %8, 0;\n"
            " @q tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], ad, bd, %4, [%5], [%6], p;\n}" ::"r"(d),
            "r"(alo), "r"(blo), "r"(dhi), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate), "r"(on)
            : "memory");
    else if constexpr (PAIR)
        asm volatile(
            "{\n .reg .pred p, q;\n .reg .b64 ad, bd;\n mov.b64 ad, {%1, %3};\n mov.b64 bd, {%2, %3};\n"
            " setp.ne.b32 p, %7, 0;\n setp.ne.b32 q, %8, 0;\n"
            " @q tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], ad, bd, %4, [%5], [%6], p;\n}" ::"r"(d),
            "r"(alo), "r"(blo), "r"(dhi), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate), "r"(on)
            : "memory");
    else if constexpr (FMT == MOE_MX_E8M0)
        asm volatile(
            "{\n .reg .pred p, q;\n .reg .b64 ad, bd;\n mov.b64 ad, {%1, %3};\n mov.b64 bd, {%2, %3};\n"
            " setp.ne.b32 p, %7, 0;\n setp.ne.b32 q, %8, 0;\n"
            " @q tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], ad, bd, %4, [%5], [%6], p;\n}" ::"r"(d),
            "r"(alo), "r"(blo), "r"(dhi), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate), "r"(on)
            : "memory");
    else
        asm volatile(
            "{\n .reg .pred p, q;\n .reg .b64 ad, bd;\n mov.b64 ad, {%1, %3};\n mov.b64 bd, {%2, %3};\n"
            " setp.ne.b32 p, %7, 0;\n setp.ne.b32 q, %8, 0;\n"
            " @q tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], ad, bd, %4, [%5], [%6], p;\n}" ::"r"(d),
            "r"(alo), "r"(blo), "r"(dhi), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate), "r"(on)
            : "memory");
}
// arrive, in both CTAs of a pair, once every MMA issued so far by this thread has completed
template <bool PAIR>
__device__ __forceinline__ void commit_if(uint32_t on, uint32_t bar) {
    if constexpr (PAIR)
        asm volatile(
            "{\n .reg .pred q;\n .reg .b16 both;\n setp.ne.b32 q, %1, 0;\n mov.b16 both, 3;\n"
            " @q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], both;\n}" ::"r"(
                bar),
            "r"(on)
            : "memory");
    else
        asm volatile(
            "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
            " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(bar),
            "r"(on)
            : "memory");
}
__device__ __forceinline__ void expect_if(uint32_t on, uint32_t bar, uint32_t bytes) {
    asm volatile(
        "{\n .reg .pred q;\n .reg .b64 st;\n setp.ne.b32 q, %2, 0;\n"
        " @q mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 st, [%0], %1;\n}" ::"r"(bar),
        "r"(bytes), "r"(on)
        : "memory");
}
__device__ __forceinline__ void copy_if(uint32_t on, uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile(
        "{\n .reg .pred q;\n setp.ne.b32 q, %4, 0;\n"
        " @q cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n}" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar), "r"(on)
        : "memory");
}

// by a whole warp; counted once a CTA
__device__ __forceinline__ void fail(const ProductArgs& a, volatile int* abort) {
    if ((threadIdx.x & 31) == 0 && atomicExch(const_cast<int*>(abort), 1) == 0) atomicAdd_system(a.timeouts, 1ull);
    __syncwarp();
}
// arrival on a barrier of another CTA of the cluster, released at CTA scope
__device__ __forceinline__ void remote_arrive(uint32_t addr) {
    asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
// bounded wait of a whole warp, the same answer in every lane
__device__ __forceinline__ bool warp_wait(uint64_t* b, uint32_t parity, volatile int* abort, unsigned long long limit_ns) {
    if (__all_sync(kAll, bar_try_wait(b, parity))) return true;
    return __all_sync(kAll, bar_wait(b, parity, limit_ns, abort));
}
struct Tile {
    int g, n, wt;  // group, rows, w row tile (a pair: the first of two)
    int64_t row0;  // first row of x and y
    int64_t xt;    // first x row tile
};

// tile t, by a whole warp: row tile t / w_units, found in the groups' running
// counts (the last g with cum[g] <= it) by two ballots, and w row tile (or pair
// of them) t % w_units
template <int NT>
__device__ __forceinline__ Tile find_tile(const ProductArgs& a, const int* cum, const int* offs, int t, int lane) {
    Tile ti;
    int q = t / a.w_units;
    ti.wt = (t - q * a.w_units) * (NT == 256 ? 2 : 1);
    ti.g = 0;
    int64_t o = 0, n = a.x_rows;
    ti.xt = 0;
    if (a.offsets) {
        const int blk = 32 * (__popc(__ballot_sync(kAll, lane * 32 < a.groups && cum[min(lane * 32, a.groups - 1)] <= q)) - 1);
        const int i = blk + lane;
        ti.g = blk + __popc(__ballot_sync(kAll, i < a.groups && cum[min(i, a.groups - 1)] <= q)) - 1;
        q -= cum[ti.g];
        const int o0 = offs[ti.g], o1 = offs[ti.g + 1];
        o = o0;
        n = o1 - o0;
        ti.xt = (o0 >> 7) + ti.g;
    }
    ti.row0 = o + (int64_t)q * NT;
    ti.n = (int)min(n - (int64_t)q * NT, (int64_t)NT);
    ti.xt += (int64_t)q * ((NT + kMxTileRows - 1) / kMxTileRows);  // NT < 128: q is 0, the product has at most NT rows
    return ti;
}

// one thread of a converged warp, the same at every call
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.b32 %0, 1, 0, p;\n}" : "=r"(p));
    return p != 0;
}

// row j of a piece: fp32 bits, or bf16 pairs
__device__ __forceinline__ void put(float* y, const uint32_t (&v)[32], int j) { *y = __uint_as_float(v[j]); }
__device__ __forceinline__ void put(__nv_bfloat16* y, const uint32_t (&v)[16], int j) {
    *reinterpret_cast<uint16_t*>(y) = (uint16_t)(v[j >> 1] >> (16 * (j & 1)));
}

// which accumulator slots a tile uses, and how often each has been used
struct Slots {
    uint32_t use[2] = {0, 0}, next = 0;
    __device__ __forceinline__ uint32_t mask(int n) const { return n > 128 ? 3u : 1u << next; }
    __device__ __forceinline__ void advance(uint32_t m) {
        if (m & 1) ++use[0];
        if (m & 2) ++use[1];
        if (m != 3) next ^= 1;
    }
};

template <int FMT, int NT, typename TY, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1) product_kernel(const ProductArgs a) {
    using C = Cfg<FMT, NT>;
    constexpr bool PAIR = C::kPair;
    static_assert(!(PAIR && SPLIT), "a pair's tile is not split");
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ uint64_t full[C::kStages], empty[C::kStages], scales_full[C::kStages], acc_full[2], acc_empty[2], drain;
    __shared__ uint32_t tmem_s;
    __shared__ volatile int abort_s, never_s;
    __shared__ int warp_sum[kThreads / 32], tile_n[kTileRing];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t smem0 = (smem_u32(smem_raw) + 1023u) & ~1023u;
    int* cum = reinterpret_cast<int*>(smem_raw + (smem0 - smem_u32(smem_raw)) + C::kStages * C::kStage);
    int* offs = cum + a.groups;

    const uint32_t rank = PAIR ? cluster_rank() : 0;  // CTA 0 issues a pair's MMAs

    if (tid == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            bar_init(&full[s], kCopyWarps);
            bar_init(&empty[s], 1);
        }
        // the four scale warps, and in CTA 0 of a pair CTA 1's forwarded
        for (int s = 0; s < C::kStages; ++s) bar_init(&scales_full[s], (PAIR && rank == 0 ? 5 : 4) + (s == 1 && a.fault));
        for (int s = 0; s < 2; ++s) {
            bar_init(&acc_full[s], 1);
            bar_init(&acc_empty[s], PAIR ? 2 * kEpiWarps : kEpiWarps);
        }
        bar_init(&drain, 1);
        abort_s = 0;
        never_s = 0;
        fence_barrier_init();
    }
    if (warp == 1) alloc_columns<PAIR>(&tmem_s, kTmemCols);
    let_next_start();
    after_previous();
    int row_tiles;
    if (a.offsets) {
        // running counts of the groups' row tiles; a thread has at most kPer groups
        const int per = (a.groups + kThreads - 1) / kThreads;
        const int g0 = tid * per;
        int first[kPer + 1], sum = 0;
#pragma unroll
        for (int j = 0; j <= kPer; ++j)
            // clamped, so that offsets which are not ascending or too large cannot lead out of x or y
            if (j <= per) {
                first[j] = min(max(a.offsets[min(g0 + j, a.groups)], 0), (int)a.x_rows);
                if (j) first[j] = max(first[j], first[j - 1]);
            }
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (j < per) sum += (first[j + 1] - first[j] + NT - 1) / NT;
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int v = __shfl_up_sync(kAll, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) warp_sum[warp] = incl;
        __syncthreads();
        int at = incl - sum;
        row_tiles = 0;
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) at += warp_sum[w];
            row_tiles += warp_sum[w];
        }
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (j < per && g0 + j < a.groups) {
                cum[g0 + j] = at;
                offs[g0 + j] = first[j];
                at += (first[j + 1] - first[j] + NT - 1) / NT;
                if (g0 + j == a.groups - 1) offs[a.groups] = first[j + 1];
            }
    } else {
        row_tiles = (int)((a.x_rows + NT - 1) / NT);
    }
    const int n_tiles = row_tiles * a.w_units;
    fence_before_sync();
    if (PAIR) cluster_sync();  // the barriers of both CTAs are ready
    else __syncthreads();
    fence_after_sync();
    const uint32_t tmem = tmem_s;
    const int parts = SPLIT ? (int)cluster_size() : 1, part = SPLIT ? (int)cluster_rank() : 0;
    const int unit = (int)blockIdx.x / (PAIR ? 2 : parts), units = (int)gridDim.x / (PAIR ? 2 : parts);
    int my_tiles = (n_tiles - unit + units - 1) / units;  // <= 0: none
    if (SPLIT) my_tiles = min(my_tiles, 1);               // there are as many clusters as tiles
    // this CTA's steps of a tile
    const int k_first = SPLIT ? (int)((int64_t)a.steps * part / parts) : 0;
    const int k_count = (SPLIT ? (int)((int64_t)a.steps * (part + 1) / parts) : a.steps) - k_first;

    // Arrival at the CTA that issues the MMAs.  CTA 1 announces no memory that another thread reads: accesses to tensor
    // memory, complete (wait::st, wait::ld) before the fence and the arrival, and copies that have landed in its own
    // shared memory, where its half of the tensor core reads them.  So it releases at CTA scope, which costs as much as
    // a relaxed arrival (7937 x 8192 x 8192 147 us in a chain of 21 calls, 4096 tokens of 512 experts 74); at cluster
    // scope it would also wait for this SM's stores of y (402 and 151).
    auto arrive_at_leader = [&](uint64_t* b) {
        if (PAIR && rank == 1) remote_arrive(leader_addr(smem_u32(b)));
        else bar_arrive(b);
    };

    if (warp == 0 || warp >= kXWarp) {
        // ---------------------------------------------------------------- copies
        const uint32_t leader = elect_one(), full0 = smem_u32(full);
        uint32_t s = 0, ph = 1, filled = 0;  // stage, parity of its release, steps begun
        bool ok = true;
        for (int i = 0; i < my_tiles && ok; ++i) {
            const Tile ti = find_tile<NT>(a, cum, offs, unit + i * units, lane);
            // this warp's one or two copies of a step: sizes, first sources, places in the stage
            uint32_t b0, b1 = 0, d0, d1 = 0;
            const uint8_t *p0, *p1 = nullptr;
            if (warp == 0) {
                if (leader) tile_n[i % kTileRing] = ti.n;
                const int wt = min(ti.wt + (int)rank, a.w_tiles - 1);  // an odd last tile: CTA 1 repeats it, and stores nothing
                p0 = a.w + ((int64_t)ti.g * a.w_tiles + wt) * a.steps * C::kTile;
                b0 = C::kTile;
                d0 = 0;
            } else {
                const uint8_t* x0 = a.x + ti.xt * a.steps * C::kTile;
                const uint8_t* x1 = x0 + (int64_t)a.steps * C::kTile;
                if (warp == kXWarp) {
                    // all rows, or this CTA's half of the MMA's N; r0 .. r1 may lie in two row tiles
                    const int n8 = (ti.n + 7) & ~7, half = PAIR ? ((ti.n + 31) & ~31) / 2 : 0;
                    const int r0 = (int)rank * half, r1 = PAIR && rank == 0 ? min(half, n8) : n8;
                    b0 = (uint32_t)max(min(r1, 128) - r0, 0) * 128u;
                    b1 = (uint32_t)max(r1 - max(r0, 128), 0) * 128u;
                    p0 = x0 + r0 * 128;
                    p1 = x1 + max(r0 - 128, 0) * 128;
                    d0 = C::kOffX;
                    d1 = C::kOffX + b0;
                } else {
                    p0 = x0 + kMxCodeBytes;
                    p1 = x1 + kMxCodeBytes;
                    b0 = C::kScaleBytes;
                    b1 = ti.n > 128 ? C::kScaleBytes : 0;
                    d0 = C::kOffXs;
                    d1 = C::kOffXs + C::kScaleBytes;
                }
            }
            if (SPLIT) p0 += (int64_t)k_first * C::kTile;
            for (int k = 0; k < k_count; ++k) {
                if (!warp_wait(&empty[s], ph, &abort_s, a.limit_ns)) {
                    fail(a, &abort_s);
                    ok = false;
                    break;
                }
                const uint32_t st = smem0 + s * C::kStage, bar = full0 + 8 * s;
                expect_if(leader, bar, b0 + b1);
                if (b0) copy_if(leader, st + d0, p0, b0, bar);
                if (PAIR && b1) copy_if(leader, st + d1, p1, b1, bar);
                p0 += C::kTile;
                if (PAIR) p1 += C::kTile;
                ++filled;
                if (++s == C::kStages) s = 0, ph ^= 1;
            }
        }
        // copies still in flight land before the CTA exits; a stage that another copy warp gave up before filling never
        // counts as full, but after that second everything has landed
        for (uint32_t i = filled > C::kStages ? filled - C::kStages : 0; i < filled; ++i)
            if (!bar_wait(&full[i % C::kStages], (i / C::kStages) & 1u, kTimeoutNs, &never_s)) break;
        __syncwarp();
    } else if (warp == 1 && rank == 1) {
        // -------------- CTA 1 of a pair: forwards its scale warps' arrivals, and so spares them the remote access
        uint32_t s = 0, ph = 0;
        const int steps = my_tiles * k_count;
        for (int it = 0; it < steps; ++it) {
            if (!warp_wait(&scales_full[s], ph, &abort_s, a.limit_ns)) {
                fail(a, &abort_s);
                break;
            }
            fence_after_sync();  // what the scales' warps stored is ordered before this warp's arrival as well
            fence_before_sync();
            if (lane == 0) arrive_at_leader(&scales_full[s]);
            __syncwarp();
            if (++s == C::kStages) s = 0, ph ^= 1;
        }
        warp_wait(&drain, 0, &never_s, kTimeoutNs);  // CTA 0's last arrival here
    } else if (warp == 1) {
        // ------------------------------------------------------------------ MMA
        const uint32_t leader = elect_one();
        uint32_t s = 0, ph = 0;
        Slots slots;
        bool ok = true;
        const uint32_t dhi = (uint32_t)(sdesc(smem0) >> 32);  // the same for every operand tile
        const uint32_t w_lo = (uint32_t)sdesc(smem0), empty0 = smem_u32(empty), acc0 = smem_u32(acc_full);
        uint32_t wd = w_lo, sc = tmem + kScaleCol;
        for (int i = 0; i < my_tiles && ok; ++i) {
            uint32_t d = 0, idesc = 0, m = 0;
            for (int k = 0; k < k_count; ++k) {
                // the scales' warps have seen the step's copies land before they arrive here
                ok = warp_wait(&scales_full[s], ph, &abort_s, a.limit_ns);
                if (k == 0 && ok) {
                    const int n = tile_n[i % kTileRing];
                    m = slots.mask(n);
                    if (m & 1) ok = warp_wait(&acc_empty[0], (slots.use[0] & 1u) ^ 1u, &abort_s, a.limit_ns);
                    if ((m & 2) && ok) ok = warp_wait(&acc_empty[1], (slots.use[1] & 1u) ^ 1u, &abort_s, a.limit_ns);
                    d = tmem + (m == 2 ? 128u : 0u);
                    idesc = PAIR ? idesc_mx<FMT>(256, (n + 31) & ~31, 0) : idesc_mx<FMT>(128, (n + 15) & ~15, 0);
                }
                if (!ok) {
                    fail(a, &abort_s);
                    break;
                }
                fence_after_sync();
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    // a column holds the scales of 64 (e4m3) or 128 (e8m0) matrix columns
                    const int atom = FMT == MOE_MX_E8M0 ? q >> 1 : q;
                    const uint32_t id = FMT == MOE_MX_E8M0 ? (q & 1) * 2 : 0;
                    mma_mx<FMT, PAIR>(leader, d, wd + 2 * q, wd + (C::kOffX >> 4) + 2 * q, dhi, idesc | id << 4 | id << 29,
                                sc + 4 * atom, sc + C::kWCols + atom * 4 * C::kXTiles, q ? 1u : (uint32_t)k);
                }
                commit_if<PAIR>(leader, empty0 + 8 * s);
                wd += C::kStage >> 4;
                sc += C::kStepCols;
                if (++s == C::kStages) s = 0, ph ^= 1, wd = w_lo, sc = tmem + kScaleCol;
            }
            if (!ok) break;
            if (m & 1) commit_if<PAIR>(leader, acc0);
            if (m & 2) commit_if<PAIR>(leader, acc0 + 8);
            slots.advance(m);
        }
        // everything issued above has completed once this commit arrives
        commit_if<PAIR>(leader, smem_u32(&drain));
        if (!warp_wait(&drain, 0, &never_s, kTimeoutNs)) fail(a, &abort_s);
    } else if (warp >= 2 && warp < kEpiWarp0) {
        // --------------------------------------------------------------- scales
        const uint32_t quarter = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        uint32_t s = 0, ph = 0;
        const int steps = my_tiles * k_count;
        for (int it = 0; it < steps; ++it) {
            if (!warp_wait(&full[s], ph, &abort_s, a.limit_ns)) {
                fail(a, &abort_s);
                break;
            }
            uint32_t wv[C::kWCols], xv[C::kXCols];
            const uint32_t st = smem0 + s * C::kStage + lane * 16;
#pragma unroll
            for (int q = 0; q < C::kAtoms; ++q) {
                const uint4 v = lds128(st + kMxCodeBytes + q * kMxAtomBytes);
                wv[4 * q] = v.x, wv[4 * q + 1] = v.y, wv[4 * q + 2] = v.z, wv[4 * q + 3] = v.w;
#pragma unroll
                for (int h = 0; h < C::kXTiles; ++h) {
                    const uint4 u = lds128(st + C::kOffXs + h * C::kScaleBytes + q * kMxAtomBytes);
                    const int c = 4 * (q * C::kXTiles + h);
                    xv[c] = u.x, xv[c + 1] = u.y, xv[c + 2] = u.z, xv[c + 3] = u.w;
                }
            }
            // the MMAs that read this stage's columns last are done: the copies into the stage waited for them
            fence_after_sync();
            const uint32_t sc = quarter + kScaleCol + s * C::kStepCols;
            store_columns(sc, wv);
            store_columns(sc + C::kWCols, xv);
            tmem_st_wait();
            fence_before_sync();
            __syncwarp();
            if (lane == 0) bar_arrive(&scales_full[s]);
            if (++s == C::kStages) s = 0, ph ^= 1;
        }
    } else {
        // ------------------------------------------------------------- epilogue
        const int q = warp & 3, half = (warp - kEpiWarp0) >> 2;
        const uint32_t trow = tmem + ((uint32_t)(32 * q) << 16);
        Slots slots;
        for (int i = 0; i < my_tiles; ++i) {
            const Tile ti = find_tile<NT>(a, cum, offs, unit + i * units, lane);
            const float alpha = a.alpha ? a.alpha[ti.g] : 1.0f;
            const uint32_t m = slots.mask(ti.n);
            bool ok = true;
            if (m & 1) ok = warp_wait(&acc_full[0], slots.use[0] & 1u, &abort_s, a.limit_ns);
            if ((m & 2) && ok) ok = warp_wait(&acc_full[1], slots.use[1] & 1u, &abort_s, a.limit_ns);
            if (!ok) {
                fail(a, &abort_s);
                break;
            }
            fence_after_sync();
            // Pieces of 32 columns, kept in the output's type until all of the tile has been read.  A large tile's slots
            // are the halves; in a small one each half has 64 columns of the slot.
            constexpr int kHalf = (NT < 128 ? NT : 128) / 2, kPieces = PAIR ? 4 : kHalf / 32;
            constexpr int kRegs = sizeof(TY) == 2 ? 16 : 32;
            constexpr int kBatch = sizeof(TY) == 2 ? kPieces : (kPieces > 2 ? 2 : kPieces);
            const int first = half * (ti.n > 128 ? 128 : kHalf);
            const int mine = min(ti.n - first, ti.n > 128 ? 128 : kHalf);  // this warp's rows, if any
            const uint32_t src = trow + (m == 2 ? 128u : 0u) + first;
            if constexpr (SPLIT) {
                // the ring is idle: the part's sums to shared memory as [row][128 features]
#pragma unroll
                for (int p = 0; p < kPieces; ++p)
                    if (32 * p < mine) {
                        uint32_t raw[32];
                        tmem_ld32(src + 32 * p, raw);
                        tmem_ld_wait();
                        const uint32_t to = smem0 + ((first + 32 * p) * 128 + 32 * q + lane) * 4;
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            asm volatile("st.shared.b32 [%0], %1;" ::"r"(to + j * 512), "r"(raw[j]) : "memory");
                    }
                continue;
            }
            const int64_t col = (int64_t)(ti.wt + (int)rank) * 128 + 32 * q + lane;
            TY* const y = static_cast<TY*>(a.y) + (ti.row0 + first) * a.y_ld + col;
            const bool in = col < a.w_rows;
#pragma unroll
            for (int p0 = 0; p0 < kPieces; p0 += kBatch) {
                uint32_t v[kBatch][kRegs];
                constexpr int kTwo = PAIR && kBatch > 1 ? 2 : 1;  // pieces read at a time
#pragma unroll
                for (int p = 0; p < kBatch; p += kTwo)
                    if (32 * (p0 + p) < mine) {
                        uint32_t raw[kTwo][32];
#pragma unroll
                        for (int t = 0; t < kTwo; ++t) tmem_ld32(src + 32 * (p0 + p + t), raw[t]);  // within the slots
                        tmem_ld_wait();
#pragma unroll
                        for (int t = 0; t < kTwo; ++t)
#pragma unroll
                            for (int j = 0; j < kRegs; ++j) {
                                if constexpr (sizeof(TY) == 2)
                                    v[p + t][j] = pack_bf16(__uint_as_float(raw[t][2 * j]) * alpha, __uint_as_float(raw[t][2 * j + 1]) * alpha);
                                else
                                    v[p + t][j] = __float_as_uint(__uint_as_float(raw[t][j]) * alpha);
                            }
                    }
                if (p0 + kBatch >= kPieces) {  // all read: the slots may be overwritten
                    fence_before_sync();
                    __syncwarp();
                    if (lane == 0) {
                        if (m & 1) arrive_at_leader(&acc_empty[0]);
                        if (m & 2) arrive_at_leader(&acc_empty[1]);
                    }
                }
                if (in) {
                    // Rows are stored in runs of 32: the longest keeps most stores going (512 groups of 80 rows x 2048 x
                    // 512: 73 us, runs of 8 82).  Where the whole product has at most 64 rows, runs of 8: few rows then
                    // take few instructions (1 row x 1024 x 256: 3.0 us, not 3.2).
                    constexpr int kRun = NT == 64 ? 8 : 32;
#pragma unroll
                    for (int p = 0; p < kBatch; ++p)
#pragma unroll
                        for (int c = 0; c < 32; c += kRun) {
                            const int rows = mine - 32 * (p0 + p) - c;
                            TY* yp = y + (int64_t)(32 * (p0 + p) + c) * a.y_ld;
                            if (rows >= kRun) {
#pragma unroll
                                for (int j = 0; j < kRun; ++j, yp += a.y_ld) put(yp, v[p], c + j);
                            } else if (rows > 0) {
#pragma unroll
                                for (int j = 0; j < kRun; ++j, yp += a.y_ld)
                                    if (j < rows) put(yp, v[p], c + j);
                            }
                        }
                }
                __syncwarp();
            }
            slots.advance(m);
        }
    }

    if constexpr (SPLIT) {
        // four features of a row a thread, a run of them for each CTA
        __syncwarp();
        cluster_sync();
        if (my_tiles > 0) {
            const Tile ti = find_tile<NT>(a, cum, offs, unit, lane);
            const float alpha = a.alpha ? a.alpha[ti.g] : 1.0f;
            const int end = ti.n * 32 * (part + 1) / parts;
            for (int i = ti.n * 32 * part / parts + tid; i < end; i += kThreads) {
                float4 sum = load_remote(smem0 + i * 16, 0);
                for (int r = 1; r < parts; ++r) {
                    const float4 v = load_remote(smem0 + i * 16, (uint32_t)r);
                    sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
                }
                const float v[4] = {sum.x * alpha, sum.y * alpha, sum.z * alpha, sum.w * alpha};
                const int64_t col = (int64_t)ti.wt * 128 + (i & 31) * 4;
                TY* const y = static_cast<TY*>(a.y) + (ti.row0 + (i >> 5)) * a.y_ld + col;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (col + j < a.w_rows) y[j] = (TY)v[j];
            }
        }
    }
    fence_before_sync();
    if (PAIR || SPLIT) cluster_sync();  // nothing of the other CTAs' is under way here any more, nor read
    else __syncthreads();
    fence_after_sync();
    if (warp == 1) free_columns<PAIR>(tmem, kTmemCols);
}

// The kernel's count of each device, pinned and mapped, set up once.
struct DeviceState {
    unsigned long long* host = nullptr;
    unsigned long long* dev = nullptr;
    int sms = 0;
};

cudaError_t device_state(DeviceState& out) {
    static std::mutex mu;
    static DeviceState states[64];
    int id = 0;
    cudaError_t e = cudaGetDevice(&id);
    if (e != cudaSuccess) return e;
    if (id < 0 || id >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    DeviceState& s = states[id];
    if (!s.host) {
        unsigned long long* p = nullptr;
        int sms = 0;
        if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, id)) != cudaSuccess) return e;
        if ((e = cudaHostAlloc(reinterpret_cast<void**>(&p), sizeof *p, cudaHostAllocMapped)) != cudaSuccess) return e;
        *p = 0;
        if ((e = cudaHostGetDevicePointer(reinterpret_cast<void**>(&s.dev), p, 0)) != cudaSuccess) {
            cudaFreeHost(p);
            return e;
        }
        s.sms = sms;
        s.host = p;
    }
    out = s;
    return cudaSuccess;
}

// Row tiles of an upper bound: a group's rows are known to the GPU only.
int64_t most_row_tiles(const ProductArgs& a, int nt) {
    if (!a.offsets) return (a.x_rows + nt - 1) / nt;
    return a.x_rows / nt + (a.groups < a.x_rows ? a.groups : a.x_rows);
}

// parts > 1: clusters of that many CTAs share a tile, one tile each
template <int FMT, int NT, typename TY, bool SPLIT = false>
cudaError_t launch_typed(ProductArgs& a, int sms, cudaStream_t st, unsigned parts = 1) {
    using C = Cfg<FMT, NT>;
    const int smem = C::kStages * C::kStage + 1024 + (a.offsets ? a.groups * 8 + 4 : 0);
    cudaError_t e = smem_limit(reinterpret_cast<const void*>(product_kernel<FMT, NT, TY, SPLIT>), smem);
    if (e != cudaSuccess) return e;
    a.w_units = C::kPair ? (a.w_tiles + 1) / 2 : a.w_tiles;
    const int64_t tiles = most_row_tiles(a, NT) * a.w_units, units = C::kPair ? sms / 2 : sms;
    if (tiles > INT32_MAX || tiles / units * a.steps > INT32_MAX / 2) return cudaErrorInvalidValue;
    const unsigned n = (unsigned)(tiles < units ? tiles : units);
    const unsigned cluster = C::kPair ? 2 : parts;
    return launch(product_kernel<FMT, NT, TY, SPLIT>, n * cluster, kThreads, smem, st, cluster, a);
}

// The variant, by sizes alone (times in us, E4M3, bf16 y; pair | one CTA):
//   - A pair's tile (256 features x 256 rows) feeds the tensor cores best: groups of 512 rows x 1024 x 2048
//     70.8 | 81.4, of 200 76.1 | 83.5.
//   - It needs more than 64 rows a group on average (a mixed batch of 80 rows a group 75.0 | 78.9, of 40 59.1 | 58.9),
//   - at least 4 steps, because its tiles cost more to begin and end (80 rows a group x 2048 x 512 91.9 | 71.0),
//   - and enough tiles for most of the SMs (512 x 4096 x 4096: 32 pairs 11.5 | 8.9; 1024 rows: 64 pairs 12.4 | 13.7).
//   - Long rows and few tiles: a cluster of 2, 4 or 8 CTAs splits a tile's steps.  That costs 1.4 us, so it takes 16
//     steps (1 row x 4096 x 4096 6.5 unsplit, 5.7 with 4) or 24 (128 rows x 1024 x 8192 12.2, 8.6; 1 row 9.9, 5.4 with
//     8; at 8 steps 4.5, 4.9).  Clusters of 8 and 4 do not fill the GPU (15 and 36 fit at a time: the bounds on tiles).
//   - Up to 64 rows in all, a shorter row tile leaves shared memory for one more step in flight: 80 experts of one
//     row 15.6 instead of 16.2.
template <int FMT, typename TY>
cudaError_t launch_rows(ProductArgs& a, int sms, cudaStream_t st) {
    if (a.steps >= (a.x_rows <= 32 ? 16 : 24)) {
        const int64_t tiles = most_row_tiles(a, 128) * a.w_tiles;
        const int parts = tiles * 8 <= sms / 2 ? 8 : tiles * 4 * 10 <= sms * 9 ? 4 : tiles * 2 <= sms ? 2 : 1;
        if (parts > 1) return launch_typed<FMT, 128, TY, true>(a, sms, st, parts);
    }
    if (a.x_rows <= 64) return launch_typed<FMT, 64, TY>(a, sms, st);
    const bool pair = a.steps >= 4 && a.x_rows > 64 * (int64_t)a.groups &&
                      most_row_tiles(a, 256) * ((a.w_tiles + 1) / 2) * 8 >= 3 * sms;
    return pair ? launch_typed<FMT, 256, TY>(a, sms, st) : launch_typed<FMT, 128, TY>(a, sms, st);
}

}  // namespace

cudaError_t mx_timeouts(uint64_t* count) {
    DeviceState ds;
    const cudaError_t e = device_state(ds);
    if (e == cudaSuccess) *count = *static_cast<volatile unsigned long long*>(ds.host);
    return e;
}

cudaError_t launch_mx_product(const moe_mx& x, const moe_mx& w, const int32_t* offsets, const float* alpha, void* y,
                              int y_type, int64_t y_ld, cudaStream_t st, bool fault) {
    DeviceState ds;
    cudaError_t e = device_state(ds);
    if (e != cudaSuccess) return e;
    ProductArgs a{};
    a.x = static_cast<const uint8_t*>(x.data_dev);
    a.w = static_cast<const uint8_t*>(w.data_dev);
    a.offsets = offsets;
    a.alpha = alpha;
    a.y = y;
    a.y_ld = y_ld;
    a.x_rows = x.rows;
    a.w_rows = w.rows;
    a.groups = w.groups;
    a.steps = (int)mx_col_tiles(x.cols);
    a.w_tiles = (int)((w.rows + kMxTileRows - 1) / kMxTileRows);
    a.timeouts = ds.dev;
    a.limit_ns = fault ? 1000000ull : kTimeoutNs;
    a.fault = fault;
    if (x.format == MOE_MX_E8M0)
        return y_type == MOE_F32 ? launch_rows<MOE_MX_E8M0, float>(a, ds.sms, st)
                                 : launch_rows<MOE_MX_E8M0, __nv_bfloat16>(a, ds.sms, st);
    return y_type == MOE_F32 ? launch_rows<MOE_MX_E4M3, float>(a, ds.sms, st)
                             : launch_rows<MOE_MX_E4M3, __nv_bfloat16>(a, ds.sms, st);
}

}  // namespace moe
