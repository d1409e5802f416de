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
// per x row tile (its used rows' codes, its scales).  The scale atoms go on to
// tensor memory with tcgen05.cp, replicated to the four lane quarters: row r
// of an atom lands in lane r % 32, column r / 32, four scale bytes a column.
//
// Warp roles of a persistent CTA (one per SM):
//   warp 0     one thread issues the copies, kStages steps ahead
//   warp 1     one thread issues scale copies, MMAs and commits
//   warps 2-5  epilogue: tensor memory -> registers -> y; warp w reads the
//              lanes of quarter w % 4
// The accumulator region holds 256 columns as two slots of 128: a tile of at
// most 128 rows takes one slot, so that its epilogue overlaps the next tile's
// MMAs; a larger one takes both.
// Every wait is bounded; one that runs out sets a status word in mapped host
// memory, and the CTA drains its MMAs and copies and frees its tensor memory.
#include <mutex>

#include "gemm_common.cuh"
#include "mx.h"

namespace moe {
namespace {

using namespace umma;
using namespace gemmc;

constexpr int kThreads = 192;
constexpr int kEpiWarp0 = 2, kEpiWarps = 4;
constexpr int kTmemCols = 512;
constexpr int kScaleBufs = 4;    // steps whose scales are in tensor memory at a time
constexpr int kScaleCol = 256;   // first scale column, behind the accumulators
constexpr unsigned long long kTimeoutNs = 1000000000ull;

struct ProductArgs {
    const uint8_t* x;
    const uint8_t* w;
    const int32_t* offsets;  // NULL: one group of x_rows rows
    const float* alpha;
    void* y;
    int64_t y_ld, x_rows, w_rows;
    int groups, steps, w_tiles;  // steps: column tiles; w_tiles: row tiles of one group of w
    int y_f32;
    int* status;
};

template <int FMT, int NT>
struct Cfg {
    static constexpr int kAtoms = FMT == MOE_MX_E8M0 ? 2 : 4;  // scale atoms of a 128 x 256 tile
    static constexpr int kScaleBytes = kAtoms * kMxAtomBytes;
    static constexpr int kTile = kMxCodeBytes + kScaleBytes;
    static constexpr int kXTiles = (NT + 127) / 128;
    // stage: w tile (codes, scales), x codes, x scales, each part 1024-byte aligned
    static constexpr int kOffX = (kTile + 1023) / 1024 * 1024;
    static constexpr int kOffXs = kOffX + NT * 128;
    static constexpr int kStage = (kOffXs + kXTiles * kScaleBytes + 1023) / 1024 * 1024;
    static constexpr int kStages = (222 * 1024 / kStage) < 8 ? (222 * 1024 / kStage) : 8;
    // scale columns of a step: kAtoms x 4 for w, then kAtoms x (4 per 128 rows) for x
    static constexpr int kWCols = kAtoms * 4, kXCols = kAtoms * 4 * kXTiles;
    static constexpr int kStepCols = kWCols + kXCols;
    static_assert(kScaleCol + kScaleBufs * kStepCols <= kTmemCols, "tensor memory");
    static_assert(kStages >= 4, "shared memory");
};

// no-swizzle shared memory descriptor of a scale atom: 32 rows of 16 bytes,
// 8-row groups 128 bytes apart
__device__ __forceinline__ uint64_t atom_desc(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)(128 >> 4) << 32 | (uint64_t)1 << 46;
}
__device__ __forceinline__ void copy_atom(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// instruction descriptor of the block-scaled kinds: e2m1 A and B, fp32 D, both
// K-major; scale type e8m0 or e4m3; `id`: first scale byte used of a column
template <int FMT>
__device__ __forceinline__ uint32_t idesc_mx(int N, uint32_t id) {
    return (id << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((FMT == MOE_MX_E8M0 ? 1u : 0u) << 23) |
           (1u << 27) | (id << 29);
}
template <int FMT>
__device__ __forceinline__ void mma_mx(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                       uint32_t accumulate) {
    if (FMT == MOE_MX_E8M0)
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
            " tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
            " tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(
                d),
            "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
            : "memory");
}

__device__ __forceinline__ void fail(const ProductArgs& a, volatile int* abort) {
    *abort = 1;
    *(volatile int*)a.status = 1;
}

struct Tile {
    int g, n, wt;      // group, rows, w row tile
    int64_t row0;      // first row of x and y
    int64_t xt;        // first x row tile
};

// tile t of the CTA's walk: row tile t / w_tiles, found by bisection in the
// groups' running counts, and w row tile t % w_tiles
template <int NT>
__device__ __forceinline__ Tile find_tile(const ProductArgs& a, const int* cum, int t) {
    Tile ti;
    int q = t / a.w_tiles;
    ti.wt = t - q * a.w_tiles;
    ti.g = 0;
    int64_t o = 0, n = a.x_rows;
    ti.xt = 0;
    if (a.offsets) {
        int lo = 0, hi = a.groups - 1;  // the last g with cum[g] <= q
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (cum[mid] <= q) lo = mid;
            else hi = mid - 1;
        }
        ti.g = lo;
        q -= cum[lo];
        o = __ldg(a.offsets + lo);
        n = __ldg(a.offsets + lo + 1) - o;
        ti.xt = o / kMxTileRows + lo;
    }
    ti.row0 = o + (int64_t)q * NT;
    ti.n = (int)(n - (int64_t)q * NT < NT ? n - (int64_t)q * NT : NT);
    ti.xt += (int64_t)q * ((NT + kMxTileRows - 1) / kMxTileRows);  // NT < 128: q is 0, the product has at most NT rows
    return ti;
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

template <int FMT, int NT>
__global__ void __launch_bounds__(kThreads, 1) product_kernel(const ProductArgs a) {
    using C = Cfg<FMT, NT>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ uint64_t full[C::kStages], empty[C::kStages], acc_full[2], acc_empty[2], drain;
    __shared__ uint32_t tmem_s;
    __shared__ volatile int abort_s, never_s;
    __shared__ int warp_sum[kThreads / 32];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t smem0 = (smem_u32(smem_raw) + 1023u) & ~1023u;
    int* cum = reinterpret_cast<int*>(smem_raw + (smem0 - smem_u32(smem_raw)) + C::kStages * C::kStage);

    if (tid == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            bar_init(&full[s], 1);
            bar_init(&empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            bar_init(&acc_full[s], 1);
            bar_init(&acc_empty[s], kEpiWarps);
        }
        bar_init(&drain, 1);
        abort_s = 0;
        never_s = 0;
        fence_barrier_init();
    }
    if (warp == 1) tmem_alloc(&tmem_s, kTmemCols);
    int row_tiles;
    if (a.offsets) {
        // running counts of the groups' row tiles
        const int per = (a.groups + kThreads - 1) / kThreads;
        const int g0 = tid * per, g1 = min(g0 + per, a.groups);
        int sum = 0;
        for (int g = g0; g < g1; ++g) sum += (a.offsets[g + 1] - a.offsets[g] + NT - 1) / NT;
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
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
        for (int g = g0; g < g1; ++g) {
            cum[g] = at;
            at += (a.offsets[g + 1] - a.offsets[g] + NT - 1) / NT;
        }
    } else {
        row_tiles = (int)((a.x_rows + NT - 1) / NT);
    }
    const int n_tiles = row_tiles * a.w_tiles;
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = tmem_s;

    if (warp == 0) {
        // ---------------------------------------------------------------- copies
        if (lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            for (int t = blockIdx.x; t < n_tiles && ok; t += gridDim.x) {
                const Tile ti = find_tile<NT>(a, cum, t);
                const uint8_t* wp = a.w + ((int64_t)ti.g * a.w_tiles + ti.wt) * a.steps * C::kTile;
                const uint8_t* xp = a.x + ti.xt * a.steps * C::kTile;
                const int n0 = min(ti.n, 128), n1 = ti.n - n0;
                const uint32_t b0 = (uint32_t)((n0 + 7) & ~7) * 128u, b1 = (uint32_t)((n1 + 7) & ~7) * 128u;
                const uint32_t bytes = C::kTile + b0 + b1 + (n1 > 0 ? 2u : 1u) * C::kScaleBytes;
                for (int k = 0; k < a.steps; ++k, ++it) {
                    const uint32_t s = it % C::kStages;
                    if (it >= C::kStages &&
                        !bar_wait(&empty[s], (it / C::kStages - 1) & 1u, kTimeoutNs, &abort_s)) {
                        fail(a, &abort_s);
                        ok = false;
                        break;
                    }
                    const uint32_t st = smem0 + s * C::kStage;
                    bar_arrive_expect_tx(&full[s], bytes);
                    bulk_g2s(st, wp + (int64_t)k * C::kTile, C::kTile, &full[s]);
                    const uint8_t* x0 = xp + (int64_t)k * C::kTile;
                    bulk_g2s(st + C::kOffX, x0, b0, &full[s]);
                    bulk_g2s(st + C::kOffXs, x0 + kMxCodeBytes, C::kScaleBytes, &full[s]);
                    if (NT > 128 && n1 > 0) {
                        const uint8_t* x1 = x0 + (int64_t)a.steps * C::kTile;
                        bulk_g2s(st + C::kOffX + 128 * 128, x1, b1, &full[s]);
                        bulk_g2s(st + C::kOffXs + C::kScaleBytes, x1 + kMxCodeBytes, C::kScaleBytes, &full[s]);
                    }
                }
            }
            // copies still in flight land before the CTA exits
            for (uint32_t i = it > C::kStages ? it - C::kStages : 0; i < it; ++i)
                bar_wait(&full[i % C::kStages], (i / C::kStages) & 1u, kTimeoutNs, &never_s);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------------ MMA
        if (lane == 0) {
            uint32_t it = 0;
            Slots slots;
            bool ok = true;
            for (int t = blockIdx.x; t < n_tiles && ok; t += gridDim.x) {
                const Tile ti = find_tile<NT>(a, cum, t);
                const uint32_t m = slots.mask(ti.n);
                for (int s = 0; s < 2 && ok; ++s)
                    if ((m >> s & 1) && !bar_wait(&acc_empty[s], (slots.use[s] & 1u) ^ 1u, kTimeoutNs, &abort_s)) ok = false;
                if (!ok) {
                    fail(a, &abort_s);
                    break;
                }
                fence_after_sync();
                const uint32_t d = tmem + (m == 2 ? 128u : 0u);
                const int N = (ti.n + 15) & ~15;
                for (int k = 0; k < a.steps; ++k, ++it) {
                    const uint32_t s = it % C::kStages;
                    if (!bar_wait(&full[s], (it / C::kStages) & 1u, kTimeoutNs, &abort_s) ||
                        // the scale buffer was last read by the MMAs of step it - kScaleBufs
                        (it >= kScaleBufs &&
                         !bar_wait(&empty[(it - kScaleBufs) % C::kStages], ((it - kScaleBufs) / C::kStages) & 1u, kTimeoutNs,
                                   &abort_s))) {
                        fail(a, &abort_s);
                        ok = false;
                        break;
                    }
                    fence_after_sync();
                    const uint32_t st = smem0 + s * C::kStage;
                    const uint32_t sc = tmem + kScaleCol + (it % kScaleBufs) * C::kStepCols;
#pragma unroll
                    for (int q = 0; q < C::kAtoms; ++q) {
                        copy_atom(sc + 4 * q, atom_desc(st + kMxCodeBytes + q * kMxAtomBytes));
                        copy_atom(sc + C::kWCols + q * 4 * C::kXTiles, atom_desc(st + C::kOffXs + q * kMxAtomBytes));
                        if (NT > 128 && ti.n > 128)
                            copy_atom(sc + C::kWCols + q * 4 * C::kXTiles + 4,
                                      atom_desc(st + C::kOffXs + C::kScaleBytes + q * kMxAtomBytes));
                    }
                    const uint64_t wd = sdesc(st), xd = sdesc(st + C::kOffX);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        // a column holds the scales of 64 (e4m3) or 128 (e8m0) matrix columns
                        const int atom = FMT == MOE_MX_E8M0 ? q >> 1 : q;
                        const uint32_t id = FMT == MOE_MX_E8M0 ? (q & 1) * 2 : 0;
                        mma_mx<FMT>(d, wd + 2 * q, xd + 2 * q, idesc_mx<FMT>(N, id), sc + 4 * atom,
                                    sc + C::kWCols + atom * 4 * C::kXTiles, (k | q) ? 1u : 0u);
                    }
                    mma_commit(&empty[s]);
                }
                if (!ok) break;
                for (int s = 0; s < 2; ++s)
                    if (m >> s & 1) mma_commit(&acc_full[s]);
                slots.advance(m);
            }
            // everything issued above has completed once this commit arrives
            mma_commit(&drain);
            if (!bar_wait(&drain, 0, kTimeoutNs, &never_s)) fail(a, &abort_s);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------- epilogue
        const int q = warp & 3;
        const uint32_t trow = tmem + ((uint32_t)(32 * q) << 16);
        Slots slots;
        for (int t = blockIdx.x; t < n_tiles; t += gridDim.x) {
            const Tile ti = find_tile<NT>(a, cum, t);
            const uint32_t m = slots.mask(ti.n);
            int ok = 1;
            if (lane == 0)
                for (int s = 0; s < 2; ++s)
                    if ((m >> s & 1) && !bar_wait(&acc_full[s], slots.use[s] & 1u, kTimeoutNs, &abort_s)) ok = 0;
            if (!__shfl_sync(0xffffffffu, ok, 0)) {
                fail(a, &abort_s);
                break;
            }
            fence_after_sync();
            const float alpha = a.alpha ? __ldg(a.alpha + ti.g) : 1.0f;
            const int64_t col = (int64_t)ti.wt * 128 + 32 * q + lane;
            const uint32_t src = trow + (m == 2 ? 128u : 0u);
            for (int c0 = 0; c0 < ti.n; c0 += 16) {
                uint32_t v[16];
                tmem_ld16(src + c0, v);
                tmem_ld_wait();
                if (col < a.w_rows) {
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (c0 + j < ti.n) {
                            const float f = __uint_as_float(v[j]) * alpha;
                            const int64_t at = (ti.row0 + c0 + j) * a.y_ld + col;
                            if (a.y_f32) static_cast<float*>(a.y)[at] = f;
                            else static_cast<__nv_bfloat16*>(a.y)[at] = __float2bfloat16_rn(f);
                        }
                }
                __syncwarp();
            }
            fence_before_sync();
            __syncwarp();
            if (lane == 0)
                for (int s = 0; s < 2; ++s)
                    if (m >> s & 1) bar_arrive(&acc_empty[s]);
            slots.advance(m);
        }
    }

    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    if (warp == 1) tmem_dealloc(tmem, kTmemCols);
}

// The kernel's status word of each device, pinned and mapped, set up once.
struct DeviceState {
    int* host = nullptr;
    int* dev = nullptr;
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
        int* p = nullptr;
        int sms = 0;
        if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, id)) != cudaSuccess) return e;
        if ((e = cudaHostAlloc(reinterpret_cast<void**>(&p), sizeof(int), cudaHostAllocMapped)) != cudaSuccess) return e;
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

template <int FMT, int NT>
cudaError_t launch_typed(ProductArgs& a, int sms, cudaStream_t st) {
    using C = Cfg<FMT, NT>;
    const int smem = C::kStages * C::kStage + 1024 + (a.offsets ? a.groups * 4 : 0);
    cudaError_t e = smem_limit(reinterpret_cast<const void*>(product_kernel<FMT, NT>), smem);
    if (e != cudaSuccess) return e;
    const int64_t row_tiles = a.offsets ? a.x_rows / NT + (a.groups < a.x_rows ? a.groups : a.x_rows)
                                        : (a.x_rows + NT - 1) / NT;
    const int64_t tiles = row_tiles * a.w_tiles;
    if (tiles > INT32_MAX) return cudaErrorInvalidValue;
    product_kernel<FMT, NT><<<(unsigned)(tiles < sms ? tiles : sms), kThreads, smem, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_mx_product(const moe_mx& x, const moe_mx& w, const int32_t* offsets, const float* alpha, void* y,
                              int y_type, int64_t y_ld, cudaStream_t st, bool* timed_out) {
    DeviceState ds;
    cudaError_t e = device_state(ds);
    if (e != cudaSuccess) return e;
    volatile int* status = ds.host;
    if (*status) {
        *status = 0;
        *timed_out = true;
        return cudaSuccess;
    }
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
    a.y_f32 = y_type == MOE_F32;
    a.status = ds.dev;
    // few rows: a short row tile leaves shared memory for more steps in flight
    const bool few = x.rows <= 64;
    if (x.format == MOE_MX_E8M0)
        return few ? launch_typed<MOE_MX_E8M0, 64>(a, ds.sms, st) : launch_typed<MOE_MX_E8M0, 256>(a, ds.sms, st);
    return few ? launch_typed<MOE_MX_E4M3, 64>(a, ds.sms, st) : launch_typed<MOE_MX_E4M3, 256>(a, ds.sms, st);
}

}  // namespace moe
