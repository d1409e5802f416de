// mx_route.cu -- routing with groups and a balance bias, the stable sort of
// the chosen pairs by expert, and the weighted combine of the experts' rows.
#include <cooperative_groups.h>

#include <cfloat>
#include <utility>

#include "mx.h"

namespace cg = cooperative_groups;

namespace moe {
namespace {

constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

// fp32 as an unsigned whole number of the same order (-inf is the smallest used)
__device__ __forceinline__ uint32_t ordered(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);  // -0 counts as 0
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
    return v;
}

struct RouteArgs {
    const void* logits;
    const float* bias;
    int32_t* idx;
    float* w;
    int64_t ld, T;
    moe_route_config c;
    uint32_t inv_group;  // e / group size = (e * inv_group) >> 20 for e < 1024
};

constexpr int kRouteWarps = 4;

// 1 / (1 + exp(-l)), within a few units of the last place
__device__ __forceinline__ float sigmoid(float l) { return __fdividef(1.0f, 1.0f + expf(-l)); }

// per-warp scratch: a score of every expert (expert e at e + e / 32, so that
// lanes a row apart do not share a bank), and the candidates of the choice
template <int NV>
struct RouteScratch {
    float score[NV * 33];
    int cand[32];
    int order[32];
};

// One warp per token; lane l holds the experts l, l + 32, ...: the row is read
// once, coalesced, and every statistic is a warp reduction on registers.
//
// The choice: no expert below t, the top_k-th largest of the 32 lanes' maxima,
// can be chosen, because top_k lanes hold one at or above t.  What is left
// (top_k to about twice as many) becomes one candidate per lane, and each
// counts the candidates before it.  A row with more than 32 left (equal
// logits) takes top_k rounds of (largest key, then lowest id) instead; rounds
// for every row, each rescanning the winner's NV keys, took 840 cycles a round
// at 512 experts.  With one token the kernel is a chain of dependent steps on
// a cold instruction cache, so the code is kept short; with thousands it is
// bound by the instructions issued.
template <typename T, int NV>
__global__ void __launch_bounds__(32 * kRouteWarps) route_kernel(const RouteArgs a) {
    __shared__ RouteScratch<NV> scratch[kRouteWarps];
    after_previous();
    let_next_start();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp;
    if (t >= a.T) return;
    RouteScratch<NV>& sh = scratch[warp];
    const moe_route_config& c = a.c;
    const int E = c.n_experts;
    const T* row = static_cast<const T*>(a.logits) + t * a.ld;

    float l[NV], ch[NV];  // logits (-inf: out) and what the choice compares
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = i * 32 + lane;
        l[i] = e < E ? to_f32(row[e]) : -INFINITY;
        ch[i] = a.bias && e < E ? a.bias[e] : 0.0f;
    }
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        l[i] = l[i] > -INFINITY && ch[i] > -INFINITY ? fminf(l[i], FLT_MAX) : -INFINITY;
        m = fmaxf(m, l[i]);
    }
    m = warp_max(m);
    const bool softmax = c.score == MOE_SCORE_SOFTMAX;
    const bool sums = c.top_groups < c.n_groups && c.group_best == 2;
    float inv_total = 1.0f;
    if (softmax && (a.bias || !c.renorm)) {
        float total = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) total += l[i] > -INFINITY ? expf(l[i] - m) : 0.0f;
        inv_total = 1.0f / warp_sum(total);
    }
    auto score = [&](float v) { return softmax ? expf(v - m) * inv_total : sigmoid(v); };
    // a score relative to exp(ref), which only scales all of them: sigmoid(v) exp(-ref) for ref <= 0 is
    // exp(v - ref) / (1 + exp(v)), and does not vanish where every logit is far below zero
    auto relative = [&](float v, float ref) {
        return softmax ? expf(v - ref) : v > 0.0f ? sigmoid(v) : expf(v - ref) / (1.0f + expf(v));
    };
#pragma unroll
    for (int i = 0; i < NV; ++i)
        ch[i] = l[i] > -INFINITY && a.bias ? score(l[i]) + ch[i] : l[i];

    if (c.top_groups < c.n_groups) {
        // each group's score by `per` lanes over shared memory, then its rank among the groups
        const int S = E / c.n_groups, G = c.n_groups;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float v = ch[i];
            if (sums && !a.bias && v > -INFINITY) v = relative(v, softmax ? m : fminf(m, 0.0f));
            sh.score[i * 33 + lane] = v;
        }
        __syncwarp();
        int per = 1;
        while (2 * per * G <= 32) per *= 2;
        const int g = lane / per, sub = lane % per;
        float b1 = -INFINITY, b2 = -INFINITY;
        if (g < G)
#pragma unroll 4
            for (int j = sub; j < S; j += per) {
                const int e = g * S + j;
                const float v = sh.score[e + (e >> 5)];
                b2 = fmaxf(b2, fminf(b1, v));
                b1 = fmaxf(b1, v);
            }
        for (int o = 1; o < per; o *= 2) {
            const float o1 = __shfl_xor_sync(kAll, b1, o), o2 = __shfl_xor_sync(kAll, b2, o);
            b2 = fmaxf(fminf(b1, o1), fmaxf(b2, o2));
            b1 = fmaxf(b1, o1);
        }
        const float gs = b1 + (c.group_best == 2 && b2 > -INFINITY ? b2 : 0.0f);
        int rank = 0;
#pragma unroll 4
        for (int q = 0; q < G; ++q) {
            const float os = __shfl_sync(kAll, gs, q * per);
            rank += os > gs || (os == gs && q < g);
        }
        const unsigned kept_lane = __ballot_sync(kAll, g < G && sub == 0 && rank < c.top_groups);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = i * 32 + lane;
            const int ge = (int)(((uint32_t)e * a.inv_group) >> 20);
            if (e < E && !((kept_lane >> (ge * per)) & 1)) ch[i] = -INFINITY;
        }
        __syncwarp();
    }

    const uint32_t none = ordered(-INFINITY);
    uint32_t key[NV], best = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        sh.score[i * 33 + lane] = ch[i];
        key[i] = ordered(ch[i]);
        best = max(best, key[i]);
    }
    // the top_k-th distinct largest lane maximum (equal ones count once, which can only lower it), and at least
    // none + 1: what is out is no candidate
    uint32_t floor_key = none + 1;
    uint32_t rest = best;
    for (int j = 0; j < c.top_k; ++j) {
        const uint32_t top = __reduce_max_sync(kAll, rest);
        floor_key = top;
        if (top <= none) break;
        if (rest == top) rest = 0;
    }
    floor_key = max(floor_key, none + 1);
    uint32_t left = 0;  // bit i: key[i] is a candidate
#pragma unroll
    for (int i = 0; i < NV; ++i) left |= (uint32_t)(key[i] >= floor_key) << i;
    int at = __popc(left);
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int v = __shfl_up_sync(kAll, at, o);
        if (lane >= o) at += v;
    }
    const int n = __shfl_sync(kAll, at, 31);
    int mine = -1;  // lane j: the j-th choice
    if (n <= 32) {
        for (at -= __popc(left); left; left &= left - 1) sh.cand[at++] = (__ffs(left) - 1) * 32 + lane;
        __syncwarp();
        const int e0 = lane < n ? sh.cand[lane] : E;
        const float s0 = lane < n ? sh.score[e0 + (e0 >> 5)] : -INFINITY;
        int rank = 0;
        for (int q = 0; q < n; ++q) {
            const float sq = __shfl_sync(kAll, s0, q);
            const int eq = __shfl_sync(kAll, e0, q);
            rank += sq > s0 || (sq == s0 && eq < e0);
        }
        if (lane < n) sh.order[rank] = e0;
        __syncwarp();
        if (lane < n && lane < c.top_k) mine = sh.order[lane];
    } else {
        for (int j = 0; j < c.top_k; ++j) {
            const uint32_t top = __reduce_max_sync(kAll, best);
            if (top == none) break;
            int first = INT_MAX;
#pragma unroll
            for (int i = NV - 1; i >= 0; --i)
                if (key[i] == top) first = i * 32 + lane;
            const int win = __reduce_min_sync(kAll, first);
            if (lane == j) mine = win;
            best = 0;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (i * 32 + lane == win) key[i] = none;
                best = max(best, key[i]);
            }
        }
    }
    const float v = mine >= 0 ? fminf(to_f32(row[mine]), FLT_MAX) : -INFINITY;

    // weights, relative to the largest chosen logit where they are renormalised
    float wt = 0.0f;
    if (c.renorm) {
        const float ref = softmax ? warp_max(v) : fminf(warp_max(v), 0.0f);
        if (mine >= 0) wt = relative(v, ref);
        const float sum = warp_sum(wt);
        if (mine >= 0) wt = wt / sum * c.scale;
    } else if (mine >= 0) {
        wt = score(v) * c.scale;
    }
    if (lane < c.top_k) {
        a.idx[t * c.top_k + lane] = mine;
        a.w[t * c.top_k + lane] = wt;
    }
}

template <typename T>
cudaError_t route_typed(const RouteArgs& a, cudaStream_t st) {
    const unsigned grid = (unsigned)((a.T + kRouteWarps - 1) / kRouteWarps);
    const int E = a.c.n_experts;
    if (E <= 128) return launch(route_kernel<T, 4>, grid, 32 * kRouteWarps, 0, st, 1, a);
    if (E <= 256) return launch(route_kernel<T, 8>, grid, 32 * kRouteWarps, 0, st, 1, a);
    if (E <= 512) return launch(route_kernel<T, 16>, grid, 32 * kRouteWarps, 0, st, 1, a);
    return launch(route_kernel<T, 32>, grid, 32 * kRouteWarps, 0, st, 1, a);
}

// ---------------------------------------------------------------------------
// dispatch
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 1024, kSortWarps = 32, kSortCtas = 16;
constexpr int kKeep = 8;  // rounds whose ranks stay in registers between the two passes

// Lanes of the warp with the same key (0 <= key < 2^bits), by one ballot a
// bit.  A match instruction does the same, but takes about 65 cycles of an SM.
__device__ __forceinline__ unsigned peers_of(int key, int bits) {
    unsigned peers = kAll;
    for (int b = 0; b < bits; ++b) {
        const unsigned set = __ballot_sync(kAll, key >> b & 1);
        peers &= key >> b & 1 ? set : ~set;
    }
    return peers;
}

// inclusive sum over a warp
__device__ __forceinline__ int warp_scan(int v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int u = __shfl_up_sync(kAll, v, o);
        if (lane >= o) v += u;
    }
    return v;
}

// Up to 1024 pairs, one a thread: one CTA, counts per (warp, expert) in bytes.
// A chain of short steps between five barriers; latency is all there is.
__global__ void __launch_bounds__(kSortThreads) dispatch_small_kernel(const int32_t* idx, int n, int top_k, int E,
                                                                      int bits, int32_t* offsets, int32_t* row_of_pair,
                                                                      int32_t* token_of_row, int32_t* group_of_row) {
    extern __shared__ uint4 cnt_raw[];  // [warps with pairs][E] bytes, then [E] first rows
    __shared__ int warp_tot[kSortWarps];
    let_next_start();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rows = (n + 31) / 32, bytes = (rows * E + 15) & ~15;
    uint8_t* cnt = reinterpret_cast<uint8_t*>(cnt_raw);
    int* first = reinterpret_cast<int*>(cnt + bytes);
    for (int i = tid; i < bytes / 16; i += blockDim.x) cnt_raw[i] = make_uint4(0, 0, 0, 0);
    after_previous();
    int key = tid < n ? idx[tid] : -1;
    if (key < 0 || key >= E) key = -1;
    __syncthreads();
    int rank = 0;
    if (warp < rows) {
        const unsigned peers = peers_of(key < 0 ? E : key, bits);
        rank = __popc(peers & ((1u << lane) - 1));
        if (key >= 0 && rank == 0) cnt[warp * E + key] = (uint8_t)__popc(peers);
    }
    __syncthreads();
    int total = 0;
    if (tid < E)
        for (int w = 0; w < rows; ++w) total += cnt[w * E + tid];
    if (key >= 0)
        for (int w = 0; w < warp; ++w) rank += cnt[w * E + key];
    const int incl = warp_scan(total, lane);
    if (lane == 31) warp_tot[warp] = incl;
    __syncthreads();
    if (warp == 0) warp_tot[lane] = warp_scan(lane < (int)blockDim.x / 32 ? warp_tot[lane] : 0, lane);
    __syncthreads();
    const int kept = warp_tot[blockDim.x / 32 - 1];
    const int at = (warp ? warp_tot[warp - 1] : 0) + incl - total;
    if (tid < E) {
        first[tid] = at;
        offsets[tid] = at;
    }
    if (tid == 0) offsets[E] = kept;
    __syncthreads();
    if (tid >= n) return;
    const int row = key >= 0 ? first[key] + rank : -1;
    row_of_pair[tid] = row;
    if (key >= 0) {
        token_of_row[row] = tid / top_k;
        group_of_row[row] = key;
    }
    if (tid >= kept) {
        token_of_row[tid] = -1;
        group_of_row[tid] = -1;
    }
}

// More pairs: the CTAs of one cluster take consecutive runs of them, and each
// warp a run of its CTA's, so that a pair's rank among its expert's pairs is
// (earlier CTAs) + (earlier warps) + (earlier rounds) + (lower lanes): stable,
// and free of atomics.  The CTAs read each other's counts per expert through
// distributed shared memory.
__global__ void __launch_bounds__(kSortThreads) dispatch_kernel(const int32_t* idx, int n, int top_k, int E, int bits,
                                                                int32_t* offsets, int32_t* row_of_pair,
                                                                int32_t* token_of_row, int32_t* group_of_row) {
    extern __shared__ int cnt[];  // [kSortWarps][E] per warp, then [E] of the CTA
    __shared__ int warp_tot[kSortWarps];
    let_next_start();
    int* const cta_cnt = cnt + kSortWarps * E;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    cg::cluster_group cluster = cg::this_cluster();
    const int me = (int)cluster.block_rank();
    const int64_t seg = ((int64_t)n + kSortCtas * kSortThreads - 1) / (kSortCtas * kSortThreads) * 32;
    const int64_t p0 = ((int64_t)me * kSortWarps + warp) * seg, p1 = p0 + seg < n ? p0 + seg : n;
    const bool keep = seg <= 32 * kKeep;
    int* mine = cnt + warp * E;
    int key_r[kKeep], rank_r[kKeep];
    auto key_at = [&](int64_t p) {
        const int e = p < p1 ? idx[p] : -1;
        return e >= 0 && e < E ? e : -1;
    };
    // rank among the warp's pairs of this expert so far; counts them
    auto take = [&](int key) {
        const unsigned peers = peers_of(key < 0 ? E : key, bits);
        const int r = key >= 0 ? mine[key] : 0, lower = __popc(peers & ((1u << lane) - 1));
        __syncwarp();
        if (key >= 0 && lower == 0) mine[key] = r + __popc(peers);
        __syncwarp();
        return r + lower;
    };
    after_previous();
    if (keep)
#pragma unroll
        for (int j = 0; j < kKeep; ++j) key_r[j] = key_at(p0 + 32 * j + lane);
    for (int i = lane; i < E; i += 32) mine[i] = 0;
    __syncwarp();
    if (keep) {
#pragma unroll
        for (int j = 0; j < kKeep; ++j)
            if (p0 + 32 * j < p1) rank_r[j] = take(key_r[j]);
    } else {
        for (int64_t p = p0 + lane; p - lane < p1; p += 32) take(key_at(p));
    }
    __syncthreads();
    int own = 0;
    if (tid < E) {
#pragma unroll 8
        for (int w = 0; w < kSortWarps; ++w) {
            const int c = cnt[w * E + tid];
            cnt[w * E + tid] = own;
            own += c;
        }
        cta_cnt[tid] = own;
    }
    cluster.sync();
    int total = 0, earlier = 0;  // of this expert: all CTAs, CTAs before this one
    if (tid < E) {
        int c[kSortCtas];  // all loads in flight: a remote one takes several hundred cycles
#pragma unroll
        for (int r = 0; r < kSortCtas; ++r) c[r] = cluster.map_shared_rank(cta_cnt, r)[tid];
#pragma unroll
        for (int r = 0; r < kSortCtas; ++r) {
            total += c[r];
            if (r < me) earlier += c[r];
        }
    }
    auto counts_read = cluster.barrier_arrive();
    const int incl = warp_scan(total, lane);
    if (lane == 31) warp_tot[warp] = incl;
    __syncthreads();
    if (warp == 0) warp_tot[lane] = warp_scan(warp_tot[lane], lane);
    __syncthreads();
    const int kept = warp_tot[kSortWarps - 1];
    if (tid < E) {
        const int at = (warp ? warp_tot[warp - 1] : 0) + incl - total;
        if (me == 0) offsets[tid] = at;
#pragma unroll 8
        for (int w = 0; w < kSortWarps; ++w) cnt[w * E + tid] += at + earlier;
    }
    if (tid == 0 && me == 0) offsets[E] = kept;
    __syncthreads();
    auto put = [&](int64_t p, int key, int row) {
        if (p >= p1) return;
        row_of_pair[p] = key >= 0 ? row : -1;
        if (key >= 0) {
            token_of_row[row] = (int)((uint32_t)p / (uint32_t)top_k);
            group_of_row[row] = key;
        }
    };
    if (keep) {
#pragma unroll
        for (int j = 0; j < kKeep; ++j)
            if (p0 + 32 * j < p1) {
                const int key = key_r[j];
                // the rank was counted from the warp's own zero: its count here is the warp's first row
                put(p0 + 32 * j + lane, key, key >= 0 ? mine[key] + rank_r[j] : -1);
            }
    } else {
        for (int64_t p = p0 + lane; p - lane < p1; p += 32) {
            const int key = key_at(p);
            put(p, key, take(key));
        }
    }
    for (int64_t r = kept + (int64_t)me * kSortThreads + tid; r < n; r += kSortCtas * kSortThreads) {
        token_of_row[r] = -1;
        group_of_row[r] = -1;
    }
    cluster.barrier_wait(std::move(counts_read));  // no CTA leaves while its counts are read
}

// ---------------------------------------------------------------------------
// combine
// ---------------------------------------------------------------------------
constexpr int kCombineThreads = 128;

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// A CTA takes 8 x 128 columns of one token, a thread 8 of them: memory-bound,
// so the loads are 16 bytes wide and four rows' are in flight at a time.
// WIDE = false: any alignment, 128 columns of a token per CTA.
template <typename TI, typename TO, bool WIDE>
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(const TI* rows, int64_t rows_ld,
                                                                  const int32_t* row_of_pair, const float* w, int top_k,
                                                                  int cols, TO* y, int64_t y_ld) {
    constexpr int V = WIDE ? 8 : 1;
    after_previous();
    let_next_start();
    const int64_t t = blockIdx.x;
    const int col = (blockIdx.y * kCombineThreads + threadIdx.x) * V;
    if (col >= cols) return;
    row_of_pair += t * top_k;
    w += t * top_k;
    float acc[V] = {};
    int j = 0;
    auto add = [&](int n) {  // n <= 4 rows from j on
        float v[4][V], wj[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = i < n ? row_of_pair[j + i] : -1;
            wj[i] = i < n ? w[j + i] : 0.0f;
#pragma unroll
            for (int q = 0; q < V; ++q) v[i][q] = 0.0f;
            if (r >= 0) {
                const TI* p = rows + r * rows_ld + col;
                if constexpr (WIDE) load8(p, v[i]);
                else v[i][0] = to_f32(*p);
            } else {
                wj[i] = 0.0f;
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int q = 0; q < V; ++q) acc[q] = fmaf(wj[i], v[i][q], acc[q]);
        j += n;
    };
    while (top_k - j >= 4) add(4);
    if (j < top_k) add(top_k - j);
    TO* out = y + t * y_ld + col;
    if constexpr (WIDE) store8(out, acc);
    else *out = (TO)acc[0];
}

// 8 columns at a time need whole, aligned 16-byte pieces in every row of both
template <typename T>
bool wide_rows(const void* p, int64_t ld, int cols) {
    return cols % 8 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * (int64_t)sizeof(T) % 16 == 0;
}

template <typename TI, typename TO>
cudaError_t combine_typed(const void* rows, int64_t rows_ld, const int32_t* row_of_pair, const float* w, int64_t T,
                          int top_k, int cols, void* y, int64_t y_ld, cudaStream_t st) {
    const bool wide = wide_rows<TI>(rows, rows_ld, cols) && wide_rows<TO>(y, y_ld, cols);
    const int per = kCombineThreads * (wide ? 8 : 1);
    const int64_t chunks = ((int64_t)cols + per - 1) / per;
    if (chunks > 65535) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)T, (unsigned)chunks);
    const TI* in = static_cast<const TI*>(rows);
    TO* out = static_cast<TO*>(y);
    return launch(wide ? combine_kernel<TI, TO, true> : combine_kernel<TI, TO, false>, grid, kCombineThreads, 0, st, 1, in,
                  rows_ld, row_of_pair, w, top_k, cols, out, y_ld);
}

}  // namespace

cudaError_t launch_route(const moe_route_config& c, const void* logits, int type, int64_t ld, const float* bias,
                         int64_t T, int32_t* idx, float* w, cudaStream_t st) {
    const int S = c.n_experts / c.n_groups;
    RouteArgs a{logits, bias, idx, w, ld, T, c, (uint32_t)(((1 << 20) + S - 1) / S)};
    return type == MOE_F32 ? route_typed<float>(a, st) : route_typed<__nv_bfloat16>(a, st);
}

size_t dispatch_workspace(int64_t, int) { return 0; }

cudaError_t launch_dispatch(const int32_t* idx, int64_t pairs, int top_k, int n_experts, int32_t* offsets,
                            int32_t* row_of_pair, int32_t* token_of_row, int32_t* group_of_row, void*,
                            cudaStream_t st) {
    int bits = 1;  // ids 0 .. n_experts, the last for a dropped pair
    while ((n_experts >> bits) != 0) ++bits;
    cudaError_t e;
    if (pairs <= kSortThreads) {
        const int n = (int)pairs, rows = (n + 31) / 32;
        const int smem = ((rows * n_experts + 15) & ~15) + n_experts * (int)sizeof(int);
        if ((e = smem_limit(reinterpret_cast<const void*>(dispatch_small_kernel), smem)) != cudaSuccess) return e;
        const int threads = ((n > n_experts ? n : n_experts) + 31) & ~31;
        return launch(dispatch_small_kernel, 1, threads, smem, st, 1, idx, n, top_k, n_experts, bits, offsets,
                      row_of_pair, token_of_row, group_of_row);
    }
    const int smem = (kSortWarps + 1) * n_experts * (int)sizeof(int);
    const void* kernel = reinterpret_cast<const void*>(dispatch_kernel);
    if ((e = smem_limit(kernel, smem)) != cudaSuccess) return e;
    // 16 CTAs are past the portable cluster size of 8
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess) return e;
    return launch(dispatch_kernel, kSortCtas, kSortThreads, smem, st, kSortCtas, idx, (int)pairs, top_k, n_experts, bits,
                  offsets, row_of_pair, token_of_row, group_of_row);
}

cudaError_t launch_combine(const void* rows, int rows_type, int64_t rows_ld, const int32_t* row_of_pair, const float* w,
                           int64_t T, int top_k, int cols, void* y, int y_type, int64_t y_ld, cudaStream_t st) {
    using bf = __nv_bfloat16;
    if (rows_type == MOE_F32)
        return y_type == MOE_F32
                   ? combine_typed<float, float>(rows, rows_ld, row_of_pair, w, T, top_k, cols, y, y_ld, st)
                   : combine_typed<float, bf>(rows, rows_ld, row_of_pair, w, T, top_k, cols, y, y_ld, st);
    return y_type == MOE_F32 ? combine_typed<bf, float>(rows, rows_ld, row_of_pair, w, T, top_k, cols, y, y_ld, st)
                             : combine_typed<bf, bf>(rows, rows_ld, row_of_pair, w, T, top_k, cols, y, y_ld, st);
}

}  // namespace moe
