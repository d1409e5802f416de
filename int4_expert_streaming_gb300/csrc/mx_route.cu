// mx_route.cu -- routing with groups and a balance bias, the stable sort of
// the chosen pairs by expert, and the weighted combine of the experts' rows.
#include <cfloat>

#include "mx.h"

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
struct RouteArgs {
    const void* logits;
    const float* bias;
    int32_t* idx;
    float* w;
    int64_t ld, T;
    moe_route_config c;
    uint32_t inv_group;  // e / group size = (e * inv_group) >> 20 for e < 1024
    int group_size, lanes_log2;  // lanes that share a group's score: the largest power of two with n_groups of it in a warp
};

constexpr int kRouteWarps = 16;  // at most, per block

__device__ __forceinline__ float from_ordered(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
__device__ __forceinline__ float warp_max(float v) { return from_ordered(__reduce_max_sync(kAll, ordered(v))); }

// 1 / (1 + exp(-l)), exp(-l) = 2^(-l log2 e), to about 2^-21 relative for |l| < 16: the choice compares fp32 sums of
// it anyway, and a short form halves this part of the kernel.  The weights take expf.
__device__ __forceinline__ float sigmoid_fast(float l) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-1.44269504f * l));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return r;
}

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
// a cold instruction cache, so the code is kept short.  With thousands (4001
// of 256 experts: 6.1 us) the warps of an SM, one token each, use 59 % of the
// issue slots while they are there, and launch and tail take as long again.
template <typename T, int NV>
__global__ void __launch_bounds__(32 * kRouteWarps) route_kernel(const RouteArgs a) {
    extern __shared__ float scratch[];  // a RouteScratch per warp
    after_previous();
    let_next_start();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = (int64_t)blockIdx.x * (blockDim.x >> 5) + warp;
    if (t >= a.T) return;
    RouteScratch<NV>& sh = reinterpret_cast<RouteScratch<NV>*>(scratch)[warp];
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
    const bool softmax = c.score == MOE_SCORE_SOFTMAX;
    const bool sums = c.top_groups < c.n_groups && c.group_best == 2;
    m = warp_max(m);
    float inv_total = 1.0f;
    if (softmax && (a.bias || !c.renorm)) {
        float total = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) total += l[i] > -INFINITY ? expf(l[i] - m) : 0.0f;
        inv_total = 1.0f / warp_sum(total);
    }
    auto score = [&](float v) { return softmax ? expf(v - m) * inv_total : sigmoid_fast(v); };
    // a score relative to exp(ref), which only scales all of them: sigmoid(v) exp(-ref) for ref <= 0 is
    // exp(v - ref) / (1 + exp(v)), and does not vanish where every logit is far below zero
    auto relative = [&](float v, float ref) {
        const float e = expf(softmax || v <= 0.0f ? v - ref : -v);
        return softmax ? e : v > 0.0f ? 1.0f / (1.0f + e) : e / (1.0f + expf(v));
    };
#pragma unroll
    for (int i = 0; i < NV; ++i)
        ch[i] = l[i] > -INFINITY && a.bias ? score(l[i]) + ch[i] : l[i];

    if (c.top_groups < c.n_groups) {
        // each group's score by `per` lanes over shared memory, then its rank among the groups
        const int S = a.group_size, G = c.n_groups, log2 = a.lanes_log2, per = 1 << log2;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float v = ch[i];
            if (sums && !a.bias && v > -INFINITY) v = relative(v, softmax ? m : fminf(m, 0.0f));
            sh.score[i * 33 + lane] = v;
        }
        __syncwarp();
        const int g = lane >> log2, sub = lane & (per - 1);
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
            const float os = __shfl_sync(kAll, gs, q << log2);
            rank += os > gs || (os == gs && q < g);
        }
        const unsigned kept_lane = __ballot_sync(kAll, g < G && sub == 0 && rank < c.top_groups);
        const bool whole = (S & 31) == 0;  // a row of 32 experts lies in one group: the test is the warp's
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = whole ? i * 32 : i * 32 + lane;
            const int ge = (int)(((uint32_t)e * a.inv_group) >> 20);
            if (e < E && !((kept_lane >> (ge << log2)) & 1)) ch[i] = -INFINITY;
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
        wt = (softmax ? expf(v - m) * inv_total : 1.0f / (1.0f + expf(-v))) * c.scale;
    }
    if (lane < c.top_k) {
        a.idx[t * c.top_k + lane] = mine;
        a.w[t * c.top_k + lane] = wt;
    }
}

template <typename T, int NV>
cudaError_t route_rows(const RouteArgs& a, cudaStream_t st) {
    // Blocks of 16 warps once they fill the GPU: starting 1000 blocks of 4 costs more than their work (4001 tokens of
    // 256 experts 7.7 -> 6.3 us); below that 4, to spread over the SMs.
    constexpr int kMost = NV == 32 ? kRouteWarps / 2 : kRouteWarps;  // within 48 KB of scratch
    const int warps = a.T >= 16 * 128 ? kMost : 4;
    return launch(route_kernel<T, NV>, (unsigned)((a.T + warps - 1) / warps), 32 * warps, warps * sizeof(RouteScratch<NV>),
                  st, 1, a);
}

template <typename T>
cudaError_t route_typed(const RouteArgs& a, cudaStream_t st) {
    const int E = a.c.n_experts;
    if (E <= 128) return route_rows<T, 4>(a, st);
    if (E <= 256) return route_rows<T, 8>(a, st);
    if (E <= 512) return route_rows<T, 16>(a, st);
    return route_rows<T, 32>(a, st);
}

// ---------------------------------------------------------------------------
// dispatch
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 1024, kSortWarps = 32, kSortCtas = 128;
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

// More pairs, two kernels: up to kSortCtas CTAs take consecutive runs of the
// pairs, and each warp a run of its CTA's.  The first counts each CTA's pairs
// per expert.  In the second a pair's place is (earlier CTAs) + (earlier warps)
// + (earlier rounds) + (lower lanes): stable, whatever runs first.  Its ranks
// within the CTA need nothing of the first kernel, so they are formed before it
// has finished; after that come the sums over the CTAs' counts and the
// scattered stores (a sector each, about one a cycle of an SM: the reason for
// many CTAs.  One cluster of 16 took 9.6 us for 40960 pairs, these 7.1).
struct SortArgs {
    const int32_t* idx;
    int n, top_k, E, bits, ctas;
    int64_t seg;  // pairs of a warp, a multiple of 32
    int32_t *offsets, *row_of_pair, *token_of_row, *group_of_row;
    int32_t* counts;  // [ctas][E]
};

// read past L1: the second kernel reads idx before it has waited for the first
__device__ __forceinline__ int sort_key(const SortArgs& a, int64_t p, int64_t end) {
    const int e = p < end ? __ldcg(a.idx + p) : -1;
    return e >= 0 && e < a.E ? e : -1;
}

__global__ void __launch_bounds__(kSortThreads) dispatch_count_kernel(const SortArgs a) {
    extern __shared__ int hist[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int e = tid; e < a.E; e += kSortThreads) hist[e] = 0;
    after_previous();
    let_next_start();  // after the wait: the next kernel may read idx at once
    const int64_t p0 = ((int64_t)blockIdx.x * kSortWarps + warp) * a.seg, p1 = min(p0 + a.seg, (int64_t)a.n);
    __syncthreads();
    for (int64_t p = p0 + lane; p - lane < p1; p += 32) {
        const int key = sort_key(a, p, p1);
        const unsigned peers = peers_of(key < 0 ? a.E : key, a.bits);
        if (key >= 0 && lane == __ffs(peers) - 1) atomicAdd(hist + key, __popc(peers));  // a sum: order does not matter
    }
    __syncthreads();
    for (int e = tid; e < a.E; e += kSortThreads) a.counts[(int64_t)blockIdx.x * a.E + e] = hist[e];
}

__global__ void __launch_bounds__(kSortThreads) dispatch_place_kernel(const SortArgs a) {
    extern __shared__ int cnt[];  // [kSortWarps][E] per warp, then [2][parts][E] sums of the counts
    __shared__ int warp_tot[kSortWarps];
    let_next_start();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, E = a.E;
    int* const sums = cnt + kSortWarps * E;
    const int64_t p0 = ((int64_t)blockIdx.x * kSortWarps + warp) * a.seg, p1 = min(p0 + a.seg, (int64_t)a.n);
    const bool keep = a.seg <= 32 * kKeep;
    int* mine = cnt + warp * E;
    int key_r[kKeep], rank_r[kKeep];
    // rank among the warp's pairs of this expert so far; counts them
    auto take = [&](int key) {
        const unsigned peers = peers_of(key < 0 ? E : key, a.bits);
        const int r = key >= 0 ? mine[key] : 0, lower = __popc(peers & ((1u << lane) - 1));
        __syncwarp();
        if (key >= 0 && lower == 0) mine[key] = r + __popc(peers);
        __syncwarp();
        return r + lower;
    };
    if (keep)
#pragma unroll
        for (int j = 0; j < kKeep; ++j) key_r[j] = sort_key(a, p0 + 32 * j + lane, p1);
    for (int i = lane; i < E; i += 32) mine[i] = 0;
    __syncwarp();
    if (keep) {
#pragma unroll
        for (int j = 0; j < kKeep; ++j)
            if (p0 + 32 * j < p1) rank_r[j] = take(key_r[j]);
    } else {
        for (int64_t p = p0 + lane; p - lane < p1; p += 32) take(sort_key(a, p, p1));
    }
    __syncthreads();
    if (tid < E) {  // the warps' first places within the CTA
        int own = 0;
#pragma unroll 8
        for (int w = 0; w < kSortWarps; ++w) {
            const int c = cnt[w * E + tid];
            cnt[w * E + tid] = own;
            own += c;
        }
    }
    after_previous();
    // each expert's pairs in all CTAs and in those before this one, by `parts` threads per expert
    int parts = 1;
    while (2 * parts * E <= kSortThreads) parts *= 2;
    const int part = tid / E, e = tid - part * E;
    if (part < parts) {
        int total = 0, earlier = 0;
#pragma unroll 20
        for (int r = part; r < a.ctas; r += parts) {
            const int c = a.counts[(int64_t)r * E + e];
            total += c;
            earlier += r < (int)blockIdx.x ? c : 0;
        }
        sums[part * E + e] = total;
        sums[(parts + part) * E + e] = earlier;
    }
    __syncthreads();
    int total = 0, earlier = 0;
    if (tid < E)
        for (int q = 0; q < parts; ++q) {
            total += sums[q * E + tid];
            earlier += sums[(parts + q) * E + tid];
        }
    const int incl = warp_scan(total, lane);
    if (lane == 31) warp_tot[warp] = incl;
    __syncthreads();
    if (warp == 0) warp_tot[lane] = warp_scan(warp_tot[lane], lane);
    __syncthreads();
    const int kept = warp_tot[kSortWarps - 1];
    int* const base = sums;  // the CTA's first place of each expert
    if (tid < E) {
        const int at = (warp ? warp_tot[warp - 1] : 0) + incl - total;
        base[tid] = at + earlier;
        if (blockIdx.x == 0) a.offsets[tid] = at;
    }
    if (tid == 0 && blockIdx.x == 0) a.offsets[E] = kept;
    __syncthreads();
    auto put = [&](int64_t p, int key, int row) {
        if (p >= p1) return;
        a.row_of_pair[p] = key >= 0 ? row : -1;
        if (key >= 0) {
            a.token_of_row[row] = (int)((uint32_t)p / (uint32_t)a.top_k);
            a.group_of_row[row] = key;
        }
    };
    if (keep) {
#pragma unroll
        for (int j = 0; j < kKeep; ++j)
            if (p0 + 32 * j < p1) {
                const int key = key_r[j];
                // the rank was counted from the warp's own zero: its count here is the warp's first place
                put(p0 + 32 * j + lane, key, key >= 0 ? base[key] + mine[key] + rank_r[j] : -1);
            }
    } else {
        for (int64_t p = p0 + lane; p - lane < p1; p += 32) {
            const int key = sort_key(a, p, p1);
            const int r = take(key);
            put(p, key, key >= 0 ? base[key] + r : -1);
        }
    }
    for (int64_t r = kept + (int64_t)blockIdx.x * kSortThreads + tid; r < a.n; r += (int64_t)gridDim.x * kSortThreads) {
        a.token_of_row[r] = -1;
        a.group_of_row[r] = -1;
    }
}

// ---------------------------------------------------------------------------
// combine
// ---------------------------------------------------------------------------
constexpr int kCombineThreads = 128;

// V consecutive values by one load or store of at most 16 bytes (eight fp32: two)
template <int V>
__device__ __forceinline__ void load_v(const float* p, float* v) {
    if constexpr (V == 8) {
        const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else if constexpr (V == 2) {
        const float2 a = *reinterpret_cast<const float2*>(p);
        v[0] = a.x, v[1] = a.y;
    } else {
        v[0] = *p;
    }
}
template <int V>
__device__ __forceinline__ void load_v(const __nv_bfloat16* p, float* v) {
    uint32_t w[(V + 1) / 2];
    if constexpr (V == 8) {
        const uint4 q = *reinterpret_cast<const uint4*>(p);
        w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
    } else if constexpr (V == 2) {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else {
        w[0] = *reinterpret_cast<const uint16_t*>(p);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
}
template <int V>
__device__ __forceinline__ void store_v(float* p, const float* v) {
    if constexpr (V == 8) {
        reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else if constexpr (V == 2) {
        *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
    } else {
        *p = v[0];
    }
}
template <int V>
__device__ __forceinline__ void store_v(__nv_bfloat16* p, const float* v) {
    uint32_t w[(V + 1) / 2];
#pragma unroll
    for (int i = 0; i < V; i += 2) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[i], i + 1 < V ? v[i + 1] : 0.0f);
        w[i / 2] = *reinterpret_cast<const uint32_t*>(&b);
    }
    if constexpr (V == 8) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else if constexpr (V == 2) *reinterpret_cast<uint32_t*>(p) = w[0];
    else *reinterpret_cast<uint16_t*>(p) = (uint16_t)w[0];
}

// A thread takes kPieces<V> pieces of V columns of one token, V as the alignment
// allows: memory-bound, so loads are wide and four rows'
// are in flight at a time.  4096 tokens of 10 rows of 2048 bf16: 32.8 us with
// V = 8 (6.1 TB/s); of 2046 with 2 38.5, of 2047 with 1 52.2: those wait for narrow loads.
template <int V>
constexpr int kPieces = V == 8 ? 1 : V == 2 ? 2 : 4;

template <typename TI, typename TO, int V>
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(const TI* rows, uint32_t n_rows,
                                                                  int64_t rows_ld, const int32_t* row_of_pair,
                                                                  const float* w, int top_k, int cols, TO* y, int64_t y_ld) {
    constexpr int U = kPieces<V>, W = U * V;
    after_previous();
    let_next_start();
    const int64_t t = blockIdx.x;
    const int col = blockIdx.y * (W * kCombineThreads) + threadIdx.x * V;  // pieces kCombineThreads * V apart
    if (col >= cols) return;
    row_of_pair += t * top_k;
    w += t * top_k;
    float acc[W] = {};
    int j = 0;
    auto add = [&](int n) {  // n <= 4 rows from j on
        float v[4][W], wj[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // Whether there is a row, kept as a condition or, where many single loads hang on it, as the index -1: the
            // compiler's order of the loads differs.  4096 x 10 bf16 rows to fp32: of 2048 32.8 us as a condition, 33.4
            // as the index, of 2046 38.5 and 43.9, of 2047 62.7 and 52.2.
            int r = i < n ? row_of_pair[j + i] : -1;
            if (V == 1 && (uint32_t)r >= n_rows) r = -1;
            const bool there = V == 1 ? r >= 0 : (uint32_t)r < n_rows;
            wj[i] = there ? w[j + i] : 0.0f;
            const TI* p = rows + (V == 1 ? (there ? r * rows_ld : 0) : (int64_t)(there ? r : 0) * rows_ld) + col;
#pragma unroll
            for (int u = 0; u < U; ++u) {
#pragma unroll
                for (int q = 0; q < V; ++q) v[i][u * V + q] = 0.0f;
                if (there && col + u * kCombineThreads * V < cols) load_v<V>(p + u * kCombineThreads * V, v[i] + u * V);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int q = 0; q < W; ++q) acc[q] = fmaf(wj[i], v[i][q], acc[q]);
        j += n;
    };
    while (top_k - j >= 4) add(4);
    if (j < top_k) add(top_k - j);
    TO* out = y + t * y_ld + col;
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (col + u * kCombineThreads * V < cols) store_v<V>(out + u * kCombineThreads * V, acc + u * V);
}

// pieces of V need whole, aligned ones in every row
template <typename T>
bool pieces_ok(const void* p, int64_t ld, int cols, int V) {
    const int64_t bytes = V * (int64_t)sizeof(T) < 16 ? V * (int64_t)sizeof(T) : 16;
    return cols % V == 0 && reinterpret_cast<uintptr_t>(p) % bytes == 0 && ld * (int64_t)sizeof(T) % bytes == 0;
}

template <typename TI, typename TO>
cudaError_t combine_typed(const void* rows, uint32_t n_rows, int64_t rows_ld, const int32_t* row_of_pair,
                          const float* w, int64_t T, int top_k, int cols, void* y, int64_t y_ld, cudaStream_t st) {
    auto both = [&](int V) { return pieces_ok<TI>(rows, rows_ld, cols, V) && pieces_ok<TO>(y, y_ld, cols, V); };
    auto run = [&](auto kernel, int per) {
        const int64_t chunks = ((int64_t)cols + per * kCombineThreads - 1) / (per * kCombineThreads);
        if (chunks > 65535) return cudaErrorInvalidValue;
        return launch(kernel, dim3((unsigned)T, (unsigned)chunks), kCombineThreads, 0, st, 1, static_cast<const TI*>(rows),
                      n_rows, rows_ld, row_of_pair, w, top_k, cols, static_cast<TO*>(y), y_ld);
    };
    if (both(8)) return run(combine_kernel<TI, TO, 8>, 8 * kPieces<8>);
    if (both(2)) return run(combine_kernel<TI, TO, 2>, 2 * kPieces<2>);
    return run(combine_kernel<TI, TO, 1>, kPieces<1>);
}

}  // namespace

cudaError_t launch_route(const moe_route_config& c, const void* logits, int type, int64_t ld, const float* bias,
                         int64_t T, int32_t* idx, float* w, cudaStream_t st) {
    const int S = c.n_experts / c.n_groups;
    int log2 = 0;
    while ((2 << log2) * c.n_groups <= 32) ++log2;
    RouteArgs a{logits, bias, idx, w, ld, T, c, (uint32_t)(((1 << 20) + S - 1) / S), S, log2};
    return type == MOE_F32 ? route_typed<float>(a, st) : route_typed<__nv_bfloat16>(a, st);
}

// CTAs of the two-kernel sort: at least one round of 32 pairs per warp each
static int sort_ctas(int64_t pairs) {
    const int64_t n = (pairs + kSortThreads - 1) / kSortThreads;
    return (int)(n < kSortCtas ? n : kSortCtas);
}

size_t dispatch_workspace(int64_t pairs, int n_experts) {
    return pairs <= kSortThreads ? 0 : (size_t)sort_ctas(pairs) * n_experts * sizeof(int32_t);
}

cudaError_t launch_dispatch(const int32_t* idx, int64_t pairs, int top_k, int n_experts, int32_t* offsets,
                            int32_t* row_of_pair, int32_t* token_of_row, int32_t* group_of_row, void* ws,
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
    SortArgs a{idx, (int)pairs, top_k, n_experts, bits, sort_ctas(pairs), 0, offsets, row_of_pair, token_of_row, group_of_row,
               static_cast<int32_t*>(ws)};
    a.seg = (pairs + (int64_t)a.ctas * kSortThreads - 1) / ((int64_t)a.ctas * kSortThreads) * 32;
    int parts = 1;
    while (2 * parts * n_experts <= kSortThreads) parts *= 2;
    const int smem = (kSortWarps + 2 * parts) * n_experts * (int)sizeof(int);
    if ((e = smem_limit(reinterpret_cast<const void*>(dispatch_place_kernel), smem)) != cudaSuccess) return e;
    e = launch(dispatch_count_kernel, a.ctas, kSortThreads, n_experts * sizeof(int), st, 1, a);
    return e != cudaSuccess ? e : launch(dispatch_place_kernel, a.ctas, kSortThreads, smem, st, 1, a);
}

cudaError_t launch_combine(const void* rows, int64_t n_rows, int rows_type, int64_t rows_ld, const int32_t* row_of_pair,
                           const float* w, int64_t T, int top_k, int cols, void* y, int y_type, int64_t y_ld, cudaStream_t st) {
    using bf = __nv_bfloat16;
    const uint32_t n = n_rows > INT32_MAX ? 1u << 31 : (uint32_t)n_rows;  // an index has no more than 31 bits
    if (rows_type == MOE_F32)
        return y_type == MOE_F32
                   ? combine_typed<float, float>(rows, n, rows_ld, row_of_pair, w, T, top_k, cols, y, y_ld, st)
                   : combine_typed<float, bf>(rows, n, rows_ld, row_of_pair, w, T, top_k, cols, y, y_ld, st);
    return y_type == MOE_F32 ? combine_typed<bf, float>(rows, n, rows_ld, row_of_pair, w, T, top_k, cols, y, y_ld, st)
                             : combine_typed<bf, bf>(rows, n, rows_ld, row_of_pair, w, T, top_k, cols, y, y_ld, st);
}

}  // namespace moe
