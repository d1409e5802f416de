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

__device__ __forceinline__ float sigmoid(float l) { return 1.0f / (1.0f + expf(-l)); }

// One warp per token; lane l holds the experts l, l + 32, ...: the row is read
// once, coalesced, and every statistic is a warp reduction on registers.  The
// top-k takes k rounds of (largest key, then lowest id) over the warp.
template <typename T, int NV>
__global__ void __launch_bounds__(32 * kRouteWarps) route_kernel(const RouteArgs a) {
    __shared__ float buf_s[kRouteWarps][NV * 33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp;
    if (t >= a.T) return;
    const moe_route_config& c = a.c;
    const int E = c.n_experts;
    const T* row = static_cast<const T*>(a.logits) + t * a.ld;

    float l[NV], ch[NV];  // logits (-inf: out) and what the choice compares
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = i * 32 + lane;
        float v = e < E ? to_f32(row[e]) : -INFINITY;
        if (!(v > -INFINITY)) v = -INFINITY;
        if (a.bias && e < E) {
            const float b = a.bias[e];
            if (!(b > -INFINITY)) v = -INFINITY;
        }
        l[i] = fminf(v, FLT_MAX);
        m = fmaxf(m, l[i]);
    }
    m = warp_max(m);
    const bool softmax = c.score == MOE_SCORE_SOFTMAX;
    const bool sums = c.top_groups < c.n_groups && c.group_best == 2;
    float total = 1.0f;
    if (softmax && (a.bias || !c.renorm)) {
        total = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) total += l[i] > -INFINITY ? expf(l[i] - m) : 0.0f;
        total = warp_sum(total);
    }
    auto score = [&](float v) { return softmax ? expf(v - m) / total : sigmoid(v); };
    // a score relative to exp(ref), which only scales all of them: sigmoid(v) exp(-ref) for ref <= 0 is
    // exp(v - ref) / (1 + exp(v)), and does not vanish where every logit is far below zero
    auto relative = [&](float v, float ref) {
        return softmax ? expf(v - ref) : v > 0.0f ? sigmoid(v) : expf(v - ref) / (1.0f + expf(v));
    };
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = i * 32 + lane;
        ch[i] = l[i];
        if (a.bias && l[i] > -INFINITY) ch[i] = score(l[i]) + a.bias[e];
    }

    if (c.top_groups < c.n_groups) {
        // each group's score by `per` lanes over shared memory, then its rank among the groups
        const int S = E / c.n_groups, G = c.n_groups;
        float* buf = buf_s[warp];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float v = ch[i];
            if (sums && !a.bias && v > -INFINITY) v = relative(v, softmax ? m : fminf(m, 0.0f));
            buf[i * 33 + lane] = v;
        }
        __syncwarp();
        int per = 1;
        while (2 * per * G <= 32) per *= 2;
        const int g = lane / per, sub = lane % per;
        float b1 = -INFINITY, b2 = -INFINITY;
        if (g < G)
            for (int j = sub; j < S; j += per) {
                const int e = g * S + j;
                const float v = buf[e + (e >> 5)];
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
    }

    // top-k: lane j keeps the j-th choice
    const uint32_t none = ordered(-INFINITY);
    uint32_t best = none;
    int at = INT_MAX;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const uint32_t k = ordered(ch[i]);
        if (k > best) best = k, at = i * 32 + lane;
    }
    int mine = -1;
    for (int j = 0; j < c.top_k; ++j) {
        const uint32_t top = __reduce_max_sync(kAll, best);
        if (top == none) break;
        const int win = __reduce_min_sync(kAll, best == top ? at : INT_MAX);
        if (lane == j) mine = win;
        if ((win & 31) == lane) {
            best = none;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (i == win >> 5) ch[i] = -INFINITY;
                const uint32_t k = ordered(ch[i]);
                if (k > best) best = k, at = i * 32 + lane;
            }
        }
        __syncwarp();
    }

    // weights, relative to the largest chosen logit where they are renormalised
    float v = -INFINITY;
    if (mine >= 0) v = fminf(to_f32(row[mine]), FLT_MAX);
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
    if (E <= 128) route_kernel<T, 4><<<grid, 32 * kRouteWarps, 0, st>>>(a);
    else if (E <= 256) route_kernel<T, 8><<<grid, 32 * kRouteWarps, 0, st>>>(a);
    else if (E <= 512) route_kernel<T, 16><<<grid, 32 * kRouteWarps, 0, st>>>(a);
    else route_kernel<T, 32><<<grid, 32 * kRouteWarps, 0, st>>>(a);
    return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// dispatch
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 1024, kSortWarps = 32;

// One CTA.  Warp w owns a run of consecutive pairs; 32 pairs at a time it
// finds equal experts by a warp match, so that a pair's rank among its
// expert's pairs is (counts of earlier warps) + (its warp's earlier rounds) +
// (lower lanes): stable, and free of atomics.
__global__ void __launch_bounds__(kSortThreads) dispatch_kernel(const int32_t* idx, int n, int top_k, int E,
                                                                int32_t* offsets, int32_t* row_of_pair,
                                                                int32_t* token_of_row, int32_t* group_of_row) {
    extern __shared__ int cnt[];  // [kSortWarps][E]
    __shared__ int warp_tot[kSortWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int i = tid; i < kSortWarps * E; i += kSortThreads) cnt[i] = 0;
    __syncthreads();
    const int64_t seg = ((int64_t)n + kSortThreads - 1) / kSortThreads * 32;
    const int64_t p0 = warp * seg, p1 = p0 + seg < n ? p0 + seg : n;
    int* mine = cnt + warp * E;
    for (int64_t p = p0 + lane; p - lane < p1; p += 32) {
        const int e = p < p1 ? idx[p] : -1;
        const int key = e >= 0 && e < E ? e : -1;
        const unsigned peers = __match_any_sync(kAll, key);
        if (key >= 0 && lane == __ffs(peers) - 1) mine[key] += __popc(peers);
        __syncwarp();
    }
    __syncthreads();
    int total = 0;
    if (tid < E)
        for (int w = 0; w < kSortWarps; ++w) {
            const int c = cnt[w * E + tid];
            cnt[w * E + tid] = total;
            total += c;
        }
    int incl = total;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int v = __shfl_up_sync(kAll, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) warp_tot[warp] = incl;
    __syncthreads();
    int before = 0, kept = 0;
    for (int w = 0; w < kSortWarps; ++w) {
        if (w < warp) before += warp_tot[w];
        kept += warp_tot[w];
    }
    const int first = before + incl - total;
    if (tid < E) {
        offsets[tid] = first;
        for (int w = 0; w < kSortWarps; ++w) cnt[w * E + tid] += first;
    }
    if (tid == 0) offsets[E] = kept;
    __syncthreads();
    for (int64_t p = p0 + lane; p - lane < p1; p += 32) {
        const int e = p < p1 ? idx[p] : -1;
        const int key = e >= 0 && e < E ? e : -1;
        const unsigned peers = __match_any_sync(kAll, key);
        int row = -1;
        if (key >= 0) {
            row = mine[key] + __popc(peers & ((1u << lane) - 1));
            token_of_row[row] = (int)(p / top_k);
            group_of_row[row] = key;
        }
        if (p < p1) row_of_pair[p] = row;
        __syncwarp();
        if (key >= 0 && lane == __ffs(peers) - 1) mine[key] += __popc(peers);
        __syncwarp();
    }
    for (int r = kept + tid; r < n; r += kSortThreads) {
        token_of_row[r] = -1;
        group_of_row[r] = -1;
    }
}

// ---------------------------------------------------------------------------
// combine
// ---------------------------------------------------------------------------
template <typename TI, typename TO>
__global__ void __launch_bounds__(256) combine_kernel(const TI* rows, int64_t rows_ld, const int32_t* row_of_pair,
                                                      const float* w, int64_t T, int top_k, int cols, TO* y,
                                                      int64_t y_ld) {
    const int per = (cols + 255) / 256;
    for (int64_t b = blockIdx.x; b < T * per; b += gridDim.x) {
        const int64_t t = b / per;
        const int col = (int)(b % per) * 256 + threadIdx.x;
        if (col >= cols) continue;
        float acc = 0.0f;
        for (int j = 0; j < top_k; ++j) {
            const int r = row_of_pair[t * top_k + j];
            if (r >= 0) acc += w[t * top_k + j] * to_f32(rows[r * rows_ld + col]);
        }
        y[t * y_ld + col] = (TO)acc;
    }
}

template <typename TI, typename TO>
cudaError_t combine_typed(const void* rows, int64_t rows_ld, const int32_t* row_of_pair, const float* w, int64_t T,
                          int top_k, int cols, void* y, int64_t y_ld, cudaStream_t st) {
    const int64_t blocks = T * ((cols + 255) / 256);
    combine_kernel<TI, TO><<<(unsigned)(blocks < 1 << 20 ? blocks : 1 << 20), 256, 0, st>>>(
        static_cast<const TI*>(rows), rows_ld, row_of_pair, w, T, top_k, cols, static_cast<TO*>(y), y_ld);
    return cudaGetLastError();
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
    const int smem = kSortWarps * n_experts * (int)sizeof(int);
    cudaError_t e = smem_limit(reinterpret_cast<const void*>(dispatch_kernel), smem);
    if (e != cudaSuccess) return e;
    dispatch_kernel<<<1, kSortThreads, smem, st>>>(idx, (int)pairs, top_k, n_experts, offsets, row_of_pair,
                                                   token_of_row, group_of_row);
    return cudaGetLastError();
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
