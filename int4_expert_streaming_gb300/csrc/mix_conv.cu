// mix_conv.cu -- short causal convolution of each channel, with the last rows
// of a sequence kept in its slot.
#include <string.h>

#include "mix.h"

namespace moe {
namespace {

constexpr int kThreads = 128;
constexpr int kTile = 32;   // rows of a CTA's piece of a sequence
constexpr int kAhead = 8;   // rows whose loads are under way at once

struct ConvArgs {
    Seqs q;
    const void *x, *w;
    const float* bias;
    void *state, *y;
    int64_t x_ld, y_ld;
    int channels, act;
    bool w_bf16;
};

// V consecutive channels of a row as they are in memory
template <typename T, int V>
struct alignas(sizeof(T) * V) Row {
    T v[V];
};
template <typename T, int V>
__device__ __forceinline__ void widen(const Row<T, V>& r, float (&f)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = (float)r.v[i];
}

// A thread takes V channels (16 bytes, or one where rows are not aligned) down
// a piece of kTile rows, the last W - 1 inputs in registers; a piece reads the
// W - 1 rows before it again.  Bound by memory: each input and output once.
// The first piece's CTAs read the old state and also write the new one, so no
// two CTAs touch a slot's channel.
template <typename T, int V, int W>
__global__ void __launch_bounds__(kThreads) conv_kernel(const __grid_constant__ ConvArgs a) {
    after_previous();
    let_next_start();
    int piece;
    const int s = a.q.find<kTile>(blockIdx.x, piece);
    const int64_t lo = a.q.start(s), hi = a.q.start(s + 1), first = lo + (int64_t)piece * kTile;
    const int slot = a.q.slot(s);
    const int c = (blockIdx.y * kThreads + threadIdx.x) * V;
    if (piece < 0 || first >= hi || slot < 0 || c >= a.channels) return;
    const int rows = (int)(hi - first < kTile ? hi - first : kTile);

    using R = Row<T, V>;
    const T* x = static_cast<const T*>(a.x) + c;
    T* y = static_cast<T*>(a.y) + first * a.y_ld + c;
    T* state = a.state ? static_cast<T*>(a.state) + (int64_t)slot * (W - 1) * a.channels + c : nullptr;
    const bool carry = state && a.q.carry(s);

    R old[W - 1];  // the slot's rows, oldest first
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
        memset(&old[i], 0, sizeof(R));
        if (piece == 0 && carry) old[i] = *reinterpret_cast<const R*>(state + (int64_t)i * a.channels);
    }
    float w[W][V], bias[V], past[W - 1][V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        bias[j] = a.bias ? a.bias[c + j] : 0.0f;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const int64_t at = (int64_t)(c + j) * W + i;
            w[i][j] = a.w_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.w)[at]) : static_cast<const float*>(a.w)[at];
        }
    }
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
        if (piece > 0) old[i] = *reinterpret_cast<const R*>(x + (first - (W - 1) + i) * a.x_ld);
        widen(old[i], past[i]);
    }
    x += first * a.x_ld;
    for (int t0 = 0; t0 < rows; t0 += kAhead) {
        R in[kAhead];
#pragma unroll
        for (int t = 0; t < kAhead; ++t)
            if (t0 + t < rows) in[t] = *reinterpret_cast<const R*>(x + (t0 + t) * a.x_ld);
#pragma unroll
        for (int t = 0; t < kAhead; ++t) {
            if (t0 + t < rows) {
                float now[V];
                widen(in[t], now);
                R out;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    float sum = bias[j];
#pragma unroll
                    for (int i = 0; i < W - 1; ++i) sum = fmaf(w[i][j], past[i][j], sum);
                    sum = fmaf(w[W - 1][j], now[j], sum);
                    out.v[j] = (T)(a.act == MOE_ACT_SILU ? silu(sum) : sum);
#pragma unroll
                    for (int i = 0; i + 1 < W - 1; ++i) past[i][j] = past[i + 1][j];
                    past[W - 2][j] = now[j];
                }
                *reinterpret_cast<R*>(y + (t0 + t) * a.y_ld) = out;
            }
        }
    }
    if (piece == 0 && state) {
        // the last W - 1 of the slot's rows and the sequence's
        const int64_t len = hi - lo;
        R next[W - 1];
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
            const int64_t at = len - (W - 1) + i;
            if (at >= 0) {
                next[i] = *reinterpret_cast<const R*>(x + at * a.x_ld);
            } else {
#pragma unroll
                for (int j = 0; j < W - 1; ++j)
                    if (j == at + W - 1) next[i] = old[j];
            }
        }
#pragma unroll
        for (int i = 0; i < W - 1; ++i) *reinterpret_cast<R*>(state + (int64_t)i * a.channels) = next[i];
    }
}

template <typename T, int V>
cudaError_t launch_width(const ConvArgs& a, int width, cudaStream_t st) {
    const dim3 grid((unsigned)a.q.pieces(kTile), (unsigned)((a.channels + kThreads * V - 1) / (kThreads * V)));
    switch (width) {
        case 2: return launch(conv_kernel<T, V, 2>, grid, kThreads, 0, st, 1, a);
        case 3: return launch(conv_kernel<T, V, 3>, grid, kThreads, 0, st, 1, a);
        default: return launch(conv_kernel<T, V, 4>, grid, kThreads, 0, st, 1, a);
    }
}

template <typename T>
cudaError_t launch_type(const ConvArgs& a, int width, cudaStream_t st) {
    constexpr int V = 16 / (int)sizeof(T);
    const bool wide = a.channels % V == 0 && a.x_ld % V == 0 && a.y_ld % V == 0 &&
                      (reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.y) |
                       reinterpret_cast<uintptr_t>(a.state)) % 16 == 0;
    return wide ? launch_width<T, V>(a, width, st) : launch_width<T, 1>(a, width, st);
}

}  // namespace

cudaError_t launch_conv(const Seqs& q, const void* x, int type, int64_t x_ld, int channels, const void* w, int w_type,
                        int width, const float* bias, int act, void* state, void* y, int64_t y_ld, cudaStream_t st) {
    ConvArgs a{q, x, w, bias, state, y, x_ld, y_ld, channels, act, w_type == MOE_BF16};
    return type == MOE_BF16 ? launch_type<__nv_bfloat16>(a, width, st) : launch_type<float>(a, width, st);
}

}  // namespace moe
