// mix_conv.cu -- short causal convolution of each channel, with the last rows
// of a sequence kept in its slot.
#include <string.h>

#include "mix.h"

namespace moe {
namespace {

constexpr int kThreads = 128;
constexpr int kAhead = 8;  // rows that are summed at a time
// Rows of a CTA's piece of a sequence, which reads the W - 1 rows before it again.  bf16, 4096 x 8192, four channels a
// thread: 30.0 us with 16, 34.0 with 32 (fewer CTAs find room).  fp32, 5003 x 1283, one channel a thread: 12.9 and 12.0.
__host__ __device__ constexpr int tile_rows(int V) { return V > 1 ? 16 : 32; }

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
struct alignas(sizeof(T) * V % 16 == 0 ? 16 : sizeof(T) * V % 8 == 0 ? 8 : sizeof(T)) Row {
    T v[V];
};
template <typename T, int V>
__device__ __forceinline__ void widen(const Row<T, V>& r, float (&f)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = (float)r.v[i];
}

// What weights and bias, and so the sums, are taken times: bf16 sums that silu follows are 2^-8 of what they stand for, as
// sigmoid_256 wants them.
template <typename T, bool SILU>
constexpr float kPart = SILU && sizeof(T) == 2 ? 1.0f / 256 : 1.0f;
template <typename T, bool SILU>
__device__ __forceinline__ float activated(float v) {
    return !SILU ? v : sizeof(T) == 2 ? v * sigmoid_256<256>(v) : silu(v);
}

// the weights of V channels, which stand one after another
template <typename T, int V, int W>
__device__ __forceinline__ void load_weights(float (&w)[W][V], const void* from, int c, float part) {
    Row<T, V * W> r;
    constexpr int kPart = V * W * sizeof(T) % 8 ? 1 : 8 / (int)sizeof(T);  // wide where c is a multiple of V: 8 bytes
    const T* p = static_cast<const T*>(from) + (int64_t)c * W;
    if (kPart > 1 && reinterpret_cast<uintptr_t>(p) % 8 == 0) {
#pragma unroll
        for (int i = 0; i < V * W / kPart; ++i)
            reinterpret_cast<Row<T, kPart>*>(r.v)[i] = reinterpret_cast<const Row<T, kPart>*>(p)[i];
    } else {
#pragma unroll
        for (int i = 0; i < V * W; ++i) r.v[i] = p[i];
    }
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
        for (int i = 0; i < W; ++i) w[i][j] = part * (float)r.v[j * W + i];
}

// A thread takes V channels (8 bytes, or one where rows are not aligned) down
// a piece of rows, the last W - 1 inputs in registers.  Wide rows are copied to
// shared memory, all of a piece at once, where each thread finds what it has
// itself copied: the loads under way are then not limited by registers.  bf16,
// 4096 x 8192: 30.4 us, 4.4 TB/s (65% of the measured copy's rate), with 61% of the
// issue slots used, for 18 instructions a value (silu's five, four products, the
// rest to load, convert and store); neither is used up, and six warps a
// scheduler do not cover every load's latency.  The first piece's CTAs read the
// old state and also write the new one, so no two CTAs touch a slot's channel.
template <typename T, int V, int W, bool SILU>
__global__ void __launch_bounds__(kThreads) conv_kernel(const __grid_constant__ ConvArgs a) {
    using R = Row<T, V>;
    constexpr bool kCopy = V > 1;
    constexpr int kTile = tile_rows(V);
    __shared__ R ring[kCopy ? kTile : 1][kThreads];
    after_previous();
    let_next_start();
    int piece;
    const int s = a.q.find<kTile>(blockIdx.x, piece);
    const int64_t lo = a.q.start(s), hi = a.q.start(s + 1), first = lo + (int64_t)piece * kTile;
    const int slot = a.q.slot(s);
    const bool carry = a.state && a.q.carry(s);
    const int c = (blockIdx.y * kThreads + threadIdx.x) * V;
    if (piece < 0 || first >= hi || slot < 0 || c >= a.channels) return;
    const int rows = (int)(hi - first < kTile ? hi - first : kTile);

    const T* x = static_cast<const T*>(a.x) + first * a.x_ld + c;
    if constexpr (kCopy) {
        const T* from = x;
        uint32_t to = (uint32_t)__cvta_generic_to_shared(&ring[0][threadIdx.x]);
#pragma unroll
        for (int group = 0; group < kTile / kAhead; ++group) {
            if (group * kAhead < rows) {
#pragma unroll
                for (int t = 0; t < kAhead; ++t, from += a.x_ld, to += sizeof(ring[0]))
                    if (group * kAhead + t < rows)
                        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(from) : "memory");
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    }
    float w[W][V], bias[V], past[W - 1][V];
    if (a.w_bf16)
        load_weights<__nv_bfloat16, V, W>(w, a.w, c, kPart<T, SILU>);
    else
        load_weights<float, V, W>(w, a.w, c, kPart<T, SILU>);
#pragma unroll
    for (int j = 0; j < V; ++j) bias[j] = a.bias ? kPart<T, SILU> * a.bias[c + j] : 0.0f;

    T* y = static_cast<T*>(a.y) + first * a.y_ld + c;
    T* state = a.state ? static_cast<T*>(a.state) + (int64_t)slot * (W - 1) * a.channels + c : nullptr;
    R old[W - 1];  // the rows before the piece, oldest first
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
        memset(&old[i], 0, sizeof(R));
        if (piece > 0)
            old[i] = *reinterpret_cast<const R*>(x + (i - (W - 1)) * a.x_ld);
        else if (carry)
            old[i] = *reinterpret_cast<const R*>(state + (int64_t)i * a.channels);
        widen(old[i], past[i]);
    }
#pragma unroll
    for (int group = 0; group < kTile / kAhead; ++group) {
        const int t0 = group * kAhead;
        if (t0 >= rows) break;
        R in[kAhead];
        if constexpr (kCopy) {
            // all groups but the ones after this
            constexpr int kGroups = kTile / kAhead;
            static_assert(kGroups <= 4, "a wait for each group");
            if (group == kGroups - 1) asm volatile("cp.async.wait_group 0;" ::: "memory");
            if (group == kGroups - 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
            if (group == kGroups - 3) asm volatile("cp.async.wait_group 2;" ::: "memory");
            if (group == kGroups - 4) asm volatile("cp.async.wait_group 3;" ::: "memory");
#pragma unroll
            for (int t = 0; t < kAhead; ++t) in[t] = ring[t0 + t][threadIdx.x];
        } else {
#pragma unroll
            for (int t = 0; t < kAhead; ++t)
                if (t0 + t < rows) in[t] = *reinterpret_cast<const R*>(x + (t0 + t) * a.x_ld);
        }
        float win[W - 1 + kAhead][V];  // and the rows before
#pragma unroll
        for (int t = 0; t < W - 1; ++t)
#pragma unroll
            for (int j = 0; j < V; ++j) win[t][j] = past[t][j];
#pragma unroll
        for (int t = 0; t < kAhead; ++t, y += a.y_ld) {
            widen(in[t], win[W - 1 + t]);
            if (t0 + t >= rows) continue;
            R out;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float sum = bias[j];
#pragma unroll
                for (int i = 0; i < W; ++i) sum = fmaf(w[i][j], win[t + i][j], sum);
                out.v[j] = (T)activated<T, SILU>(sum);
            }
            *reinterpret_cast<R*>(y) = out;
        }
#pragma unroll
        for (int t = 0; t < W - 1; ++t)
#pragma unroll
            for (int j = 0; j < V; ++j) past[t][j] = win[kAhead + t][j];
    }
    if (piece == 0 && state) {
        // the last W - 1 of the slot's rows and the sequence's
        const int64_t len = hi - lo;
        R last[W - 1];
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
            const int64_t at = len - (W - 1) + i;
            if (at >= 0) {
                last[i] = *reinterpret_cast<const R*>(x + at * a.x_ld);
            } else {
#pragma unroll
                for (int j = 0; j < W - 1; ++j)
                    if (j == at + W - 1) last[i] = old[j];
            }
        }
#pragma unroll
        for (int i = 0; i < W - 1; ++i) *reinterpret_cast<R*>(state + (int64_t)i * a.channels) = last[i];
    }
}

// A batch in which every row is a sequence: a thread takes V channels of one.  What does not depend on the slot is loaded
// before that is known.  64 rows of 8192 channels, bf16: 3.4 us a call, 6.5 by the kernel above.
template <typename T, int V, int W, bool SILU>
__global__ void __launch_bounds__(kThreads) conv_step_kernel(const __grid_constant__ ConvArgs a) {
    using R = Row<T, V>;
    after_previous();
    const int s = blockIdx.x, c = (blockIdx.y * kThreads + threadIdx.x) * V;
    if (c >= a.channels) return;
    const int slot = a.q.slot(s);
    const bool carry = a.state && a.q.carry(s);
    const R in = *reinterpret_cast<const R*>(static_cast<const T*>(a.x) + s * a.x_ld + c);
    float w[W][V], rows[W][V];
    if (a.w_bf16)
        load_weights<__nv_bfloat16, V, W>(w, a.w, c, kPart<T, SILU>);
    else
        load_weights<float, V, W>(w, a.w, c, kPart<T, SILU>);
    float bias[V];
#pragma unroll
    for (int j = 0; j < V; ++j) bias[j] = a.bias ? kPart<T, SILU> * a.bias[c + j] : 0.0f;
    if (slot < 0) return;
    T* state = a.state ? static_cast<T*>(a.state) + (int64_t)slot * (W - 1) * a.channels + c : nullptr;
    R old[W - 1];
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
        memset(&old[i], 0, sizeof(R));
        if (carry) old[i] = *reinterpret_cast<const R*>(state + (int64_t)i * a.channels);
        widen(old[i], rows[i]);
    }
    widen(in, rows[W - 1]);
    R out;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        float sum = bias[j];
#pragma unroll
        for (int i = 0; i < W; ++i) sum = fmaf(w[i][j], rows[i][j], sum);
        out.v[j] = (T)activated<T, SILU>(sum);
    }
    *reinterpret_cast<R*>(static_cast<T*>(a.y) + s * a.y_ld + c) = out;
    let_next_start();  // not earlier: 64 x 8192 in a chain of calls 3.4 us, at the kernel's start 4.4
    if (state) {
#pragma unroll
        for (int i = 0; i + 1 < W - 1; ++i) *reinterpret_cast<R*>(state + (int64_t)i * a.channels) = old[i + 1];
        *reinterpret_cast<R*>(state + (int64_t)(W - 2) * a.channels) = in;
    }
}

template <typename T, int V, int W>
cudaError_t launch_act(const ConvArgs& a, cudaStream_t st) {
    const unsigned columns = (unsigned)((a.channels + kThreads * V - 1) / (kThreads * V));
    if (!a.q.offsets && a.q.per == 1) {
        const dim3 grid((unsigned)a.q.n, columns);
        if (a.act == MOE_ACT_SILU) return launch(conv_step_kernel<T, V, W, true>, grid, kThreads, 0, st, 1, a);
        return launch(conv_step_kernel<T, V, W, false>, grid, kThreads, 0, st, 1, a);
    }
    const dim3 grid((unsigned)a.q.pieces(tile_rows(V)), columns);
    if (a.act == MOE_ACT_SILU) return launch(conv_kernel<T, V, W, true>, grid, kThreads, 0, st, 1, a);
    return launch(conv_kernel<T, V, W, false>, grid, kThreads, 0, st, 1, a);
}

template <typename T, int V>
cudaError_t launch_width(const ConvArgs& a, int width, cudaStream_t st) {
    if (width == 2) return launch_act<T, V, 2>(a, st);
    if (width == 3) return launch_act<T, V, 3>(a, st);
    return launch_act<T, V, 4>(a, st);
}

template <typename T>
cudaError_t launch_type(const ConvArgs& a, int width, cudaStream_t st) {
    constexpr int V = 8 / (int)sizeof(T);
    const bool wide = a.channels % V == 0 && a.x_ld % V == 0 && a.y_ld % V == 0 &&
                      (reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.y) |
                       reinterpret_cast<uintptr_t>(a.state)) % 8 == 0;
    return wide ? launch_width<T, V>(a, width, st) : launch_width<T, 1>(a, width, st);
}

}  // namespace

cudaError_t launch_conv(const Seqs& q, const void* x, int type, int64_t x_ld, int channels, const void* w, int w_type,
                        int width, const float* bias, int act, void* state, void* y, int64_t y_ld, cudaStream_t st) {
    ConvArgs a{q, x, w, bias, state, y, x_ld, y_ld, channels, act, w_type == MOE_BF16};
    return type == MOE_BF16 ? launch_type<__nv_bfloat16>(a, width, st) : launch_type<float>(a, width, st);
}

}  // namespace moe
