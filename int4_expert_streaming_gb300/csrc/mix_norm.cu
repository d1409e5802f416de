// mix_norm.cu -- norms of heads with the position rotation or a gate.
#include <string.h>

#include "mix.h"

namespace moe {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kThreads = 256;
constexpr int kTable = 4096;  // angles of a CTA at most

struct NormArgs {
    moe_head_norm_config c;
    moe_heads a, b;
    const int32_t* pos;
    const float* inv_freq;
    int64_t rows;   // T * heads
    int heads;      // a's and b's
    int per_block;  // rows of a CTA
};

// sin and cos of pos * f: the product is reduced to a part of a turn in fp64
// (a few operations an angle; relative to 2^31 turns that leaves 2^-21), the
// rest is fp32.
__device__ __forceinline__ float2 turn(int pos, float f) {
    double t = (double)pos * ((double)f * 0.15915494309189535);
    t -= rint(t);
    float2 r;
    sincospif(2.0f * (float)t, &r.y, &r.x);
    return r;
}

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[2 * j] = __uint_as_float(w[j] << 16);
        v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// E values of a head for each thread, P for each load: E = P * chunks, and the
// chunk i of lane l begins at (l + LANES * i) * P.
template <typename T, int P>
struct Piece;
template <typename T>
struct Piece<T, 8> {
    static __device__ __forceinline__ void load(const T* p, float (&v)[8]) { load8(p, v); }
    static __device__ __forceinline__ void store(T* p, const float (&v)[8]) { store8(p, v); }
};
template <typename T>
struct Piece<T, 1> {
    static __device__ __forceinline__ void load(const T* p, float (&v)[1]) { v[0] = (float)*p; }
    static __device__ __forceinline__ void store(T* p, const float (&v)[1]) { *p = (T)v[0]; }
};

// LANES threads take one head, in CH chunks of P values each: P = 8 where every
// address allows wide loads, one value otherwise (then also rotations whose
// halves are not a multiple of 8).  The partner of a rotated value is read
// again (it is in the first-level cache) rather than passed between threads.
// All reads of a head come before its first write, so y may be x.  sin and cos
// are found once for each token of a CTA, for all its heads.  Bound by memory.
template <typename T, int LANES, int CH, int P>
__global__ void __launch_bounds__(kThreads) norm_kernel(const __grid_constant__ NormArgs g) {
    extern __shared__ float2 table[];  // [token of the CTA][pair]
    after_previous();
    let_next_start();
    const int64_t row0 = (int64_t)blockIdx.x * g.per_block;
    const int64_t end = row0 + g.per_block < g.rows ? row0 + g.per_block : g.rows;
    const int64_t token0 = row0 / g.heads;
    const int half = g.c.rot_dim / 2, D = g.c.dim;
    if (half) {
        const int tokens = (int)((end - 1) / g.heads - token0) + 1;
        for (int i = threadIdx.x; i < tokens * half; i += kThreads)
            table[i] = turn(g.pos[token0 + i / half], g.inv_freq[i % half]);
        __syncthreads();
    }
    const int lane = threadIdx.x % LANES;
    const int first = (int)(row0 - token0 * g.heads);
    for (int r = threadIdx.x / LANES; r < g.per_block; r += kThreads / LANES) {
        const bool there = row0 + r < end;
        // rows past the last redo the last one's sums: every thread of a warp takes part in the shuffles
        const int at = first + (there ? r : (int)(end - 1 - row0));
        const int token = at / g.heads;
        int h = at - token * g.heads;
        const moe_heads& t = h < g.a.heads ? g.a : g.b;
        h -= h < g.a.heads ? 0 : g.a.heads;
        const T* x = static_cast<const T*>(t.x_dev) + (token0 + token) * t.x_ld + h * t.x_head;
        float v[CH][P], sum = 0;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int e = (lane + LANES * i) * P;
#pragma unroll
            for (int j = 0; j < P; ++j) v[i][j] = 0;
            if (e < D) Piece<T, P>::load(x + e, v[i]);
#pragma unroll
            for (int j = 0; j < P; ++j) sum = fmaf(v[i][j], v[i][j], sum);
        }
        float factor = 1;
        if (g.c.norm != MOE_NORM_NONE) {
#pragma unroll
            for (int d = LANES / 2; d; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
            factor = 1.0f / sqrtf((g.c.norm == MOE_NORM_RMS ? sum / (float)D : sum) + g.c.eps);
        }
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int e = (lane + LANES * i) * P;
            if (e >= D) continue;
            float w[P];
            if (t.weight_dev) Piece<float, P>::load(t.weight_dev + e, w);
            float o[P];
            auto scaled = [&](float value, float weight) {
                return value * factor * (t.weight_dev ? g.c.weight_offset + weight : 1.0f);
            };
            if (e < g.c.rot_dim && (P == 1 || g.c.pairs == MOE_ROT_HALVES)) {
                // the other value of each pair
                int f;
                bool second;
                if (g.c.pairs == MOE_ROT_HALVES) {
                    second = e >= half;
                    f = second ? e - half : e + half;
                } else {
                    second = e & 1;
                    f = e ^ 1;
                }
                float u[P], wu[P];
                Piece<T, P>::load(x + f, u);
                if (t.weight_dev) Piece<float, P>::load(t.weight_dev + f, wu);
                const int pair = g.c.pairs == MOE_ROT_HALVES ? (second ? f : e) : e / 2;
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    const float2 cs = table[token * half + pair + j];
                    const float z = scaled(v[i][j], w[j]), other = scaled(u[j], wu[j]);
                    o[j] = fmaf(z, cs.x, second ? other * cs.y : -(other * cs.y));
                }
            } else {
#pragma unroll
                for (int j = 0; j < P; ++j) o[j] = scaled(v[i][j], w[j]);
                if (P > 1 && e < g.c.rot_dim) {
#pragma unroll
                    for (int j = 0; j + 1 < P; j += 2)
                        if (e + j < g.c.rot_dim) {
                            const float2 cs = table[token * half + (e + j) / 2];
                            const float z = o[j], y = o[j + 1];
                            o[j] = fmaf(z, cs.x, -(y * cs.y));
                            o[j + 1] = fmaf(y, cs.x, z * cs.y);
                        }
                }
            }
#pragma unroll
            for (int j = 0; j < P; ++j) v[i][j] = o[j];
        }
        if (t.gate_dev) {
            const T* gate = static_cast<const T*>(t.gate_dev) + (token0 + token) * t.gate_ld + h * t.gate_head;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int e = (lane + LANES * i) * P;
                if (e < D) {
                    float u[P];
                    Piece<T, P>::load(gate + e, u);
#pragma unroll
                    for (int j = 0; j < P; ++j) v[i][j] *= silu(u[j]);
                }
            }
        }
        __syncwarp();  // every lane has read its partners
        if (there) {
            T* y = static_cast<T*>(t.y_dev) + (token0 + token) * t.y_ld + h * t.y_head;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int e = (lane + LANES * i) * P;
                if (e < D) Piece<T, P>::store(y + e, v[i]);
            }
        }
    }
}

template <typename T, int LANES, int CH, int P>
cudaError_t launch_rows(NormArgs& g, cudaStream_t st) {
    constexpr int kPass = kThreads / LANES;  // rows a CTA has under way
    const int half = g.c.rot_dim / 2;
    // Few rows: one pass a CTA, so that more of them start at once.
    int passes = g.rows >= (int64_t)kPass * 152 * 8 ? 4 : 1;
    auto angles = [&](int p) {
        const int rows = p * kPass, tokens = rows / g.heads + 2;
        return (tokens < rows ? tokens : rows) * half;
    };
    while (passes > 1 && angles(passes) > kTable) passes >>= 1;
    g.per_block = passes * kPass;
    const unsigned grid = (unsigned)((g.rows + g.per_block - 1) / g.per_block);
    return launch(norm_kernel<T, LANES, CH, P>, dim3(grid), kThreads, (size_t)angles(passes) * sizeof(float2), st, 1, g);
}

template <typename T>
bool wide(const moe_heads& t, int D) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(t.x_dev) | reinterpret_cast<uintptr_t>(t.y_dev) |
                         reinterpret_cast<uintptr_t>(t.gate_dev) | reinterpret_cast<uintptr_t>(t.weight_dev);
    const int64_t n = t.x_ld | t.x_head | t.y_ld | t.y_head | (t.gate_dev ? t.gate_ld | t.gate_head : 0);
    return D % 8 == 0 && at % 16 == 0 && n % (16 / (int)sizeof(T)) == 0;
}

template <typename T>
cudaError_t launch_type(NormArgs& g, bool second, cudaStream_t st) {
    const int D = g.c.dim;
    const bool halves = g.c.pairs == MOE_ROT_ADJACENT || g.c.rot_dim % 16 == 0;
    if (halves && wide<T>(g.a, D) && (!second || wide<T>(g.b, D))) {
        if (D <= 64) return launch_rows<T, 8, 1, 8>(g, st);
        if (D <= 128) return launch_rows<T, 16, 1, 8>(g, st);
        if (D <= 256) return launch_rows<T, 32, 1, 8>(g, st);
        return launch_rows<T, 32, 2, 8>(g, st);
    }
    if (D <= 128) return launch_rows<T, 32, 4, 1>(g, st);
    return launch_rows<T, 32, 16, 1>(g, st);
}

}  // namespace

cudaError_t launch_head_norm(const moe_head_norm_config& c, const moe_heads& a, const moe_heads* b, const int32_t* pos,
                             const float* inv_freq, int64_t T, cudaStream_t st) {
    NormArgs g{c, a, b ? *b : moe_heads{}, pos, inv_freq, T * (a.heads + (b ? b->heads : 0)),
               a.heads + (b ? b->heads : 0), 0};
    return a.type == MOE_BF16 ? launch_type<__nv_bfloat16>(g, b != nullptr, st) : launch_type<float>(g, b != nullptr, st);
}

}  // namespace moe
