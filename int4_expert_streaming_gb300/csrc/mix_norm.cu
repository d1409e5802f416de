// mix_norm.cu -- norms of heads with the position rotation or a gate.
#include <string.h>

#include "mix.h"

namespace moe {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kThreads = 256;

struct NormArgs {
    moe_head_norm_config c;
    moe_heads a, b;
    const int32_t* pos;
    const float* inv_freq;
    int64_t T;
    uint32_t inverse_a, inverse_b;  // 2^32 / heads, rounded up
    unsigned first_blocks;          // the CTAs with heads of a
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

// P consecutive values as they are in memory
template <typename T, int P>
struct Raw {
    uint32_t w[P * sizeof(T) / 4 ? P * sizeof(T) / 4 : 1];
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (P == 1) {
            if constexpr (sizeof(T) == 4)
                w[0] = __float_as_uint(*reinterpret_cast<const float*>(p));
            else
                w[0] = (uint32_t)*reinterpret_cast<const unsigned short*>(p) << 16;
        } else {
#pragma unroll
            for (int i = 0; i < (int)(P * sizeof(T)) / 16; ++i)
                reinterpret_cast<uint4*>(w)[i] = reinterpret_cast<const uint4*>(p)[i];
        }
    }
    __device__ __forceinline__ void get(float (&v)[P]) const {
        if constexpr (P == 1) {
            v[0] = __uint_as_float(w[0]);
        } else if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < P; ++i) v[i] = __uint_as_float(w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < P / 2; ++i) {
                v[2 * i] = __uint_as_float(w[i] << 16);
                v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        }
    }
};
template <typename T, int P>
__device__ __forceinline__ void store(T* p, const float (&v)[P]) {
    if constexpr (P == 1) {
        *p = (T)v[0];
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < P / 4; ++i)
            reinterpret_cast<float4*>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    } else {
        uint32_t w[P / 2];
#pragma unroll
        for (int i = 0; i < P / 2; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
#pragma unroll
        for (int i = 0; i < P / 8; ++i)
            reinterpret_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
}

// LANES threads take one head, in CH chunks of P values each (chunk i of lane l
// begins at (l + LANES * i) * P): P = 8 where every address allows wide loads,
// one value otherwise (then also rotations whose halves are not a multiple of
// 8).  They take U heads at a time, all of whose loads are under way together.
// A CTA has heads of one tensor only; its lanes keep their part of the weights.
// The partner of a rotated value comes from its lane (CH = 1), else it is read
// again.  All reads of a head come before its first write, so y may be x.  sin
// and cos are found once for each token of a CTA, for all its heads, behind the
// loads.  Bound by memory.
template <typename T, int LANES, int CH, int P, int U, bool ROT, bool GATE>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 && U > 1 && !GATE ? 4 : 1) norm_kernel(const __grid_constant__ NormArgs g) {
    extern __shared__ float2 table[];  // [token of the CTA][pair]
    after_previous();
    let_next_start();
    constexpr int kPass = kThreads / LANES;
    const bool second = blockIdx.x >= g.first_blocks;
    const moe_heads& t = second ? g.b : g.a;
    const uint32_t inverse = second ? g.inverse_b : g.inverse_a;  // of the heads, 32 bits behind the point, rounded up
    const int64_t row0 = (int64_t)(blockIdx.x - (second ? g.first_blocks : 0)) * (kPass * U), rows = g.T * t.heads;
    const int here = (int)(rows - row0 < kPass * U ? rows - row0 : kPass * U);
    const int64_t token0 = row0 / t.heads;
    const int half = g.c.rot_dim / 2, D = g.c.dim, lane = threadIdx.x % LANES;
    const int first = (int)(row0 - token0 * t.heads);

    // token (of the CTA's) and head of a thread's u-th row; rows past the last redo the last one's sums: every thread of a
    // warp takes part in the shuffles.  Found again where needed: it is two instructions, and registers are CTAs
    auto place = [&](int u, int& token, int& h) {
        const int r = threadIdx.x / LANES + u * kPass;
        const uint32_t at = first + (r < here ? r : here - 1);  // below heads + 128, so the product is exact
        token = t.heads == 1 ? at : __umulhi(at, inverse);
        h = at - token * t.heads;
    };
    Raw<T, P> x[U][CH], gate[U][CH];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        int token, h;
        place(u, token, h);
        const T* from = static_cast<const T*>(t.x_dev) + (token0 + token) * t.x_ld + h * t.x_head;
        const T* gfrom = static_cast<const T*>(t.gate_dev) + (token0 + token) * t.gate_ld + h * t.gate_head;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int e = (lane + LANES * i) * P;
            memset(&x[u][i], 0, sizeof x[u][i]);
            if (e < D) {
                x[u][i].load(from + e);
                if (GATE && t.gate_dev) gate[u][i].load(gfrom + e);
            }
        }
    }
    float w[CH][P];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int e = (lane + LANES * i) * P;
#pragma unroll
        for (int j = 0; j < P; ++j) w[i][j] = 1;
        if (t.weight_dev && e < D) {
            Raw<float, P> r;
            r.load(t.weight_dev + e);
            r.get(w[i]);
#pragma unroll
            for (int j = 0; j < P; ++j) w[i][j] += g.c.weight_offset;
        }
    }
    if (ROT) {
        const int tokens = (first + here - 1) / t.heads + 1;
        for (int i = threadIdx.x; i < tokens * half; i += kThreads)
            table[i] = turn(g.pos[token0 + i / half], g.inv_freq[i % half]);
        __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        int token, h;
        place(u, token, h);
        float v[CH][P], sum = 0;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            x[u][i].get(v[i]);
#pragma unroll
            for (int j = 0; j < P; ++j) sum = fmaf(v[i][j], v[i][j], sum);
        }
        float factor = 1;
        if (g.c.norm != MOE_NORM_NONE) {
#pragma unroll
            for (int d = LANES / 2; d; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
            factor = rsqrtf((g.c.norm == MOE_NORM_RMS ? sum / (float)D : sum) + g.c.eps);
        }
#pragma unroll
        for (int i = 0; i < CH; ++i)
#pragma unroll
            for (int j = 0; j < P; ++j) v[i][j] = v[i][j] * factor * w[i][j];
        if constexpr (ROT) {
            const float2* cs = table + token * half;
            if (P > 1 && g.c.pairs == MOE_ROT_ADJACENT) {
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    const int e = (lane + LANES * i) * P;
#pragma unroll
                    for (int j = 0; j + 1 < P; j += 2)
                        if (e + j < g.c.rot_dim) {
                            const float2 r = cs[(e + j) / 2];
                            const float p = v[i][j], q = v[i][j + 1];
                            v[i][j] = fmaf(p, r.x, -(q * r.y));
                            v[i][j + 1] = fmaf(q, r.x, p * r.y);
                        }
                }
            } else if constexpr (CH == 1 && P > 1) {
                const int e = lane * P;
                const bool upper = e >= half;
                const int partner = (upper ? e - half : e + half) / P;
                float q[P];
#pragma unroll
                for (int j = 0; j < P; ++j) q[j] = __shfl_sync(kAll, v[0][j], partner, LANES);
                if (e < g.c.rot_dim) {
                    const float4* r = reinterpret_cast<const float4*>(cs + (upper ? e - half : e));
#pragma unroll
                    for (int j = 0; j < P; j += 2) {
                        const float4 f = r[j / 2];
                        v[0][j] = fmaf(v[0][j], f.x, upper ? q[j] * f.y : -(q[j] * f.y));
                        v[0][j + 1] = fmaf(v[0][j + 1], f.z, upper ? q[j + 1] * f.w : -(q[j + 1] * f.w));
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    const int e = (lane + LANES * i) * P;
                    if (e >= g.c.rot_dim) continue;
                    const bool halves = g.c.pairs == MOE_ROT_HALVES, upper = halves ? e >= half : e & 1;
                    const int f = halves ? (upper ? e - half : e + half) : e ^ 1;
                    const int pair = halves ? (upper ? f : e) : e / 2;
                    Raw<T, P> other;
                    Raw<float, P> wr;
                    float q[P], wq[P];
                    other.load(static_cast<const T*>(t.x_dev) + (token0 + token) * t.x_ld + h * t.x_head + f);
                    other.get(q);
                    if (t.weight_dev) wr.load(t.weight_dev + f), wr.get(wq);
#pragma unroll
                    for (int j = 0; j < P; ++j) {
                        const float2 r = cs[pair + j];
                        q[j] *= factor * (t.weight_dev ? g.c.weight_offset + wq[j] : 1.0f);
                        v[i][j] = fmaf(v[i][j], r.x, upper ? q[j] * r.y : -(q[j] * r.y));
                    }
                }
                __syncwarp();  // every lane has read its partners
            }
        }
        if (GATE && t.gate_dev) {
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                float z[P];
                gate[u][i].get(z);
#pragma unroll
                for (int j = 0; j < P; ++j) v[i][j] *= sizeof(T) == 2 ? silu_bf16(z[j]) : silu(z[j]);
            }
        }
        if (threadIdx.x / LANES + u * kPass < here) {
            T* y = static_cast<T*>(t.y_dev) + (token0 + token) * t.y_ld + h * t.y_head;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int e = (lane + LANES * i) * P;
                if (e < D) store<T, P>(y + e, v[i]);
            }
        }
    }
}

template <typename T, int LANES, int CH, int P, int U, bool ROT, bool GATE>
cudaError_t launch_heads(NormArgs& g, cudaStream_t st) {
    constexpr int kRows = kThreads / LANES * U;  // heads of a CTA
    auto tokens = [](int heads) { return heads == 0 ? 0 : kRows / heads + 2 < kRows ? kRows / heads + 2 : kRows; };
    const int most = tokens(g.a.heads) > tokens(g.b.heads) ? tokens(g.a.heads) : tokens(g.b.heads);
    const size_t table = ROT ? (size_t)most * (g.c.rot_dim / 2) * sizeof(float2) : 0;
    g.first_blocks = (unsigned)((g.T * g.a.heads + kRows - 1) / kRows);
    const unsigned grid = g.first_blocks + (unsigned)((g.T * g.b.heads + kRows - 1) / kRows);
    return launch(norm_kernel<T, LANES, CH, P, U, ROT, GATE>, dim3(grid), kThreads, table, st, 1, g);
}

// Few heads: one at a time, so that more CTAs start at once.
template <typename T, int LANES, int CH, int P>
cudaError_t launch_rows(NormArgs& g, cudaStream_t st) {
    constexpr int kMany = CH == 1 && P > 1 ? 4 : 1;
    const bool many = g.T * (g.a.heads + g.b.heads) >= (int64_t)(kThreads / LANES) * 152 * 8;
    const bool gate = g.a.gate_dev || g.b.gate_dev;
    if (g.c.rot_dim) {
        if (gate) return launch_heads<T, LANES, CH, P, 1, true, true>(g, st);
        return many ? launch_heads<T, LANES, CH, P, kMany, true, false>(g, st) : launch_heads<T, LANES, CH, P, 1, true, false>(g, st);
    }
    if (gate)
        return many ? launch_heads<T, LANES, CH, P, kMany, false, true>(g, st) : launch_heads<T, LANES, CH, P, 1, false, true>(g, st);
    return many ? launch_heads<T, LANES, CH, P, kMany, false, false>(g, st) : launch_heads<T, LANES, CH, P, 1, false, false>(g, st);
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
    auto inverse = [](int heads) { return (uint32_t)((UINT64_C(1) << 32) / heads + 1); };
    NormArgs g{c, a, b ? *b : moe_heads{}, pos, inv_freq, T, inverse(a.heads), b ? inverse(b->heads) : 0, 0};
    return a.type == MOE_BF16 ? launch_type<__nv_bfloat16>(g, b != nullptr, st) : launch_type<float>(g, b != nullptr, st);
}

}  // namespace moe
