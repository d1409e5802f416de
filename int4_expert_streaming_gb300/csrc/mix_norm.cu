// mix_norm.cu -- norms of heads with the position rotation or a gate.
#include <string.h>

#include "mix.h"

namespace moe {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kThreads = 256;
constexpr int kHalves = 1, kAdjacent = 2;  // rotations

struct NormArgs {
    moe_head_norm_config c;
    moe_heads a, b;
    const int32_t* pos;
    const float* inv_freq;
    int64_t T;
    uint32_t inverse_a, inverse_b;  // 2^32 / heads, rounded up
    unsigned first_blocks;          // the CTAs with heads of a
    float part;                     // of the sum of squares in the norm: 1 / dim, or 1
};

// sin and cos of pos * f.  The angle in turns is reduced to a part of one
// before it is rounded: pos f / 2 pi as a sum of two fp32, exact to 2^-26 of a
// turn up to the 16 millionth position and f of 1; beyond, in fp64, whose few
// operations cost as much as the rest of the kernel where every angle takes them.
__device__ __forceinline__ float2 turn(int pos, float f) {
    constexpr double kTurns = 0.15915494309189535;  // 1 / 2 pi
    constexpr float kHigh = (float)kTurns, kRest = (float)(kTurns - (double)kHigh);
    float t;
    if ((uint32_t)pos + (1u << 24) <= 1u << 25 && fabsf(f) <= 1.0f) {
        const float p = (float)pos, high = f * kHigh, rest = fmaf(f, kHigh, -high) + f * kRest;
        const float whole = p * high;
        t = (whole - rintf(whole)) + fmaf(p, rest, fmaf(p, high, -whole));
        t -= rintf(t);
    } else {
        double d = (double)pos * ((double)f * kTurns);
        t = (float)(d - rint(d));
    }
    float2 r;
    sincospif(2.0f * t, &r.y, &r.x);
    return r;
}

// P consecutive values as they are in memory: one, four or eight
template <typename T, int P>
struct Raw {
    static constexpr int kWords = P == 1 ? 1 : P * (int)sizeof(T) / 4;
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (P == 1) {
            if constexpr (sizeof(T) == 4)
                w[0] = __float_as_uint(*reinterpret_cast<const float*>(p));
            else
                w[0] = (uint32_t)*reinterpret_cast<const unsigned short*>(p) << 16;
        } else if constexpr (kWords == 2) {
            const uint2 q = *reinterpret_cast<const uint2*>(p);
            w[0] = q.x, w[1] = q.y;
        } else {
#pragma unroll
            for (int i = 0; i < kWords; i += 4) {
                const uint4 q = reinterpret_cast<const uint4*>(p)[i / 4];
                w[i] = q.x, w[i + 1] = q.y, w[i + 2] = q.z, w[i + 3] = q.w;
            }
        }
    }
    // as pairs; one value with a zero
    __device__ __forceinline__ void get2(f32x2* v) const {
        if constexpr (P == 1) {
            v[0] = both(__uint_as_float(w[0]), 0.0f);
        } else if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < P / 2; ++i) v[i] = both(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
        } else {
#pragma unroll
            for (int i = 0; i < P / 2; ++i) v[i] = both_of(w[i]);
        }
    }
    __device__ __forceinline__ void get(float* v) const {
        if constexpr (P == 1 || sizeof(T) == 4) {
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
__device__ __forceinline__ void store(T* p, const float* v) {
    if constexpr (P == 1) {
        *p = (T)v[0];
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < P; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    } else {
        uint32_t w[P / 2];
#pragma unroll
        for (int i = 0; i < P / 2; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
        if constexpr (P == 4)
            *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        else
            *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// LANES threads take one head, in CH chunks of P values each.  P = 8 where
// every address allows wide loads: a chunk is eight values in a row, but in the
// part that turns by halves two pieces of four, the same place of both halves,
// so that pairs meet in a thread.  P = 1
// otherwise (then also rotations whose halves are not a multiple of 4), and the
// partner of a rotated value is read again.  The threads take U heads at a
// time, all of whose loads are under way together.  A CTA has heads of one
// tensor only; its lanes keep their part of the weights.  All reads of a head
// come before its first write, so y may be x.  sin and cos are found once for
// each token of a CTA, for all its heads, behind the loads.  bf16: 4096 tokens of
// 32 gated heads of 128 17.8 us, 83% of the measured copy's rate; of 16 and 2 heads
// of 256, 64 values of them rotated, 18.1 us, 61%, with 68% of the issue slots
// used: neither is used up, and seven warps a scheduler do not cover every load's
// latency and the barrier behind the angles.  P = 1: 4096 tokens of 16 heads of 80, 20
// values of them rotated, 22 us (24 of them, by P = 8: 6.7).  Two or more pieces of work a CTA one after another cost 2 to 11% more.
template <typename T, int LANES, int CH, int P, int U, int ROT, bool GATE>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 && U > 1 ? (GATE ? 3 : 4) : 1)
    norm_kernel(const __grid_constant__ NormArgs g) {
    extern __shared__ float2 table[];  // [token of the CTA][pair]
    after_previous();
    let_next_start();
    constexpr int kPass = kThreads / LANES, kPiece = P == 8 && ROT == kHalves ? 4 : P, kPieces = P / kPiece;
    const bool second = blockIdx.x >= g.first_blocks;
    const moe_heads& t = second ? g.b : g.a;
    const uint32_t inverse = second ? g.inverse_b : g.inverse_a;  // of the heads, 32 bits behind the point, rounded up
    const int64_t row0 = (int64_t)(blockIdx.x - (second ? g.first_blocks : 0)) * (kPass * U), rows = g.T * t.heads;
    const int here = (int)(rows - row0 < kPass * U ? rows - row0 : kPass * U);
    // 64-bit division is a hundred instructions before the first load
    const int64_t token0 = rows <= UINT32_MAX ? (uint32_t)row0 / (uint32_t)t.heads : row0 / t.heads;
    const int half = g.c.rot_dim / 2, D = g.c.dim, lane = threadIdx.x % LANES;
    const int first = (int)(row0 - token0 * t.heads);
    constexpr bool halves = ROT == kHalves;

    // token (of the CTA's) and head of a thread's u-th row; rows past the last redo the last one's sums: every thread of a
    // warp takes part in the shuffles.  Found again where needed: it is two instructions, and registers are CTAs
    auto place = [&](int u, int& token, int& h) {
        const int r = threadIdx.x / LANES + u * kPass;
        const uint32_t at = first + (r < here ? r : here - 1);  // below heads + 128, so the product is exact
        token = t.heads == 1 ? at : __umulhi(at, inverse);
        h = at - token * t.heads;
    };
    // where piece p of chunk i begins
    auto at = [&](int i, int p) {
        const int c = lane + LANES * i;
        if (P == 8 && halves && c < g.c.rot_dim / 8) return 4 * c + p * half;
        return c * P + p * kPiece;
    };
    Raw<T, kPiece> x[U][CH][kPieces], gate[U][CH][kPieces];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        int token, h;
        place(u, token, h);
        const T* from = static_cast<const T*>(t.x_dev) + (token0 + token) * t.x_ld + h * t.x_head;
        const T* gfrom = static_cast<const T*>(t.gate_dev) + (token0 + token) * t.gate_ld + h * t.gate_head;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            memset(&x[u][i], 0, sizeof x[u][i]);
            if ((lane + LANES * i) * P < D) {
#pragma unroll
                for (int p = 0; p < kPieces; ++p) {
                    x[u][i][p].load(from + at(i, p));
                    if (GATE && t.gate_dev) gate[u][i][p].load(gfrom + at(i, p));
                }
            }
        }
    }
    // the lane's part of the weights, two values a register pair
    constexpr int kTwos = P == 1 ? 1 : P / 2;
    f32x2 w[CH][kTwos];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        float f[P];
#pragma unroll
        for (int j = 0; j < P; ++j) f[j] = 1;
        if (t.weight_dev && (lane + LANES * i) * P < D) {
#pragma unroll
            for (int p = 0; p < kPieces; ++p) {
                Raw<float, kPiece> r;
                r.load(t.weight_dev + at(i, p));
                r.get(&f[p * kPiece]);
            }
#pragma unroll
            for (int j = 0; j < P; ++j) f[j] += g.c.weight_offset;
        }
#pragma unroll
        for (int j = 0; j < kTwos; ++j) w[i][j] = both(f[P == 1 ? 0 : 2 * j], P == 1 ? 0.0f : f[2 * j + 1]);
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
        f32x2 v2[CH][kTwos], sum2 = 0;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
#pragma unroll
            for (int p = 0; p < kPieces; ++p) x[u][i][p].get2(&v2[i][p * kPiece / 2]);
#pragma unroll
            for (int j = 0; j < kTwos; ++j) sum2 = fma2(v2[i][j], v2[i][j], sum2);
        }
        float sum = apart(sum2).x + apart(sum2).y, factor = 1;
        if (g.c.norm != MOE_NORM_NONE) {
#pragma unroll
            for (int d = LANES / 2; d; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
            factor = rsqrtf(fmaf(sum, g.part, g.c.eps));
        }
        constexpr bool kParts = GATE && sizeof(T) == 2;  // the gate as 2^8 / (1 + e^-z) times z, and the 2^-8 here
        if (kParts && t.gate_dev) factor *= 1.0f / 256;
        float v[CH][P];
#pragma unroll
        for (int i = 0; i < CH; ++i)
#pragma unroll
            for (int j = 0; j < kTwos; ++j) {
                const float2 f = apart(mul2(mul2(v2[i][j], both(factor, factor)), w[i][j]));
                v[i][P == 1 ? 0 : 2 * j] = f.x;
                if (P > 1) v[i][2 * j + 1] = f.y;
            }
        if constexpr (ROT && P == 8) {
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int c = lane + LANES * i;
                const float2* cs = table + token * half + 4 * c;  // of the chunk's four pairs, either way
                if (halves) {
                    if (c < g.c.rot_dim / 8) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float2 r = cs[j];
                            const float p = v[i][j], q = v[i][4 + j];
                            v[i][j] = fmaf(p, r.x, -(q * r.y));
                            v[i][4 + j] = fmaf(q, r.x, p * r.y);
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (8 * c + 2 * j < g.c.rot_dim) {
                            const float2 r = cs[j];
                            const float p = v[i][2 * j], q = v[i][2 * j + 1];
                            v[i][2 * j] = fmaf(p, r.x, -(q * r.y));
                            v[i][2 * j + 1] = fmaf(q, r.x, p * r.y);
                        }
                }
            }
        } else if constexpr (ROT) {
            const float2* cs = table + token * half;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int e = lane + LANES * i;
                if (e >= g.c.rot_dim) continue;
                const bool upper = halves ? e >= half : e & 1;
                const int f = halves ? (upper ? e - half : e + half) : e ^ 1;
                Raw<T, 1> other;
                float q;
                other.load(static_cast<const T*>(t.x_dev) + (token0 + token) * t.x_ld + h * t.x_head + f);
                other.get(&q);
                q *= factor * (t.weight_dev ? g.c.weight_offset + t.weight_dev[f] : 1.0f);
                const float2 r = cs[halves ? (upper ? f : e) : e / 2];
                v[i][0] = fmaf(v[i][0], r.x, upper ? q * r.y : -(q * r.y));
            }
            __syncwarp();  // every lane has read its partners
        }
        if (GATE && t.gate_dev) {
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                float z[P];
#pragma unroll
                for (int p = 0; p < kPieces; ++p) gate[u][i][p].get(&z[p * kPiece]);
#pragma unroll
                for (int j = 0; j < P; ++j) v[i][j] = kParts ? v[i][j] * sigmoid_256<1>(z[j]) * z[j] : v[i][j] * silu(z[j]);
            }
        }
        if (threadIdx.x / LANES + u * kPass < here) {
            T* y = static_cast<T*>(t.y_dev) + (token0 + token) * t.y_ld + h * t.y_head;
#pragma unroll
            for (int i = 0; i < CH; ++i)
                if ((lane + LANES * i) * P < D) {
#pragma unroll
                    for (int p = 0; p < kPieces; ++p) store<T, kPiece>(y + at(i, p), &v[i][p * kPiece]);
                }
        }
    }
}

template <typename T, int LANES, int CH, int P, int U, int ROT, bool GATE>
cudaError_t launch_heads(NormArgs& g, cudaStream_t st) {
    constexpr int kRows = kThreads / LANES * U;  // heads of a CTA
    auto tokens = [](int heads) { return heads == 0 ? 0 : kRows / heads + 2 < kRows ? kRows / heads + 2 : kRows; };
    const int most = tokens(g.a.heads) > tokens(g.b.heads) ? tokens(g.a.heads) : tokens(g.b.heads);
    const size_t table = ROT ? (size_t)most * (g.c.rot_dim / 2) * sizeof(float2) : 0;
    g.first_blocks = (unsigned)((g.T * g.a.heads + kRows - 1) / kRows);
    const unsigned grid = g.first_blocks + (unsigned)((g.T * g.b.heads + kRows - 1) / kRows);
    return launch(norm_kernel<T, LANES, CH, P, U, ROT, GATE>, dim3(grid), kThreads, table, st, 1, g);
}

template <typename T, int LANES, int CH, int P, int U>
cudaError_t launch_rows(NormArgs& g, cudaStream_t st) {
    const bool gate = g.a.gate_dev || g.b.gate_dev;
    if (g.c.rot_dim && g.c.pairs == MOE_ROT_HALVES)
        return gate ? launch_heads<T, LANES, CH, P, U, kHalves, true>(g, st) : launch_heads<T, LANES, CH, P, U, kHalves, false>(g, st);
    if (g.c.rot_dim)
        return gate ? launch_heads<T, LANES, CH, P, U, kAdjacent, true>(g, st) : launch_heads<T, LANES, CH, P, U, kAdjacent, false>(g, st);
    return gate ? launch_heads<T, LANES, CH, P, U, 0, true>(g, st) : launch_heads<T, LANES, CH, P, U, 0, false>(g, st);
}

// Heads of up to 16 LANES values.  Sixteen values a thread and two heads at a time: what a head costs beside its values
// (its place, its sum's exchange) is then small, and loads of 64 bytes a thread are under way.  Few heads: eight values
// and one head, so that more threads start at once.  bf16 heads of 128, in us, 8 and 2 x 16 values a thread: 64 heads
// 1.35 and 1.57, 4096 heads 1.64 and 1.73, 8192 heads 2.30 and 1.75, 65536 heads 7.1 and 4.4; gated, 4096 heads 1.8 and
// 2.4, 8192 heads 2.9 and 2.5; of 256, rotated, 1024 heads 2.1 and 2.9, 8192 heads 4.4 and 3.5; of 64, 8192 heads 1.60
// and 1.73, 16384 heads 2.3 and 1.7.
template <typename T, int LANES>
cudaError_t launch_wide(NormArgs& g, cudaStream_t st) {
    if (LANES < 32 && g.T * (g.a.heads + g.b.heads) < (int64_t)(kThreads / LANES) * 190)
        return launch_rows<T, LANES < 32 ? 2 * LANES : 32, LANES < 32 ? 1 : 2, 8, 1>(g, st);
    return launch_rows<T, LANES, 2, 8, LANES < 32 ? 2 : 1>(g, st);
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
    const bool halves = g.c.pairs == MOE_ROT_ADJACENT || g.c.rot_dim % 8 == 0;
    if (halves && wide<T>(g.a, D) && (!second || wide<T>(g.b, D))) {
        if (D <= 64) return launch_wide<T, 4>(g, st);
        if (D <= 128) return launch_wide<T, 8>(g, st);
        if (D <= 256) return launch_wide<T, 16>(g, st);
        return launch_wide<T, 32>(g, st);
    }
    if (D <= 128) return launch_rows<T, 32, 4, 1, 1>(g, st);
    return launch_rows<T, 32, 16, 1, 1>(g, st);
}

}  // namespace

cudaError_t launch_head_norm(const moe_head_norm_config& c, const moe_heads& a, const moe_heads* b, const int32_t* pos,
                             const float* inv_freq, int64_t T, cudaStream_t st) {
    auto inverse = [](int heads) { return (uint32_t)((UINT64_C(1) << 32) / heads + 1); };
    NormArgs g{c, a, b ? *b : moe_heads{}, pos, inv_freq, T, inverse(a.heads), b ? inverse(b->heads) : 0, 0,
               c.norm == MOE_NORM_RMS ? 1.0f / (float)c.dim : 1.0f};
    return a.type == MOE_BF16 ? launch_type<__nv_bfloat16>(g, b != nullptr, st) : launch_type<float>(g, b != nullptr, st);
}

}  // namespace moe
