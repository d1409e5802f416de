// mix_delta.cu -- the gated delta rule: token by token for short runs, in
// chunks of 64 tokens on the tensor cores for long ones.
#include <cuda_fp16.h>
#include <string.h>

#include "mix.h"

namespace moe {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kC = kDeltaChunk;

// ------------------------------------------------------------------ //
// token by token                                                       //
// ------------------------------------------------------------------ //
// With S' = e^g S:  u = beta (v - S' k),  S <- S' + u k^T,  o = S' q + u (k q):
// all sums over k_dim of one token (S' k, S' q, k q) are formed together.
// Eight threads share a row of S and keep it in registers over the tokens of
// the run; a warp has four rows twice.  Bound by reading and writing S.
constexpr int kStepRows = 32;  // rows of S of a CTA of four warps

template <int KD>
__global__ void __launch_bounds__(128) steps_kernel(const __grid_constant__ DeltaArgs a) {
    after_previous();
    let_next_start();
    constexpr int kJ = KD / 32;  // float4 of a thread's part of a row
    const int dk = a.c.k_dim, dv = a.c.v_dim, Hv = a.c.v_heads;
    const int blocks = (dv + kStepRows - 1) / kStepRows;
    const int s = blockIdx.x / blocks, h = blockIdx.y, kh = h / (Hv / a.c.k_heads);
    const int64_t lo = a.q.start(s), hi = a.q.start(s + 1);
    const int slot = a.q.slot(s);
    if (lo >= hi || hi - lo > a.longer_than || slot < 0) return;
    const int lane = threadIdx.x & 31, sub = lane & 7;
    const int d0 = (blockIdx.x % blocks) * kStepRows + (threadIdx.x >> 5) * 8 + (lane >> 3);  // and d0 + 4

    float* state = a.state ? a.state + ((int64_t)slot * Hv + h) * dv * dk : nullptr;
    float4 S[2][kJ];
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
            const int at = 4 * (sub + 8 * j), d = d0 + 4 * p;
            S[p][j] = make_float4(0, 0, 0, 0);
            if (state && at < dk && d < dv && a.q.carry(s))
                S[p][j] = *reinterpret_cast<const float4*>(state + (int64_t)d * dk + at);
        }

    struct In {
        float4 k[kJ], q[kJ];
        float v[2], g, beta;
    };
    auto four = [](const __nv_bfloat16* p, bool wide) {
        uint2 w;
        if (wide) {
            w = *reinterpret_cast<const uint2*>(p);
        } else {
            unsigned short t[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) t[i] = reinterpret_cast<const unsigned short*>(p)[i];
            memcpy(&w, t, 8);
        }
        return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                           __uint_as_float(w.y & 0xffff0000u));
    };
    auto load = [&](int64_t t, In& in) {
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
            const int at = 4 * (sub + 8 * j);
            in.k[j] = in.q[j] = make_float4(0, 0, 0, 0);
            if (at < dk) {
                in.k[j] = four(a.kr + t * a.k_ld + kh * dk + at, a.wide);
                in.q[j] = four(a.qr + t * a.q_ld + kh * dk + at, a.wide);
            }
        }
#pragma unroll
        for (int p = 0; p < 2; ++p) in.v[p] = d0 + 4 * p < dv ? __bfloat162float(a.vr[t * a.v_ld + h * dv + d0 + 4 * p]) : 0;
        in.g = a.g[t * Hv + h];
        in.beta = a.beta[t * Hv + h];
    };
    In next;
    load(lo, next);
    for (int64_t t = lo; t < hi; ++t) {
        const In in = next;
        if (t + 1 < hi) load(t + 1, next);
        const float decay = expf(in.g);
        float sk[2] = {0, 0}, sq[2] = {0, 0}, kq = 0;
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
            const float4 k = in.k[j], q = in.q[j];
            kq = fmaf(k.x, q.x, fmaf(k.y, q.y, fmaf(k.z, q.z, fmaf(k.w, q.w, kq))));
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                float4& r = S[p][j];
                r.x *= decay, r.y *= decay, r.z *= decay, r.w *= decay;
                sk[p] = fmaf(r.x, k.x, fmaf(r.y, k.y, fmaf(r.z, k.z, fmaf(r.w, k.w, sk[p]))));
                sq[p] = fmaf(r.x, q.x, fmaf(r.y, q.y, fmaf(r.z, q.z, fmaf(r.w, q.w, sq[p]))));
            }
        }
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) {
            kq += __shfl_xor_sync(kAll, kq, d);
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                sk[p] += __shfl_xor_sync(kAll, sk[p], d);
                sq[p] += __shfl_xor_sync(kAll, sq[p], d);
            }
        }
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const float u = in.beta * (in.v[p] - sk[p]);
#pragma unroll
            for (int j = 0; j < kJ; ++j) {
                S[p][j].x = fmaf(u, in.k[j].x, S[p][j].x);
                S[p][j].y = fmaf(u, in.k[j].y, S[p][j].y);
                S[p][j].z = fmaf(u, in.k[j].z, S[p][j].z);
                S[p][j].w = fmaf(u, in.k[j].w, S[p][j].w);
            }
            if (sub == 0 && d0 + 4 * p < dv)
                a.o[t * a.o_ld + h * dv + d0 + 4 * p] = __float2bfloat16_rn(a.c.scale * fmaf(u, kq, sq[p]));
        }
    }
    if (state) {
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int j = 0; j < kJ; ++j) {
                const int at = 4 * (sub + 8 * j), d = d0 + 4 * p;
                if (at < dk && d < dv) *reinterpret_cast<float4*>(state + (int64_t)d * dk + at) = S[p][j];
            }
    }
}

// ------------------------------------------------------------------ //
// chunks                                                               //
// ------------------------------------------------------------------ //
// A chunk of 64 tokens with the state S before it, G_i the sum of g up to
// token i, L_ij = e^(G_i - G_j) for j <= i:
//   A_ij = beta_i L_ij (k_i k_j), j < i         T = (1 + A)^-1 diag(beta)
//   U = T (V - e^G K S^T)                       the chunk's updates
//   O = scale (e^G Q S^T + (L_ij q_i k_j) U)    S <- e^(G_63) S + U^T (e^(G_63 - G) K)
// All exponents are of differences that are 0 or less.  T and P = L q k do not
// depend on S: prepare_kernel finds them for all chunks at once.  chunks_kernel
// then goes through a sequence's chunks one after another.
//
// Numbers enter the products as fp16.  K and Q are bf16, exact in fp16 once a
// row is scaled by a power of two that brings its largest value to 2^14 (values
// 2^-28 below that lose bits).  S, V - e^G K S^T, T and the updates are sums in
// fp32 and enter as two fp16 numbers each, high and rest, together 22 bits,
// again scaled by row or column; the product of the two rests is left out.
// What only goes into o, which is rounded to bf16, enters by its high number.
//
// Workspace, per chunk and k head: K16 and Q16 [64 x KD] fp16; per chunk and v
// head: T high, T rest, P [64 x 64] fp16 and the factors of Factors.  Rows are
// stored with their 16-byte pieces exchanged (piece p of row r at p ^ (r & 7)),
// ready to be copied to shared memory and read from there without conflicts.
struct Factors {
    float ks[kC];  // e^G_i times the scale of k's row
    float t[kC];   // scale of T's row
    float p[kC];   // scale of P's row, times the factor on o
    float qs[kC];  // e^G_i times the scale of q's row, times the factor on o
    float left[kC];  // e^(G_63 - G_i) times the scale of k's row
    float all[4];  // e^G_63
};
constexpr int kSquare = kC * kC * 2;
constexpr int kHeadBytes = (3 * kSquare + (int)sizeof(Factors) + 127) / 128 * 128;

__host__ __device__ constexpr int padded_dim(int k_dim) { return k_dim <= 64 ? 64 : 128; }
__host__ __device__ constexpr int pair_bytes(int KD) { return 2 * kC * KD * 2; }

__device__ __forceinline__ uint32_t smem_at(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void ldmatrix(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void ldmatrix_trans(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ uint32_t transposed(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }

// The power of two that brings a largest magnitude to [2^14, 2^15), and its
// inverse.  `e`: the magnitude's exponent field, kept within what both allow.
__device__ __forceinline__ int field(float m) { return max((int)(__float_as_uint(m) >> 23), 16); }
__device__ __forceinline__ float up(int e) { return __uint_as_float((uint32_t)(268 - e) << 23); }    // 2^(14 - (e - 127))
__device__ __forceinline__ float down(int e) {                                                        // 2^(e - 127 - 14)
    return e > 14 ? __uint_as_float((uint32_t)(e - 14) << 23) : 0.0f;
}

// byte of 16-byte piece p of row r, in rows of N pieces
template <int N>
__device__ __forceinline__ int piece_at(int r, int p) {
    return (r * N + (p ^ (r & 7))) * 16;
}

// rows r0 .. r0+15, pieces p, p+1: the fragment of a left operand (16 x 16)
template <int N>
__device__ __forceinline__ uint32_t left_at(uint32_t base, int r0, int p, int lane) {
    return base + piece_at<N>(r0 + (lane & 15), p + (lane >> 4));
}
// the same block read the other way: as right operand with rows of the memory as its columns, or (transposed) as left
// operand with columns of the memory as its rows
template <int N>
__device__ __forceinline__ uint32_t right_at(uint32_t base, int r0, int p, int lane) {
    return base + piece_at<N>(r0 + (lane & 7) + ((lane >> 4) << 3), p + ((lane >> 3) & 1));
}

constexpr int kPitch = kC + 4;  // floats of a row of A

template <int KD>
struct PrepareShared {
    uint8_t k[kC * KD * 2], q[kC * KD * 2];
    float A[2][kC][kPitch];  // two v heads at a time: A, then T
    float k_scale[kC], q_scale[kC];
    float g_high[2][kC], g_rest[2][kC], beta[2][kC];
};

__device__ __forceinline__ uint4 eight(const __nv_bfloat16* p, bool wide) {
    uint4 w;
    if (wide) return *reinterpret_cast<const uint4*>(p);
    unsigned short t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = reinterpret_cast<const unsigned short*>(p)[i];
    memcpy(&w, t, 16);
    return w;
}

// One chunk and k head: K16 and Q16; then for its v heads, two at a time, the
// factors, P and T.  (1 + A)^-1 by substitution down each of its 64 columns, a
// thread a column, in fp32.
template <int KD>
__global__ void __launch_bounds__(128) prepare_kernel(const __grid_constant__ DeltaArgs a) {
    extern __shared__ uint8_t raw[];
    PrepareShared<KD>& m = *reinterpret_cast<PrepareShared<KD>*>(raw);
    after_previous();
    let_next_start();
    int c;
    const int s = a.q.find<kC>(blockIdx.x, c);
    const int64_t lo = a.q.start(s), hi = a.q.start(s + 1);
    if (c < 0 || hi - lo <= a.longer_than || (int64_t)c * kC >= hi - lo || a.q.slot(s) < 0) return;
    const int64_t row0 = lo + (int64_t)c * kC;
    const int rows = (int)(hi - row0 < kC ? hi - row0 : kC);
    const int kh = blockIdx.y, Hk = a.c.k_heads, Hv = a.c.v_heads, share = Hv / Hk, dk = a.c.k_dim;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint8_t* pair = a.ws + ((int64_t)blockIdx.x * Hk + kh) * pair_bytes(KD);
    uint8_t* heads = a.ws + a.q_pieces * Hk * pair_bytes(KD) + ((int64_t)blockIdx.x * Hv + kh * share) * kHeadBytes;

    // rows of K and Q: KD / 8 threads a row
    constexpr int kRow = KD / 8, kPass = 128 / kRow, kN = kC / kPass;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        const __nv_bfloat16* src = (which ? a.qr + row0 * a.q_ld : a.kr + row0 * a.k_ld) + kh * dk;
        const int64_t ld = which ? a.q_ld : a.k_ld;
        const int p = tid % kRow;
        uint4 w[kN];
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int r = tid / kRow + i * kPass;
            w[i] = make_uint4(0, 0, 0, 0);
            if (r < rows && p * 8 < dk) w[i] = eight(src + r * ld + p * 8, a.wide);
        }
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int r = tid / kRow + i * kPass;
            const uint32_t v[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
            uint32_t top = 0;  // of the magnitudes' bits, which order as the magnitudes do
#pragma unroll
            for (int j = 0; j < 4; ++j) top = __vmaxu2(top, v[j] & 0x7fff7fffu);
            top = max(top >> 16, top & 0xffffu);
#pragma unroll
            for (int d = 1; d < kRow; d <<= 1) top = max(top, __shfl_xor_sync(kAll, top, d));
            const int e = max((int)(top >> 7), 16);
            const float f = up(e);
            uint4 h;
            uint32_t* hw = reinterpret_cast<uint32_t*>(&h);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                hw[j] = pack(__uint_as_float(v[j] << 16) * f, __uint_as_float(v[j] & 0xffff0000u) * f);
            *reinterpret_cast<uint4*>(pair + which * (kC * KD * 2) + piece_at<kRow>(r, p)) = h;
            *reinterpret_cast<uint4*>((which ? m.q : m.k) + piece_at<kRow>(r, p)) = w[i];
            if (p == 0) (which ? m.q_scale : m.k_scale)[r] = down(e);
        }
    }
    __syncthreads();

    // K K^T and Q K^T, rows 16 warp .. +15, columns up to the diagonal block
    float kk[8][4], qk[8][4];
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) kk[n][i] = qk[n][i] = 0;
    const uint32_t k_at = smem_at(m.k), q_at = smem_at(m.q);
#pragma unroll
    for (int t = 0; t < KD / 16; ++t) {
        uint32_t ka[4], qa[4];
        ldmatrix(ka, left_at<kRow>(k_at, 16 * warp, 2 * t, lane));
        ldmatrix(qa, left_at<kRow>(q_at, 16 * warp, 2 * t, lane));
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            if (n > warp) continue;
            uint32_t b[4];
            ldmatrix(b, right_at<kRow>(k_at, 16 * n, 2 * t, lane));
            mma_bf16(kk[2 * n], ka, b[0], b[1]);
            mma_bf16(kk[2 * n + 1], ka, b[2], b[3]);
            mma_bf16(qk[2 * n], qa, b[0], b[1]);
            mma_bf16(qk[2 * n + 1], qa, b[2], b[3]);
        }
    }

    for (int h0 = 0; h0 < share; h0 += 2) {
        const int count = min(2, share - h0);
        // sums of g in fp64 (64 additions), kept as two floats: differences of far sums stay exact
        if (warp < count) {
            const int h = kh * share + h0 + warp;
            double G[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = 2 * lane + i;
                float g = 0, beta = 0;
                if (r < rows) {
                    g = a.g[(row0 + r) * Hv + h];
                    beta = a.beta[(row0 + r) * Hv + h];
                    if (g < -120.0f) g = -120.0f;  // e^-120 is 0 in fp32, and -inf has no differences
                }
                G[i] = g;
                m.beta[warp][r] = beta;
            }
            G[1] += G[0];
            double before = G[1];
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const double o = __shfl_up_sync(kAll, before, d);
                if (lane >= d) before += o;
            }
            before = __shfl_up_sync(kAll, before, 1);
            if (lane == 0) before = 0;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                G[i] += before;
                m.g_high[warp][2 * lane + i] = (float)G[i];
                m.g_rest[warp][2 * lane + i] = (float)(G[i] - (double)(float)G[i]);
            }
        }
        __syncthreads();
        for (int b = 0; b < count; ++b) {
            uint8_t* out = heads + (int64_t)(h0 + b) * kHeadBytes;
            Factors& f = *reinterpret_cast<Factors*>(out + 3 * kSquare);
            const float *gh = m.g_high[b], *gr = m.g_rest[b];
            if (tid < kC) {
                const float e = expf(gh[tid] + gr[tid]);
                const float rest = expf((gh[kC - 1] - gh[tid]) + (gr[kC - 1] - gr[tid]));
                f.ks[tid] = e * m.k_scale[tid];
                f.qs[tid] = e * m.q_scale[tid] * a.c.scale;
                f.left[tid] = rest * m.k_scale[tid];
                if (tid == kC - 1) f.all[0] = e;
            }
            float top[2] = {0, 0};
            float P[8][4];
#pragma unroll
            for (int n = 0; n < 8; ++n) {
                if (n > 2 * warp + 1) continue;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = 16 * warp + (lane >> 2) + 8 * (i >> 1), j = 8 * n + 2 * (lane & 3) + (i & 1);
                    const float L = j <= r ? expf((gh[r] - gh[j]) + (gr[r] - gr[j])) : 0.0f;
                    m.A[b][r][j] = j < r ? m.beta[b][r] * L * kk[n][i] : 0.0f;
                    P[n][i] = j <= r ? L * qk[n][i] : 0.0f;
                    top[i >> 1] = fmaxf(top[i >> 1], fabsf(P[n][i]));
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                top[i] = fmaxf(top[i], __shfl_xor_sync(kAll, top[i], 1));
                top[i] = fmaxf(top[i], __shfl_xor_sync(kAll, top[i], 2));
                const int r = 16 * warp + (lane >> 2) + 8 * i, e = field(top[i]);
                const float scale = up(e);
                if ((lane & 3) == 0) f.p[r] = down(e) * a.c.scale;
#pragma unroll
                for (int n = 0; n < 8; ++n)
                    if (n <= 2 * warp + 1)
                        *reinterpret_cast<uint32_t*>(out + 2 * kSquare + piece_at<8>(r, n) + 4 * (lane & 3)) =
                            pack(P[n][2 * i] * scale, P[n][2 * i + 1] * scale);
            }
        }
        __syncthreads();
        const int b = tid >> 6, col = tid & 63;
        float t[kC];
        if (b < count) {
#pragma unroll
            for (int i = 0; i < kC; ++i) {
                float sum[4] = {i == col ? 1.0f : 0.0f, 0, 0, 0};
#pragma unroll
                for (int j = 0; j < i; j += 4) {
                    const float4 r = *reinterpret_cast<const float4*>(&m.A[b][i][j]);
                    sum[0] = fmaf(-r.x, t[j], sum[0]);
                    if (j + 1 < i) sum[1] = fmaf(-r.y, t[j + 1], sum[1]);
                    if (j + 2 < i) sum[2] = fmaf(-r.z, t[j + 2], sum[2]);
                    if (j + 3 < i) sum[3] = fmaf(-r.w, t[j + 3], sum[3]);
                }
                t[i] = (sum[0] + sum[1]) + (sum[2] + sum[3]);
            }
        }
        __syncthreads();
        if (b < count) {
            const float beta = m.beta[b][col];
#pragma unroll
            for (int i = 0; i < kC; ++i) m.A[b][i][col] = t[i] * beta;
        }
        __syncthreads();
        // rows of T out: eight threads a row
        for (int r = tid >> 3; r < count * kC; r += 16) {
            const int which = r / kC, row = r % kC, p = tid & 7;
            uint8_t* out = heads + (int64_t)(h0 + which) * kHeadBytes;
            const float4 x = *reinterpret_cast<const float4*>(&m.A[which][row][8 * p]);
            const float4 y = *reinterpret_cast<const float4*>(&m.A[which][row][8 * p + 4]);
            const float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
            float top = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(v[j]));
#pragma unroll
            for (int d = 1; d < 8; d <<= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, d));
            const int e = field(top);
            const float scale = up(e);
            uint32_t high[4], rest[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float u0 = v[2 * j] * scale, u1 = v[2 * j + 1] * scale;
                high[j] = pack(u0, u1);
                const float2 h = unpack(high[j]);
                rest[j] = pack(u0 - h.x, u1 - h.y);
            }
            *reinterpret_cast<uint4*>(out + piece_at<8>(row, p)) = make_uint4(high[0], high[1], high[2], high[3]);
            *reinterpret_cast<uint4*>(out + kSquare + piece_at<8>(row, p)) = make_uint4(rest[0], rest[1], rest[2], rest[3]);
            if (p == 0) reinterpret_cast<Factors*>(out + 3 * kSquare)->t[row] = down(e);
        }
        __syncthreads();
    }
}

// the right operand's fragment (16 x 8) of two accumulator blocks c: as high numbers and rests
struct Fragment {
    uint32_t high[2], rest[2];
};
__device__ __forceinline__ Fragment split(const float (&c)[4], float f0, float f1) {
    Fragment r;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float x = c[2 * i] * f0, y = c[2 * i + 1] * f1;
        const uint32_t w = pack(x, y);
        const float2 h = unpack(w);
        r.high[i] = transposed(w);
        r.rest[i] = transposed(pack(x - h.x, y - h.y));
    }
    return r;
}
__device__ __forceinline__ void split_high(uint32_t (&high)[2], const float (&c)[4], float f0, float f1) {
#pragma unroll
    for (int i = 0; i < 2; ++i) high[i] = transposed(pack(c[2 * i] * f0, c[2 * i + 1] * f1));
}
// exponent fields of the two columns' largest magnitudes over N accumulator blocks
template <int N>
__device__ __forceinline__ void fields(int (&e)[2], const float (&c)[N][4]) {
    float m0 = 0, m1 = 0;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        m0 = fmaxf(m0, fmaxf(fabsf(c[n][0]), fabsf(c[n][2])));
        m1 = fmaxf(m1, fmaxf(fabsf(c[n][1]), fabsf(c[n][3])));
    }
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) {
        m0 = fmaxf(m0, __shfl_xor_sync(kAll, m0, d));
        m1 = fmaxf(m1, __shfl_xor_sync(kAll, m1, d));
    }
    e[0] = field(m0);
    e[1] = field(m1);
}

template <int KD, int NT, int NW>
struct ChunkShape {
    static constexpr int kCols = NW * NT * 8;            // columns of V of a CTA
    static constexpr int kVPitch = kCols * 2 + 16;       // bytes of a row; the 16 keep 8 rows on different banks
    static constexpr int kStage = pair_bytes(KD) + kHeadBytes + kC * kVPitch;
    static constexpr int kStages = 3;
    static constexpr int kBytes = kStages * kStage;
};

// A CTA takes one sequence, v head and kCols columns of V; each warp keeps S^T
// for its NT * 8 columns [KD x 8 NT] in registers, as accumulators of the
// state's product, and needs nothing of the other warps: they share the tiles
// in shared memory only, copied two chunks ahead.  An accumulator becomes the
// right operand of the next product by one transposition of each 8 x 8 block.
template <int KD, int NT, int NW>
__global__ void __launch_bounds__(NW * 32, 1) chunks_kernel(const __grid_constant__ DeltaArgs a) {
    using Shape = ChunkShape<KD, NT, NW>;
    extern __shared__ __align__(128) uint8_t raw[];
    after_previous();
    let_next_start();
    constexpr int kM = KD / 16, kRow = KD / 8;
    const int dk = a.c.k_dim, dv = a.c.v_dim, Hk = a.c.k_heads, Hv = a.c.v_heads;
    const int blocks = (dv + Shape::kCols - 1) / Shape::kCols;
    const int s = blockIdx.x / blocks, h = blockIdx.y, kh = h / (Hv / Hk);
    const int64_t lo = a.q.start(s), hi = a.q.start(s + 1), len = hi - lo;
    const int slot = a.q.slot(s);
    if (len <= 0 || len <= a.longer_than || slot < 0) return;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int first = (blockIdx.x % blocks) * Shape::kCols;  // column of V
    const int chunks = (int)((len + kC - 1) / kC);
    const int64_t piece = a.q.piece_of<kC>(s);
    const uint32_t base = smem_at(raw);

    auto copy16 = [](uint32_t to, const void* from, bool there) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there ? 16 : 0) : "memory");
    };
    auto fetch = [&](int c) {
        if (c < chunks) {
            const uint32_t to = base + (c % Shape::kStages) * Shape::kStage;
            const uint8_t* pair = a.ws + ((piece + c) * Hk + kh) * pair_bytes(KD);
            const uint8_t* head = a.ws + a.q_pieces * Hk * pair_bytes(KD) + ((piece + c) * Hv + h) * kHeadBytes;
            for (int i = tid * 16; i < pair_bytes(KD); i += NW * 512) copy16(to + i, pair + i, true);
            for (int i = tid * 16; i < kHeadBytes; i += NW * 512) copy16(to + pair_bytes(KD) + i, head + i, true);
            const int64_t row0 = lo + (int64_t)c * kC;
            for (int i = tid; i < kC * (Shape::kCols / 8); i += NW * 32) {
                const int r = i / (Shape::kCols / 8), d = first + i % (Shape::kCols / 8) * 8;
                const bool there = row0 + r < hi && d < dv;
                const __nv_bfloat16* from = there ? a.vr + (row0 + r) * a.v_ld + h * dv + d : a.vr;
                const uint32_t at = (uint32_t)(pair_bytes(KD) + kHeadBytes + r * Shape::kVPitch + (d - first) * 2);
                if (a.wide) {
                    copy16(to + at, from, there);
                } else {
                    *reinterpret_cast<uint4*>(raw + (c % Shape::kStages) * Shape::kStage + at) =
                        there ? eight(from, false) : make_uint4(0, 0, 0, 0);
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    fetch(0);
    fetch(1);

    // S^T: rows 16 m + lane / 4 (+ 8) of k_dim, columns d0 + 8 n (+ 1) of v_dim
    float S[NT][kM][4];
    const int d0 = first + warp * NT * 8 + 2 * (lane & 3);
    float* state = a.state ? a.state + ((int64_t)slot * Hv + h) * dv * dk : nullptr;
    const bool carry = state && a.q.carry(s);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int m = 0; m < kM; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int d = d0 + 8 * n + (i & 1), k = 16 * m + (lane >> 2) + 8 * (i >> 1);
                S[n][m][i] = carry && d < dv && k < dk ? state[(int64_t)d * dk + k] : 0.0f;
            }

    for (int c = 0; c < chunks; ++c) {
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncthreads();  // chunk c is there for all, and all are done with chunk c - 1
        fetch(c + 2);
        const uint8_t* stage = raw + (c % Shape::kStages) * Shape::kStage;
        const uint32_t K16 = base + (c % Shape::kStages) * Shape::kStage, Q16 = K16 + kC * KD * 2;
        const uint32_t T_high = K16 + pair_bytes(KD), T_rest = T_high + kSquare, P16 = T_rest + kSquare;
        const Factors& f = *reinterpret_cast<const Factors*>(stage + pair_bytes(KD) + 3 * kSquare);
        const uint8_t* V = stage + pair_bytes(KD) + kHeadBytes;
        const int r0 = lane >> 2;

        // K S^T and Q S^T
        float x[NT][4][4], qs[NT][4][4];
        int e_s[NT][2];
        float s_up[NT][2], s_down[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            fields(e_s[n], S[n]);
#pragma unroll
            for (int i = 0; i < 2; ++i) s_up[n][i] = up(e_s[n][i]), s_down[n][i] = down(e_s[n][i]);
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) x[n][m][i] = qs[n][m][i] = 0;
        }
#pragma unroll
        for (int t = 0; t < kM; ++t) {
            Fragment b[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) b[n] = split(S[n][t], s_up[n][0], s_up[n][1]);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                uint32_t w[4];
                ldmatrix(w, left_at<kRow>(K16, 16 * m, 2 * t, lane));
#pragma unroll
                for (int n = 0; n < NT; ++n) mma_f16(x[n][m], w, b[n].high[0], b[n].high[1]);
#pragma unroll
                for (int n = 0; n < NT; ++n) mma_f16(x[n][m], w, b[n].rest[0], b[n].rest[1]);
                ldmatrix(w, left_at<kRow>(Q16, 16 * m, 2 * t, lane));
#pragma unroll
                for (int n = 0; n < NT; ++n) mma_f16(qs[n][m], w, b[n].high[0], b[n].high[1]);
            }
        }
        // X = V - e^G K S^T
        float x_up[NT][2], x_down[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int r = 16 * m + r0 + 8 * i;
                    const uint32_t v = *reinterpret_cast<const uint32_t*>(V + r * Shape::kVPitch + (d0 - first + 8 * n) * 2);
                    const float ks = f.ks[r];
                    x[n][m][2 * i] = fmaf(-ks * s_down[n][0], x[n][m][2 * i], __uint_as_float(v << 16));
                    x[n][m][2 * i + 1] = fmaf(-ks * s_down[n][1], x[n][m][2 * i + 1], __uint_as_float(v & 0xffff0000u));
                }
            int e[2];
            fields(e, x[n]);
#pragma unroll
            for (int i = 0; i < 2; ++i) x_up[n][i] = up(e[i]), x_down[n][i] = down(e[i]);
        }
        // U = T X
        float u[NT][4][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) u[n][m][i] = 0;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            Fragment b[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) b[n] = split(x[n][t], x_up[n][0], x_up[n][1]);
#pragma unroll
            for (int m = t; m < 4; ++m) {
                uint32_t w[4];
                ldmatrix(w, left_at<8>(T_high, 16 * m, 2 * t, lane));
#pragma unroll
                for (int n = 0; n < NT; ++n) mma_f16(u[n][m], w, b[n].high[0], b[n].high[1]);
#pragma unroll
                for (int n = 0; n < NT; ++n) mma_f16(u[n][m], w, b[n].rest[0], b[n].rest[1]);
                ldmatrix(w, left_at<8>(T_rest, 16 * m, 2 * t, lane));
#pragma unroll
                for (int n = 0; n < NT; ++n) mma_f16(u[n][m], w, b[n].high[0], b[n].high[1]);
            }
        }
        float u_up[NT][2], u_down[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) u[n][m][i] *= f.t[16 * m + r0 + 8 * (i >> 1)] * x_down[n][i & 1];
            int e[2];
            fields(e, u[n]);
#pragma unroll
            for (int i = 0; i < 2; ++i) u_up[n][i] = up(e[i]), u_down[n][i] = down(e[i]);
        }
        // o
        float pu[NT][4][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) pu[n][m][i] = 0;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            uint32_t b[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) split_high(b[n], u[n][t], u_up[n][0], u_up[n][1]);
#pragma unroll
            for (int m = t; m < 4; ++m) {
                uint32_t w[4];
                ldmatrix(w, left_at<8>(P16, 16 * m, 2 * t, lane));
#pragma unroll
                for (int n = 0; n < NT; ++n) mma_f16(pu[n][m], w, b[n][0], b[n][1]);
            }
        }
        const int64_t row0 = lo + (int64_t)c * kC;
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = 16 * m + r0 + 8 * i;
                const float fq = f.qs[r], fp = f.p[r];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const float y0 = fmaf(fq * s_down[n][0], qs[n][m][2 * i], fp * u_down[n][0] * pu[n][m][2 * i]);
                    const float y1 = fmaf(fq * s_down[n][1], qs[n][m][2 * i + 1], fp * u_down[n][1] * pu[n][m][2 * i + 1]);
                    const int d = d0 + 8 * n;
                    if (row0 + r < hi && d < dv) {
                        __nv_bfloat16* o = a.o + (row0 + r) * a.o_ld + h * dv + d;
                        const __nv_bfloat162 v = __floats2bfloat162_rn(y0, y1);
                        if (a.o_pairs) {
                            *reinterpret_cast<__nv_bfloat162*>(o) = v;
                        } else {
                            o[0] = v.x;
                            o[1] = v.y;
                        }
                    }
                }
            }
        // S <- e^G_63 S + U^T (e^(G_63 - G) K), the sum in units of the updates' scale
        const float all = f.all[0];
        float l_up[NT][2], l_down[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) u[n][m][i] *= f.left[16 * m + r0 + 8 * (i >> 1)];
            int e[2];
            fields(e, u[n]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                e[i] = max(e[i], e_s[n][i] - 60);  // S stays finite in these units; updates 2^-60 of it do not count
                l_up[n][i] = up(e[i]), l_down[n][i] = down(e[i]);
            }
#pragma unroll
            for (int m = 0; m < kM; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) S[n][m][i] *= all * l_up[n][i & 1];
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            Fragment b[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) b[n] = split(u[n][t], l_up[n][0], l_up[n][1]);
#pragma unroll
            for (int m = 0; m < kM; ++m) {
                uint32_t w[4];
                ldmatrix_trans(w, right_at<kRow>(K16, 16 * t, 2 * m, lane));
#pragma unroll
                for (int n = 0; n < NT; ++n) mma_f16(S[n][m], w, b[n].high[0], b[n].high[1]);
#pragma unroll
                for (int n = 0; n < NT; ++n) mma_f16(S[n][m], w, b[n].rest[0], b[n].rest[1]);
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int m = 0; m < kM; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) S[n][m][i] *= l_down[n][i & 1];
    }
    if (state) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int m = 0; m < kM; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int d = d0 + 8 * n + (i & 1), k = 16 * m + (lane >> 2) + 8 * (i >> 1);
                    if (d < dv && k < dk) state[(int64_t)d * dk + k] = S[n][m][i];
                }
    }
}

template <int KD, int NT, int NW>
cudaError_t launch_shape(const DeltaArgs& a, cudaStream_t st) {
    using Shape = ChunkShape<KD, NT, NW>;
    const int blocks = (a.c.v_dim + Shape::kCols - 1) / Shape::kCols;
    if (cudaError_t e = cudaFuncSetAttribute(chunks_kernel<KD, NT, NW>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             Shape::kBytes))
        return e;
    return launch(chunks_kernel<KD, NT, NW>, dim3((unsigned)(a.q.n * blocks), (unsigned)a.c.v_heads), NW * 32,
                  Shape::kBytes, st, 1, a);
}

template <int KD>
cudaError_t launch_chunked(const DeltaArgs& a, cudaStream_t st) {
    if (cudaError_t e = cudaFuncSetAttribute(prepare_kernel<KD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)sizeof(PrepareShared<KD>)))
        return e;
    if (cudaError_t e = launch(prepare_kernel<KD>, dim3((unsigned)a.q_pieces, (unsigned)a.c.k_heads), 128,
                               sizeof(PrepareShared<KD>), st, 1, a))
        return e;
    return launch_shape<KD, 1, 4>(a, st);
}

}  // namespace

size_t delta_workspace(const moe_delta_config& c, int64_t T, int n) {
    return (size_t)(T / kC + n) *
           ((size_t)c.k_heads * pair_bytes(padded_dim(c.k_dim)) + (size_t)c.v_heads * kHeadBytes);
}

cudaError_t launch_delta_steps(const DeltaArgs& a, cudaStream_t st) {
    const int blocks = (a.c.v_dim + kStepRows - 1) / kStepRows;
    const dim3 grid((unsigned)(a.q.n * blocks), (unsigned)a.c.v_heads);
    if (a.c.k_dim <= 64) return launch(steps_kernel<64>, grid, 128, 0, st, 1, a);
    return launch(steps_kernel<128>, grid, 128, 0, st, 1, a);
}

cudaError_t launch_delta_chunks(const DeltaArgs& a, cudaStream_t st) {
    return padded_dim(a.c.k_dim) == 64 ? launch_chunked<64>(a, st) : launch_chunked<128>(a, st);
}

}  // namespace moe
