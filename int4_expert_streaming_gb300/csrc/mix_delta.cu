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
// kLanes threads share a row of S and keep it in registers over the tokens of
// the run, kRows rows each.  Bound by reading and writing S: its loads are
// issued before anything else is waited for, together with the first tokens'.
constexpr int kLanes = 16, kRows = 2;
constexpr int kStepRows = 128 / kLanes * kRows;  // rows of S of a CTA of four warps

// KD / kLanes values of a row of K or Q, still packed
template <int KD>
struct Token {
    static constexpr int kE = KD / kLanes;  // values of a thread: 8 or 4
    uint32_t k[kE / 2], q[kE / 2];
    __nv_bfloat16 v[kRows];
    float g, beta;
};
__device__ __forceinline__ void packed(uint32_t (&w)[4], const __nv_bfloat16* p, bool wide) {
    if (wide) {
        *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(p);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = reinterpret_cast<const unsigned short*>(p)[2 * i] | (uint32_t)reinterpret_cast<const unsigned short*>(p)[2 * i + 1] << 16;
    }
}
__device__ __forceinline__ void packed(uint32_t (&w)[2], const __nv_bfloat16* p, bool wide) {
    if (wide) {
        *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(p);
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            w[i] = reinterpret_cast<const unsigned short*>(p)[2 * i] | (uint32_t)reinterpret_cast<const unsigned short*>(p)[2 * i + 1] << 16;
    }
}

template <int KD>
__global__ void __launch_bounds__(128) steps_kernel(const __grid_constant__ DeltaArgs a) {
    after_previous();
    let_next_start();
    constexpr int kE = KD / kLanes;
    const int dk = a.c.k_dim, dv = a.c.v_dim, Hv = a.c.v_heads;
    const int blocks = (dv + kStepRows - 1) / kStepRows;
    const int s = blockIdx.x / blocks, h = blockIdx.y, kh = h / (Hv / a.c.k_heads);
    const int64_t lo = a.q.start(s), hi = a.q.start(s + 1);
    const int slot = a.q.slot(s);
    const bool carry = a.state && a.q.carry(s);
    if (lo >= hi || hi - lo > a.longer_than || slot < 0) return;
    const int lane = threadIdx.x % kLanes, at = lane * kE;
    const int d0 = (blockIdx.x % blocks) * kStepRows + threadIdx.x / kLanes * kRows;
    const bool in_k = at < dk;

    auto load = [&](int64_t t, Token<KD>& in) {
#pragma unroll
        for (int i = 0; i < kE / 2; ++i) in.k[i] = in.q[i] = 0;
        if (in_k) {
            packed(in.k, a.kr + t * a.k_ld + kh * dk + at, a.wide);
            packed(in.q, a.qr + t * a.q_ld + kh * dk + at, a.wide);
        }
#pragma unroll
        for (int p = 0; p < kRows; ++p) in.v[p] = d0 + p < dv ? a.vr[t * a.v_ld + h * dv + d0 + p] : __nv_bfloat16(0.0f);
        in.g = a.g[t * Hv + h];
        in.beta = a.beta[t * Hv + h];
    };
    float* state = a.state ? a.state + (((int64_t)slot * Hv + h) * dv + d0) * dk + at : nullptr;
    float S[kRows][kE];
#pragma unroll
    for (int p = 0; p < kRows; ++p)
#pragma unroll
        for (int i = 0; i < kE; i += 4) {
            const bool there = carry && in_k && d0 + p < dv;
            *reinterpret_cast<float4*>(&S[p][i]) =
                there ? *reinterpret_cast<const float4*>(state + p * dk + i) : make_float4(0, 0, 0, 0);
        }
    Token<KD> next[2];
    load(lo, next[0]);
    if (lo + 1 < hi) load(lo + 1, next[1]);
    for (int64_t t = lo; t < hi; ++t) {
        const Token<KD> in = next[0];
        next[0] = next[1];
        if (t + 2 < hi) load(t + 2, next[1]);
        const float decay = expf(in.g);
        float k[kE], q[kE], sk[kRows], sq[kRows], kq = 0;
#pragma unroll
        for (int i = 0; i < kE / 2; ++i) {
            k[2 * i] = __uint_as_float(in.k[i] << 16), k[2 * i + 1] = __uint_as_float(in.k[i] & 0xffff0000u);
            q[2 * i] = __uint_as_float(in.q[i] << 16), q[2 * i + 1] = __uint_as_float(in.q[i] & 0xffff0000u);
        }
#pragma unroll
        for (int i = 0; i < kE; ++i) kq = fmaf(k[i], q[i], kq);
#pragma unroll
        for (int p = 0; p < kRows; ++p) {
            sk[p] = sq[p] = 0;
#pragma unroll
            for (int i = 0; i < kE; ++i) {
                S[p][i] *= decay;
                sk[p] = fmaf(S[p][i], k[i], sk[p]);
                sq[p] = fmaf(S[p][i], q[i], sq[p]);
            }
        }
#pragma unroll
        for (int d = 1; d < kLanes; d <<= 1) {
            kq += __shfl_xor_sync(kAll, kq, d);
#pragma unroll
            for (int p = 0; p < kRows; ++p) {
                sk[p] += __shfl_xor_sync(kAll, sk[p], d);
                sq[p] += __shfl_xor_sync(kAll, sq[p], d);
            }
        }
        float o[kRows];
#pragma unroll
        for (int p = 0; p < kRows; ++p) {
            const float u = in.beta * (__bfloat162float(in.v[p]) - sk[p]);
#pragma unroll
            for (int i = 0; i < kE; ++i) S[p][i] = fmaf(u, k[i], S[p][i]);
            o[p] = a.c.scale * fmaf(u, kq, sq[p]);
        }
        if (lane < kRows && d0 + lane < dv)
            a.o[t * a.o_ld + h * dv + d0 + lane] = __float2bfloat16_rn(lane ? o[kRows - 1] : o[0]);
    }
    if (state && in_k) {
#pragma unroll
        for (int p = 0; p < kRows; ++p)
            if (d0 + p < dv) {
#pragma unroll
                for (int i = 0; i < kE; i += 4)
                    *reinterpret_cast<float4*>(state + p * dk + i) = *reinterpret_cast<const float4*>(&S[p][i]);
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
    float all;       // e^G_63
    // how large things can get, from what came before: V - e^G K S^T over the largest of S, beside V; U over the
    // largest of that; and `left` itself
    float most_ks, most_t, most_left;
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
constexpr int kOne = 141;  // the exponent field of which both are 1
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

constexpr int kPitch = kC + 4;  // floats of a row of A and T: rows of 8 lanes are on different banks
constexpr int kPrepare = 256;   // threads: four warps for each of two v heads

template <int KD>
struct PrepareShared {
    float A[2][kC][kPitch];
    union {
        uint8_t kq[2][kC * KD * 2];  // K and Q, bf16; then
        float T[2][kC][kPitch];      // the lower blocks; the upper ones hold what their lower ones are made of
    };
    float k_scale[kC], q_scale[kC], k_sum[kC], q_top[kC];
    float g_high[2][kC], g_rest[2][kC], beta[2][kC];
    float before[2][4][kC];  // e^(G_16w - G_j), j < 16 w
    unsigned most[2];        // bits of the largest row sum of |T|
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

// left[16 x 16] right[16 x 16] (rows of kPitch floats), added to acc: columns 0..7 and 8..15 as accumulator blocks.  Each
// number enters as two of 11 bits; the product of the two rests is left out, which leaves 2^-22.
__device__ __forceinline__ void halves(float x, uint32_t& high, uint32_t& rest) {
    high = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;  // to nearest
    rest = (__float_as_uint(x - __uint_as_float(high)) + 0x1000u) & 0xffffe000u;
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
__device__ __forceinline__ void block_product(float (&acc)[2][4], const float* left, const float* right, int lane) {
    const float *l0 = left + (lane >> 2) * kPitch + (lane & 3), *r0 = right + (lane & 3) * kPitch + (lane >> 2);
#pragma unroll
    for (int k = 0; k < 16; k += 8) {
        uint32_t ah[4], ar[4], bh[2][2], br[2][2];
#pragma unroll
        for (int i = 0; i < 4; ++i) halves(l0[(i & 1) * 8 * kPitch + k + (i >> 1) * 4], ah[i], ar[i]);
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) halves(r0[(k + 4 * i) * kPitch + 8 * n], bh[n][i], br[n][i]);
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            mma_tf32(acc[n], ar, bh[n]);
            mma_tf32(acc[n], ah, br[n]);
            mma_tf32(acc[n], ah, bh[n]);
        }
    }
}
__device__ __forceinline__ void block_store(float* to, const float (&acc)[2][4], float sign, int lane) {
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i)
            *reinterpret_cast<float2*>(to + ((lane >> 2) + 8 * i) * kPitch + 8 * n + (lane & 3) * 2) =
                make_float2(sign * acc[n][2 * i], sign * acc[n][2 * i + 1]);
}
// the four warps of one of the two heads
__device__ __forceinline__ void head_barrier(int b) {
    if (b)
        asm volatile("bar.sync 2, 128;" ::: "memory");
    else
        asm volatile("bar.sync 1, 128;" ::: "memory");
}

// One chunk and two v heads of a k head: K16 and Q16, the factors, P and T.
// (1 + A)^-1 by blocks of 16: the four on the diagonal by substitution in fp32,
// a lane a column; then T_10 and T_32, and of those the lower left quarter, by
//   (T_11 0; T_21 T_22) with T_21 = -T_22 A_21 T_11.
// Bound by issuing instructions.
template <int KD>
__global__ void __launch_bounds__(kPrepare, 3) prepare_kernel(const __grid_constant__ DeltaArgs a) {
    extern __shared__ __align__(128) uint8_t raw[];
    PrepareShared<KD>& m = *reinterpret_cast<PrepareShared<KD>*>(raw);
    after_previous();
    let_next_start();
    int c;
    const int s = a.q.find<kC>(blockIdx.x, c);
    const int64_t lo = a.q.start(s), hi = a.q.start(s + 1);
    if (c < 0 || hi - lo <= a.longer_than || (int64_t)c * kC >= hi - lo || a.q.slot(s) < 0) return;
    const int64_t row0 = lo + (int64_t)c * kC;
    const int rows = (int)(hi - row0 < kC ? hi - row0 : kC);
    const int Hk = a.c.k_heads, Hv = a.c.v_heads, share = Hv / Hk, dk = a.c.k_dim;
    const int twos = (share + 1) / 2, kh = blockIdx.y / twos, h0 = blockIdx.y % twos * 2;
    const int tid = threadIdx.x, lane = tid & 31, warp = (tid >> 5) & 3, b = tid >> 7;  // b: which of two heads
    const bool there = h0 + b < share;
    const int h = kh * share + h0 + (there ? b : 0);
    uint8_t* pair = a.ws + ((int64_t)blockIdx.x * Hk + kh) * pair_bytes(KD);
    uint8_t* out = a.ws + a.q_pieces * Hk * pair_bytes(KD) + ((int64_t)blockIdx.x * Hv + h) * kHeadBytes;
    Factors& f = *reinterpret_cast<Factors*>(out + 3 * kSquare);

    float g[2] = {0, 0}, beta2[2] = {0, 0};  // of two neighbouring tokens a lane, in the first warp
    if (warp == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = 2 * lane + i;
            if (r < rows) {
                g[i] = a.g[(row0 + r) * Hv + h];
                beta2[i] = a.beta[(row0 + r) * Hv + h];
            }
        }
    }
    // rows of K (the first four warps) and Q: KD / 8 threads a row
    constexpr int kRow = KD / 8, kPass = 128 / kRow, kN = kC / kPass;
    {
        const __nv_bfloat16* src = (b ? a.qr + row0 * a.q_ld : a.kr + row0 * a.k_ld) + kh * dk;
        const int64_t ld = b ? a.q_ld : a.k_ld;
        const int p = tid % kRow, r0 = (tid & 127) / kRow;
        uint4 w[kN];
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int r = r0 + i * kPass;
            w[i] = make_uint4(0, 0, 0, 0);
            if (r < rows && p * 8 < dk) w[i] = eight(src + r * ld + p * 8, a.wide);
        }
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int r = r0 + i * kPass;
            const uint32_t v[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
            *reinterpret_cast<uint4*>(m.kq[b] + piece_at<kRow>(r, p)) = w[i];
            uint32_t top = 0;  // of the magnitudes' bits, which order as the magnitudes do
#pragma unroll
            for (int j = 0; j < 4; ++j) top = __vmaxu2(top, v[j] & 0x7fff7fffu);
            top = max(top >> 16, top & 0xffffu);
#pragma unroll
            for (int d = 1; d < kRow; d <<= 1) top = max(top, __shfl_xor_sync(kAll, top, d));
            const int e = max((int)(top >> 7), 16);
            const float f = up(e);
            uint4 w16;
            uint32_t* hw = reinterpret_cast<uint32_t*>(&w16);
            float sum = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float x = __uint_as_float(v[j] << 16), y = __uint_as_float(v[j] & 0xffff0000u);
                hw[j] = pack(x * f, y * f);
                sum += fabsf(x) + fabsf(y);
            }
            if (h0 == 0) *reinterpret_cast<uint4*>(pair + b * (kC * KD * 2) + piece_at<kRow>(r, p)) = w16;
            if (!b) {
#pragma unroll
                for (int d = 1; d < kRow; d <<= 1) sum += __shfl_xor_sync(kAll, sum, d);
            }
            if (p == 0) {
                (b ? m.q_scale : m.k_scale)[r] = down(e);
                (b ? m.q_top : m.k_sum)[r] = b ? __uint_as_float(top << 16) : sum;
            }
        }
    }
    // sums of g in fp64 (64 additions), kept as two floats: differences of far sums stay exact
    if (warp == 0) {
        double G[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            G[i] = g[i] < -120.0f ? -120.0f : g[i];  // e^-120 is 0 in fp32, and -inf has no differences
            m.beta[b][2 * lane + i] = beta2[i];
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
            m.g_high[b][2 * lane + i] = (float)G[i];
            m.g_rest[b][2 * lane + i] = (float)(G[i] - (double)(float)G[i]);
        }
        if (lane == 0) m.most[b] = 0;
    }
    __syncthreads();

    const float *gh = m.g_high[b], *gr = m.g_rest[b];
    const uint32_t k_at = smem_at(m.kq[0]), q_at = smem_at(m.kq[1]);
    if (there) {
        // e^(G_i - G_j) = e^(G_i - G_16w) e^(G_16w - G_j) in the blocks left of the diagonal ones, both 1 or less
        float most_k = fmaxf(m.k_sum[lane], m.k_sum[lane + 32]);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) most_k = fmaxf(most_k, __shfl_xor_sync(kAll, most_k, d));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int j = lane + 32 * i;
            if (j < 16 * warp) m.before[b][warp][j] = expf((gh[16 * warp] - gh[j]) + (gr[16 * warp] - gr[j]));
        }
        __syncwarp();
        if (warp == 0) {  // which has the shortest rows below
            float most_ks = 0, most_left = 0;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = lane + 32 * i;
                const float e = expf(gh[r] + gr[r]);
                const float left = expf((gh[kC - 1] - gh[r]) + (gr[kC - 1] - gr[r])) * m.k_scale[r];
                f.ks[r] = e * m.k_scale[r];
                f.qs[r] = e * m.q_scale[r] * a.c.scale;
                f.left[r] = left;
                most_ks = fmaxf(most_ks, e * m.k_sum[r]);
                most_left = fmaxf(most_left, left);
                if (r == kC - 1) f.all = e;
            }
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                most_ks = fmaxf(most_ks, __shfl_xor_sync(kAll, most_ks, d));
                most_left = fmaxf(most_left, __shfl_xor_sync(kAll, most_left, d));
            }
            if (lane == 0) f.most_ks = most_ks, f.most_left = most_left;
        }
        // A and P, rows 16 warp .. +15, columns up to the diagonal block
        float after[2], beta[2], p_up[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = 16 * warp + (lane >> 2) + 8 * i;
            after[i] = expf((gh[r] - gh[16 * warp]) + (gr[r] - gr[16 * warp]));
            beta[i] = m.beta[b][r];
            // |q_i k_j| is at most the largest of q_i times the sum of k_j; a bound will do for 11 bits
            const int e = field(2.0f * m.q_top[r] * most_k);
            p_up[i] = up(e);
            if ((lane & 3) == 0) f.p[r] = down(e) * a.c.scale;
        }
        auto decay = [&](int n, float (&L)[2][2]) {
            const int j = 8 * n + 2 * (lane & 3);
            if (n >= 2 * warp) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int r = 16 * warp + (lane >> 2) + 8 * i;
                    L[i][0] = j <= r ? expf((gh[r] - gh[j]) + (gr[r] - gr[j])) : 0.0f;
                    L[i][1] = j + 1 <= r ? expf((gh[r] - gh[j + 1]) + (gr[r] - gr[j + 1])) : 0.0f;
                }
            } else {
                const float2 e = *reinterpret_cast<const float2*>(&m.before[b][warp][j]);
#pragma unroll
                for (int i = 0; i < 2; ++i) L[i][0] = after[i] * e.x, L[i][1] = after[i] * e.y;
            }
        };
#pragma unroll
        for (int which = 0; which < 2; ++which) {  // K K^T, then Q K^T
            float acc[8][4];
#pragma unroll
            for (int n = 0; n < 8; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[n][i] = 0;
#pragma unroll
            for (int t = 0; t < KD / 16; ++t) {
                uint32_t l[4];
                ldmatrix(l, left_at<kRow>(which ? q_at : k_at, 16 * warp, 2 * t, lane));
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    if (n > warp) continue;
                    uint32_t w[4];
                    ldmatrix(w, right_at<kRow>(k_at, 16 * n, 2 * t, lane));
                    mma_bf16(acc[2 * n], l, w[0], w[1]);
                    mma_bf16(acc[2 * n + 1], l, w[2], w[3]);
                }
            }
#pragma unroll
            for (int n = 0; n < 8; ++n) {
                if (n > 2 * warp + 1) continue;
                const int j = 8 * n + 2 * (lane & 3);
                float L[2][2];
                decay(n, L);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int r = 16 * warp + (lane >> 2) + 8 * i;
                    const float by = which ? p_up[i] : beta[i];
                    float v0 = by * (L[i][0] * acc[n][2 * i]), v1 = by * (L[i][1] * acc[n][2 * i + 1]);
                    if (n >= 2 * warp) {  // nothing from above the diagonal, also where a product is not a number
                        if (j + !which > r) v0 = 0;
                        if (j + 1 + !which > r) v1 = 0;
                    }
                    if (which)
                        *reinterpret_cast<uint32_t*>(out + 2 * kSquare + piece_at<8>(r, n) + 4 * (lane & 3)) = pack(v0, v1);
                    else
                        *reinterpret_cast<float2*>(&m.A[b][r][j]) = make_float2(v0, v1);
                }
            }
        }
    }
    __syncthreads();  // all are done with K and Q, where T goes
    if (there) {
        // the diagonal block
        if (lane < 16) {
            const float* A = &m.A[b][16 * warp][16 * warp];
            float t[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float sum[2] = {i == lane ? 1.0f : 0.0f, 0};
#pragma unroll
                for (int j = 0; j < i; j += 4) {
                    const float4 r = *reinterpret_cast<const float4*>(A + i * kPitch + j);
                    sum[0] = fmaf(-r.x, t[j], sum[0]);
                    if (j + 1 < i) sum[1] = fmaf(-r.y, t[j + 1], sum[1]);
                    if (j + 2 < i) sum[0] = fmaf(-r.z, t[j + 2], sum[0]);
                    if (j + 3 < i) sum[1] = fmaf(-r.w, t[j + 3], sum[1]);
                }
                t[i] = sum[0] + sum[1];
                m.T[b][16 * warp + i][16 * warp + lane] = t[i];
            }
        }
        head_barrier(b);
        auto A = [&](int i, int k) { return &m.A[b][16 * i][16 * k]; };
        auto T = [&](int i, int k) { return &m.T[b][16 * i][16 * k]; };
        if ((warp & 1) == 0) {  // T_10, T_32
            const int i = warp + 1;
            float acc[2][4] = {}, acc2[2][4] = {};
            block_product(acc, A(i, warp), T(warp, warp), lane);
            block_store(T(warp, i), acc, 1.0f, lane);  // above the diagonal, where nothing else stands
            __syncwarp();
            block_product(acc2, T(i, i), T(warp, i), lane);
            block_store(T(i, warp), acc2, -1.0f, lane);
        }
        head_barrier(b);
        {  // W = A_21 T_11, to the upper right quarter: blocks (0, 2), (0, 3), (1, 2), (1, 3)
            const int i = 2 + (warp >> 1), j = warp & 1;
            float acc[2][4] = {};
            block_product(acc, A(i, 1), T(1, j), lane);
            if (j == 0) block_product(acc, A(i, 0), T(0, 0), lane);
            block_store(T(j, i), acc, 1.0f, lane);
        }
        head_barrier(b);
        {  // the lower left quarter: -T_22 W
            const int i = 2 + (warp >> 1), j = warp & 1;
            float acc[2][4] = {};
            block_product(acc, T(i, i), T(j, i), lane);
            if (i == 3) block_product(acc, T(3, 2), T(j, 2), lane);
            block_store(T(i, j), acc, -1.0f, lane);
        }
        head_barrier(b);
        {
            // rows of T diag(beta) out: eight threads a row
            const int p = tid & 7;
            float beta[8], most = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) beta[j] = m.beta[b][8 * p + j];
            for (int row = (tid & 127) >> 3; row < kC; row += 16) {
                const float4 x = *reinterpret_cast<const float4*>(&m.T[b][row][8 * p]);
                const float4 y = *reinterpret_cast<const float4*>(&m.T[b][row][8 * p + 4]);
                float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w}, top = 0, sum = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    v[j] = (p >> 1) <= (row >> 4) ? v[j] * beta[j] : 0.0f;  // above the diagonal blocks stand other things
                    top = fmaxf(top, fabsf(v[j]));
                    sum += fabsf(v[j]);
                }
#pragma unroll
                for (int d = 1; d < 8; d <<= 1) {
                    top = fmaxf(top, __shfl_xor_sync(kAll, top, d));
                    sum += __shfl_xor_sync(kAll, sum, d);
                }
                most = fmaxf(most, sum);
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
                if (p == 0) f.t[row] = down(e);
            }
            if (p == 0) atomicMax(&m.most[b], __float_as_uint(most));
        }
        head_barrier(b);
        if ((tid & 127) == 0) f.most_t = __uint_as_float(m.most[b]);
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
// Exponent fields of two columns' largest magnitudes, of which each lane has its rows' as the high halves of floats in one
// word.  The same word for the 8 lanes of a column pair.
__device__ __forceinline__ uint32_t columns_max(uint32_t w) {
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) w = __vmaxu2(w, __shfl_xor_sync(kAll, w, d));
    return w;
}
__device__ __forceinline__ float first_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float second_of(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

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

    int unit[NT][2];  // S stands in units of down(unit), by column
#pragma unroll
    for (int n = 0; n < NT; ++n) unit[n][0] = unit[n][1] = kOne;
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

        // Scales.  S's is from its largest value.  Those of V - e^G K S^T, U and what goes into S are from bounds that
        // follow from it: fp16 has room for a bound that is 2^10 too large without loss, and reductions over the
        // columns in mid-chunk would be on the path from one chunk to the next.
        float s_up[NT][2], s_down[NT][2], x_up[NT][2], x_down[NT][2], u_up[NT][2], u_down[NT][2], l_up[NT][2], grow[NT][2];
        uint32_t v[NT][4][2];
        const float most_ks = f.most_ks, most_t = f.most_t, most_left = f.most_left, all = f.all;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float m0 = 0, m1 = 0;
#pragma unroll
            for (int m = 0; m < kM; ++m) {
                m0 = fmaxf(m0, fmaxf(fabsf(S[n][m][0]), fabsf(S[n][m][2])));
                m1 = fmaxf(m1, fmaxf(fabsf(S[n][m][1]), fabsf(S[n][m][3])));
            }
            const uint32_t ms = columns_max(__byte_perm(__float_as_uint(m0), __float_as_uint(m1), 0x7632));
            uint32_t mv = 0;
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    v[n][m][i] = *reinterpret_cast<const uint32_t*>(V + (16 * m + r0 + 8 * i) * Shape::kVPitch + (d0 - first + 8 * n) * 2);
                    mv = __vmaxu2(mv, v[n][m][i] & 0x7fff7fffu);
                }
            mv = columns_max(mv);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float top = i ? second_of(ms) : first_of(ms);  // rounded down, but within its power of two
                const int e = field(top);
                s_up[n][i] = up(e);
                s_down[n][i] = down(e) * down(unit[n][i]);
                // a power of two above each bound; 2^14 stands for it
                const float x = (i ? second_of(mv) : first_of(mv)) + most_ks * (2.0f * top * down(unit[n][i]));
                const float u = x * most_t, l = u * most_left;
                const int ex = field(2.0f * x), eu = field(2.0f * u);
                x_up[n][i] = up(ex), x_down[n][i] = down(ex);
                u_up[n][i] = up(eu), u_down[n][i] = down(eu);
                // S has to stay finite in the new units, and its change of units a number of fp32; what updates lose by
                // that is 2^-60 of S, or 2^-100 of what they were made for before
                const int el = min(max(field(2.0f * l), max(e + unit[n][i] - kOne - 60, unit[n][i] - 120)), 254);
                l_up[n][i] = up(el);
                grow[n][i] = all * __uint_as_float((uint32_t)(127 + min(max(unit[n][i] - el, -126), 127)) << 23);
                unit[n][i] = el;
            }
        }

        // K S^T and Q S^T
        float x[NT][4][4], qs[NT][4][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) x[n][m][i] = qs[n][m][i] = 0;
#pragma unroll
        for (int t = 0; t < kM; ++t) {
            Fragment b[NT];
            uint32_t kw[4][4], qw[4][4];
#pragma unroll
            for (int m = 0; m < 4; ++m) ldmatrix(kw[m], left_at<kRow>(K16, 16 * m, 2 * t, lane));
#pragma unroll
            for (int n = 0; n < NT; ++n) b[n] = split(S[n][t], s_up[n][0], s_up[n][1]);
#pragma unroll
            for (int m = 0; m < 4; ++m) ldmatrix(qw[m], left_at<kRow>(Q16, 16 * m, 2 * t, lane));
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int m = 0; m < 4; ++m) mma_f16(x[n][m], kw[m], b[n].high[0], b[n].high[1]);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int m = 0; m < 4; ++m) mma_f16(qs[n][m], qw[m], b[n].high[0], b[n].high[1]);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int m = 0; m < 4; ++m) mma_f16(x[n][m], kw[m], b[n].rest[0], b[n].rest[1]);
        }
        // X = V - e^G K S^T
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float ks = f.ks[16 * m + r0 + 8 * i];
                    x[n][m][2 * i] = fmaf(-ks * s_down[n][0], x[n][m][2 * i], first_of(v[n][m][i]));
                    x[n][m][2 * i + 1] = fmaf(-ks * s_down[n][1], x[n][m][2 * i + 1], second_of(v[n][m][i]));
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
            uint32_t high[4][4], rest[4][4];
#pragma unroll
            for (int m = t; m < 4; ++m) {
                ldmatrix(high[m], left_at<8>(T_high, 16 * m, 2 * t, lane));
                ldmatrix(rest[m], left_at<8>(T_rest, 16 * m, 2 * t, lane));
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) b[n] = split(x[n][t], x_up[n][0], x_up[n][1]);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int m = t; m < 4; ++m) mma_f16(u[n][m], high[m], b[n].high[0], b[n].high[1]);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int m = t; m < 4; ++m) mma_f16(u[n][m], rest[m], b[n].high[0], b[n].high[1]);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int m = t; m < 4; ++m) mma_f16(u[n][m], high[m], b[n].rest[0], b[n].rest[1]);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) u[n][m][i] *= f.t[16 * m + r0 + 8 * (i >> 1)] * x_down[n][i & 1];

        // S <- e^G_63 S + U^T (e^(G_63 - G) K)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int m = 0; m < kM; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) S[n][m][i] *= grow[n][i & 1];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            Fragment b[NT];
            const float l0 = f.left[16 * t + r0], l1 = f.left[16 * t + r0 + 8];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float left[4] = {u[n][t][0] * l0, u[n][t][1] * l0, u[n][t][2] * l1, u[n][t][3] * l1};
                b[n] = split(left, l_up[n][0], l_up[n][1]);
            }
#pragma unroll
            for (int half = 0; half < kM; half += 4) {
                uint32_t w[4][4];
#pragma unroll
                for (int m = 0; m < 4; ++m) ldmatrix_trans(w[m], right_at<kRow>(K16, 16 * t, 2 * (half + m), lane));
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int m = 0; m < 4; ++m) mma_f16(S[n][half + m], w[m], b[n].high[0], b[n].high[1]);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int m = 0; m < 4; ++m) mma_f16(S[n][half + m], w[m], b[n].rest[0], b[n].rest[1]);
            }
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
            uint32_t b[NT][2], w[4][4];
#pragma unroll
            for (int n = 0; n < NT; ++n) split_high(b[n], u[n][t], u_up[n][0], u_up[n][1]);
#pragma unroll
            for (int m = t; m < 4; ++m) ldmatrix(w[m], left_at<8>(P16, 16 * m, 2 * t, lane));
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int m = t; m < 4; ++m) mma_f16(pu[n][m], w[m], b[n][0], b[n][1]);
        }
        const int64_t row0 = lo + (int64_t)c * kC;
        const int rows = (int)(hi - row0 < kC ? hi - row0 : kC);
        __nv_bfloat16* o = a.o + (row0 + r0) * a.o_ld + h * dv + d0;
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = 16 * m + 8 * i;
                const float fq = f.qs[r + r0], fp = f.p[r + r0];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const float y0 = fmaf(fq * s_down[n][0], qs[n][m][2 * i], fp * u_down[n][0] * pu[n][m][2 * i]);
                    const float y1 = fmaf(fq * s_down[n][1], qs[n][m][2 * i + 1], fp * u_down[n][1] * pu[n][m][2 * i + 1]);
                    if (r + r0 < rows && d0 + 8 * n < dv) {
                        const __nv_bfloat162 y = __floats2bfloat162_rn(y0, y1);
                        if (a.o_pairs) {
                            *reinterpret_cast<__nv_bfloat162*>(o + r * a.o_ld + 8 * n) = y;
                        } else {
                            o[r * a.o_ld + 8 * n] = y.x;
                            o[r * a.o_ld + 8 * n + 1] = y.y;
                        }
                    }
                }
            }
    }
    if (state) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int m = 0; m < kM; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int d = d0 + 8 * n + (i & 1), k = 16 * m + (lane >> 2) + 8 * (i >> 1);
                    if (d < dv && k < dk) state[(int64_t)d * dk + k] = S[n][m][i] * down(unit[n][i & 1]);
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
    if (cudaError_t e = launch(prepare_kernel<KD>, dim3((unsigned)a.q_pieces, (unsigned)(a.c.k_heads * ((a.c.v_heads / a.c.k_heads + 1) / 2))),
                               kPrepare,
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
