// mix_delta.cu -- the gated delta rule token by token, for short runs (long
// ones: mix_chunks.cu).

#include "mix.h"

namespace moe {
namespace {

constexpr unsigned kAll = 0xffffffffu;
// With S' = e^g S:  u = beta (v - S' k),  S <- S' + u k^T,  o = S' q + u (k q):
// all sums over k_dim of one token (S' k, S' q, k q) are formed together.
// Eight threads share a row of S and keep it in registers over the tokens of
// the run, four rows each.  One token is bound by reading and writing S: its
// loads are issued before anything else is waited for, together with the first
// token's.  A run is a chain: its state's loads, then one token after another, of
// about 350 instructions a warp (38% of the slots with 2.6 warps a scheduler);
// products go two at a time, and four rows share what is unpacked of k and q.  64
// sequences, 32 heads, 128 x 128: one token each (256 MB of states) 42.6 us, 89% of
// the measured copy's rate; four tokens for each of 16 sequences 19.3 us, in three
// rounds of CTAs.  Before decays near 1 had a way of their own 42.4 and 18.6, then
// with two rows a thread 43.7 and 21.7, with sixteen threads a row 50.7 and 24.5.
constexpr int kLanes = 8, kRows = 4;
constexpr int kStepRows = 128 / kLanes * kRows;  // rows of S of a CTA

// KD / 8 values of a row of K or Q, still packed
template <int KD>
struct Token {
    static constexpr int kE = KD / kLanes;  // values of a thread: 16 or 8
    uint32_t k[kE / 2], q[kE / 2];
    uint32_t v[kRows / 2];  // of two rows each
    float g, beta;
};
template <int N>
__device__ __forceinline__ void packed(uint32_t (&w)[N], const __nv_bfloat16* p, bool wide) {
    if (wide) {
        if constexpr (N == 2) {
            *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(p);
        } else {
#pragma unroll
            for (int i = 0; i < N; i += 4) *reinterpret_cast<uint4*>(w + i) = *reinterpret_cast<const uint4*>(p + 2 * i);
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            w[i] = reinterpret_cast<const unsigned short*>(p)[2 * i] | (uint32_t)reinterpret_cast<const unsigned short*>(p)[2 * i + 1] << 16;
    }
}

template <int KD>
__global__ void __launch_bounds__(128) steps_kernel(const __grid_constant__ DeltaArgs a) {
    after_previous();
    constexpr int kE = KD / kLanes;
    const int dk = a.c.k_dim, dv = a.c.v_dim, Hv = a.c.v_heads;
    const int blocks = (dv + kStepRows - 1) / kStepRows;
    const int s = blockIdx.x / blocks, h = blockIdx.y, kh = h / (Hv / a.c.k_heads);
    const int64_t lo = a.q.start(s), hi = a.q.start(s + 1);
    const int slot = a.q.slot(s);
    const bool carry = a.state && a.q.carry(s);
    if (lo >= hi || hi - lo > a.longer_than || slot < 0) return;
    // a thread's values of a row of S, in pieces of 8 (k_dim is a multiple of that)
    constexpr int kPiece = 8;
    const int lane = threadIdx.x % kLanes;
    auto at = [&](int i) { return (lane + kLanes * (i / kPiece)) * kPiece + i % kPiece; };
    const int d0 = (blockIdx.x % blocks) * kStepRows + threadIdx.x / kLanes * kRows;
    const bool in_v = d0 < dv;  // and the other rows: v_dim is a multiple of 8

    // of the token whose loads come next
    const __nv_bfloat16 *kp = a.kr + lo * a.k_ld + kh * dk, *qp = a.qr + lo * a.q_ld + kh * dk, *vp = a.vr + lo * a.v_ld + h * dv + d0;
    const float *gp = a.g + lo * Hv + h, *bp = a.beta + lo * Hv + h;
    auto load = [&](Token<KD>& in) {
#pragma unroll
        for (int i = 0; i < kE; i += kPiece) {
            uint32_t k[kPiece / 2] = {}, q[kPiece / 2] = {};
            if (at(i) < dk) {
                packed(k, kp + at(i), a.wide);
                packed(q, qp + at(i), a.wide);
            }
#pragma unroll
            for (int j = 0; j < kPiece / 2; ++j) in.k[i / 2 + j] = k[j], in.q[i / 2 + j] = q[j];
        }
#pragma unroll
        for (int p = 0; p < kRows / 2; ++p) {
            in.v[p] = 0;
            if (in_v)
                in.v[p] = a.wide ? reinterpret_cast<const uint32_t*>(vp)[p]
                                 : reinterpret_cast<const unsigned short*>(vp)[2 * p] |
                                       (uint32_t)reinterpret_cast<const unsigned short*>(vp)[2 * p + 1] << 16;
        }
        in.g = *gp;
        in.beta = *bp;
        kp += a.k_ld, qp += a.q_ld, vp += a.v_ld, gp += Hv, bp += Hv;
    };
    float* state = a.state ? a.state + (((int64_t)slot * Hv + h) * dv + d0) * dk : nullptr;
    f32x2 S[kRows][kE / 2];
#pragma unroll
    for (int p = 0; p < kRows; ++p)
#pragma unroll
        for (int i = 0; i < kE; i += 4) {
            S[p][i / 2] = S[p][i / 2 + 1] = 0;
            if (carry && at(i) < dk && in_v) {
                const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(state + p * dk + at(i));
                S[p][i / 2] = v.x, S[p][i / 2 + 1] = v.y;
            }
        }
    Token<KD> next;
    load(next);
    // the next 16 tokens' rows to L1, eight threads a token: without this four tokens for each of 16 sequences take 0.8 us more
    const int ahead = 1 + threadIdx.x / 8, part = threadIdx.x % 8;
    if (ahead < hi - lo) {
        const void* line = nullptr;
        if (part < 2 && part * 64 < dk) line = a.kr + (lo + ahead) * a.k_ld + kh * dk + part * 64;
        if (part / 2 == 1 && part % 2 * 64 < dk) line = a.qr + (lo + ahead) * a.q_ld + kh * dk + part % 2 * 64;
        if (part == 4) line = a.vr + (lo + ahead) * a.v_ld + h * dv + (blockIdx.x % blocks) * kStepRows;
        if (part == 5) line = a.g + (lo + ahead) * Hv + h;
        if (part == 6) line = a.beta + (lo + ahead) * Hv + h;
        if (line) asm volatile("prefetch.global.L1 [%0];" ::"l"(line));
    }
    __nv_bfloat16* o = a.o + lo * a.o_ld + h * dv + d0 + lane;
    for (int tokens = (int)(hi - lo); tokens > 0; --tokens) {
        const Token<KD> in = next;
        if (tokens > 1) load(next);
        // S <- e^g S.  Decays near 1 as S + (e^g - 1) S: with one fp32 of e^-0.00001, off by the same at every token, S was 2^-10
        // off after 16384 of them.  16 runs of 4 19.3 us instead of 18.6; with the sums in both branches 20.9
        const bool near = fabsf(in.g) < 0.25f;
        const float by = near ? expm1f(in.g) : expf(in.g);
        const f32x2 bys = both(by, by);
        if (near) {
#pragma unroll
            for (int p = 0; p < kRows; ++p)
#pragma unroll
                for (int i = 0; i < kE / 2; ++i) S[p][i] = fma2(S[p][i], bys, S[p][i]);
        } else {
#pragma unroll
            for (int p = 0; p < kRows; ++p)
#pragma unroll
                for (int i = 0; i < kE / 2; ++i) S[p][i] = mul2(S[p][i], bys);
        }
        f32x2 k[kE / 2], q[kE / 2], kq2 = 0, sk2[kRows], sq2[kRows];
#pragma unroll
        for (int i = 0; i < kE / 2; ++i) {
            k[i] = both_of(in.k[i]), q[i] = both_of(in.q[i]);
            kq2 = fma2(k[i], q[i], kq2);
        }
#pragma unroll
        for (int p = 0; p < kRows; ++p) {
            sk2[p] = sq2[p] = 0;
#pragma unroll
            for (int i = 0; i < kE / 2; ++i) {
                sk2[p] = fma2(S[p][i], k[i], sk2[p]);
                sq2[p] = fma2(S[p][i], q[i], sq2[p]);
            }
        }
        float sk[kRows], sq[kRows], kq = apart(kq2).x + apart(kq2).y;
#pragma unroll
        for (int p = 0; p < kRows; ++p) sk[p] = apart(sk2[p]).x + apart(sk2[p]).y, sq[p] = apart(sq2[p]).x + apart(sq2[p]).y;
#pragma unroll
        for (int d = 1; d < kLanes; d <<= 1) {
            kq += __shfl_xor_sync(kAll, kq, d);
#pragma unroll
            for (int p = 0; p < kRows; ++p) {
                sk[p] += __shfl_xor_sync(kAll, sk[p], d);
                sq[p] += __shfl_xor_sync(kAll, sq[p], d);
            }
        }
        float y[kRows];
#pragma unroll
        for (int p = 0; p < kRows; ++p) {
            const float u = in.beta * (__uint_as_float(p & 1 ? in.v[p / 2] & 0xffff0000u : in.v[p / 2] << 16) - sk[p]);
            const f32x2 us = both(u, u);
#pragma unroll
            for (int i = 0; i < kE / 2; ++i) S[p][i] = fma2(us, k[i], S[p][i]);
            y[p] = a.c.scale * fmaf(u, kq, sq[p]);
        }
        float mine = y[0];
#pragma unroll
        for (int p = 1; p < kRows; ++p) mine = lane == p ? y[p] : mine;
        if (lane < kRows && in_v) *o = __float2bfloat16_rn(mine);
        o += a.o_ld;
    }
    let_next_start();  // at the kernel's start 16 runs of 4 take 0.7 us more, one token 0.2
    if (state && in_v) {
#pragma unroll
        for (int p = 0; p < kRows; ++p)
#pragma unroll
            for (int i = 0; i < kE; i += 4)
                if (at(i) < dk)
                    *reinterpret_cast<ulonglong2*>(state + p * dk + at(i)) = make_ulonglong2(S[p][i / 2], S[p][i / 2 + 1]);
    }
}

}  // namespace

cudaError_t launch_delta_steps(const DeltaArgs& a, cudaStream_t st) {
    const int blocks = (a.c.v_dim + kStepRows - 1) / kStepRows;
    const dim3 grid((unsigned)(a.q.n * blocks), (unsigned)a.c.v_heads);
    if (a.c.k_dim <= 64) return launch(steps_kernel<64>, grid, 128, 0, st, 1, a);
    return launch(steps_kernel<128>, grid, 128, 0, st, 1, a);
}

}  // namespace moe
