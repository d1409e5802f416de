// mix_delta.cu -- the gated delta rule token by token, for short runs (long
// ones: mix_chunks.cu).

#include "mix.h"

namespace moe {
namespace {

constexpr unsigned kAll = 0xffffffffu;
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

}  // namespace

cudaError_t launch_delta_steps(const DeltaArgs& a, cudaStream_t st) {
    const int blocks = (a.c.v_dim + kStepRows - 1) / kStepRows;
    const dim3 grid((unsigned)(a.q.n * blocks), (unsigned)a.c.v_heads);
    if (a.c.k_dim <= 64) return launch(steps_kernel<64>, grid, 128, 0, st, 1, a);
    return launch(steps_kernel<128>, grid, 128, 0, st, 1, a);
}

}  // namespace moe
