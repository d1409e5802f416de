// mix.h -- the operators between two expert layers (short convolution, head
// norms, gated delta rule): launchers, and how a batch's sequences are found.
#pragma once

#include "mx.h"

namespace moe {

// Rows up to which a sequence of the delta rule runs token by token.  In us, token by token and in a chunk, of 24 and of 32
// rows: 32 heads of 128 x 128, one run 16.3 and 17.4, 20.7 and 17.3; 16 runs 66 and 65, 84 and 66; 64 runs 247 and 242, 319 and 243.
// 8 heads of 128 x 128, one run 16.2 and 17.0, 20.6 and 17.0; 64 runs 67 and 66, 84 and 66.  16 heads of 64 x 96, one run 11.7 and
// 14.7, 14.6 and 14.7; 64 runs 83 and 91, 104 and 92.  Of 64 x 64, 16 runs 17.2 and 24.3, 21.1 and 24.4, and equal at 40 rows.  So
// smaller heads could go to 32 rows; the bound is the same for all, as a sequence's results may depend on its length alone.
constexpr int kDeltaShort = 24;
constexpr int kDeltaChunk = 64;

// A batch's sequences (moe_seqs).  Lists on the device are not trusted: rows
// are clamped to 0..T and a slot outside 0..slots-1 reads as -1.
struct Seqs {
    const int32_t* offsets;  // NULL: sequence s has rows s * per .. s * per + per - 1
    const int32_t* slot_of;
    const int32_t* carry_of;
    int n, per;
    int64_t T;
    int64_t slots;  // INT64_MAX without a state

    __device__ __forceinline__ int64_t start(int s) const {
        if (!offsets) return (int64_t)s * per;
        const int64_t o = offsets[s];
        return o < 0 ? 0 : o > T ? T : o;
    }
    __device__ __forceinline__ int slot(int s) const {
        const int v = slot_of ? slot_of[s] : s;
        return v < 0 || v >= slots ? -1 : v;
    }
    __device__ __forceinline__ bool carry(int s) const { return !carry_of || carry_of[s] != 0; }

    // Pieces of `size` rows: sequence s has its pieces at start(s) / size + s and after (consecutive sequences never
    // overlap, see MxRows); `pieces` is their number at most.  The sequence whose pieces begin at or before `piece`,
    // found by a whole warp, 32 sequences a step.
    int64_t pieces(int size) const { return offsets ? T / size + n : (int64_t)n * ((per + size - 1) / size); }
    template <int SIZE>
    __device__ __forceinline__ int find(int64_t piece, int& index) const {
        if (!offsets) {
            const int each = (per + SIZE - 1) / SIZE;
            index = (int)(piece % each);
            return (int)(piece / each);
        }
        int lo = 0, left = n;
        while (left > 1) {
            const int step = (left + 31) >> 5, at = (threadIdx.x & 31) * step;
            const bool before = at < left && start(lo + at) / SIZE + lo + at <= piece;
            const int k = __popc(__ballot_sync(0xffffffffu, before));
            const int skip = k > 1 ? (k - 1) * step : 0;
            lo += skip;
            left = min(step, left - skip);
        }
        index = (int)(piece - (start(lo) / SIZE + lo));
        return lo;
    }
    template <int SIZE>
    __device__ __forceinline__ int64_t piece_of(int s) const {
        return offsets ? start(s) / SIZE + s : (int64_t)s * ((per + SIZE - 1) / SIZE);
    }
};

// v / (1 + exp(-v)).  expf, not one multiplication and ex2: that loses |v| 2^-24 of the value, too much for fp32 results
// from v = -8 on.  Below -80 it is v exp(v), in two steps: 1 / (1 + exp(-v)) would be below what rcp.approx.ftz gives from -87.3 on,
// and v times it is a normal number down to -91.8.
__device__ __forceinline__ float silu(float v) {
    if (v < -80.0f) {
        const float half = expf(0.5f * v);
        return v * half * half;
    }
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + expf(-v)));
    return v * r;
}

// For results that are rounded to bf16: silu(v) = 2^-8 v times this, relative 2^-21 + |v| 2^-24, a fifth of the instructions.
// Numerator and denominator are 2^-8 of the formula's: rcp.approx.ftz gives 0 for 2^126 and more, which 1 + exp(-v) reaches while
// v / (1 + exp(-v)) is still 1e-36.  This way what is 2^-126 or more is there.  x: v / TIMES; who calls puts the 2^-8 where it
// costs no instruction a value (one more cost the convolution of prompts 3%).
template <int TIMES>
__device__ __forceinline__ float sigmoid_256(float x) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(fmaf(-1.44269504f * TIMES, x, -8.0f)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f / 256 + e));
    return r;
}

// Two fp32 numbers in a 64-bit register: one instruction multiplies and adds both.
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 both(float x, float y) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 apart(f32x2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// two bf16 as they are in memory
__device__ __forceinline__ f32x2 both_of(uint32_t w) { return both(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)); }

// mix_conv.cu
cudaError_t launch_conv(const Seqs& q, const void* x, int type, int64_t x_ld, int channels, const void* w, int w_type,
                        int width, const float* bias, int act, void* state, void* y, int64_t y_ld, cudaStream_t st);
// mix_norm.cu
cudaError_t launch_head_norm(const moe_head_norm_config& c, const moe_heads& a, const moe_heads* b, const int32_t* pos,
                             const float* inv_freq, int64_t T, cudaStream_t st);
// mix_delta.cu, mix_chunks.cu
struct DeltaArgs {
    moe_delta_config c;
    Seqs q;
    const __nv_bfloat16 *qr, *kr, *vr;
    int64_t q_ld, k_ld, v_ld, o_ld;
    const float *g, *beta;
    float* state;
    __nv_bfloat16* o;
    uint8_t* ws;
    int longer_than;  // the chunked kernels leave out sequences of so many rows or fewer, the stepping one those of more
    int64_t q_pieces;  // of kDeltaChunk rows
    bool wide;         // q, k and v rows are aligned for 16-byte loads
    bool o_pairs;      // o's for stores of two values
};
size_t delta_workspace(const moe_delta_config& c, int64_t T, int n);
cudaError_t launch_delta_steps(const DeltaArgs& a, cudaStream_t st);
cudaError_t launch_delta_chunks(const DeltaArgs& a, cudaStream_t st);

}  // namespace moe
