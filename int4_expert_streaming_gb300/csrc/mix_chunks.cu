// mix_chunks.cu -- the gated delta rule in chunks of 64 tokens on the tensor
// cores, for long runs (short ones: mix_delta.cu).
//
// A chunk with the state S before it, G_i the sum of g up to token i, L_ij =
// e^(G_i - G_j) for j <= i:
//   A_ij = beta_i L_ij (k_i k_j), j < i         T = (1 + A)^-1 diag(beta)
//   X = V - e^G K S^T                           U = T X, the chunk's updates
//   O = scale (e^G Q S^T + P U), P_ij = L_ij q_i k_j
//   S <- e^(G_63) S + U^T (e^(G_63 - G) K)
// All exponents are of differences that are 0 or less.  T and P T do not depend
// on S: prepare_kernel finds them for all chunks at once.  chunks_kernel then
// goes through a sequence's chunks one after another, three products each:
//   (K; Q) S^T,   (T; P T) X,   K^T U
//
// Numbers enter the products as fp16.  K and Q are bf16, exact in fp16 once a
// row is scaled by a power of two that brings its largest value to 2^14 (values
// 2^-28 below that lose bits).  S, X, T, P, P T and the updates are sums in fp32
// and enter as two fp16 numbers each, high and rest, together 22 bits, in units
// that bring their largest value or a bound of it to 2^14: all 22 bits are there
// down to 2^-16 of that, so a bound may be generous.  The product of two rests is
// left out.  What goes into o alone has both numbers too: with the high ones
// only, o was off by 2^-12 of |S| |q|, more than its rounding to bf16 where sums
// cancel in it (a key that is written over).  That costs 4096 tokens with 32 heads of
// 128 178 us instead of 165, 64 prompts of 64 256 instead of 252.
#include <cuda_fp16.h>
#include <string.h>

#include "mix.h"
namespace moe {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kC = kDeltaChunk;

// Workspace, per chunk and k head: K16 and Q16, panels of 64 columns of 128 rows
// (K's, then Q's).  Per chunk and v head: T high, P T high, T rest and P T rest
// [64 x 64 each], and the factors.  At the end the sequences (Taken).  Rows are of 128 bytes with their 16-byte pieces
// exchanged (piece p of row r at p ^ (r & 7)): read from shared memory without
// conflicts.
struct Factors {
    float ks[kC];    // e^G_i times the unit of k's row
    float left[kC];  // e^(G_63 - G_i) times the unit of k's row
    float qs[kC];    // e^G_i times the unit of q's row, times the factor on o
    float pt[kC];    // units of P T's row and of T, times the factor on o
    float all, rest; // e^G_63: their sum
    float t;         // unit of T
    // how large things can get: X over the largest of S, beside V; what goes into S over the largest of X
    float most_ks, most_l;
};
constexpr int kSquare = kC * 128;
constexpr int kPanel = 2 * kSquare;
constexpr int kHeadTiles = 4 * kSquare;
constexpr int kHeadBytes = (kHeadTiles + (int)sizeof(Factors) + 127) / 128 * 128;

constexpr int kSorted = 512;
// A sequence as chunks_kernel takes it, in one load: lists, slot and offsets one after another cost a CTA 1 us (64 prompts of
// 64 tokens, 32 heads, 256 us: 16 us more)
struct alignas(16) Taken {
    int lo, hi, slot;  // rows; slot -1: not taken
    uint32_t piece;    // its first chunk's place; bit 31: it goes on from its slot
};

__host__ __device__ constexpr int padded_dim(int k_dim) { return k_dim <= 64 ? 64 : 128; }
__host__ __device__ constexpr int pair_bytes(int KD) { return KD / 64 * kPanel; }

__device__ __forceinline__ uint32_t smem_at(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void ldmatrix(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void ldmatrix_trans(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void stmatrix(uint32_t at, uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(w0), "r"(w1), "r"(w2), "r"(w3) : "memory");
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

// two numbers as the high ones and what is left of them
__device__ __forceinline__ uint32_t halved(float x, float y, uint32_t& rest) {
    const uint32_t high = pack(x, y);
    const float2 h = unpack(high);
    rest = pack(x - h.x, y - h.y);
    return high;
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
// the same block as right operand, with rows of the memory as its columns
template <int N>
__device__ __forceinline__ uint32_t right_at(uint32_t base, int r0, int p, int lane) {
    return base + piece_at<N>(r0 + (lane & 7) + ((lane >> 4) << 3), p + ((lane >> 3) & 1));
}


// the same in K16 over Q16, piece p of a row of KD / 8: rows r0 .. r0+15, pieces p, p+1, as left operand; and, transposed,
// with the pieces' columns as its rows
__device__ __forceinline__ uint32_t rows_at(uint32_t base, int r0, int p, int lane) {
    return left_at<8>(base + (p >> 3) * kPanel, r0, p & 7, lane);
}
__device__ __forceinline__ uint32_t columns_at(uint32_t base, int r0, int p, int lane) {
    return right_at<8>(base + (p >> 3) * kPanel, r0, p & 7, lane);
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
    unsigned top[2], most[2];  // bits of the largest |T| and of the largest row sum
    float left[2];             // the largest e^(G_63 - G_i) times the unit of k's row
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
// to 2^-22 of the value, and 0 below 2^-126
__device__ __forceinline__ float exp2_of(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// the four warps of one of the two heads
__device__ __forceinline__ void head_barrier(int b) {
    if (b)
        asm volatile("bar.sync 2, 128;" ::: "memory");
    else
        asm volatile("bar.sync 1, 128;" ::: "memory");
}

__device__ __forceinline__ Taken* taken_of(const DeltaArgs& a, int pair, int head) {
    return reinterpret_cast<Taken*>(a.ws + a.q_pieces * ((int64_t)a.c.k_heads * pair + (int64_t)a.c.v_heads * head));
}
// The sequences first .. first + kPrepare - 1 to their places.  Longest first,
// so that their CTAs start first and the last to start are short (9001 rows in 24
// sequences: 132 us, in their own order 141).  Above kSorted sequences, where the
// comparisons would take longer than a chunk, they stand in their own order: no one
// of so many is long beside the whole.
__device__ __forceinline__ void list_sequences(const DeltaArgs& a, int first, int* lens) {
    const int n = a.q.n, s = first + threadIdx.x;
    const bool sorted = n <= kSorted;
    if (sorted) {
        for (int i = threadIdx.x; i < n; i += kPrepare) lens[i] = (int)(a.q.start(i + 1) - a.q.start(i));
        __syncthreads();
    }
    if (s >= n) return;
    const int64_t lo = a.q.start(s), len = a.q.start(s + 1) - lo;
    int place = s;
    if (sorted) {
        place = 0;
        for (int j = 0; j < n; ++j) place += lens[j] > lens[s] || (lens[j] == lens[s] && j < s);
    }
    const int slot = len > a.longer_than ? a.q.slot(s) : -1;
    taken_of(a, pair_bytes(padded_dim(a.c.k_dim)), kHeadBytes)[place] =
        {(int)lo, (int)(lo + len), slot, (uint32_t)a.q.piece_of<kC>(s) | (a.state && a.q.carry(s) ? 1u << 31 : 0u)};
}

// One chunk and two v heads of a k head: K16 and Q16, the factors, T and P T.
// (1 + A)^-1 by blocks of 16: the four on the diagonal by substitution in fp32,
// a lane a column; then T_10 and T_32, and of those the lower left quarter, by
//   (T_11 0; T_21 T_22) with T_21 = -T_22 A_21 T_11.
// Two heads a CTA, since they share K and Q; three CTAs an SM.  4096 tokens, 16
// and 32 heads of 128: 52 us of the call's 178, with 48% of the issue slots and
// 68% of shared memory's rate in use and a tenth of the time in barriers.
template <int KD>
__global__ void __launch_bounds__(kPrepare, 3) prepare_kernel(const __grid_constant__ DeltaArgs a) {
    extern __shared__ __align__(128) uint8_t raw[];
    PrepareShared<KD>& m = *reinterpret_cast<PrepareShared<KD>*>(raw);
    after_previous();
    if (blockIdx.x >= a.q_pieces) {
        if (blockIdx.y == 0) list_sequences(a, (int)(blockIdx.x - a.q_pieces) * kPrepare, reinterpret_cast<int*>(raw));
        return;
    }
    int c;
    const int s = a.q.find<kC>(blockIdx.x, c);
    const int64_t lo = a.q.start(s), hi = a.q.start(s + 1);
    if (c < 0 || hi - lo <= a.longer_than || (int64_t)c * kC >= hi - lo || a.q.slot(s) < 0) return;
    const int64_t row0 = lo + (int64_t)c * kC;
    const int rows = (int)(hi - row0 < kC ? hi - row0 : kC);
    const int Hk = a.c.k_heads, Hv = a.c.v_heads, share = Hv / Hk, dk = a.c.k_dim;
    const int twos = (share + 1) / 2, kh = blockIdx.y / twos, h0 = blockIdx.y % twos * 2;
    // b: which of two heads.  A head's later warps have more to do (T is triangular); the second head's are numbered from
    // the back, so that each scheduler has one of many blocks and one of few
    const int tid = threadIdx.x, lane = tid & 31, b = tid >> 7, warp = b ? 7 - (tid >> 5) : tid >> 5;
    const bool there = h0 + b < share;
    const int h = kh * share + h0 + (there ? b : 0);
    uint8_t* pair = a.ws + ((int64_t)blockIdx.x * Hk + kh) * pair_bytes(KD);
    uint8_t* out = a.ws + a.q_pieces * Hk * pair_bytes(KD) + ((int64_t)blockIdx.x * Hv + h) * kHeadBytes;
    Factors& f = *reinterpret_cast<Factors*>(out + kHeadTiles);

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
        // the rows' largest magnitudes, whose bits order as they do: two rows a word
        uint32_t tops[kN / 2];
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const uint32_t v[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
            *reinterpret_cast<uint4*>(m.kq[b] + piece_at<kRow>(r0 + i * kPass, p)) = w[i];
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) top = __vmaxu2(top, v[j] & 0x7fff7fffu);
            top = max(top >> 16, top & 0xffffu);
            if (i & 1)
                tops[i / 2] |= top << 16;
            else
                tops[i / 2] = top;
        }
#pragma unroll
        for (int i = 0; i < kN / 2; ++i)
#pragma unroll
            for (int d = 1; d < kRow; d <<= 1) tops[i] = __vmaxu2(tops[i], __shfl_xor_sync(kAll, tops[i], d));
        float sums[kN];
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int r = r0 + i * kPass;
            const uint32_t v[4] = {w[i].x, w[i].y, w[i].z, w[i].w}, top = i & 1 ? tops[i / 2] >> 16 : tops[i / 2] & 0xffffu;
            const int e = max((int)(top >> 7), 16);
            const float f = up(e);
            uint4 w16;
            uint32_t* hw = reinterpret_cast<uint32_t*>(&w16);
            sums[i] = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float x = __uint_as_float(v[j] << 16), y = __uint_as_float(v[j] & 0xffff0000u);
                hw[j] = pack(x * f, y * f);
                sums[i] += fabsf(x) + fabsf(y);
            }
            if (h0 == 0) *reinterpret_cast<uint4*>(pair + (p >> 3) * kPanel + piece_at<8>(b * kC + r, p & 7)) = w16;
            if (p == 0) {
                (b ? m.q_scale : m.k_scale)[r] = down(e);
                if (b) m.q_top[r] = __uint_as_float(top << 16);
            }
        }
        if (!b) {  // sums of the rows of K: half of the rows stay with a lane at each step, until it has one
            int rest = kN, mine = 0;
#pragma unroll
            for (int d = 1; d < kRow; d <<= 1) {
                if (rest > 1) {
                    rest /= 2;
                    const bool high = p & d;
#pragma unroll
                    for (int i = 0; i < kN / 2; ++i)
                        if (i < rest) {
                            const float other = __shfl_xor_sync(kAll, high ? sums[i] : sums[i + rest], d);
                            sums[i] = (high ? sums[i + rest] : sums[i]) + other;
                        }
                    mine += high ? rest : 0;
                } else {
                    sums[0] += __shfl_xor_sync(kAll, sums[0], d);
                }
            }
            m.k_sum[r0 + mine * kPass] = sums[0];
        }
    }
    // sums of g in fp64 (64 additions), in powers of two, kept as two floats: differences of far sums stay exact
    if (warp == 0) {
        double G[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            G[i] = (g[i] < -120.0f ? -120.0f : g[i]) * 1.4426950408889634;  // e^-120 is 0 in fp32, and -inf has no differences
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
        if (lane == 0) m.most[b] = m.top[b] = 0;
    }
    __syncthreads();

    const float *gh = m.g_high[b], *gr = m.g_rest[b];
    uint32_t P[8][2], Pr[8][2];  // of blocks up to the diagonal one, as left operands' fragments: high numbers and rests
    float p_down[2];
    const uint32_t k_at = smem_at(m.kq[0]), q_at = smem_at(m.kq[1]);
    if (there) {
        // e^(G_i - G_j) = e^(G_i - G_16w) e^(G_16w - G_j) in the blocks left of the diagonal ones, both 1 or less
        float most_k = fmaxf(m.k_sum[lane], m.k_sum[lane + 32]);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) most_k = fmaxf(most_k, __shfl_xor_sync(kAll, most_k, d));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int j = lane + 32 * i;
            if (j < 16 * warp) m.before[b][warp][j] = exp2_of((gh[16 * warp] - gh[j]) + (gr[16 * warp] - gr[j]));
        }
        __syncwarp();
        if (warp == 0) {  // which has the shortest rows below
            float most_ks = 0, most_left = 0;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = lane + 32 * i;
                const float e = exp2_of(gh[r] + gr[r]);
                const float left = exp2_of((gh[kC - 1] - gh[r]) + (gr[kC - 1] - gr[r])) * m.k_scale[r];
                f.ks[r] = e * m.k_scale[r];
                f.qs[r] = e * m.q_scale[r] * a.c.scale;
                f.left[r] = left;
                most_ks = fmaxf(most_ks, e * m.k_sum[r]);
                most_left = fmaxf(most_left, left);
                if (r == kC - 1) {
                    // Every chunk takes S times this: what one fp32 of e^-0.001 is off by, the same for each, would be 2^-13 of S
                    // after 4096 of them.  For decays that leave a state in place so long, 1 + (e^G - 1) as two fp32.
                    const float less = expm1f((gh[r] + gr[r]) * 0.69314718f);
                    f.all = fabsf(less) < 0.25f ? 1.0f + less : e;
                    f.rest = fabsf(less) < 0.25f ? less - (f.all - 1.0f) : 0.0f;
                }
            }
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                most_ks = fmaxf(most_ks, __shfl_xor_sync(kAll, most_ks, d));
                most_left = fmaxf(most_left, __shfl_xor_sync(kAll, most_left, d));
            }
            if (lane == 0) f.most_ks = most_ks, m.left[b] = most_left;
        }
        // A and P, rows 16 warp .. +15, columns up to the diagonal block
        float after[2], beta[2], p_up[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = 16 * warp + (lane >> 2) + 8 * i;
            after[i] = exp2_of((gh[r] - gh[16 * warp]) + (gr[r] - gr[16 * warp]));
            beta[i] = m.beta[b][r];
            // |q_i k_j| is at most the largest of q_i times the sum of k_j
            const int e = field(2.0f * m.q_top[r] * most_k);
            p_up[i] = up(e);
            p_down[i] = down(e);
        }
        float diagonal[2][2][2];  // of the diagonal block's halves
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = 16 * warp + (lane >> 2) + 8 * i, j = 16 * warp + 8 * n + 2 * (lane & 3);
                diagonal[n][i][0] = j <= r ? exp2_of((gh[r] - gh[j]) + (gr[r] - gr[j])) : 0.0f;
                diagonal[n][i][1] = j + 1 <= r ? exp2_of((gh[r] - gh[j + 1]) + (gr[r] - gr[j + 1])) : 0.0f;
            }
        auto decay = [&](int n, float (&L)[2][2]) {
            const int j = 8 * n + 2 * (lane & 3);
            if (n >= 2 * warp) {
#pragma unroll
                for (int i = 0; i < 2; ++i) L[i][0] = diagonal[n & 1][i][0], L[i][1] = diagonal[n & 1][i][1];
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
                        P[n][i] = halved(v0, v1, Pr[n][i]);
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
        // T diag(beta) in units of its largest value, eight threads a row; to shared memory too, over A
        const int p = tid & 7;
        float beta[8], v[4][8], top = 0, most = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) beta[j] = m.beta[b][8 * p + j];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = ((tid & 127) >> 3) + 16 * i;
            const float4 x = *reinterpret_cast<const float4*>(&m.T[b][row][8 * p]);
            const float4 y = *reinterpret_cast<const float4*>(&m.T[b][row][8 * p + 4]);
            const float t[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
            float sum = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[i][j] = (p >> 1) <= i ? t[j] * beta[j] : 0.0f;  // above the diagonal blocks stand other things
                top = fmaxf(top, fabsf(v[i][j]));
                sum += fabsf(v[i][j]);
            }
#pragma unroll
            for (int d = 1; d < 8; d <<= 1) sum += __shfl_xor_sync(kAll, sum, d);
            most = fmaxf(most, sum);
        }
        const unsigned tops = __reduce_max_sync(kAll, __float_as_uint(top)), mosts = __reduce_max_sync(kAll, __float_as_uint(most));
        if (lane == 0) {
            atomicMax(&m.top[b], tops);
            atomicMax(&m.most[b], mosts);
        }
        head_barrier(b);
        const int e = field(__uint_as_float(m.top[b]));
        const float t_up = up(e);
        uint8_t* T16 = reinterpret_cast<uint8_t*>(m.A[b]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = ((tid & 127) >> 3) + 16 * i;
            uint32_t high[4], rest[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) high[j] = halved(v[i][2 * j] * t_up, v[i][2 * j + 1] * t_up, rest[j]);
            const uint4 h4 = make_uint4(high[0], high[1], high[2], high[3]), r4 = make_uint4(rest[0], rest[1], rest[2], rest[3]);
            *reinterpret_cast<uint4*>(T16 + piece_at<8>(row, p)) = h4;
            *reinterpret_cast<uint4*>(T16 + kSquare + piece_at<8>(row, p)) = r4;
            *reinterpret_cast<uint4*>(out + piece_at<8>(row, p)) = h4;
            *reinterpret_cast<uint4*>(out + 2 * kSquare + piece_at<8>(row, p)) = r4;
        }
        if ((tid & 127) == 0) f.t = down(e), f.most_l = __uint_as_float(m.most[b]) * m.left[b];
        head_barrier(b);
        let_next_start();  // at the kernel's start: the same (one prompt of 4096 178 us, 24 ragged 132)
        // P T, rows 16 warp .. +15
        const uint32_t t_at = smem_at(T16);
        float acc[8][4];
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[n][i] = 0;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            if (t > warp) continue;
            const uint32_t l[4] = {P[2 * t][0], P[2 * t][1], P[2 * t + 1][0], P[2 * t + 1][1]};
            const uint32_t lr[4] = {Pr[2 * t][0], Pr[2 * t][1], Pr[2 * t + 1][0], Pr[2 * t + 1][1]};
#pragma unroll
            for (int n = 0; n <= t; ++n) {
                uint32_t w[4], wr[4];
                ldmatrix_trans(w, left_at<8>(t_at, 16 * t, 2 * n, lane));
                ldmatrix_trans(wr, left_at<8>(t_at + kSquare, 16 * t, 2 * n, lane));
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    mma_f16(acc[2 * n + m], lr, w[2 * m], w[2 * m + 1]);
                    mma_f16(acc[2 * n + m], l, wr[2 * m], wr[2 * m + 1]);
                    mma_f16(acc[2 * n + m], l, w[2 * m], w[2 * m + 1]);
                }
            }
        }
        // to rows of memory over T, whose last readers were before the barriers, and from there 16 bytes a thread
        uint8_t* rows16 = reinterpret_cast<uint8_t*>(m.T[b]) + warp * 2 * 16 * 128;
        uint32_t high[8][2], rest[8][2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float largest = 0;
#pragma unroll
            for (int n = 0; n < 8; ++n) largest = fmaxf(largest, fmaxf(fabsf(acc[n][2 * i]), fabsf(acc[n][2 * i + 1])));
            largest = fmaxf(largest, __shfl_xor_sync(kAll, largest, 1));
            largest = fmaxf(largest, __shfl_xor_sync(kAll, largest, 2));
            const int r = 16 * warp + (lane >> 2) + 8 * i, er = field(largest);
            const float by = up(er);
#pragma unroll
            for (int n = 0; n < 8; ++n) high[n][i] = halved(acc[n][2 * i] * by, acc[n][2 * i + 1] * by, rest[n][i]);
            if ((lane & 3) == 0) f.pt[r] = down(er) * p_down[i] * (down(e) * a.c.scale);
        }
#pragma unroll
        for (int n = 0; n < 8; n += 2) {
            const uint32_t at = left_at<8>(smem_at(rows16), 0, n, lane);
            stmatrix(at, high[n][0], high[n][1], high[n + 1][0], high[n + 1][1]);
            stmatrix(at + 16 * 128, rest[n][0], rest[n][1], rest[n + 1][0], rest[n + 1][1]);
        }
        __syncwarp();
#pragma unroll
        for (int i = lane * 16; i < 16 * 128; i += 32 * 16) {
            *reinterpret_cast<uint4*>(out + kSquare + warp * 16 * 128 + i) = *reinterpret_cast<const uint4*>(rows16 + i);
            *reinterpret_cast<uint4*>(out + 3 * kSquare + warp * 16 * 128 + i) = *reinterpret_cast<const uint4*>(rows16 + 16 * 128 + i);
        }
    }
}


// ------------------------------------------------------------------ //
// the chunks of a sequence                                             //
// ------------------------------------------------------------------ //

// Two accumulator blocks (16 x 8) side by side, times f, as a left operand's fragment (16 x 16): high numbers and rests.
// Accumulators and left operands have the same places, so nothing moves between threads.
struct Fragment {
    uint32_t high[4], rest[4];
};
__device__ __forceinline__ void split(Fragment& r, const float (&c0)[4], const float (&c1)[4], float f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float(&c)[4] = i < 2 ? c0 : c1;
        r.high[i] = halved(c[2 * (i & 1)] * f, c[2 * (i & 1) + 1] * f, r.rest[i]);
    }
}
__device__ __forceinline__ uint32_t transposed(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ float warp_max(float v) { return __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(v))); }
__device__ __forceinline__ void put4(uint32_t at, const uint32_t (&w)[4]) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
}
__device__ __forceinline__ void put4(uint32_t at, const float (&w)[4]) {
    asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(at), "f"(w[0]), "f"(w[1]), "f"(w[2]), "f"(w[3]) : "memory");
}
__device__ __forceinline__ void get4(uint32_t (&w)[4], uint32_t at) {
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void get4(float (&w)[4], uint32_t at) {
    asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(w[0]), "=f"(w[1]), "=f"(w[2]), "=f"(w[3]) : "r"(at) : "memory");
}

constexpr int kVector = 32 * 16;  // bytes: 16 of each thread of a warp

template <int KD, int PAIRS>  // pairs of warps with S
struct ChunkShape {
    static constexpr int kCols = 16 * PAIRS;       // columns of V of a CTA
    static constexpr int kVPitch = kCols * 2 + 16;  // bytes of a row; the 16 keep 8 rows on different banks
    static constexpr int kHalf = PAIRS * 2 * 32;   // threads with S, and as many for o
    static constexpr int kTiles = KD / 32;         // 16 x 16 blocks of a warp's half of S^T
    // a stage: K and Q, T and P T, V; two of them, and of the factors
    static constexpr int kV = pair_bytes(KD) + kHeadTiles;
    static constexpr int kStage = kV + kC * kVPitch;
    static constexpr int kFactors = kHeadBytes - kHeadTiles;
    // handed on by each warp with S: its half of S, high numbers and rests, and its tokens' X
    static constexpr int kX = 2 * kTiles * kVector, kHand = kX + 4 * kVector;
    // exchanged in a pair, by each warp: sums for the other's tokens, then what goes into S (high, rest)
    static constexpr int kSwap = 4 * kVector;
    static constexpr int kOffFactors = 2 * kStage, kOffHands = kOffFactors + 2 * kFactors;
    static constexpr int kOffSwap = kOffHands + 2 * PAIRS * kHand;
    static constexpr int kBytes = kOffSwap + 2 * PAIRS * kSwap;
    static_assert(kBytes <= 227 * 1024, "shared memory of a CTA");
    // barriers beside the CTA's: of a pair, and for S and X that are handed on
    static constexpr int kPairBarrier = 1, kHandedS = 1 + PAIRS, kHandedX = 1 + 2 * PAIRS;
    // registers of a thread with S and of one for o, where the same number for both would be too few for S
    static constexpr int kMost = 168, kLeast = 88;
    static_assert(PAIRS == 2 || 2 * kHalf * 128 == kHalf * (kMost + kLeast), "registers of the launch");
};

// The 16 tokens numbered g = 0, 1 of a warp's half q of a pair: 0..15 and 48..63, or 16..31 and 32..47; T is triangular,
// and this way both have as many of its blocks.
__device__ __forceinline__ int group_of(int q, int g) { return q ? 1 + g : 3 * g; }

// A CTA takes one sequence, v head and kCols columns of V.  A pair of warps
// keeps S for 16 columns [16 x KD] in registers, each warp half of k_dim, as
// accumulators of the state's product.  S is the left operand of the next
// product as it stands: only K, T and K^T come from shared memory, each by
// fragments of half the size that the other way round would need.  Between the
// three products of a chunk the pair exchanges what both need: sums over their
// halves of k_dim, X of their tokens, and what goes into S.  As many more warps form
// o, from the S and X that they are handed, and copy the tiles of the next chunk.
//
// The way from chunk to chunk bounds this where there are few sequences and
// heads: 4096 tokens with 32 heads are 64 chunks one after another on 128 CTAs,
// 125 us, 3700 cycles a chunk: S's largest value and K S^T 1400, X 550, U 700, its
// conversion 450, S 650.  The warps for o are at work for nearly as long: Q S^T 1500
// beside the copies, P T X 1200.  The tensor pipe is busy for 54% of the time,
// shared memory for 72%.  Half of k_dim (half of the first and last product) saves
// 850.  The same chunk by tcgen05 with S in tensor memory, the four products by one
// thread, was built when this way took 116 us, and took 144: three trips to the
// tensor core and back of 500 to 600 cycles each, and a fence and a barrier of 230
// to 450 before each.
template <int KD, int PAIRS>
__global__ void __launch_bounds__(2 * ChunkShape<KD, PAIRS>::kHalf, 1) chunks_kernel(const __grid_constant__ DeltaArgs a) {
    using Shape = ChunkShape<KD, PAIRS>;
    constexpr int kPairs = PAIRS, kCols = Shape::kCols, kHalf = Shape::kHalf, kVPitch = Shape::kVPitch;
    extern __shared__ __align__(128) uint8_t raw[];
    __shared__ float2 units[2 * kPairs];                     // of S and of X
    __shared__ float2 found[2 * kPairs];                     // by a warp for the other of its pair: largest of S and of V
    after_previous();
    constexpr int kT = Shape::kTiles, kN = 2 * kT;
    const int dk = a.c.k_dim, dv = a.c.v_dim, Hk = a.c.k_heads, Hv = a.c.v_heads;
    // blocks of columns, heads, and slowest the sequences
    const int blocks = (dv + kCols - 1) / kCols;
    Taken taken;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(taken.lo), "=r"(taken.hi), "=r"(taken.slot), "=r"(taken.piece)
                 : "l"(taken_of(a, pair_bytes(KD), kHeadBytes) + blockIdx.x / (blocks * Hv)) : "memory");
    const int h = blockIdx.x / blocks % Hv, kh = h / (Hv / Hk), slot = taken.slot;
    if (slot < 0) return;
    const int64_t lo = taken.lo, hi = taken.hi, len = hi - lo;
    const int tid = threadIdx.x, lane = tid & 31, warp = (tid >> 5) % (2 * kPairs), p = warp >> 1, q = warp & 1;
    const int first = (blockIdx.x % blocks) * kCols;  // column of V
    const int chunks = (int)((len + kC - 1) / kC);
    const int64_t piece = taken.piece & 0x7fffffffu;
    const uint32_t base = smem_at(raw);
    const uint32_t hands = base + Shape::kOffHands + lane * 16;
    const int r0 = lane >> 2, c0 = 2 * (lane & 3);

    if (tid >= kHalf) {
        if (PAIRS > 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Shape::kLeast));
        auto copy16 = [](uint32_t to, const void* from, bool there) {
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there ? 16 : 0) : "memory");
        };
        const int t = tid - kHalf;
        constexpr int kFetches = 8, kFirst = 2;
        // Copies of chunk c: K and Q, T and P T by eighths, the factors and V with the first.  All at once hold the warp up for
        // 1000 cycles, so they stand between the products: 4096 tokens 178 us, with half of them before the products 181.
        auto fetch = [&](int c, int part) {
            if (c >= chunks) return;
            const uint32_t to = base + (c & 1) * Shape::kStage;
            const uint8_t* pair = a.ws + ((piece + c) * Hk + kh) * pair_bytes(KD);
            const uint8_t* head = a.ws + a.q_pieces * Hk * pair_bytes(KD) + ((piece + c) * Hv + h) * kHeadBytes;
#pragma unroll
            for (int i = 0; i < pair_bytes(KD) / 8; i += kHalf * 16) {
                const int at = part * (pair_bytes(KD) / 8) + i + t * 16;
                if (kHalf * 16 <= pair_bytes(KD) / 8 || t * 16 < pair_bytes(KD) / 8) copy16(to + at, pair + at, true);
            }
#pragma unroll
            for (int i = 0; i < kHeadTiles / 8; i += kHalf * 16) {
                const int at = part * (kHeadTiles / 8) + i + t * 16;
                copy16(to + pair_bytes(KD) + at, head + at, true);
            }
            if (part) return;
            for (int i = t * 16; i < Shape::kFactors; i += kHalf * 16)
                copy16(base + Shape::kOffFactors + (c & 1) * Shape::kFactors + i, head + kHeadTiles + i, true);
            const int64_t row0 = lo + (int64_t)c * kC;
#pragma unroll
            for (int i = t; i < kC * (kCols / 8); i += kHalf) {
                const int r = i / (kCols / 8), d = first + i % (kCols / 8) * 8;
                const bool there = row0 + r < hi && d < dv;
                const __nv_bfloat16* from = there ? a.vr + (row0 + r) * a.v_ld + h * dv + d : a.vr;
                const uint32_t at = (uint32_t)(Shape::kV + r * kVPitch + (d - first) * 2);
                if (a.wide) {
                    copy16(to + at, from, there);
                } else {
                    *reinterpret_cast<uint4*>(raw + (c & 1) * Shape::kStage + at) =
                        there ? eight(from, false) : make_uint4(0, 0, 0, 0);
                }
            }
        };
        float o[4][4];  // of this warp's two groups of 16 tokens
        auto put = [&](int c) {  // to memory
            const int64_t row0 = lo + (int64_t)c * kC;
            const int rows = (int)(hi - row0 < kC ? hi - row0 : kC), d = first + 16 * p + c0;
            __nv_bfloat16* to = a.o + row0 * a.o_ld + h * dv + d;
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const int r = 16 * group_of(q, n >> 1) + 8 * (n & 1) + r0;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const __nv_bfloat162 y = __floats2bfloat162_rn(o[n][2 * i], o[n][2 * i + 1]);
                    const uint32_t w = transposed(*reinterpret_cast<const uint32_t*>(&y));  // a token's two columns
                    if (r < rows && d + 8 * i < dv) {
                        __nv_bfloat16* at = to + r * a.o_ld + 8 * i;
                        if (a.o_pairs) {
                            *reinterpret_cast<uint32_t*>(at) = w;
                        } else {
                            reinterpret_cast<unsigned short*>(at)[0] = (unsigned short)w;
                            reinterpret_cast<unsigned short*>(at)[1] = (unsigned short)(w >> 16);
                        }
                    }
                }
            }
        };
        for (int i = 0; i < kFetches; ++i) fetch(0, i);
        for (int c = 0; c < chunks; ++c) {
            asm volatile("cp.async.wait_all;" ::: "memory");
            __syncthreads();  // chunk c is there; nobody reads chunk c - 1 or what was handed on in it
#pragma unroll
            for (int i = 0; i < kFirst; ++i) fetch(c + 1, i);
            const uint32_t stage = base + (c & 1) * Shape::kStage, hand = hands + 2 * p * Shape::kHand;
            const Factors& f = *reinterpret_cast<const Factors*>(raw + Shape::kOffFactors + (c & 1) * Shape::kFactors);
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[n][i] = 0;
            // Q S^T, in the units of each half of k_dim, then P T X
#pragma unroll
            for (int part = 0; part < 3; ++part) {
                if (part == 0) asm volatile("bar.sync %0, 128;" ::"r"(Shape::kHandedS + p) : "memory");
                if (part == 2) asm volatile("bar.sync %0, 128;" ::"r"(Shape::kHandedX + p) : "memory");
                float acc[4][4];
#pragma unroll
                for (int n = 0; n < 4; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[n][i] = 0;
                if (part < 2) {
#pragma unroll
                    for (int t = 0; t < kT; ++t) {
                        if (kFirst + part * kT + t < kFetches) fetch(c + 1, kFirst + part * kT + t);
                        uint32_t x[4], rest[4];
                        get4(x, hand + part * Shape::kHand + t * kVector);
                        get4(rest, hand + part * Shape::kHand + (kT + t) * kVector);
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            uint32_t w[4];
                            ldmatrix(w, columns_at(stage, kC + 16 * group_of(q, g), 2 * (part * kT + t), lane));
                            mma_f16(acc[2 * g], x, w[0], w[1]);
                            mma_f16(acc[2 * g + 1], x, w[2], w[3]);
                            mma_f16(acc[2 * g], rest, w[0], w[1]);
                            mma_f16(acc[2 * g + 1], rest, w[2], w[3]);
                        }
                    }
                } else {
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        if (kFirst + 2 * kT + t < kFetches) fetch(c + 1, kFirst + 2 * kT + t);
                        uint32_t x[4], rest[4];
                        const int owner = t == 1 || t == 2;
                        get4(x, hand + owner * Shape::kHand + Shape::kX + t / 2 * kVector);
                        get4(rest, hand + owner * Shape::kHand + Shape::kX + (2 + t / 2) * kVector);
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            if (group_of(q, g) < t) continue;
                            const uint32_t at = right_at<8>(stage + pair_bytes(KD) + kSquare, 16 * group_of(q, g), 2 * t, lane);
                            uint32_t w[4];
                            ldmatrix(w, at + 2 * kSquare);
                            mma_f16(acc[2 * g], x, w[0], w[1]);
                            mma_f16(acc[2 * g + 1], x, w[2], w[3]);
                            ldmatrix(w, at);
                            mma_f16(acc[2 * g], rest, w[0], w[1]);
                            mma_f16(acc[2 * g + 1], rest, w[2], w[3]);
                            mma_f16(acc[2 * g], x, w[0], w[1]);
                            mma_f16(acc[2 * g + 1], x, w[2], w[3]);
                        }
                    }
                }
                const float2 unit = units[2 * p + (part < 2 ? part : 0)];
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const float2 by = *reinterpret_cast<const float2*>((part < 2 ? f.qs : f.pt) + 16 * group_of(q, n >> 1) + 8 * (n & 1) + c0);
                    const float b0 = by.x * (part < 2 ? unit.x : unit.y), b1 = by.y * (part < 2 ? unit.x : unit.y);
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[n][i] = fmaf(i & 1 ? b1 : b0, acc[n][i], o[n][i]);
                }
            }
            put(c);
        }
        return;
    }

    if (PAIRS > 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Shape::kMost));
    const uint32_t swap = base + Shape::kOffSwap + lane * 16;
    const uint32_t my_swap = swap + warp * Shape::kSwap, its_swap = swap + (warp ^ 1) * Shape::kSwap;
    const uint32_t hand = hands + warp * Shape::kHand, its_hand = hands + (warp ^ 1) * Shape::kHand;
    auto pair_barrier = [&]() { asm volatile("bar.sync %0, 64;" ::"r"(Shape::kPairBarrier + p) : "memory"); };
    auto handed = [&](int barrier) { asm volatile("bar.arrive %0, 128;" ::"r"(barrier + p) : "memory"); };
    // S: rows d0, d0 + 8 of v_dim, columns k0 + 8 n (+ 1) of k_dim, in units of down(unit)
    const int d0 = first + 16 * p + r0, k0 = q * (KD / 2) + c0;
    float S[kN][4];
    int unit = kOne;
    const bool carry = taken.piece >> 31;
    float* state = a.state ? a.state + ((int64_t)slot * Hv + h) * dv * dk : nullptr;
#pragma unroll
    for (int n = 0; n < kN; ++n)
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            const int d = d0 + 4 * i, k = k0 + 8 * n;
            const float2 v = carry && d < dv && k < dk ? *reinterpret_cast<const float2*>(state + (int64_t)d * dk + k) : make_float2(0, 0);
            S[n][i] = v.x, S[n][i + 1] = v.y;
        }
    auto largest_of_s = [&]() {
        float most = 0;
#pragma unroll
        for (int n = 0; n < kN; ++n)
            most = fmaxf(most, fmaxf(fmaxf(fabsf(S[n][0]), fabsf(S[n][1])), fmaxf(fabsf(S[n][2]), fabsf(S[n][3]))));
        return warp_max(most);
    };
    // groups of 16 tokens: this warp's, then the other's
    const int group[4] = {group_of(q, 0), group_of(q, 1), group_of(q ^ 1, 0), group_of(q ^ 1, 1)};

    for (int c = 0; c < chunks; ++c) {
        __syncthreads();
        const uint32_t stage = base + (c & 1) * Shape::kStage, T_high = stage + pair_bytes(KD), T_rest = T_high + 2 * kSquare;
        const Factors& f = *reinterpret_cast<const Factors*>(raw + Shape::kOffFactors + (c & 1) * Shape::kFactors);

        // V of this warp's tokens, turned: two groups of 16 tokens by 16 columns
        uint32_t v[2][4], bits = 0;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            ldmatrix_trans(v[g], stage + Shape::kV + (16 * group[g] + (lane & 15)) * kVPitch + 32 * p + (lane >> 4) * 16);
#pragma unroll
            for (int i = 0; i < 4; ++i) bits = __vmaxu2(bits, v[g][i] & 0x7fff7fffu);
        }
        bits = __reduce_max_sync(kAll, max(bits & 0xffff0000u, bits << 16));
        // This half's part of K S^T, for the other's tokens first.  S's unit is from its largest value: a bound from the chunk
        // before leaves few bits of a state that was cleared there.
        const float most = largest_of_s();
        const int e_s = field(most);
        const float s_up = up(e_s), s_down = down(e_s) * down(unit);
        float x[8][4];
        Fragment b[kT];
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[n][i] = 0;
        auto times_k = [&](int t, int g) {  // two groups of tokens
            uint32_t w[2][4];
#pragma unroll
            for (int m = 0; m < 2; ++m) ldmatrix(w[m], columns_at(stage, 16 * group[g + m], 2 * (q * kT + t), lane));
#pragma unroll
            for (int m = 0; m < 4; ++m) mma_f16(x[2 * g + m], b[t].high, w[m >> 1][2 * (m & 1)], w[m >> 1][2 * (m & 1) + 1]);
#pragma unroll
            for (int m = 0; m < 4; ++m) mma_f16(x[2 * g + m], b[t].rest, w[m >> 1][2 * (m & 1)], w[m >> 1][2 * (m & 1) + 1]);
        };
#pragma unroll
        for (int t = 0; t < kT; ++t) {
            split(b[t], S[2 * t], S[2 * t + 1], s_up);
            put4(hand + t * kVector, b[t].high);
            put4(hand + (kT + t) * kVector, b[t].rest);
            times_k(t, 2);
        }
        if (lane == 0) found[warp] = make_float2(most, __uint_as_float(bits)), units[warp].x = s_down;
        handed(Shape::kHandedS);
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const float send[4] = {x[4 + n][0] * s_down, x[4 + n][1] * s_down, x[4 + n][2] * s_down, x[4 + n][3] * s_down};
            put4(my_swap + n * kVector, send);
        }
        pair_barrier();
#pragma unroll
        for (int t = 0; t < kT; ++t) times_k(t, 0);
        const float2 its = found[warp ^ 1];
        const float s_most = fmaxf(most, its.x), bound = fmaf(f.most_ks, s_most * down(unit), fmaxf(__uint_as_float(bits), its.y));
        const float l_bound = bound * f.most_l;
        const int e_x = field(2.0f * bound);
        const float x_up = up(e_x), x_down = down(e_x);
        // S has to stay finite in the new units, and its change of units a number of fp32; what updates lose by that is 2^-60
        // of S, or 2^-100 of what they were made for before
        const int next = min(max(field(2.0f * l_bound), max(field(s_most) + unit - kOne - 60, unit - 120)), 254);
        const float units_by = __uint_as_float((uint32_t)(127 + min(max(unit - next, -126), 127)) << 23);
        const float grow = f.all * units_by, grow_rest = f.rest * units_by;
        const float to_l = f.t * x_down * up(next);
        if (lane == 0) units[warp].y = x_down;
        unit = next;

        // X = V - e^G K S^T of this warp's tokens
        Fragment X[2];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const int n = 2 * g + m;
                float other[4];
                get4(other, its_swap + n * kVector);
                const float2 ks = *reinterpret_cast<const float2*>(f.ks + 16 * group[g] + 8 * m + c0);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t w = v[g][m + 2 * (i >> 1)];
                    x[n][i] = fmaf(i & 1 ? -ks.y : -ks.x, fmaf(x[n][i], s_down, other[i]), __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16));
                }
            }
            split(X[g], x[2 * g], x[2 * g + 1], x_up);
            put4(hand + Shape::kX + g * kVector, X[g].high);
            put4(hand + Shape::kX + (2 + g) * kVector, X[g].rest);
        }
        handed(Shape::kHandedX);
        // U = T X of this warp's tokens, first what its own X bring: two sums a block, the second of what the rests bring
        float u[4][4], u2[4][4];
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) u[n][i] = u2[n][i] = 0;
        auto times_t = [&](int out, const Fragment& in, int t) {
            uint32_t high[4], rest[4];
            ldmatrix(high, right_at<8>(T_high, 16 * group[out], 2 * t, lane));
            ldmatrix(rest, right_at<8>(T_rest, 16 * group[out], 2 * t, lane));
            mma_f16(u[2 * out], in.high, high[0], high[1]);
            mma_f16(u[2 * out + 1], in.high, high[2], high[3]);
            mma_f16(u2[2 * out], in.high, rest[0], rest[1]);
            mma_f16(u2[2 * out + 1], in.high, rest[2], rest[3]);
            mma_f16(u2[2 * out], in.rest, high[0], high[1]);
            mma_f16(u2[2 * out + 1], in.rest, high[2], high[3]);
        };
        times_t(0, X[0], group[0]);
        times_t(1, X[0], group[0]);
        times_t(1, X[1], group[1]);
        pair_barrier();
        {
            Fragment theirs[2];
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                get4(theirs[g].high, its_hand + Shape::kX + g * kVector);
                get4(theirs[g].rest, its_hand + Shape::kX + (2 + g) * kVector);
            }
            times_t(1, theirs[0], group[2]);  // group 1 for 3, or 0 for 2
            if (q)
                times_t(0, theirs[0], group[2]);  // 0 for 1
            else
                times_t(1, theirs[1], group[3]);  // 2 for 3
        }
        // U^T (e^(G_63 - G) K) in the new units, with this warp's tokens first: a sum of its own.  The tensor core's additions
        // round towards zero, and eight a chunk into S itself took 2^-22 of it a chunk
        float grown[kN][4];
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) grown[n][i] = S[n][i] * grow_rest;
        auto times_k_turned = [&](const Fragment& l, int t) {
            uint32_t w[kT][4];
#pragma unroll
            for (int n = 0; n < kT; ++n) ldmatrix_trans(w[n], rows_at(stage, 16 * t, 2 * (q * kT + n), lane));
#pragma unroll
            for (int n = 0; n < kT; ++n) {
                mma_f16(grown[2 * n], l.high, w[n][0], w[n][1]);
                mma_f16(grown[2 * n + 1], l.high, w[n][2], w[n][3]);
            }
#pragma unroll
            for (int n = 0; n < kT; ++n) {
                mma_f16(grown[2 * n], l.rest, w[n][0], w[n][1]);
                mma_f16(grown[2 * n + 1], l.rest, w[n][2], w[n][3]);
            }
        };
        Fragment L[2];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const int n = 2 * g + m;
                const float2 left = *reinterpret_cast<const float2*>(f.left + 16 * group[g] + 8 * m + c0);
                const float l0 = left.x * to_l, l1 = left.y * to_l;
#pragma unroll
                for (int i = 0; i < 4; ++i) u[n][i] = (u[n][i] + u2[n][i]) * (i & 1 ? l1 : l0);
            }
            split(L[g], u[2 * g], u[2 * g + 1], 1.0f);
            put4(my_swap + 2 * g * kVector, L[g].high);
            put4(my_swap + (2 * g + 1) * kVector, L[g].rest);
        }
        times_k_turned(L[0], group[0]);
        times_k_turned(L[1], group[1]);
        pair_barrier();
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            get4(L[g].high, its_swap + 2 * g * kVector);
            get4(L[g].rest, its_swap + (2 * g + 1) * kVector);
        }
        times_k_turned(L[0], group[2]);
        times_k_turned(L[1], group[3]);
        // S <- e^G_63 S + that
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) S[n][i] = fmaf(S[n][i], grow, grown[n][i]);
    }
    let_next_start();  // not earlier: 64 prompts of 64 255.5 us, at the kernel's start 256.5; 24 ragged 131.8 and 132.4
    if (state) {
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                const int d = d0 + 4 * i, k = k0 + 8 * n;
                if (d < dv && k < dk)
                    *reinterpret_cast<float2*>(state + (int64_t)d * dk + k) = make_float2(S[n][i] * down(unit), S[n][i + 1] * down(unit));
            }
    }
}

template <int KD, int PAIRS>
cudaError_t launch_chunks(const DeltaArgs& a, cudaStream_t st) {
    using Shape = ChunkShape<KD, PAIRS>;
    const auto kernel = chunks_kernel<KD, PAIRS>;
    if (PAIRS > 2) {  // the warps with S wait for registers that the others give back: the launch must have them
        cudaFuncAttributes f;
        if (cudaError_t e = cudaFuncGetAttributes(&f, kernel)) return e;
        if (f.numRegs * 2 < Shape::kMost + Shape::kLeast) return cudaErrorLaunchOutOfResources;
    }
    if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape::kBytes)) return e;
    const int64_t blocks = (a.c.v_dim + Shape::kCols - 1) / Shape::kCols;
    return launch(kernel, dim3((unsigned)(a.q.n * a.c.v_heads * blocks)), 2 * Shape::kHalf, Shape::kBytes, st, 1, a);
}
template <int KD>
cudaError_t launch_chunked(const DeltaArgs& a, cudaStream_t st) {
    const int twos = (a.c.v_heads / a.c.k_heads + 1) / 2;
    constexpr int kShared = (int)sizeof(PrepareShared<KD>);
    if (cudaError_t e = cudaFuncSetAttribute(prepare_kernel<KD>, cudaFuncAttributeMaxDynamicSharedMemorySize, kShared)) return e;
    if (cudaError_t e = launch(prepare_kernel<KD>, dim3((unsigned)(a.q_pieces + (a.q.n + kPrepare - 1) / kPrepare), (unsigned)(a.c.k_heads * twos)), kPrepare, kShared,
                               st, 1, a))
        return e;
    // Four pairs take 1.6 to 1.8 times as long for a chunk as two, so they pay where the CTAs of two would be more than the
    // SMs (and are twos).  Four pairs and two, in us: 32 heads of 128, 64 prompts of 64 tokens 259 and 298, 16 of 256 182 and 195, 2 of
    // 2048 173 and 179, one of 4096 (128 CTAs of two pairs) 286 and 178; 16 heads of 64, 8 of 512 52 and 55, 5 of 1024 (160 CTAs)
    // 78 and 82, 4 of 1024 (128) 73 and 53.
    constexpr int kSMs = 152;  // of a GB300
    const int64_t columns = (a.c.v_dim + 31) / 32, ctas = a.q.n * a.c.v_heads * columns;
    return ctas > kSMs && columns % 2 == 0 ? launch_chunks<KD, 4>(a, st) : launch_chunks<KD, 2>(a, st);
}

}  // namespace

size_t delta_workspace(const moe_delta_config& c, int64_t T, int n) {
    return (size_t)(T / kC + n) *
               ((size_t)c.k_heads * pair_bytes(padded_dim(c.k_dim)) + (size_t)c.v_heads * kHeadBytes) +
           (size_t)n * sizeof(Taken);
}

cudaError_t launch_delta_chunks(const DeltaArgs& a, cudaStream_t st) {
    return padded_dim(a.c.k_dim) == 64 ? launch_chunked<64>(a, st) : launch_chunked<128>(a, st);
}

}  // namespace moe
