// mx_quantise.cu -- rows to microscaled 4-bit floats and back.
#include <cuda_fp4.h>
#include <cuda_fp8.h>
#include <string.h>

#include "mx.h"

namespace moe {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kThreads = 256;

// 16 consecutive columns of a row for each of 16 threads, as they were loaded:
// unpacked only when they are needed, so that the next row's loads can be under
// way.  Rows that are not aligned for 16-byte loads are loaded value by value,
// thread c taking columns c, c + 16, ..., so that the threads' loads share
// sectors, and change hands in shared memory (pitch 17: no bank conflicts).
// 16384 rows of 2047 columns to e8m0: bf16 23.7 us, fp32 26.5 (of 2048: 15.1 and 24.7), to e4m3 30.3 and 30.0 (19.0 and
// 25.2; the bf16 form spills 16 bytes).
constexpr int kSwap = 16 * 17;  // floats of a row

template <typename T, bool WIDE>
struct Raw {
    uint4 q[sizeof(T)];  // 16 values
    // p: column 0 of the 256; n: of them in the row (256 or fewer); c: this thread's place
    __device__ __forceinline__ void load(const T* p, int n, int c) {
        constexpr int kPer = 16 / (int)sizeof(T);  // values of a quad
        if (WIDE && n >= 16 * c + 16) {
#pragma unroll
            for (int i = 0; i < (int)sizeof(T); ++i) q[i] = reinterpret_cast<const uint4*>(p + 16 * c)[i];
        } else {
#pragma unroll
            for (int i = 0; i < (int)sizeof(T); ++i) {
                T t[kPer];
#pragma unroll
                for (int j = 0; j < kPer; ++j) {
                    const int col = WIDE ? 16 * c + i * kPer + j : 16 * (i * kPer + j) + c;
                    t[j] = col < n ? p[col] : (T)0.0f;
                }
                memcpy(&q[i], t, 16);
            }
        }
    }
    // swap: the row's kSwap floats, used where the loads were not wide (by all 16 threads)
    __device__ __forceinline__ void get(float (&v)[16], int c, float* swap) const {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T); ++i) {
            const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (sizeof(T) == 4) {
                    v[4 * i + j] = __uint_as_float(w[j]);
                } else {
                    v[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
                    v[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
                }
            }
        }
        if constexpr (!WIDE) {
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 16; ++j) swap[17 * j + c] = v[j];
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = swap[17 * c + j];
        }
    }
};

__device__ __forceinline__ void store8(float* p, int n, const float (&v)[8]) {
    if (n >= 8) {
        reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = v[i];
    }
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, int n, const float (&v)[8]) {
    if (n >= 8) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
            w[j] = *reinterpret_cast<const uint32_t*>(&b);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = __float2bfloat16_rn(v[i]);
    }
}

struct QuantArgs {
    uint8_t* data;
    MxRows rows;
    const void* src;
    const int32_t* src_row;
    const float* tscale;
    void* dst;
    int64_t ld, src_rows;
    int cols, col_tiles;
    bool wide;
};

constexpr int kRows = kThreads / 16;  // rows of a block's step: 16 threads share a row's 256 columns

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_abs(float a, float b, float c) {  // of the magnitudes; NaN if any is
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// g / (1 + exp(-g)) * u, exp(-g) = 2^(-g log2 e); both units are good to about 2^-22, far below a code's spacing
__device__ __forceinline__ float silu_mul(float g, float u) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-1.44269504f * g));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return g * r * u;
}
// eight values to e2m1 codes, the first in the lowest nibble
__device__ __forceinline__ uint32_t codes8(const float* v) {
    uint32_t r;
    asm("{\n .reg .b8 a, b, c, d;\n"
        " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
        " mov.b32 %0, {a, b, c, d};\n}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// byte offset of a chunk's 8 code bytes in its tile, and of its scale bytes' word
__device__ __forceinline__ uint32_t code_at(int in, int c16) {
    const int c = c16 >> 1;  // 16-byte chunk of the tile's row
    return (uint32_t)(in * 128 + ((c ^ (in & 7)) << 4) + ((c16 & 1) << 3));
}
__device__ __forceinline__ uint32_t scale_at(int in, int atom) {
    return (uint32_t)(kMxCodeBytes + atom * kMxAtomBytes + (in & 31) * 16 + (in >> 5) * 4);
}

// A block takes 16 rows of one column tile at a time, a thread 16 columns of a
// row, so 16 threads write one row's 128 bytes of codes, and the scale bytes of
// four blocks go out as one word.  Row maps and tile addresses need no
// division.  With many rows a block goes through several sets of 16, and loads
// the next set's values before it works on this one's.  SwiGLU of 40960 x 512
// bf16 to e4m3 takes 19.4 us for 96 MB (4.9 TB/s): two special-function
// operations a value take 10 us of that, about 300 instructions per 16 values
// as long again, and neither overlaps the loads fully.
//
// Both formats divide by a scale before the rounding to e2m1.  A power of two
// is an exact multiply.  The e4m3 scale takes a reciprocal and one residual
// step: r = x / d to a few units of the last place, then
// r + (x - r d) / d, the remainder exact in one fma.  Where x / d is itself a
// short number, as a tie between two codes is, the result is exactly that.
template <typename T, int FMT, bool SWIGLU, bool WIDE>
__global__ void __launch_bounds__(kThreads) quantise_kernel(const QuantArgs a) {
    after_previous();
    let_next_start();
    __shared__ float swap_s[WIDE ? 1 : kRows * kSwap];
    const int c16 = threadIdx.x & 15;
    float* const swap = swap_s + (WIDE ? 0 : (threadIdx.x >> 4) * kSwap);
    const int col = blockIdx.y * kMxTileCols;
    const int64_t stride = (int64_t)gridDim.x * kRows, first = (int64_t)blockIdx.x * kRows;
    int64_t r = first + (threadIdx.x >> 4);
    Raw<T, WIDE> x, up;
    bool live;
    // the row's values: they do not wait for its place in the tiles
    auto fetch = [&](int64_t row) {
        const int64_t from = row < a.rows.rows ? (a.src_row ? a.src_row[row] : row) : -1;
        live = (uint64_t)from < (uint64_t)a.src_rows;  // -1 is not
        const int n = live ? a.cols - col : 0;
        const T* p = static_cast<const T*>(a.src) + (live ? from * a.ld + col : 0);
        x.load(p, n, c16);
        if (SWIGLU) up.load(p + a.cols, n, c16);
    };
    fetch(r);
    for (int64_t at = first; at < a.rows.rows; at += stride, r += stride) {
        int g = 0, in = 0;
        int64_t tile = 0;
        const bool mine = live && a.rows.place(r, g, tile, in);
        float v[16];
        x.get(v, c16, swap);
        if (SWIGLU) {
            float u[16];
            up.get(u, c16, swap);
            if (at + stride < a.rows.rows) fetch(r + stride);
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = silu_mul(v[j], u[j]);
        } else if (at + stride < a.rows.rows) {
            fetch(r + stride);
        }
        float amax = 0.0f;
#pragma unroll
        for (int j = 0; j < 16; j += 2) amax = max_abs(amax, v[j], v[j + 1]);
        if (FMT == MOE_MX_E8M0) amax = max_nan(amax, __shfl_xor_sync(kAll, amax, 1));
        const bool finite = amax <= 3.402823466e38f;
        uint32_t byte;
        if (FMT == MOE_MX_E8M0) {
            // floor(log2 amax) is the exponent field less 127 (subnormals end at the lower bound either way)
            int e = (int)(__float_as_uint(amax) >> 23) - 127 - 2;
            if (e < -127) e = -127;
            const float inv = __uint_as_float((uint32_t)(127 - e) << 23);  // 2^-e, normal for e in -127..125
            byte = (uint32_t)(e + 127);
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] *= inv;
        } else {
            const float t = a.tscale && mine ? a.tscale[g] : 1.0f;
            // a block of zeros has scale 0 also where t is 0
            const __nv_fp8_storage_t s =
                __nv_cvt_float_to_fp8(__fdiv_rn(amax, amax > 0.0f ? 6.0f * t : 1.0f), __NV_SATFINITE, __NV_E4M3);
            byte = s;
            const float d = __half2float(__half(__nv_cvt_fp8_to_halfraw(s, __NV_E4M3))) * t;
            const float inv = d > 0.0f ? __frcp_rn(d) : 0.0f;
            if (inv >= 1e30f) {  // scales so small that a remainder could be subnormal, or the reciprocal infinite
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] = __fdiv_rn(v[j], d);
            } else if (SWIGLU) {  // the activation is not exact to the last place either
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] *= inv;
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float q = v[j] * inv;
                    v[j] = fmaf(fmaf(-q, d, v[j]), inv, q);
                }
            }
        }
        uint32_t out[2] = {codes8(v), codes8(v + 8)};
        if (!finite) {
            byte = FMT == MOE_MX_E8M0 ? 255 : 127;
            out[0] = out[1] = 0;
        }
        // join the bytes of four consecutive blocks
        constexpr int kBlock = FMT == MOE_MX_E8M0 ? 2 : 1;  // threads per block
        uint32_t word = byte;
        word |= __shfl_down_sync(kAll, word, kBlock) << 8;
        word |= __shfl_down_sync(kAll, word, 2 * kBlock) << 16;
        if (!mine) continue;
        uint8_t* base = a.data + (tile * a.col_tiles + blockIdx.y) * (int64_t)mx_tile_bytes(FMT);
        *reinterpret_cast<uint2*>(base + code_at(in, c16)) = make_uint2(out[0], out[1]);
        if (c16 % (4 * kBlock) == 0)
            *reinterpret_cast<uint32_t*>(base + scale_at(in, c16 / (4 * kBlock))) = word;
    }
}

// Eight columns a lane, so that a warp reads a row's 128 bytes of codes and
// writes its 256 numbers in whole lines.  A warp takes ROWS rows: its first
// lanes look their places up together, and all rows' codes are loaded before
// the first is needed.  Eight rows a warp where that still fills the GPU
// (40960 x 512 to bf16: 11.5 us, with two 14.1), else one (64 rows of 2048
// columns: 1.7 us instead of 2.9).  Bound by the instructions issued (84 % of
// the slots at 16384 x 2048, 14.5 us; rows that are not aligned take 32).
__device__ __forceinline__ __half2 e2m1_pair(uint32_t byte) {
    return __half2(__nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)(byte & 0xffu), __NV_E2M1));
}

template <typename T, int FMT, int ROWS>
__global__ void __launch_bounds__(kThreads) dequantise_kernel(const QuantArgs a) {
    after_previous();
    let_next_start();
    const int lane = threadIdx.x & 31, col = blockIdx.y * kMxTileCols, n = a.cols - col;  // columns of the row from here on
    const int64_t r0 = ((int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * ROWS;
    const int b = FMT == MOE_MX_E8M0 ? lane >> 2 : lane >> 1;
    int g = 0, in = 0;
    int64_t tile = 0;
    const bool there = lane < ROWS && r0 + lane < a.rows.rows && a.rows.place(r0 + lane, g, tile, in);
    const float t_own = there && a.tscale ? a.tscale[g] : 1.0f;
    const unsigned live = __ballot_sync(kAll, there);
    uint32_t codes[ROWS], byte[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int in_i = __shfl_sync(kAll, in, i);
        const int64_t tile_i = __shfl_sync(kAll, tile, i);
        codes[i] = byte[i] = 0;
        if (!(live >> i & 1)) continue;
        const uint8_t* base = a.data + (tile_i * a.col_tiles + blockIdx.y) * (int64_t)mx_tile_bytes(FMT);
        codes[i] = *reinterpret_cast<const uint32_t*>(base + in_i * 128 + (((lane >> 2) ^ (in_i & 7)) << 4) + (lane & 3) * 4);
        byte[i] = base[scale_at(in_i, b >> 2) + (b & 3)];
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const float t = __shfl_sync(kAll, t_own, i);
        if (!(live >> i & 1)) continue;
        float s;
        if (FMT == MOE_MX_E8M0)
            s = byte[i] == 255 ? __uint_as_float(0x7fffffffu)
                               : byte[i] ? __uint_as_float(byte[i] << 23) : __uint_as_float(0x400000u);
        else
            s = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte[i], __NV_E4M3)));
        T* const row = static_cast<T*>(a.dst) + (r0 + i) * a.ld + col;
        if (a.wide) {
            float v[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const __half2 h = e2m1_pair(codes[i] >> (8 * j));
                v[2 * j] = __low2float(h) * s;
                v[2 * j + 1] = __high2float(h) * s;
            }
            if (a.tscale)
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] *= t;
            store8(row + 8 * lane, n - 8 * lane, v);
        } else {
            // columns 32 j + lane, from the lane that holds them: stores of neighbours share sectors
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int from = 4 * j + (lane >> 3), c = 32 * j + lane;
                const uint32_t word = __shfl_sync(kAll, codes[i], from);
                const float sj = __shfl_sync(kAll, s, from);
                const float v = __low2float(e2m1_pair(word >> (4 * (lane & 7)) & 15u)) * sj;
                if (c < n) row[c] = (T)(a.tscale ? v * t : v);
            }
        }
    }
}

dim3 grid_of(const QuantArgs& a, int rows) {
    return dim3((unsigned)((a.rows.rows + rows - 1) / rows), (unsigned)a.col_tiles);
}
int sm_count() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 1;  // the launch itself will say what is wrong
    return sms;
}
// Blocks that stay and walk: four of 256 threads on an SM with SwiGLU, as many as fit at a time (40960 x 512: 19.5 us,
// with six 23.5); eight without, where less work hides less of the loads (16384 x 2048 bf16 to e8m0: 15.2 us, with
// four 18.5).
dim3 walk_grid(const QuantArgs& a, bool swiglu) {
    dim3 g = grid_of(a, kRows);
    const unsigned most = (unsigned)(((swiglu ? 4 : 8) * sm_count() + a.col_tiles - 1) / a.col_tiles);
    if (g.x > most) g.x = most;
    return g;
}

template <typename T, int FMT>
cudaError_t dequantise_rows(const QuantArgs& a, cudaStream_t st) {
    constexpr int kWarps = kThreads / 32;
    if (a.rows.rows * a.col_tiles >= (int64_t)8 * kWarps * sm_count())
        return launch(dequantise_kernel<T, FMT, 8>, grid_of(a, 8 * kWarps), kThreads, 0, st, 1, a);
    return launch(dequantise_kernel<T, FMT, 1>, grid_of(a, kWarps), kThreads, 0, st, 1, a);
}

template <typename T, int FMT>
cudaError_t quantise_act(const QuantArgs& a, int act, cudaStream_t st) {
    const bool swiglu = act == MOE_ACT_SWIGLU;
    return launch(a.wide ? (swiglu ? quantise_kernel<T, FMT, true, true> : quantise_kernel<T, FMT, false, true>)
                         : (swiglu ? quantise_kernel<T, FMT, true, false> : quantise_kernel<T, FMT, false, false>),
                  walk_grid(a, swiglu), kThreads, 0, st, 1, a);
}

// whole 16-byte loads or stores need every 16-column chunk of every row aligned
bool wide_ok(const void* p, int64_t ld, int64_t second, int type) {
    const int64_t size = type == MOE_F32 ? 4 : 2;
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * size % 16 == 0 && second * size % 16 == 0;
}

}  // namespace

cudaError_t launch_mx_quantise(const moe_mx& m, const MxRows& rows, const void* src, int64_t src_rows, int type,
                               int64_t ld, int act, const int32_t* src_row, const float* tscale, cudaStream_t st) {
    QuantArgs a{};
    a.data = static_cast<uint8_t*>(m.data_dev);
    a.rows = rows;
    a.src = src;
    a.src_rows = src_rows;
    a.src_row = src_row;
    a.tscale = tscale;
    a.ld = ld;
    a.cols = m.cols;
    a.col_tiles = (int)mx_col_tiles(m.cols);
    a.wide = wide_ok(src, ld, act == MOE_ACT_SWIGLU ? m.cols : 0, type);
    if (rows.rows / kRows >= INT32_MAX || a.col_tiles > 65535) return cudaErrorInvalidValue;
    if (type == MOE_F32) {
        if (m.format == MOE_MX_E8M0) return quantise_act<float, MOE_MX_E8M0>(a, act, st);
        return quantise_act<float, MOE_MX_E4M3>(a, act, st);
    }
    if (m.format == MOE_MX_E8M0) return quantise_act<__nv_bfloat16, MOE_MX_E8M0>(a, act, st);
    return quantise_act<__nv_bfloat16, MOE_MX_E4M3>(a, act, st);
}

cudaError_t launch_mx_dequantise(const moe_mx& m, const MxRows& rows, const float* tscale, void* dst, int type,
                                 int64_t ld, cudaStream_t st) {
    QuantArgs a{};
    a.data = static_cast<uint8_t*>(m.data_dev);
    a.rows = rows;
    a.tscale = tscale;
    a.dst = dst;
    a.ld = ld;
    a.cols = m.cols;
    a.col_tiles = (int)mx_col_tiles(m.cols);
    a.wide = wide_ok(dst, ld, 0, type);
    if (rows.rows * a.col_tiles / 8 >= INT32_MAX || a.col_tiles > 65535) return cudaErrorInvalidValue;
    if (type == MOE_F32) {
        if (m.format == MOE_MX_E8M0) return dequantise_rows<float, MOE_MX_E8M0>(a, st);
        return dequantise_rows<float, MOE_MX_E4M3>(a, st);
    }
    if (m.format == MOE_MX_E8M0)
        return dequantise_rows<__nv_bfloat16, MOE_MX_E8M0>(a, st);
    return dequantise_rows<__nv_bfloat16, MOE_MX_E4M3>(a, st);
}

}  // namespace moe
