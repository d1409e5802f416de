// mx_quantise.cu -- rows to microscaled 4-bit floats and back.
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "mx.h"

namespace moe {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kThreads = 256;
constexpr int kChunk = 16;  // columns of a thread: one E4M3 block, half an E8M0 block

__device__ __forceinline__ void load16(const float* p, int n, bool wide, float (&v)[16]) {
    if (wide && n >= 16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 q = reinterpret_cast<const float4*>(p)[i];
            v[4 * i] = q.x, v[4 * i + 1] = q.y, v[4 * i + 2] = q.z, v[4 * i + 3] = q.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = i < n ? p[i] : 0.0f;
    }
}
__device__ __forceinline__ void load16(const __nv_bfloat16* p, int n, bool wide, float (&v)[16]) {
    if (wide && n >= 16) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint4 q = reinterpret_cast<const uint4*>(p)[i];
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
                v[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = i < n ? __bfloat162float(p[i]) : 0.0f;
    }
}
__device__ __forceinline__ void store16(float* p, int n, bool wide, const float (&v)[16]) {
    if (wide && n >= 16) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            reinterpret_cast<float4*>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (i < n) p[i] = v[i];
    }
}
__device__ __forceinline__ void store16(__nv_bfloat16* p, int n, bool wide, const float (&v)[16]) {
    if (wide && n >= 16) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(v[8 * i + 2 * j], v[8 * i + 2 * j + 1]);
                w[j] = *reinterpret_cast<const uint32_t*>(&b);
            }
            reinterpret_cast<uint4*>(p)[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
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
    int64_t ld;
    int cols, col_tiles;
    bool wide;
};

constexpr int kRows = kThreads / 16;  // rows of a block: 16 threads share a row's 256 columns

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float silu_mul(float g, float u) { return __fdividef(g, 1.0f + __expf(-g)) * u; }

// byte offset of a chunk's 8 code bytes in its tile, and of its scale bytes' word
__device__ __forceinline__ uint32_t code_at(int in, int c16) {
    const int c = c16 >> 1;  // 16-byte chunk of the tile's row
    return (uint32_t)(in * 128 + ((c ^ (in & 7)) << 4) + ((c16 & 1) << 3));
}
__device__ __forceinline__ uint32_t scale_at(int in, int atom) {
    return (uint32_t)(kMxCodeBytes + atom * kMxAtomBytes + (in & 31) * 16 + (in >> 5) * 4);
}

// A block takes 16 rows of one column tile, a thread 16 columns of a row, so
// 16 threads write one row's 128 bytes of codes, and the scale bytes of four
// blocks go out as one word.  Row maps and tile addresses need no division.
//
// Both formats divide by a scale before the rounding to e2m1.  A power of two
// is an exact multiply.  The e4m3 scale takes a reciprocal and one residual
// step: r = x / d to a few units of the last place, then
// r + (x - r d) / d, the remainder exact in one fma.  Where x / d is itself a
// short number, as a tie between two codes is, the result is exactly that.
template <typename T, int FMT, bool SWIGLU>
__global__ void __launch_bounds__(kThreads) quantise_kernel(const QuantArgs a) {
    after_previous();
    let_next_start();
    const int c16 = threadIdx.x & 15;
    const int64_t r = (int64_t)blockIdx.x * kRows + (threadIdx.x >> 4);
    int g = 0, in = 0;
    int64_t tile = 0;
    bool live = r < a.rows.rows;
    int64_t from = live ? (a.src_row ? a.src_row[r] : r) : -1;
    live = live && a.rows.place(r, g, tile, in) && from >= 0;
    float v[16];
    const int col = blockIdx.y * kMxTileCols + c16 * kChunk, n = live ? a.cols - col : 0;
    const T* p = static_cast<const T*>(a.src) + (live ? from * a.ld + col : 0);
    load16(p, n, a.wide, v);
    if (SWIGLU) {
        float u[16];
        load16(p + a.cols, n, a.wide, u);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = silu_mul(v[i], u[i]);
    }
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) amax = max_nan(amax, fabsf(v[i]));
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
        for (int i = 0; i < 16; ++i) v[i] *= inv;
    } else {
        const float t = a.tscale && live ? a.tscale[g] : 1.0f;
        const __nv_fp8_storage_t s =
            __nv_cvt_float_to_fp8(__fdiv_rn(amax, 6.0f * t), __NV_SATFINITE, __NV_E4M3);
        byte = s;
        const float d = __half2float(__half(__nv_cvt_fp8_to_halfraw(s, __NV_E4M3))) * t;
        const float inv = d > 0.0f ? __frcp_rn(d) : 0.0f;
        if (inv < 1e30f) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float q = v[i] * inv;
                v[i] = fmaf(fmaf(-q, d, v[i]), inv, q);
            }
        } else {  // scales so small that the remainder could be subnormal
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = __fdiv_rn(v[i], d);
        }
    }
    uint32_t out[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t w = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = make_float2(v[8 * h + 2 * i], v[8 * h + 2 * i + 1]);
            w |= (uint32_t)__nv_cvt_float2_to_fp4x2(f, __NV_E2M1, cudaRoundNearest) << (8 * i);
        }
        out[h] = w;
    }
    if (!finite) {
        byte = FMT == MOE_MX_E8M0 ? 255 : 127;
        out[0] = out[1] = 0;
    }
    // join the bytes of four consecutive blocks
    constexpr int kStep = FMT == MOE_MX_E8M0 ? 2 : 1;  // threads per block
    uint32_t word = byte;
    word |= __shfl_down_sync(kAll, word, kStep) << 8;
    word |= __shfl_down_sync(kAll, word, 2 * kStep) << 16;
    if (!live) return;
    uint8_t* base = a.data + (tile * a.col_tiles + blockIdx.y) * (int64_t)mx_tile_bytes(FMT);
    *reinterpret_cast<uint2*>(base + code_at(in, c16)) = make_uint2(out[0], out[1]);
    if (c16 % (4 * kStep) == 0) *reinterpret_cast<uint32_t*>(base + scale_at(in, c16 / (4 * kStep))) = word;
}

template <typename T, int FMT>
__global__ void __launch_bounds__(kThreads) dequantise_kernel(const QuantArgs a) {
    after_previous();
    let_next_start();
    const int c16 = threadIdx.x & 15;
    const int64_t r = (int64_t)blockIdx.x * kRows + (threadIdx.x >> 4);
    int g, in;
    int64_t tile;
    const int col = blockIdx.y * kMxTileCols + c16 * kChunk, n = a.cols - col;
    if (r >= a.rows.rows || n <= 0 || !a.rows.place(r, g, tile, in)) return;
    const uint8_t* base = a.data + (tile * a.col_tiles + blockIdx.y) * (int64_t)mx_tile_bytes(FMT);
    const int b = FMT == MOE_MX_E8M0 ? c16 >> 1 : c16;
    const uint2 q = *reinterpret_cast<const uint2*>(base + code_at(in, c16));
    const uint32_t byte = base[scale_at(in, b >> 2) + (b & 3)];
    float s;
    if (FMT == MOE_MX_E8M0)
        s = byte == 255 ? __uint_as_float(0x7fffffffu) : byte ? __uint_as_float(byte << 23) : __uint_as_float(0x400000u);
    else
        s = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3)));
    const float t = a.tscale ? a.tscale[g] : 1.0f;
    float v[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t two = ((i < 4 ? q.x : q.y) >> (8 * (i & 3))) & 0xffu;
        const __half2 h = __half2(__nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)two, __NV_E2M1));
        v[2 * i] = __low2float(h) * s * t;
        v[2 * i + 1] = __high2float(h) * s * t;
    }
    store16(static_cast<T*>(a.dst) + r * a.ld + col, n, a.wide, v);
}

dim3 grid_of(const QuantArgs& a) { return dim3((unsigned)((a.rows.rows + kRows - 1) / kRows), (unsigned)a.col_tiles); }

template <typename T, int FMT>
cudaError_t quantise_act(const QuantArgs& a, int act, cudaStream_t st) {
    if (act == MOE_ACT_SWIGLU) return launch(quantise_kernel<T, FMT, true>, grid_of(a), kThreads, 0, st, 1, a);
    return launch(quantise_kernel<T, FMT, false>, grid_of(a), kThreads, 0, st, 1, a);
}

// whole 16-byte loads or stores need every 16-column chunk of every row aligned
bool wide_ok(const void* p, int64_t ld, int64_t second, int type) {
    const int64_t size = type == MOE_F32 ? 4 : 2;
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * size % 16 == 0 && second * size % 16 == 0;
}

}  // namespace

cudaError_t launch_mx_quantise(const moe_mx& m, const MxRows& rows, const void* src, int type, int64_t ld, int act,
                               const int32_t* src_row, const float* tscale, cudaStream_t st) {
    QuantArgs a{};
    a.data = static_cast<uint8_t*>(m.data_dev);
    a.rows = rows;
    a.src = src;
    a.src_row = src_row;
    a.tscale = tscale;
    a.ld = ld;
    a.cols = m.cols;
    a.col_tiles = (int)mx_col_tiles(m.cols);
    a.wide = wide_ok(src, ld, act == MOE_ACT_SWIGLU ? m.cols : 0, type);
    if ((rows.rows + kRows - 1) / kRows > INT32_MAX || a.col_tiles > 65535) return cudaErrorInvalidValue;
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
    if ((rows.rows + kRows - 1) / kRows > INT32_MAX || a.col_tiles > 65535) return cudaErrorInvalidValue;
    if (type == MOE_F32) {
        if (m.format == MOE_MX_E8M0) return launch(dequantise_kernel<float, MOE_MX_E8M0>, grid_of(a), kThreads, 0, st, 1, a);
        return launch(dequantise_kernel<float, MOE_MX_E4M3>, grid_of(a), kThreads, 0, st, 1, a);
    }
    if (m.format == MOE_MX_E8M0)
        return launch(dequantise_kernel<__nv_bfloat16, MOE_MX_E8M0>, grid_of(a), kThreads, 0, st, 1, a);
    return launch(dequantise_kernel<__nv_bfloat16, MOE_MX_E4M3>, grid_of(a), kThreads, 0, st, 1, a);
}

}  // namespace moe
