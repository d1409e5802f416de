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
            const float4 q = __ldg(reinterpret_cast<const float4*>(p) + i);
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
            const uint4 q = __ldg(reinterpret_cast<const uint4*>(p) + i);
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
    int cols, chunks;  // chunks: 16-column chunks of a padded row, a multiple of 16
    bool wide;
};

// byte offset of a chunk's 8 code bytes in its tile, and of its scale bytes' word
__device__ __forceinline__ uint32_t code_at(int in, int c16) {
    const int c = c16 >> 1;  // 16-byte chunk of the tile's row
    return (uint32_t)(in * 128 + ((c ^ (in & 7)) << 4) + ((c16 & 1) << 3));
}
__device__ __forceinline__ uint32_t scale_at(int in, int atom) {
    return (uint32_t)(kMxCodeBytes + atom * kMxAtomBytes + (in & 31) * 16 + (in >> 5) * 4);
}

// A thread takes 16 columns of a row, 16 threads one row of a tile: 128 bytes
// of codes, and the scale bytes of four blocks joined into one word.
template <typename T, int FMT, bool SWIGLU>
__global__ void __launch_bounds__(kThreads) quantise_kernel(const QuantArgs a) {
    const int64_t item = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t r = item / a.chunks;
    const int ck = (int)(item % a.chunks);
    int g = 0, in = 0;
    int64_t tile = 0;
    bool live = r < a.rows.rows && a.rows.place(r, g, tile, in);
    int64_t from = live ? (a.src_row ? a.src_row[r] : r) : -1;
    live = from >= 0;
    float v[16];
    const int col = ck * kChunk, n = live ? a.cols - col : 0;
    const T* p = static_cast<const T*>(a.src) + (live ? from * a.ld + col : 0);
    load16(p, n, a.wide, v);
    if (SWIGLU) {
        float u[16];
        load16(p + a.cols, n, a.wide, u);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = v[i] / (1.0f + expf(-v[i])) * u[i];
    }
    float amax = 0.0f;
    bool finite = true;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        amax = fmaxf(amax, fabsf(v[i]));
        finite = finite && fabsf(v[i]) <= 3.402823466e38f;
    }
    uint32_t byte;
    uint32_t out[2];
    if (FMT == MOE_MX_E8M0) {
        amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, 1));
        finite = finite & (__shfl_xor_sync(kAll, (int)finite, 1) != 0);
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
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = d > 0.0f ? __fdiv_rn(v[i], d) : 0.0f;
    }
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
    uint8_t* base = a.data + (tile * (a.chunks / 16) + (ck >> 4)) * (int64_t)mx_tile_bytes(FMT);
    const int c16 = ck & 15;
    *reinterpret_cast<uint2*>(base + code_at(in, c16)) = make_uint2(out[0], out[1]);
    if (c16 % (4 * kStep) == 0) *reinterpret_cast<uint32_t*>(base + scale_at(in, c16 / (4 * kStep))) = word;
}

template <typename T, int FMT>
__global__ void __launch_bounds__(kThreads) dequantise_kernel(const QuantArgs a) {
    const int64_t item = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t r = item / a.chunks;
    const int ck = (int)(item % a.chunks);
    int g, in;
    int64_t tile;
    const int n = a.cols - ck * kChunk;
    if (r >= a.rows.rows || n <= 0 || !a.rows.place(r, g, tile, in)) return;
    const uint8_t* base = a.data + (tile * (a.chunks / 16) + (ck >> 4)) * (int64_t)mx_tile_bytes(FMT);
    const int c16 = ck & 15, b = FMT == MOE_MX_E8M0 ? c16 >> 1 : c16;
    const uint2 q = __ldg(reinterpret_cast<const uint2*>(base + code_at(in, c16)));
    const uint32_t byte = __ldg(base + scale_at(in, b >> 2) + (b & 3));
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
    store16(static_cast<T*>(a.dst) + r * a.ld + ck * kChunk, n, a.wide, v);
}

unsigned grid_of(const QuantArgs& a) { return (unsigned)((a.rows.rows * a.chunks + kThreads - 1) / kThreads); }

template <typename T, int FMT>
void quantise_act(const QuantArgs& a, int act, cudaStream_t st) {
    if (act == MOE_ACT_SWIGLU)
        quantise_kernel<T, FMT, true><<<grid_of(a), kThreads, 0, st>>>(a);
    else
        quantise_kernel<T, FMT, false><<<grid_of(a), kThreads, 0, st>>>(a);
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
    a.chunks = (int)mx_col_tiles(m.cols) * 16;
    a.wide = wide_ok(src, ld, act == MOE_ACT_SWIGLU ? m.cols : 0, type);
    if ((rows.rows * a.chunks + kThreads - 1) / kThreads > INT32_MAX) return cudaErrorInvalidValue;
    if (type == MOE_F32) {
        if (m.format == MOE_MX_E8M0) quantise_act<float, MOE_MX_E8M0>(a, act, st);
        else quantise_act<float, MOE_MX_E4M3>(a, act, st);
    } else {
        if (m.format == MOE_MX_E8M0) quantise_act<__nv_bfloat16, MOE_MX_E8M0>(a, act, st);
        else quantise_act<__nv_bfloat16, MOE_MX_E4M3>(a, act, st);
    }
    return cudaGetLastError();
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
    a.chunks = (int)mx_col_tiles(m.cols) * 16;
    a.wide = wide_ok(dst, ld, 0, type);
    if ((rows.rows * a.chunks + kThreads - 1) / kThreads > INT32_MAX) return cudaErrorInvalidValue;
    if (type == MOE_F32) {
        if (m.format == MOE_MX_E8M0) dequantise_kernel<float, MOE_MX_E8M0><<<grid_of(a), kThreads, 0, st>>>(a);
        else dequantise_kernel<float, MOE_MX_E4M3><<<grid_of(a), kThreads, 0, st>>>(a);
    } else {
        if (m.format == MOE_MX_E8M0) dequantise_kernel<__nv_bfloat16, MOE_MX_E8M0><<<grid_of(a), kThreads, 0, st>>>(a);
        else dequantise_kernel<__nv_bfloat16, MOE_MX_E4M3><<<grid_of(a), kThreads, 0, st>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace moe
