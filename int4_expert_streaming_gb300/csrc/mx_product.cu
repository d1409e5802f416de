// mx_product.cu -- y = alpha * X W^T of two microscaled 4-bit matrices, dense
// or grouped: a plain tiled form on the CUDA cores.
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "mx.h"

namespace moe {
namespace {

constexpr int kT = 64, kK = 32;  // tile rows and columns, columns of a step

struct ProductArgs {
    const uint8_t* x;
    const uint8_t* w;
    const int32_t* offsets;  // NULL: one group of x_rows rows
    const float* alpha;
    void* y;
    int64_t y_ld, x_rows, w_rows;
    int groups, cols, col_tiles, y_f32;
};

template <int FMT>
__device__ __forceinline__ float value(const uint8_t* data, int64_t row_tile, int in, int col, int col_tiles) {
    const uint8_t* base = data + (row_tile * col_tiles + col / kMxTileCols) * (int64_t)mx_tile_bytes(FMT);
    const int c = col % kMxTileCols, b = c / (FMT == MOE_MX_E8M0 ? 32 : 16);
    const uint32_t two = base[in * 128 + (((c >> 5) ^ (in & 7)) << 4) + ((c & 31) >> 1)];
    const uint32_t byte = base[kMxCodeBytes + (b >> 2) * kMxAtomBytes + (in & 31) * 16 + (in >> 5) * 4 + (b & 3)];
    const __half2 h = __half2(__nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)two, __NV_E2M1));
    float s;
    if (FMT == MOE_MX_E8M0)
        s = byte == 255 ? __uint_as_float(0x7fffffffu) : byte ? __uint_as_float(byte << 23) : __uint_as_float(0x400000u);
    else
        s = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3)));
    return (col & 1 ? __high2float(h) : __low2float(h)) * s;
}

// Block (n tile, y tile): the group of y tile j is found by bisection, since
// group g's tiles can start at offsets[g] / 64 + g without overlap.
template <int FMT>
__global__ void __launch_bounds__(256) product_kernel(const ProductArgs a) {
    __shared__ float xs[kK][kT + 1], ws[kK][kT + 1];
    int g = 0;
    int64_t o = 0, n = a.x_rows, j = blockIdx.y;
    if (a.offsets) {
        int lo = 0, hi = a.groups - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (a.offsets[mid] / kT + mid <= j) lo = mid;
            else hi = mid - 1;
        }
        g = lo;
        o = a.offsets[g];
        n = a.offsets[g + 1] - o;
        j -= o / kT + g;
    }
    const int64_t r0 = j * kT, c0 = (int64_t)blockIdx.x * kT;
    if (r0 >= n) return;
    const int64_t xt = a.offsets ? o / kMxTileRows + g : 0;
    const int64_t wt = g * ((a.w_rows + kMxTileRows - 1) / kMxTileRows);
    float acc[4][4] = {};
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int k0 = 0; k0 < a.cols; k0 += kK) {
        for (int i = threadIdx.x; i < kT * kK; i += 256) {
            const int k = i % kK, q = i / kK;
            const int64_t xr = r0 + q, wr = c0 + q;
            xs[k][q] = xr < n && k0 + k < a.cols
                           ? value<FMT>(a.x, xt + xr / kMxTileRows, (int)(xr % kMxTileRows), k0 + k, a.col_tiles) : 0.0f;
            ws[k][q] = wr < a.w_rows && k0 + k < a.cols
                           ? value<FMT>(a.w, wt + wr / kMxTileRows, (int)(wr % kMxTileRows), k0 + k, a.col_tiles) : 0.0f;
        }
        __syncthreads();
#pragma unroll 4
        for (int k = 0; k < kK; ++k) {
            float xv[4], wv[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) xv[i] = xs[k][ty + 16 * i], wv[i] = ws[k][tx + 16 * i];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[i][q] += xv[i] * wv[q];
        }
        __syncthreads();
    }
    const float alpha = a.alpha ? a.alpha[g] : 1.0f;
    for (int i = 0; i < 4; ++i)
        for (int q = 0; q < 4; ++q) {
            const int64_t r = r0 + ty + 16 * i, c = c0 + tx + 16 * q;
            if (r >= n || c >= a.w_rows) continue;
            const float v = acc[i][q] * alpha;
            if (a.y_f32) static_cast<float*>(a.y)[(o + r) * a.y_ld + c] = v;
            else static_cast<__nv_bfloat16*>(a.y)[(o + r) * a.y_ld + c] = __float2bfloat16_rn(v);
        }
}

}  // namespace

cudaError_t launch_mx_product(const moe_mx& x, const moe_mx& w, const int32_t* offsets, const float* alpha, void* y,
                              int y_type, int64_t y_ld, cudaStream_t st) {
    ProductArgs a{static_cast<const uint8_t*>(x.data_dev), static_cast<const uint8_t*>(w.data_dev), offsets, alpha, y,
                  y_ld, x.rows, w.rows, w.groups, x.cols, (int)mx_col_tiles(x.cols), y_type == MOE_F32};
    const int64_t tiles = offsets ? x.rows / kT + w.groups : (x.rows + kT - 1) / kT;
    if (tiles > 65535) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)((w.rows + kT - 1) / kT), (unsigned)tiles);
    if (x.format == MOE_MX_E8M0) product_kernel<MOE_MX_E8M0><<<grid, 256, 0, st>>>(a);
    else product_kernel<MOE_MX_E4M3><<<grid, 256, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace moe
