// mx.h -- the context-free operators (routing with groups, pair sort,
// microscaled 4-bit matrices, combine): launchers and the tile layout shared
// by their kernels.
#pragma once

#include <cuda_bf16.h>

#include "moe_internal.h"

namespace moe {

constexpr int kMxTileRows = 128, kMxTileCols = 256;
constexpr int kMxCodeBytes = 16384;  // codes of one tile
constexpr int kMxAtomBytes = 512;    // scales of 128 rows x 4 blocks

__host__ __device__ inline int mx_block(int format) { return format == MOE_MX_E8M0 ? 32 : 16; }
__host__ __device__ inline int mx_tile_bytes(int format) {
    return kMxCodeBytes + kMxAtomBytes * (kMxTileCols / 4 / mx_block(format));
}
__host__ __device__ inline int64_t mx_col_tiles(int cols) { return (cols + kMxTileCols - 1) / kMxTileCols; }

// Launches are programmatic dependents of the kernel before them on the
// stream: a kernel's CTAs may be set up while that one still runs, and wait
// (after_previous) before they touch memory; every thread that does so waits.
// Memory is read by plain loads: the read-only path may not be used for data
// that changes during the kernel's life.  let_next_start allows the same to the
// kernel after it.  Between two small
// kernels this hides most of the launch.
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t st, unsigned cluster,
                   const A&... args) {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = threads;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// Where the rows of a matrix stand: row tile and row within it.  Ragged
// groups start at row tile offsets[g] / 128 + g: consecutive groups then never
// overlap, because floor((o + n) / 128) + 1 - floor(o / 128) >= ceil(n / 128).
struct MxRows {
    const int32_t* group_of_row;  // ragged only
    const int32_t* offsets;
    int64_t rows;       // rows to walk
    int64_t per_group;  // uniform: rows per group
    int groups;
    __device__ __forceinline__ bool place(int64_t r, int& g, int64_t& tile, int& in) const {
        int64_t q;
        if (group_of_row) {
            g = group_of_row[r];
            if (g < 0 || g >= groups) return false;
            const int o = offsets[g];
            q = r - o;
            if (o < 0 || q < 0) return false;  // maps that do not belong together: nothing is written out of range
            tile = (o >> 7) + g + (q >> 7);
        } else if (rows == per_group) {
            g = 0;
            q = r;
            tile = r >> 7;
        } else {
            g = (int)(r / per_group);
            q = r - g * per_group;
            tile = g * ((per_group + kMxTileRows - 1) >> 7) + (q >> 7);
        }
        in = (int)(q & (kMxTileRows - 1));
        return true;
    }
};

// mx_route.cu
cudaError_t launch_route(const moe_route_config& c, const void* logits, int type, int64_t ld, const float* bias,
                         int64_t T, int32_t* idx, float* w, cudaStream_t st);
size_t dispatch_workspace(int64_t pairs, int n_experts);
cudaError_t launch_dispatch(const int32_t* idx, int64_t pairs, int top_k, int n_experts, int32_t* offsets,
                            int32_t* row_of_pair, int32_t* token_of_row, int32_t* group_of_row, void* ws,
                            cudaStream_t st);
cudaError_t launch_combine(const void* rows, int64_t n_rows, int rows_type, int64_t rows_ld, const int32_t* row_of_pair,
                           const float* w, int64_t T, int top_k, int cols, void* y, int y_type, int64_t y_ld, cudaStream_t st);
// mx_quantise.cu
cudaError_t launch_mx_quantise(const moe_mx& m, const MxRows& rows, const void* src, int64_t src_rows, int type,
                               int64_t ld, int act, const int32_t* src_row, const float* tscale, cudaStream_t st);
cudaError_t launch_mx_dequantise(const moe_mx& m, const MxRows& rows, const float* tscale, void* dst, int type,
                                 int64_t ld, cudaStream_t st);
// mx_product.cu; fault: with a wait that nothing ends, and short limits
cudaError_t launch_mx_product(const moe_mx& x, const moe_mx& w, const int32_t* offsets, const float* alpha, void* y,
                              int y_type, int64_t y_ld, cudaStream_t st, bool fault);
cudaError_t mx_timeouts(uint64_t* count);  // of the current device

}  // namespace moe
