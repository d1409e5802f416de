// mx_api.cu -- C entries of the context-free operators: argument checks, then
// one launcher each (see include/moe.h).
#include "mx.h"

namespace moe {
namespace {

thread_local bool g_fault = false;  // moe_mx_set_fault

// the descriptor's shape, not its address
bool mx_ok(const moe_mx* m) {
    return m && m->rows >= 0 && m->cols >= 1 && m->groups >= 1 && m->groups <= 1024 &&
           (m->format == MOE_MX_E8M0 || m->format == MOE_MX_E4M3) && (m->ragged == 0 || m->ragged == 1) &&
           m->rows <= (INT64_C(1) << 31) - 1 && m->cols <= 1 << 23 &&
           (m->ragged ? m->rows : m->rows * m->groups) <= (INT64_C(1) << 40);
}

int check_mx(const moe_mx* m, const char* name) {
    if (!mx_ok(m)) return fail_global(MOE_EINVAL, "%s: bad matrix descriptor", name);
    if (m->rows > 0 && (!m->data_dev || reinterpret_cast<uintptr_t>(m->data_dev) % 128))
        return fail_global(MOE_EINVAL, "%s: data_dev must be set and 128-byte aligned", name);
    return MOE_OK;
}

MxRows rows_of(const moe_mx* m, const int32_t* group_of_row, const int32_t* offsets) {
    MxRows r;
    r.group_of_row = m->ragged ? group_of_row : nullptr;
    r.offsets = offsets;
    r.rows = m->ragged ? m->rows : m->rows * m->groups;
    r.per_group = m->rows;
    r.groups = m->groups;
    return r;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_route(const moe_route_config* c, const void* logits, int32_t type, int64_t ld, const float* bias,
                         int64_t T, int32_t* idx, float* w, void* stream) {
    return guarded([&]() -> int {
        if (!c) return fail_global(MOE_EINVAL, "moe_route: cfg is NULL");
        if (c->n_experts < 1 || c->n_experts > 1024)
            return fail_global(MOE_EINVAL, "moe_route: n_experts=%d outside 1..1024", c->n_experts);
        if (c->n_groups < 1 || c->n_groups > 32 || c->n_experts % c->n_groups)
            return fail_global(MOE_EINVAL, "moe_route: n_groups=%d must be 1..32 and divide n_experts=%d", c->n_groups,
                               c->n_experts);
        if (c->top_groups < 1 || c->top_groups > c->n_groups)
            return fail_global(MOE_EINVAL, "moe_route: top_groups=%d outside 1..n_groups", c->top_groups);
        if (c->top_k < 1 || c->top_k > 32 || c->top_k > c->top_groups * (c->n_experts / c->n_groups))
            return fail_global(MOE_EINVAL, "moe_route: top_k=%d outside 1..min(32, experts of top_groups)", c->top_k);
        if (c->group_best < 1 || c->group_best > 2)
            return fail_global(MOE_EINVAL, "moe_route: group_best=%d must be 1 or 2", c->group_best);
        if (c->score != MOE_SCORE_SOFTMAX && c->score != MOE_SCORE_SIGMOID)
            return fail_global(MOE_EINVAL, "moe_route: unknown score %d", c->score);
        if (!type_ok(type)) return fail_global(MOE_EINVAL, "moe_route: unknown logits type %d", type);
        if (T < 0 || T > INT32_MAX) return fail_global(MOE_EINVAL, "moe_route: T=%lld out of range", (long long)T);
        if (ld < c->n_experts) return fail_global(MOE_EINVAL, "moe_route: ld=%lld below n_experts", (long long)ld);
        if (T == 0) return MOE_OK;
        if (!logits || !idx || !w) return fail_global(MOE_EINVAL, "moe_route: logits, idx and w are required");
        return launched(launch_route(*c, logits, type, ld, bias, T, idx, w, static_cast<cudaStream_t>(stream)),
                        "moe_route");
    });
}

static bool dispatch_ok(int64_t T, int32_t k, int32_t E) {
    return T >= 0 && k >= 1 && E >= 1 && E <= 1024 && T <= INT32_MAX && T * k <= INT32_MAX;
}

extern "C" size_t moe_dispatch_workspace(int64_t T, int32_t top_k, int32_t n_experts) {
    return dispatch_ok(T, top_k, n_experts) ? dispatch_workspace(T * top_k, n_experts) : 0;
}

extern "C" int moe_dispatch(const int32_t* idx, int64_t T, int32_t top_k, int32_t n_experts, int32_t* offsets,
                            int32_t* row_of_pair, int32_t* token_of_row, int32_t* group_of_row, void* ws,
                            size_t ws_bytes, void* stream) {
    return guarded([&]() -> int {
        if (!dispatch_ok(T, top_k, n_experts))
            return fail_global(MOE_EINVAL, "moe_dispatch: T=%lld, top_k=%d or n_experts=%d out of range", (long long)T,
                               top_k, n_experts);
        if (!offsets) return fail_global(MOE_EINVAL, "moe_dispatch: offsets is required");
        if (T > 0 && (!idx || !row_of_pair || !token_of_row || !group_of_row))
            return fail_global(MOE_EINVAL, "moe_dispatch: idx and the three row maps are required");
        const size_t need = dispatch_workspace(T * top_k, n_experts);
        if (ws_bytes < need || (need && (!ws || reinterpret_cast<uintptr_t>(ws) % 16)))
            return fail_global(MOE_EINVAL, "moe_dispatch: needs %zu bytes of 16-byte aligned workspace, got %zu", need,
                               ws_bytes);
        return launched(launch_dispatch(idx, T * top_k, top_k, n_experts, offsets, row_of_pair, token_of_row,
                                        group_of_row, ws, static_cast<cudaStream_t>(stream)),
                        "moe_dispatch");
    });
}

extern "C" size_t moe_mx_bytes(const moe_mx* m) {
    if (!mx_ok(m)) return 0;
    const int64_t tiles = m->ragged ? m->rows / kMxTileRows + m->groups
                                    : m->groups * ((m->rows + kMxTileRows - 1) / kMxTileRows);
    return (size_t)tiles * (size_t)mx_col_tiles(m->cols) * (size_t)mx_tile_bytes(m->format);
}

// the row maps of a ragged matrix, and none for a uniform one
static int check_maps(const moe_mx* m, const int32_t* group_of_row, const int32_t* offsets, const char* name) {
    if (m->ragged && m->rows > 0 && (!group_of_row || !offsets))
        return fail_global(MOE_EINVAL, "%s: a ragged matrix needs group_of_row and offsets", name);
    if (!m->ragged && (group_of_row || offsets))
        return fail_global(MOE_EINVAL, "%s: group_of_row and offsets go with a ragged matrix", name);
    return MOE_OK;
}

extern "C" int moe_mx_quantise_rows(const moe_mx* m, const void* src, int64_t src_rows, int32_t type, int64_t ld,
                                    int32_t act, const int32_t* src_row, const int32_t* group_of_row,
                                    const int32_t* offsets, const float* tscale, void* stream) {
    return guarded([&]() -> int {
        int rc = check_mx(m, "moe_mx_quantise");
        if (rc || (rc = check_maps(m, group_of_row, offsets, "moe_mx_quantise"))) return rc;
        if (!type_ok(type)) return fail_global(MOE_EINVAL, "moe_mx_quantise: unknown source type %d", type);
        if (act != MOE_ACT_NONE && act != MOE_ACT_SWIGLU)
            return fail_global(MOE_EINVAL, "moe_mx_quantise: unknown activation %d", act);
        if (ld < (int64_t)m->cols * (act == MOE_ACT_SWIGLU ? 2 : 1))
            return fail_global(MOE_EINVAL, "moe_mx_quantise: src_ld=%lld is shorter than a source row", (long long)ld);
        if (tscale && m->format != MOE_MX_E4M3)
            return fail_global(MOE_EINVAL, "moe_mx_quantise: tensor scales go with MOE_MX_E4M3");
        if (src_rows < 0) return fail_global(MOE_EINVAL, "moe_mx_quantise: src_rows=%lld", (long long)src_rows);
        const MxRows rows = rows_of(m, group_of_row, offsets);
        if (rows.rows == 0) return MOE_OK;
        if (!src && src_rows > 0) return fail_global(MOE_EINVAL, "moe_mx_quantise: src is required");
        return launched(launch_mx_quantise(*m, rows, src, src_rows, type, ld, act, src_row, tscale,
                                           static_cast<cudaStream_t>(stream)),
                        "moe_mx_quantise");
    });
}

extern "C" int moe_mx_quantise(const moe_mx* m, const void* src, int32_t type, int64_t ld, int32_t act,
                               const int32_t* src_row, const int32_t* group_of_row, const int32_t* offsets,
                               const float* tscale, void* stream) {
    return moe_mx_quantise_rows(m, src, INT64_MAX, type, ld, act, src_row, group_of_row, offsets, tscale, stream);
}

extern "C" int moe_mx_dequantise(const moe_mx* m, const int32_t* group_of_row, const int32_t* offsets,
                                 const float* tscale, void* dst, int32_t type, int64_t ld, void* stream) {
    return guarded([&]() -> int {
        int rc = check_mx(m, "moe_mx_dequantise");
        if (rc || (rc = check_maps(m, group_of_row, offsets, "moe_mx_dequantise"))) return rc;
        if (!type_ok(type)) return fail_global(MOE_EINVAL, "moe_mx_dequantise: unknown type %d", type);
        if (ld < m->cols)
            return fail_global(MOE_EINVAL, "moe_mx_dequantise: dst_ld=%lld is shorter than a row", (long long)ld);
        const MxRows rows = rows_of(m, group_of_row, offsets);
        if (rows.rows == 0) return MOE_OK;
        if (!dst) return fail_global(MOE_EINVAL, "moe_mx_dequantise: dst is required");
        return launched(launch_mx_dequantise(*m, rows, tscale, dst, type, ld, static_cast<cudaStream_t>(stream)),
                        "moe_mx_dequantise");
    });
}

extern "C" int moe_mx_product(const moe_mx* x, const moe_mx* w, const int32_t* offsets, const float* alpha, void* y,
                              int32_t type, int64_t y_ld, void* stream) {
    return guarded([&]() -> int {
        int rc = check_mx(x, "moe_mx_product: x");
        if (rc || (rc = check_mx(w, "moe_mx_product: w"))) return rc;
        if (w->ragged) return fail_global(MOE_EINVAL, "moe_mx_product: w must be uniform");
        if (x->format != w->format || x->cols != w->cols)
            return fail_global(MOE_EINVAL, "moe_mx_product: x and w differ in format or cols");
        if (x->groups != w->groups || (!x->ragged && x->groups != 1))
            return fail_global(MOE_EINVAL, "moe_mx_product: x must be ragged with w's groups, or uniform with one group");
        if ((x->ragged != 0) != (offsets != nullptr) && x->rows > 0)
            return fail_global(MOE_EINVAL, "moe_mx_product: offsets go with a ragged x");
        if (!type_ok(type)) return fail_global(MOE_EINVAL, "moe_mx_product: unknown type %d", type);
        if (y_ld < w->rows) return fail_global(MOE_EINVAL, "moe_mx_product: y_ld=%lld below w's rows", (long long)y_ld);
        if (x->rows == 0 || w->rows == 0) return MOE_OK;
        if (!y) return fail_global(MOE_EINVAL, "moe_mx_product: y is required");
        return launched(
            launch_mx_product(*x, *w, offsets, alpha, y, type, y_ld, static_cast<cudaStream_t>(stream), g_fault),
            "moe_mx_product");
    });
}

extern "C" int moe_mx_timeouts(uint64_t* count) {
    return guarded([&]() -> int {
        if (!count) return fail_global(MOE_EINVAL, "moe_mx_timeouts: count is NULL");
        return launched(mx_timeouts(count), "moe_mx_timeouts");
    });
}

extern "C" int moe_mx_set_fault(uint32_t fault_flags) {
    return guarded([&]() -> int {
        if (fault_flags & ~MOE_FAULT_DEVICE_WAIT)
            return fail_global(MOE_EINVAL, "moe_mx_set_fault: only MOE_FAULT_DEVICE_WAIT applies");
        g_fault = fault_flags != 0;
        return MOE_OK;
    });
}

extern "C" int moe_combine_rows(const void* rows, int64_t n_rows, int32_t rows_type, int64_t rows_ld,
                                const int32_t* row_of_pair, const float* w, int64_t T, int32_t top_k, int32_t cols,
                                void* y, int32_t y_type, int64_t y_ld, void* stream) {
    return guarded([&]() -> int {
        if (T < 0 || T > INT32_MAX || top_k < 1 || cols < 1 || cols > 1 << 22 || T * top_k > INT32_MAX)
            return fail_global(MOE_EINVAL, "moe_combine: T=%lld, top_k=%d or cols=%d out of range", (long long)T, top_k,
                               cols);
        if (!type_ok(rows_type) || !type_ok(y_type)) return fail_global(MOE_EINVAL, "moe_combine: unknown element type");
        if (rows_ld < cols || y_ld < cols) return fail_global(MOE_EINVAL, "moe_combine: a stride is shorter than a row");
        if (n_rows < 0) return fail_global(MOE_EINVAL, "moe_combine: n_rows=%lld", (long long)n_rows);
        if (T == 0) return MOE_OK;
        if ((!rows && n_rows > 0) || !row_of_pair || !w || !y)
            return fail_global(MOE_EINVAL, "moe_combine: rows, row_of_pair, w and y are required");
        return launched(launch_combine(rows, n_rows, rows_type, rows_ld, row_of_pair, w, T, top_k, cols, y, y_type, y_ld,
                                       static_cast<cudaStream_t>(stream)),
                        "moe_combine");
    });
}

extern "C" int moe_combine(const void* rows, int32_t rows_type, int64_t rows_ld, const int32_t* row_of_pair,
                           const float* w, int64_t T, int32_t top_k, int32_t cols, void* y, int32_t y_type,
                           int64_t y_ld, void* stream) {
    return moe_combine_rows(rows, INT64_MAX, rows_type, rows_ld, row_of_pair, w, T, top_k, cols, y, y_type, y_ld, stream);
}

// The device that a call made now would run on, -1 where there is none; for the Python module, which compares tensors with it.
extern "C" int moe_binding_device(void) {
    int dev = -1;
    return cudaGetDevice(&dev) == cudaSuccess ? dev : -1;
}
