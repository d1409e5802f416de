// mix_api.cu -- C entries of the operators between two expert layers: argument
// checks, then one launcher each (see include/moe.h).
#include "mix.h"

namespace moe {
namespace {

// The batch that a call is given; per = T where it has no list of sequences.
int check_seqs(const moe_seqs* seqs, int64_t T, bool has_state, int64_t slots, const char* name, Seqs& q) {
    if (T < 0 || T > INT32_MAX) return fail_global(MOE_EINVAL, "%s: T=%lld out of range", name, (long long)T);
    if (has_state && (slots < 0 || slots > INT32_MAX))
        return fail_global(MOE_EINVAL, "%s: slots=%lld out of range", name, (long long)slots);
    q = Seqs{nullptr, nullptr, nullptr, 1, (int)T, T, has_state ? slots : INT64_MAX};
    if (seqs) {
        if (seqs->n < 0 || seqs->n > 1 << 20)
            return fail_global(MOE_EINVAL, "%s: n=%d sequences, outside 0..2^20", name, seqs->n);
        if (!seqs->offsets_dev && seqs->n != T)
            return fail_global(MOE_EINVAL, "%s: without offsets every row is a sequence: n=%d, T=%lld", name, seqs->n,
                               (long long)T);
        if (seqs->max_len < 0) return fail_global(MOE_EINVAL, "%s: max_len=%d", name, seqs->max_len);
        q.offsets = seqs->offsets_dev;
        q.slot_of = seqs->slot_dev;
        q.carry_of = seqs->carry_dev;
        q.n = seqs->n;
        if (!q.offsets) q.per = 1;
    }
    if (has_state && !q.slot_of && slots < q.n)
        return fail_global(MOE_EINVAL, "%s: %d sequences, %lld slots", name, q.n, (long long)slots);
    return MOE_OK;
}

bool aligned(const void* p, unsigned n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

bool delta_ok(const moe_delta_config* c) {
    return c && c->k_heads >= 1 && c->v_heads >= c->k_heads && c->v_heads <= 1024 && c->v_heads % c->k_heads == 0 &&
           c->k_dim >= 8 && c->k_dim <= 128 && c->k_dim % 8 == 0 && c->v_dim >= 8 && c->v_dim <= 128 && c->v_dim % 8 == 0;
}
// whether no sequence is long enough for chunks
bool all_short(int64_t T, int32_t max_len) { return T <= kDeltaShort || (max_len >= 1 && max_len <= kDeltaShort); }

int check_heads(const moe_heads& t, const moe_head_norm_config* c, int64_t T, const char* name) {
    if (!type_ok(t.type)) return fail_global(MOE_EINVAL, "moe_head_norm: unknown type %d of %s", t.type, name);
    if (t.heads < 1 || t.heads > 32768) return fail_global(MOE_EINVAL, "moe_head_norm: %d heads of %s", t.heads, name);
    const int64_t ld[] = {t.x_ld, t.y_ld, t.gate_dev ? t.gate_ld : t.x_ld},
                  head[] = {t.x_head, t.y_head, t.gate_dev ? t.gate_head : t.x_head};
    for (int i = 0; i < 3; ++i)
        if (ld[i] < 0 || head[i] < 0)
            return fail_global(MOE_EINVAL, "moe_head_norm: a stride of %s is negative", name);
    if ((t.heads > 1 && t.y_head < c->dim) || (T > 1 && t.y_ld < c->dim))
        return fail_global(MOE_EINVAL, "moe_head_norm: a stride of %s' y is shorter than a head", name);
    if (T > 0 && (!t.x_dev || !t.y_dev)) return fail_global(MOE_EINVAL, "moe_head_norm: x and y of %s are required", name);
    if (t.x_dev == t.y_dev && T > 0 && (t.x_ld != t.y_ld || t.x_head != t.y_head))
        return fail_global(MOE_EINVAL, "moe_head_norm: %s: y is x, but with other strides", name);
    return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_conv(const moe_seqs* seqs, const void* x, int32_t type, int64_t x_ld, int64_t T, int32_t channels,
                        const void* w, int32_t w_type, int32_t width, const float* bias, int32_t act, void* state,
                        int64_t slots, void* y, int64_t y_ld, void* stream) {
    return guarded([&]() -> int {
        Seqs q;
        if (int rc = check_seqs(seqs, T, state != nullptr, slots, "moe_conv", q)) return rc;
        if (!type_ok(type) || !type_ok(w_type)) return fail_global(MOE_EINVAL, "moe_conv: unknown element type");
        if (channels < 1 || channels > 1 << 22)
            return fail_global(MOE_EINVAL, "moe_conv: channels=%d outside 1..2^22", channels);
        if (width < 2 || width > 4) return fail_global(MOE_EINVAL, "moe_conv: width=%d outside 2..4", width);
        if (act != MOE_ACT_NONE && act != MOE_ACT_SILU) return fail_global(MOE_EINVAL, "moe_conv: unknown activation %d", act);
        if (x_ld < channels || y_ld < channels)
            return fail_global(MOE_EINVAL, "moe_conv: a stride is shorter than a row");
        if (T == 0 || q.n == 0) return MOE_OK;
        if (!x || !w || !y) return fail_global(MOE_EINVAL, "moe_conv: x, w and y are required");
        if (x == y) return fail_global(MOE_EINVAL, "moe_conv: y may not be x");
        return launched(launch_conv(q, x, type, x_ld, channels, w, w_type, width, bias, act, state, y, y_ld,
                                    static_cast<cudaStream_t>(stream)),
                        "moe_conv");
    });
}

extern "C" int moe_head_norm(const moe_head_norm_config* c, const moe_heads* a, const moe_heads* b, const int32_t* pos,
                             const float* inv_freq, int64_t T, void* stream) {
    return guarded([&]() -> int {
        if (!c || !a) return fail_global(MOE_EINVAL, "moe_head_norm: cfg and a are required");
        if (c->dim < 1 || c->dim > 512) return fail_global(MOE_EINVAL, "moe_head_norm: dim=%d outside 1..512", c->dim);
        if (c->norm < MOE_NORM_NONE || c->norm > MOE_NORM_L2)
            return fail_global(MOE_EINVAL, "moe_head_norm: unknown norm %d", c->norm);
        if (c->rot_dim < 0 || c->rot_dim > c->dim || c->rot_dim % 2)
            return fail_global(MOE_EINVAL, "moe_head_norm: rot_dim=%d must be even and within 0..dim", c->rot_dim);
        if (c->pairs != MOE_ROT_HALVES && c->pairs != MOE_ROT_ADJACENT)
            return fail_global(MOE_EINVAL, "moe_head_norm: unknown pairs %d", c->pairs);
        if (!(c->eps >= 0)) return fail_global(MOE_EINVAL, "moe_head_norm: eps must be 0 or more");
        if (T < 0 || T > INT32_MAX) return fail_global(MOE_EINVAL, "moe_head_norm: T=%lld out of range", (long long)T);
        if (int rc = check_heads(*a, c, T, "a")) return rc;
        if (b) {
            if (int rc = check_heads(*b, c, T, "b")) return rc;
            if (a->type != b->type) return fail_global(MOE_EINVAL, "moe_head_norm: a and b differ in type");
            if (T > 0 && a->y_dev == b->y_dev) return fail_global(MOE_EINVAL, "moe_head_norm: a and b have the same y");
        }
        if (T * ((int64_t)a->heads + (b ? b->heads : 0)) > INT64_C(1) << 33)
            return fail_global(MOE_EINVAL, "moe_head_norm: more than 2^33 heads in all");
        if (T == 0) return MOE_OK;
        if (c->rot_dim && (!pos || !inv_freq))
            return fail_global(MOE_EINVAL, "moe_head_norm: a rotation needs pos and inv_freq");
        return launched(launch_head_norm(*c, *a, b, pos, inv_freq, T, static_cast<cudaStream_t>(stream)), "moe_head_norm");
    });
}

extern "C" size_t moe_delta_workspace(const moe_delta_config* c, int64_t T, int32_t n, int32_t max_len) {
    if (!delta_ok(c) || T < 0 || T > INT32_MAX || n < 0 || n > 1 << 20 || all_short(T, max_len)) return 0;
    return delta_workspace(*c, T, n);
}

extern "C" int moe_delta(const moe_delta_config* c, const moe_seqs* seqs, const void* q, int64_t q_ld, const void* k,
                         int64_t k_ld, const void* v, int64_t v_ld, const float* g, const float* beta, float* state,
                         int64_t slots, void* o, int64_t o_ld, int64_t T, void* ws, size_t ws_bytes, void* stream) {
    return guarded([&]() -> int {
        if (!delta_ok(c))
            return fail_global(MOE_EINVAL, "moe_delta: heads must be 1..1024, v_heads a multiple of k_heads, k_dim and "
                                           "v_dim multiples of 8 within 8..128");
        DeltaArgs a{};
        if (int rc = check_seqs(seqs, T, state != nullptr, slots, "moe_delta", a.q)) return rc;
        const int64_t kd = (int64_t)c->k_heads * c->k_dim, vd = (int64_t)c->v_heads * c->v_dim;
        if (q_ld < kd || k_ld < kd || v_ld < vd || o_ld < vd)
            return fail_global(MOE_EINVAL, "moe_delta: a stride is shorter than a row");
        if (!aligned(state, 16)) return fail_global(MOE_EINVAL, "moe_delta: state_dev must be 16-byte aligned");
        if (T == 0 || a.q.n == 0) return MOE_OK;
        if (!q || !k || !v || !g || !beta || !o)
            return fail_global(MOE_EINVAL, "moe_delta: q, k, v, g, beta and o are required");
        if ((int64_t)a.q.n * c->v_heads * ((c->v_dim + 31) / 32) > INT32_MAX)
            return fail_global(MOE_EINVAL, "moe_delta: n=%d sequences are too many for %d heads", a.q.n, c->v_heads);
        const int32_t max_len = !seqs ? 0 : seqs->offsets_dev ? seqs->max_len : 1;
        const bool chunks = !all_short(T, max_len);
        const size_t need = chunks ? delta_workspace(*c, T, a.q.n) : 0;
        if (need && (ws_bytes < need || !ws || !aligned(ws, 128)))
            return fail_global(MOE_EINVAL, "moe_delta: needs %zu bytes of 128-byte aligned workspace, got %zu", need,
                               ws_bytes);
        a.c = *c;
        a.qr = static_cast<const __nv_bfloat16*>(q);
        a.kr = static_cast<const __nv_bfloat16*>(k);
        a.vr = static_cast<const __nv_bfloat16*>(v);
        a.q_ld = q_ld, a.k_ld = k_ld, a.v_ld = v_ld, a.o_ld = o_ld;
        a.g = g, a.beta = beta, a.state = state;
        a.o = static_cast<__nv_bfloat16*>(o);
        a.ws = static_cast<uint8_t*>(ws);
        a.q_pieces = a.q.pieces(kDeltaChunk);
        a.wide = (q_ld | k_ld | v_ld) % 8 == 0 && aligned(q, 16) && aligned(k, 16) && aligned(v, 16);
        a.o_pairs = o_ld % 2 == 0 && aligned(o, 4);
        const cudaStream_t st = static_cast<cudaStream_t>(stream);
        a.longer_than = chunks ? kDeltaShort : INT32_MAX;
        // one sequence of all rows is known to be long
        if (!chunks || seqs)
            if (int rc = launched(launch_delta_steps(a, st), "moe_delta")) return rc;
        return chunks ? launched(launch_delta_chunks(a, st), "moe_delta") : MOE_OK;
    });
}
