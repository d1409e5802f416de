"""The operators without a context, as far as they go without a GPU: shapes and sizes, refusals (nothing is launched for
a bad argument), and the plain definitions' own properties."""
import ctypes

import numpy as np
import pytest

import _mx_oracle as mxo
import int4_expert_streaming_gb300 as moe


@pytest.fixture(scope="module")
def lib():
    moe.build()
    return moe.load_library()


P = 1 << 20  # an address that is never read: every call here is refused before any GPU work


def refused(rc, word):
    assert rc == moe.MOE_EINVAL
    assert word in moe.moe_last_error(None), moe.moe_last_error(None)


@pytest.mark.parametrize("fmt,tile", [(moe.MOE_MX_E8M0, 17408), (moe.MOE_MX_E4M3, 18432)])
def test_matrix_bytes(lib, fmt, tile):
    m = moe.moe_mx
    assert moe.moe_mx_bytes(m(None, 1, 1, 1, fmt, 0)) == tile
    assert moe.moe_mx_bytes(m(None, 129, 257, 3, fmt, 0)) == 3 * 2 * 2 * tile
    assert moe.moe_mx_bytes(m(None, 129, 257, 3, fmt, 1)) == (1 + 3) * 2 * tile
    assert moe.moe_mx_bytes(m(None, 0, 256, 4, fmt, 0)) == 0
    assert moe.moe_mx_bytes(m(None, 1 << 20, 8192, 1024, fmt, 0)) == 1024 * 8192 * 32 * tile  # past 32 bits
    for bad in (m(None, -1, 1, 1, fmt, 0), m(None, 1, 0, 1, fmt, 0), m(None, 1, 1, 0, fmt, 0), m(None, 1, 1, 1025, fmt, 0),
                m(None, 1, 1, 1, 2, 0), m(None, 1, 1, 1, fmt, 2)):
        assert moe.moe_mx_bytes(bad) == 0
    assert lib.moe_mx_bytes(None) == 0


@pytest.mark.parametrize("field,value,word", [
    ("n_experts", 0, "n_experts"), ("n_experts", 1025, "n_experts"), ("n_groups", 3, "n_groups"),
    ("n_groups", 64, "n_groups"), ("top_groups", 0, "top_groups"), ("top_groups", 9, "top_groups"), ("top_k", 0, "top_k"),
    ("top_k", 33, "top_k"), ("group_best", 3, "group_best"), ("score", 2, "score")])
def test_route_refuses_bad_config(lib, field, value, word):
    cfg = moe.make_route_config(256, 8, n_groups=8, top_groups=4)
    setattr(cfg, field, value)
    refused(lib.moe_route(cfg, P, moe.MOE_F32, 1024, None, 4, P, P, None), word)


def test_route_refuses_bad_arguments(lib):
    cfg = moe.make_route_config(64, 8, n_groups=8, top_groups=1)
    refused(lib.moe_route(None, P, 0, 64, None, 4, P, P, None), "cfg")
    refused(lib.moe_route(cfg, P, 2, 64, None, 4, P, P, None), "type")
    refused(lib.moe_route(cfg, P, 0, 63, None, 4, P, P, None), "ld")
    refused(lib.moe_route(cfg, P, 0, 64, None, -1, P, P, None), "T=")
    refused(lib.moe_route(cfg, None, 0, 64, None, 4, P, P, None), "required")
    refused(lib.moe_route(cfg, P, 0, 64, None, 4, None, P, None), "required")
    cfg.top_k = 9  # one group of eight stays
    refused(lib.moe_route(cfg, P, 0, 64, None, 4, P, P, None), "top_k")
    assert lib.moe_route(moe.make_route_config(64, 8), None, 0, 64, None, 0, None, None, None) == moe.MOE_OK  # no tokens


def test_dispatch_refuses_bad_arguments(lib):
    def call(T=4, k=2, E=8, idx=P, off=P, rop=P, tor=P, gor=P, ws=P, size=1 << 40):
        return lib.moe_dispatch(idx, T, k, E, off, rop, tor, gor, ws, size, None)
    refused(call(T=-1), "range")
    refused(call(k=0), "range")
    refused(call(E=1025), "range")
    refused(call(T=1 << 30, k=2), "range")
    refused(call(off=None), "offsets")
    refused(call(rop=None), "required")
    assert moe.moe_dispatch_workspace(-1, 2, 8) == 0
    need = moe.moe_dispatch_workspace(1 << 16, 10, 512)
    if need:
        refused(call(T=1 << 16, k=10, E=512, size=need - 1), "workspace")
        refused(call(T=1 << 16, k=10, E=512, ws=P + 8), "workspace")


def test_matrix_calls_refuse_bad_arguments(lib):
    E8, E4 = moe.MOE_MX_E8M0, moe.MOE_MX_E4M3
    m = moe.moe_mx(P, 4, 64, 1, E8, 0)
    r = moe.moe_mx(P, 4, 64, 2, E8, 1)

    def q(m=m, src=P, kind=0, ld=64, act=0, src_row=None, gor=None, off=None, ts=None):
        return lib.moe_mx_quantise(m, src, kind, ld, act, src_row, gor, off, ts, None)
    refused(q(m=moe.moe_mx(P, 4, 0, 1, E8, 0)), "descriptor")
    refused(q(m=moe.moe_mx(P + 64, 4, 64, 1, E8, 0)), "aligned")
    refused(q(m=moe.moe_mx(None, 4, 64, 1, E8, 0)), "aligned")
    refused(q(kind=7), "type")
    refused(q(act=2), "activation")
    refused(q(ld=63), "src_ld")
    refused(q(act=1, ld=127), "src_ld")
    refused(q(ts=P), "E4M3")
    refused(q(gor=P, off=P), "ragged")
    refused(q(m=r, gor=P), "ragged")
    refused(q(src=None), "src")
    assert q(m=moe.moe_mx(None, 0, 64, 1, E8, 0), src=None) == moe.MOE_OK  # no rows

    def d(m=m, gor=None, off=None, dst=P, kind=0, ld=64):
        return lib.moe_mx_dequantise(m, gor, off, None, dst, kind, ld, None)
    refused(d(ld=63), "dst_ld")
    refused(d(kind=2), "type")
    refused(d(dst=None), "dst")
    refused(d(m=r, off=P), "ragged")

    w = moe.moe_mx(P, 32, 64, 1, E8, 0)

    def p(x=m, w=w, off=None, y=P, kind=0, ld=32):
        return lib.moe_mx_product(x, w, off, None, y, kind, ld, None)
    refused(p(w=moe.moe_mx(P, 32, 64, 1, E8, 1)), "uniform")
    refused(p(w=moe.moe_mx(P, 32, 64, 1, E4, 0)), "format")
    refused(p(w=moe.moe_mx(P, 32, 65, 1, E8, 0)), "cols")
    refused(p(x=r), "groups")
    refused(p(x=moe.moe_mx(P, 4, 64, 2, E8, 0), w=moe.moe_mx(P, 32, 64, 2, E8, 0)), "ragged")
    refused(p(off=P), "offsets")
    refused(p(x=r, w=moe.moe_mx(P, 32, 64, 2, E8, 0)), "offsets")
    refused(p(kind=3), "type")
    refused(p(ld=31), "y_ld")
    refused(p(y=None), "y is")
    assert p(x=moe.moe_mx(None, 0, 64, 1, E8, 0), y=None) == moe.MOE_OK

    def c(T=2, k=2, cols=8, kind=0, ld=8, yk=0, yld=8, rows=P):
        return lib.moe_combine(rows, kind, ld, P, P, T, k, cols, P, yk, yld, None)
    refused(c(T=-1), "range")
    refused(c(k=0), "range")
    refused(c(cols=0), "range")
    refused(c(kind=2), "type")
    refused(c(yk=-1), "type")
    refused(c(ld=7), "stride")
    refused(c(yld=7), "stride")
    refused(c(rows=None), "required")
    assert c(T=0, rows=None) == moe.MOE_OK


def test_binding_refuses_host_and_wrong_tensors(lib):
    torch = pytest.importorskip("torch")
    cfg = moe.make_route_config(16, 2)
    l, i, w = torch.zeros(3, 16), torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2)
    with pytest.raises(ValueError):
        moe.moe_route(cfg, l, None, i, w)
    with pytest.raises(ValueError):
        moe.make_mx(moe.MOE_MX_E8M0, 4, 64, data=torch.zeros(17408, dtype=torch.uint8))
    with pytest.raises(ValueError):
        moe.make_mx(5, 4, 64, data=torch.zeros(17408, dtype=torch.uint8))
    with pytest.raises(ValueError):
        moe.moe_combine(l, i, w, torch.zeros(3, 16))


# ---- the plain definitions themselves -------------------------------------

def test_nearest_even_on_both_tables():
    assert list(mxo.nearest_even(mxo.E2M1, [0, .25, .26, .75, 1.25, 1.75, 2.5, 3.5, 5, 5.1, 6, 99])) == \
        [0, 0, 1, 2, 2, 4, 4, 6, 6, 7, 7, 7]
    assert mxo.E4M3[126] == 448 and mxo.E4M3[8] == 2.0 ** -6 and mxo.E4M3[1] == 2.0 ** -9
    mid = (mxo.E4M3[:-1] + mxo.E4M3[1:]) / 2
    assert all(i % 2 == 0 for i in mxo.nearest_even(mxo.E4M3, mid))


@pytest.mark.parametrize("fmt", [0, 1])
def test_quantising_a_representable_matrix_is_exact(fmt):
    """Values code * scale whose block holds a code of 6 (E4M3) or 4 (E8M0) come back unchanged."""
    rng = np.random.default_rng(fmt)
    B = mxo.BLOCK[fmt]
    code = rng.integers(0, 16, (5, 512)).astype(np.uint8)
    code[:, ::B] = 7 if fmt else 6
    byte = (rng.integers(100, 150, (5, 512 // B)) if fmt == 0 else rng.integers(8, 126, (5, 512 // B))).astype(np.uint8)
    x = mxo.values(code, byte, fmt)
    if fmt == 0:
        code[code & 7 == 7] -= 1  # 6 and 4 share a binade: both keep the scale
        x = mxo.values(code, byte, fmt)
    c2, b2 = mxo.quantise(x.astype(np.float32), fmt)
    assert np.array_equal(mxo.values(c2, b2, fmt), x) and np.array_equal(b2, byte)


@pytest.mark.parametrize("fmt", [0, 1])
def test_tiles_round_trip_in_the_plain_definition(fmt):
    rng = np.random.default_rng(3)
    offsets, group = np.array([0, 3, 3, 140, 141]), np.array([0] * 3 + [2] * 137 + [3])
    rt, ir = mxo.ragged_place(offsets, group)
    assert len(set(zip(rt, ir))) == 141 and rt.max() < 141 // 128 + 4
    code = rng.integers(0, 16, (141, 512)).astype(np.uint8)
    byte = rng.integers(0, 255, (141, 512 // mxo.BLOCK[fmt])).astype(np.uint8)
    raw = mxo.write_tiles(code, byte, rt, ir, 141 // 128 + 4, fmt)
    c2, b2 = mxo.read_tiles(raw, rt, ir, 512, fmt)
    assert np.array_equal(c2, code) and np.array_equal(b2, byte)


def test_ragged_groups_never_share_a_row_tile():
    rng = np.random.default_rng(0)
    for _ in range(200):
        n = rng.choice([0, 1, 127, 128, 129, 255, 256, 300], rng.integers(1, 12))
        off = np.concatenate([[0], np.cumsum(n)])
        for g in range(len(n)):
            last = off[g] // 128 + g + -(-n[g] // 128)
            assert last <= (off[g + 1] // 128 + g + 1 if g + 1 < len(n) else off[-1] // 128 + len(n))


def test_config_struct_matches_the_header():
    assert ctypes.sizeof(moe.moe_route_config) == 32 and ctypes.sizeof(moe.moe_mx) == 32
