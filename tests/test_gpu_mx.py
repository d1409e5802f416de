"""The operators without a context on the GPU against plain definitions in 64 bits (_mx_oracle): routing with groups,
pair sort, microscaled 4-bit matrices, their product dense and grouped, combine.

Whole numbers, codes, scale bytes and read-back values have to be equal.  Tolerances of the others, from the arithmetic:
  route weights   exp of a rounded difference (|l - m| < 32: 2^-20 in the argument at most), a sum and a quotient:
                  4e-6 relative
  product         every code product is exact in fp32, one accumulation rounds or truncates an operand at most 2^-21
                  of the running magnitude per 64 columns, and the magnitude is at most S = sum |x w|:
                  (K / 64 + 2) * 2^-21 * S before the rounding of y
  combine         k fused or separate products and sums: (k + 1) * 2^-23 * sum |w row| before the rounding of y
A result y in the output's type then lies between the roundings of (exact - bound) and (exact + bound), rounding being
monotone; no further allowance is made for it.
"""
import numpy as np
import pytest

import _mx_oracle as mxo

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

import int4_expert_streaming_gb300 as moe  # noqa: E402

E8, E4 = moe.MOE_MX_E8M0, moe.MOE_MX_E4M3


@pytest.fixture(scope="module", autouse=True)
def _built():
    moe.build()
    moe.load_library()


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def within(got, ref, bound):
    """Where got (fp32 or bf16) is a rounding of some number within bound of ref (both fp64)."""
    lo, hi = (ref - bound).to(got.dtype).double(), (ref + bound).to(got.dtype).double()
    return (got.double() >= lo) & (got.double() <= hi)


def i32(*shape, fill=-7):
    return torch.full(shape, fill, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------------------
# route
# ---------------------------------------------------------------------------

def separated(logits, bias, G, top_groups, best, k, sigmoid):
    """Rows whose choice hangs on no rounding: the group scores, and the best k + 1 scores of the groups that stay, are
    either equal or further apart than fp32 can blur."""
    l = logits.astype(np.float64)
    s = 1 / (1 + np.exp(-l)) if sigmoid else np.exp(l - l.max(1, keepdims=True))
    if not sigmoid:
        s /= s.sum(1, keepdims=True)
    c = s if bias is None else s + bias
    g = np.sort(c.reshape(len(l), G, -1), 2)[:, :, -best:].sum(2)
    kept = np.zeros(g.shape, bool)
    np.put_along_axis(kept, np.argsort(-g, 1, kind="stable")[:, :top_groups], True, 1)
    inside = np.where(np.repeat(kept, l.shape[1] // G, 1), l if bias is None else c, -np.inf)

    def ok(v):
        v = np.sort(v, 1)
        with np.errstate(invalid="ignore"):
            d = np.diff(v, axis=1)
        return ((d == 0) | (d > 4e-6 * np.abs(v[:, -1:])) | ~np.isfinite(d)).all(1)
    return logits[ok(np.sort(inside, 1)[:, -(k + 1):]) & ok(g)]


def run_route(cfg, logits, bias):
    T = logits.shape[0]
    idx, w = i32(T, cfg.top_k), torch.full((T, cfg.top_k), float("nan"), device="cuda")
    moe.moe_route(cfg, logits, bias, idx, w, torch.cuda.current_stream())
    torch.cuda.synchronize()
    return idx.cpu().numpy(), w.cpu().numpy()


ROUTES = [  # E, k, G, top_groups, best
    (1, 1, 1, 1, 1), (7, 7, 1, 1, 1), (64, 6, 8, 3, 1), (160, 6, 8, 3, 2), (256, 8, 8, 4, 2), (256, 8, 1, 1, 1),
    (512, 10, 1, 1, 1), (1024, 32, 32, 9, 2), (1023, 5, 31, 2, 1), (33, 2, 11, 2, 2), (32, 3, 32, 4, 2)]


@pytest.mark.parametrize("E,k,G,tg,best", ROUTES)
@pytest.mark.parametrize("score", [moe.MOE_SCORE_SOFTMAX, moe.MOE_SCORE_SIGMOID])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_matches_definition(E, k, G, tg, best, score, biased, dtype):
    rng = np.random.default_rng(E * 7 + k + 100 * biased + score)
    sigmoid = score == moe.MOE_SCORE_SIGMOID
    logits = np.round(rng.normal(0, 1.5, (400, E)) * 16) / 16  # exact in bf16; equal logits are common
    bias = (np.round(rng.normal(0, .2, E) * 8) / 8).astype(np.float32) if biased else None
    logits = separated(logits, bias, G, tg, best, k, sigmoid)[:37].astype(np.float32)
    assert len(logits) >= 1
    for renorm, scale in ((True, 2.5), (False, 1.0)):
        cfg = moe.make_route_config(E, k, G, tg, best, score, renorm, scale)
        ld = E + 3
        buf = torch.full((len(logits), ld), float("nan"), dtype=dtype, device="cuda")
        buf[:, :E] = cuda(logits).to(dtype)
        got_i, got_w = run_route(cfg, buf[:, :E], None if bias is None else cuda(bias))
        ref_i, ref_w = mxo.route(logits, bias, k, G, tg, best, sigmoid, renorm, scale)
        assert np.array_equal(got_i, ref_i)
        np.testing.assert_allclose(got_w, ref_w, rtol=4e-6, atol=0)


@pytest.mark.parametrize("score", [moe.MOE_SCORE_SOFTMAX, moe.MOE_SCORE_SIGMOID])
@pytest.mark.parametrize("biased", [False, True])
def test_route_masks_and_extremes(score, biased):
    """Rows with nothing left, with fewer experts than top_k, of the type's lowest value, with NaN, infinities, and
    logits far below zero (weights must not vanish together)."""
    E, k, G, tg, best = 64, 4, 8, 2, 2
    sigmoid = score == moe.MOE_SCORE_SIGMOID
    rows = []
    base = (np.arange(E) * 37 % E).astype(np.float64) / 8
    ninf = np.full(E, -np.inf)
    rows.append(ninf)
    rows.append(np.full(E, np.nan))
    few = ninf.copy(); few[[5, 60]] = [1.0, -2.0]; rows.append(few)
    one = ninf.copy(); one[17] = -500.0; rows.append(one)
    low = np.full(E, np.finfo(np.float32).min); low[3] = 0.0; rows.append(low)
    rows.append(np.full(E, np.finfo(np.float32).min))
    nan = base.copy(); nan[::3] = np.nan; rows.append(nan)
    inf = base.copy(); inf[9] = np.inf; rows.append(inf)
    rows.append(base - 200)
    rows.append(base * 0)
    logits = np.array(rows, np.float32)
    bias = None
    if biased:
        bias = (np.arange(E) % 5 / 4).astype(np.float32)
        bias[7] = -np.inf
        bias[8] = np.nan
    cfg = moe.make_route_config(E, k, G, tg, best, score, True, 1.0)
    got_i, got_w = run_route(cfg, cuda(logits), None if bias is None else cuda(bias))
    ref_i, ref_w = mxo.route(logits, bias, k, G, tg, best, sigmoid, True, 1.0)
    assert np.array_equal(got_i, ref_i)
    np.testing.assert_allclose(got_w, ref_w, rtol=4e-6, atol=1e-37)
    assert (got_i[0] == -1).all() and (got_w[0] == 0).all()
    live = got_i[:, 0] >= 0
    np.testing.assert_allclose(got_w[live].sum(1), 1, rtol=1e-6)


@pytest.mark.parametrize("E,k", [(512, 10), (1024, 32), (100, 3)])
def test_route_of_many_tokens_is_the_route_of_each(E, k):
    torch.manual_seed(0)
    logits = torch.randn(5003, E, device="cuda")
    cfg = moe.make_route_config(E, k)
    all_i, all_w = run_route(cfg, logits, None)
    for t in (0, 1, 4999, 5002):
        i, w = run_route(cfg, logits[t:t + 1], None)
        assert np.array_equal(i[0], all_i[t]) and np.array_equal(w[0], all_w[t])
    again = run_route(cfg, logits, None)
    assert np.array_equal(again[0], all_i) and np.array_equal(again[1], all_w)


# ---------------------------------------------------------------------------
# dispatch and combine
# ---------------------------------------------------------------------------

def run_dispatch(idx, E, stream=None):
    T, k = idx.shape
    off, rop, tor, gor = i32(E + 1), i32(T, k), i32(T * k), i32(T * k)
    ws = torch.full((max(1, moe.moe_dispatch_workspace(T, k, E)),), 0xAB, dtype=torch.uint8, device="cuda")
    moe.moe_dispatch(cuda(idx), E, off, rop, tor, gor, ws, stream)
    torch.cuda.synchronize()
    return [v.cpu().numpy() for v in (off, rop, tor, gor)]


@pytest.mark.parametrize("T,k,E", [(0, 4, 16), (1, 1, 1), (1, 10, 512), (3, 5, 1024), (64, 8, 256), (257, 7, 33),
                                   (1000, 10, 512), (4096, 10, 512), (20011, 8, 1024), (100003, 2, 3)])
@pytest.mark.parametrize("kind", ["spread", "one", "dropped", "none"])
def test_dispatch_matches_definition(T, k, E, kind):
    rng = np.random.default_rng(T + E)
    idx = rng.integers(0, E, (T, k)).astype(np.int32)
    if kind == "one":
        idx[:] = E - 1
    elif kind == "dropped":
        idx[rng.random((T, k)) < 0.4] = -1
        idx[rng.random((T, k)) < 0.1] = E  # any id out of range is dropped
    elif kind == "none":
        idx[:] = -1
    for got, ref in zip(run_dispatch(idx, E), mxo.dispatch(idx, E)):
        assert np.array_equal(got, ref)


@pytest.mark.parametrize("T,k,cols", [(1, 1, 1), (1, 10, 2048), (5, 3, 77), (300, 10, 512), (17, 8, 2051), (64, 32, 96)])
@pytest.mark.parametrize("tin", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tout", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pad", [0, 5, 8])
def test_combine_matches_definition(T, k, cols, tin, tout, pad):
    rng = np.random.default_rng(T * cols + k)
    n = T * k + 3
    rows = torch.full((n, cols + pad), float("nan"), dtype=tin, device="cuda")
    rows[:, :cols] = cuda(rng.normal(0, 1, (n, cols)).astype(np.float32)).to(tin)
    row = rng.permutation(n)[:T * k].reshape(T, k).astype(np.int32)
    row[rng.random((T, k)) < 0.2] = -1
    row[T // 2] = -1  # a token without pairs
    w = rng.random((T, k)).astype(np.float32)
    y = torch.full((T, cols + pad), 3.0, dtype=tout, device="cuda")
    moe.moe_combine(rows[:, :cols], cuda(row), cuda(w), y[:, :cols], torch.cuda.current_stream())
    torch.cuda.synchronize()
    r = rows[:, :cols].double().cpu().numpy()
    terms = np.where((row >= 0)[..., None], w.astype(np.float64)[..., None] * r[np.maximum(row, 0)], 0)
    ref = terms.sum(1)
    lim = (k + 1) * 2.0 ** -23 * np.abs(terms).sum(1)
    assert within(y[:, :cols].cpu(), torch.from_numpy(ref), torch.from_numpy(lim)).all()
    assert (y[:, cols:] == 3.0).all()  # nothing past a row's end


# ---------------------------------------------------------------------------
# quantise and dequantise
# ---------------------------------------------------------------------------

def special(rng, rows, cols, fmt):
    """Values over many binades with exact ties, zero blocks, subnormals, and a few NaN and infinities."""
    x = rng.normal(0, 1, (rows, cols)) * np.exp2(rng.integers(-20, 8, (rows, 1)))
    x = np.where(rng.random(x.shape) < 0.3, np.round(x * 8) / 8, x)
    x[rng.random(rows) < 0.1] = 0
    if rows > 2:
        x[1, :min(16, cols)] = 0
        x[2] *= 1e-38
    x = x.astype(np.float32)
    if rows > 6:
        x[4, cols // 2] = np.nan
        x[5, 0] = np.inf
        x[6, cols - 1] = -np.inf
    return x


def bf16_of(x):
    return torch.from_numpy(x).to(torch.bfloat16).float().numpy()


@pytest.mark.parametrize("fmt", [E8, E4])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 16), (3, 31), (7, 256), (130, 257), (9, 2048), (300, 100)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pad", [0, 3, 8])
def test_quantise_bytes_match_definition(fmt, rows, cols, dtype, pad):
    rng = np.random.default_rng(rows * 31 + cols + fmt)
    x = special(rng, rows, cols, fmt)
    if dtype is torch.bfloat16:
        x = bf16_of(x)
    src = torch.full((rows, cols + pad), float("nan"), dtype=dtype, device="cuda")
    src[:, :cols] = cuda(x).to(dtype)
    m = moe.make_mx(fmt, rows, cols)
    m._data.fill_(0xEE)
    t = cuda(np.array([0.37 / 3], np.float32)) if fmt == E4 and pad else None
    moe.moe_mx_quantise(m, src[:, :cols], tensor_scale=t, stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    rt, ir = mxo.uniform_place(1, rows)
    code, byte = mxo.read_tiles(m._data.cpu().numpy(), rt, ir, cols, fmt)
    tt = None if t is None else np.full(rows, t.item(), np.float32)
    rcode, rbyte = mxo.quantise(x, fmt, tt)
    assert np.array_equal(byte, rbyte)
    # the sign of a zero code may differ: -0 and 0 are the same value
    zero = (code & 7 == 0) & (rcode & 7 == 0)
    assert np.array_equal(np.where(zero, 0, code), np.where(zero, 0, rcode))
    # rows past the last are not written
    raw = m._data.cpu().numpy().reshape(-1, mxo.tile_bytes(fmt))
    if rows % 128:
        assert (raw[-1, (rows % 128) * 128:16384] == 0xEE).all()
    # and back
    for dt in (torch.float32, torch.bfloat16):
        out = torch.full((rows, cols + pad), 5.0, dtype=dt, device="cuda")
        moe.moe_mx_dequantise(m, out[:, :cols], tensor_scale=t)
        ref = torch.from_numpy(mxo.values(code, byte, fmt)[:, :cols]).float()
        if t is not None:
            ref = ref * t.cpu()
        assert torch.equal(torch.nan_to_num(out[:, :cols].cpu(), 9e9), torch.nan_to_num(ref.to(dt), 9e9))
        assert (out[:, cols:] == 5.0).all()


@pytest.mark.parametrize("fmt", [E8, E4])
def test_quantise_ragged_gather_with_left_out_rows(fmt):
    rng = np.random.default_rng(8)
    E, cols, tokens = 9, 300, 50
    n = np.array([0, 1, 128, 0, 129, 3, 260, 0, 5])
    offsets = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    group = np.repeat(np.arange(E), n).astype(np.int32)
    R = len(group)
    src_row = rng.integers(0, tokens, R).astype(np.int32)
    rows_alloc = R + 4
    group_p = np.concatenate([group, [-1] * 4]).astype(np.int32)
    src_p = np.concatenate([src_row, [-1] * 4]).astype(np.int32)
    src_p[7] = -1
    x = rng.normal(0, 1, (tokens, cols)).astype(np.float32)
    t = rng.uniform(0.5, 2, E).astype(np.float32) if fmt == E4 else None
    m = moe.make_mx(fmt, rows_alloc, cols, groups=E, ragged=True)
    m._data.fill_(0xEE)
    moe.moe_mx_quantise(m, cuda(x), src_row=cuda(src_p), group_of_row=cuda(group_p), offsets=cuda(offsets),
                        tensor_scale=None if t is None else cuda(t))
    rt, ir = mxo.ragged_place(offsets, group)
    code, byte = mxo.read_tiles(m._data.cpu().numpy(), rt, ir, cols, fmt)
    rcode, rbyte = mxo.quantise(x[src_row], fmt, None if t is None else t[group])
    there = np.arange(R) != 7
    zero = (code & 7 == 0) & (rcode & 7 == 0)
    assert np.array_equal(byte[there], rbyte[there])
    assert np.array_equal(np.where(zero, 0, code)[there], np.where(zero, 0, rcode)[there])
    assert (code[7] == 0xE).all()
    out = torch.full((rows_alloc, cols), 5.0, device="cuda")
    moe.moe_mx_dequantise(m, out, group_of_row=cuda(group_p), offsets=cuda(offsets))
    assert np.array_equal(out.cpu().numpy()[:R][there], mxo.values(code[there], byte[there], fmt)[:, :cols].astype(np.float32))
    assert (out[R:] == 5.0).all()


@pytest.mark.parametrize("fmt", [E8, E4])
@pytest.mark.parametrize("cols", [512, 33])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_swiglu_then_quantise(fmt, cols, dtype):
    """The activation is fp32 with an exp that is not exact, so a value next to a boundary may fall on either side:
    each value is within its block's rounding step of the definition's activation, and nearly all are the same."""
    rng = np.random.default_rng(cols)
    src = cuda(rng.normal(0, 2, (70, 2 * cols)).astype(np.float32)).to(dtype)
    m = moe.make_mx(fmt, 70, cols)
    moe.moe_mx_quantise(m, src, act=moe.MOE_ACT_SWIGLU)
    out = torch.empty((70, cols), device="cuda")
    moe.moe_mx_dequantise(m, out)
    s = src.double().cpu().numpy()
    x = s[:, :cols] / (1 + np.exp(-s[:, :cols])) * s[:, cols:]
    code, byte = mxo.quantise(x.astype(np.float32), fmt)
    ref = mxo.values(code, byte, fmt)[:, :cols]
    got = out.double().cpu().numpy()
    assert (got != ref).mean() < 1e-3
    C, B = -(-cols // 256) * 256, mxo.BLOCK[fmt]
    a = np.zeros((70, C))
    a[:, :cols] = np.abs(x)
    a = np.repeat(a.reshape(70, -1, B).max(2), B, 1)[:, :cols]
    assert (np.abs(got - x) <= a * (0.26 if fmt == E8 else 0.2) + 2.0 ** -8).all()


# ---------------------------------------------------------------------------
# product
# ---------------------------------------------------------------------------

def random_matrix(rng, rows, cols, fmt, spread=3):
    """Codes and scale bytes of rows x cols, zero past cols; scales over a few binades around 1."""
    C, B = -(-cols // 256) * 256, mxo.BLOCK[fmt]
    code = rng.integers(0, 16, (rows, C)).astype(np.uint8)
    code[:, cols:] = 0
    lo, hi = (127 - spread, 127 + spread) if fmt == E8 else (56 - 8 * spread, 56 + 8 * spread)
    byte = rng.integers(lo, hi, (rows, C // B)).astype(np.uint8)
    byte[:, -(-cols // B):] = 0
    return code, byte


def check_product(fmt, n, N, K, ydt, seed=0, alpha=False, pad=0, extra_rows=0, stream=None, spread=3):
    """Grouped product with the group sizes n (an int: dense) against the definition, byte images written by the
    oracle: everything outside the matrices' own rows holds NaN scales."""
    rng = np.random.default_rng(seed)
    dense = isinstance(n, int)
    sizes = np.array([n] if dense else n)
    E, R = len(sizes), int(sizes.sum())
    offsets = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    group = np.repeat(np.arange(E), sizes)
    xc, xb = random_matrix(rng, R, K, fmt, spread)
    wc, wb = random_matrix(rng, E * N, K, fmt, spread)
    kw = dict(data=None)
    rows = R + extra_rows
    if dense:
        place, tiles = mxo.uniform_place(1, R), -(-rows // 128)
    else:
        place, tiles = mxo.ragged_place(offsets, group), rows // 128 + E
    x = moe.make_mx(fmt, rows, K, groups=E, ragged=not dense,
                    data=cuda(mxo.write_tiles(xc, xb, *place, tiles, fmt)))
    w = moe.make_mx(fmt, N, K, groups=E,
                    data=cuda(mxo.write_tiles(wc, wb, *mxo.uniform_place(E, N), E * -(-N // 128), fmt)))
    a = rng.uniform(0.5, 2, E).astype(np.float32) if alpha else None
    y = torch.full((rows, N + pad), 77.0, dtype=ydt, device="cuda")
    moe.moe_mx_product(x, w, y[:, :N], offsets=None if dense else cuda(offsets), alpha=None if a is None else cuda(a),
                       stream=stream)
    torch.cuda.synchronize()
    xv = torch.from_numpy(mxo.values(xc, xb, fmt)).cuda()
    wv = torch.from_numpy(mxo.values(wc, wb, fmt)).cuda().view(E, N, -1)
    ref = torch.zeros((R, N), dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(ref)
    for e in range(E):
        s = slice(offsets[e], offsets[e + 1])
        ref[s] = xv[s] @ wv[e].T
        mag[s] = xv[s].abs() @ wv[e].abs().T
        if a is not None:
            ref[s] *= float(a[e])
            mag[s] *= float(a[e])
    got = y[:R, :N]
    bad = ~within(got, ref, (K / 64 + 2) * 2.0 ** -21 * mag)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:5].tolist(), got[bad][:5].tolist(), ref[bad][:5].tolist())
    assert (y[:R, N:] == 77.0).all() and (y[R:] == 77.0).all()
    return y


@pytest.mark.parametrize("fmt", [E8, E4])
@pytest.mark.parametrize("R,N,K", [(1, 1, 1), (1, 128, 256), (1, 1024, 2048), (2, 129, 300), (17, 64, 64), (16, 256, 512),
                                   (33, 100, 31), (127, 130, 1000), (128, 128, 256), (129, 384, 257), (200, 200, 4096),
                                   (257, 513, 768), (300, 1000, 513)])
@pytest.mark.parametrize("ydt", [torch.float32, torch.bfloat16])
def test_dense_product_matches_definition(fmt, R, N, K, ydt):
    check_product(fmt, R, N, K, ydt, seed=R + N + K, alpha=True)


@pytest.mark.parametrize("fmt", [E8, E4])
@pytest.mark.parametrize("R,N,K", [(1300, 4000, 1100), (2049, 8192 - 3, 1024), (700, 12000, 1024), (769, 3000, 2048)])
def test_large_dense_product_matches_definition(fmt, R, N, K):
    """Enough tiles for pairs of CTAs, an odd last feature tile, row tiles of every remainder."""
    check_product(fmt, R, N, K, torch.bfloat16, alpha=True)


@pytest.mark.parametrize("fmt", [E8, E4])
@pytest.mark.parametrize("sizes,N,K", [(1, 1024, 8192), (1, 300, 4096), (7, 4096, 4100), (33, 1000, 6400), (128, 1024, 8192),
                                       (200, 130, 6300), (300, 1024, 6144 + 255), ([1, 0, 3], 500, 8000), ([40, 90], 127, 7000)])
@pytest.mark.parametrize("ydt", [torch.float32, torch.bfloat16])
def test_long_rows_split_over_a_cluster(fmt, sizes, N, K, ydt):
    """Few tiles and many steps: clusters of 2, 4 and 8 CTAs share a tile, with steps that do not divide evenly."""
    check_product(fmt, sizes, N, K, ydt, alpha=True, pad=3)


@pytest.mark.parametrize("fmt", [E8, E4])
@pytest.mark.parametrize("sizes", [[400, 0, 1, 255, 256, 257, 129, 128, 127, 700, 33, 16, 0, 512], [300] * 9])
@pytest.mark.parametrize("ydt", [torch.float32, torch.bfloat16])
def test_large_groups_match_definition(fmt, sizes, ydt):
    check_product(fmt, sizes, 1500, 1024, ydt, alpha=True, extra_rows=3)


@pytest.mark.parametrize("fmt", [E8, E4])
@pytest.mark.parametrize("pad", [1, 4, 8])
def test_product_into_strided_rows(fmt, pad):
    check_product(fmt, 70, 200, 320, torch.bfloat16, pad=pad)
    check_product(fmt, 70, 200, 320, torch.float32, pad=pad)


@pytest.mark.parametrize("fmt", [E8, E4])
@pytest.mark.parametrize("sizes", [[1], [0, 0, 5, 0], [1] * 30, [0, 1, 127, 128, 129, 0, 255, 256, 257, 2],
                                   [300, 0, 0, 1, 16, 15, 17, 500], [0] * 511 + [3], [0, 0]])
@pytest.mark.parametrize("N,K", [(128, 256), (200, 520)])
def test_grouped_product_matches_definition(fmt, sizes, N, K):
    check_product(fmt, sizes, N, K, torch.bfloat16, seed=len(sizes), alpha=True)
    check_product(fmt, sizes, N, K, torch.float32, seed=len(sizes), extra_rows=9)


@pytest.mark.parametrize("fmt", [E8, E4])
def test_decode_batches_of_a_large_expert_set(fmt):
    """A few rows over 256 experts: rows a group 0 to 3, wide and deep matrices."""
    sizes = np.zeros(256, int)
    sizes[np.random.default_rng(5).integers(0, 256, 40)] += 1
    sizes[200] = 3
    check_product(fmt, list(sizes), 256, 2048, torch.bfloat16, alpha=True)


@pytest.mark.parametrize("fmt", [E8, E4])
def test_scales_over_the_whole_range_of_the_format(fmt):
    """Scale bytes from the smallest to the largest: each result is still the exact sum's rounding within the bound."""
    check_product(fmt, 40, 130, 512, torch.float32, spread=30 if fmt == E8 else 6)


@pytest.mark.parametrize("fmt", [E8, E4])
def test_a_nan_scale_reaches_its_row_or_column_and_no_other(fmt):
    rng = np.random.default_rng(2)
    R, N, K = 40, 140, 512
    xc, xb = random_matrix(rng, R, K, fmt)
    wc, wb = random_matrix(rng, N, K, fmt)
    nan = 255 if fmt == E8 else 127
    xb[7, 3] = nan
    wb[131, 0] = nan
    x = moe.make_mx(fmt, R, K, data=cuda(mxo.write_tiles(xc, xb, *mxo.uniform_place(1, R), 1, fmt)))
    w = moe.make_mx(fmt, N, K, data=cuda(mxo.write_tiles(wc, wb, *mxo.uniform_place(1, N), 2, fmt)))
    y = torch.empty((R, N), device="cuda")
    moe.moe_mx_product(x, w, y)
    nans = torch.isnan(y).cpu().numpy()
    want = np.zeros((R, N), bool)
    want[7], want[:, 131] = True, True
    assert np.array_equal(nans, want)


def test_product_is_the_same_every_time_and_on_another_stream():
    a = check_product(E4, [0, 5, 40, 1], 300, 2048, torch.float32, seed=3)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = check_product(E4, [0, 5, 40, 1], 300, 2048, torch.float32, seed=3, stream=s)
    assert torch.equal(a, b)
    for _ in range(3):
        assert torch.equal(a, check_product(E4, [0, 5, 40, 1], 300, 2048, torch.float32, seed=3))


def test_matrices_past_32_bits():
    """A weight set of 5 GB: the first and the last group's rows come back and multiply as any other's."""
    G, N, K, fmt = 513, 2048, 8448, E8
    torch.manual_seed(1)
    src = torch.randn(64, K, device="cuda").to(torch.bfloat16)
    row = (torch.arange(G * N, device="cuda", dtype=torch.int32) * 5) % 64
    w = moe.make_mx(fmt, N, K, groups=G)
    assert w._data.numel() > 1 << 32
    moe.moe_mx_quantise(w, src, src_row=row)
    small = moe.make_mx(fmt, 64, K)
    moe.moe_mx_quantise(small, src)
    ref = torch.empty((64, K), dtype=torch.bfloat16, device="cuda")
    moe.moe_mx_dequantise(small, ref)
    back = torch.empty((G * N, K), dtype=torch.bfloat16, device="cuda")  # 17 GB
    moe.moe_mx_dequantise(w, back)
    for r0 in (0, 12345, G * N // 2, G * N - 64):
        assert torch.equal(back[r0:r0 + 64], ref[row[r0:r0 + 64].long()])
    del back
    offsets = torch.full((G + 1,), 3, dtype=torch.int32, device="cuda")
    offsets[0], offsets[-1] = 0, 8
    group = torch.tensor([0] * 3 + [G - 1] * 5, dtype=torch.int32, device="cuda")
    x = moe.make_mx(fmt, 8, K, groups=G, ragged=True)
    moe.moe_mx_quantise(x, src[:8], group_of_row=group, offsets=offsets)
    y = torch.empty((8, N), device="cuda")
    moe.moe_mx_product(x, w, y, offsets=offsets)
    v = ref.double()
    for r, g in enumerate(group.tolist()):
        wr = v[row[g * N:(g + 1) * N].long()]
        want, mag = wr @ v[r], wr.abs() @ v[r].abs()
        assert within(y[r], want, (K / 64 + 2) * 2.0 ** -21 * mag).all()


def test_calls_can_be_captured_in_a_graph():
    rng = np.random.default_rng(0)
    R, N, K = 5, 256, 512
    src = cuda(rng.normal(0, 1, (R, K)).astype(np.float32))
    w = moe.make_mx(E4, N, K)
    moe.moe_mx_quantise(w, cuda(rng.normal(0, 1, (N, K)).astype(np.float32)))
    x = moe.make_mx(E4, R, K)
    y = torch.zeros((R, N), device="cuda")
    moe.moe_mx_quantise(x, src)
    moe.moe_mx_product(x, w, y)
    want = y.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_mx_quantise(x, src, stream=torch.cuda.current_stream())
        moe.moe_mx_product(x, w, y, stream=torch.cuda.current_stream())
    src *= 2
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want * 2)
