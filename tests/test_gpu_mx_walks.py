"""The operators without a context at sizes where their kernels go round: many tiles a CTA, many sets of rows a block, more
than a million pairs; and in the parts of the formats, and the combinations of arguments, that the small cases leave out.

Reference and tolerances as in test_gpu_mx (products: the bound of their accumulation; bytes: equal)."""
import threading

import numpy as np
import pytest

import _mx_oracle as mxo

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

import int4_expert_streaming_gb300 as moe  # noqa: E402
from test_gpu_mx import E4, E8, check_product, cuda, run_dispatch, within  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    moe.build()
    moe.load_library()


# ---------------------------------------------------------------------------
# product: about 20 tiles a CTA (152 CTAs, 76 pairs)
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", [E8, E4])
@pytest.mark.parametrize("K", [200, 700])
@pytest.mark.parametrize("ydt", [torch.float32, torch.bfloat16])
def test_many_tiles_of_few_rows(fmt, K, ydt):
    check_product(fmt, [1, 0, 2, 1] * 15, 8200, K, ydt, alpha=True)  # 45 row tiles x 65


@pytest.mark.parametrize("fmt", [E8, E4])
@pytest.mark.parametrize("K", [256, 768])
@pytest.mark.parametrize("ydt", [torch.float32, torch.bfloat16])
def test_many_tiles_of_one_cta(fmt, K, ydt):
    check_product(fmt, [60, 1, 128, 0, 129, 33] * 50, 1400, K, ydt, alpha=True, extra_rows=5)  # 300 row tiles x 11


@pytest.mark.parametrize("fmt", [E8, E4])
@pytest.mark.parametrize("ydt", [torch.float32, torch.bfloat16])
def test_many_tiles_of_a_pair(fmt, ydt):
    check_product(fmt, [300, 256, 90, 0, 257, 1, 128, 129] * 10, 4000, 1024, ydt, alpha=True)  # 100 row tiles x 16


# ---------------------------------------------------------------------------
# product: scales of the whole range
# ---------------------------------------------------------------------------

def product_of(xc, xb, wc, wb, fmt):
    (R, C), N = xc.shape, wc.shape[0]
    x = moe.make_mx(fmt, R, C, data=cuda(mxo.write_tiles(xc, xb, *mxo.uniform_place(1, R), -(-R // 128), fmt)))
    w = moe.make_mx(fmt, N, C, data=cuda(mxo.write_tiles(wc, wb, *mxo.uniform_place(1, N), -(-N // 128), fmt)))
    y = torch.full((R, N), 77.0, device="cuda")
    moe.moe_mx_product(x, w, y)
    xv, wv = mxo.values(xc, xb, fmt), mxo.values(wc, wb, fmt)
    ref, mag = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    bound = (C / 64 + 2) * 2.0 ** -21 * mag
    assert within(y.cpu(), torch.from_numpy(ref), torch.from_numpy(bound)).all()


@pytest.mark.parametrize("R", [40, 300])
def test_product_of_every_e4m3_scale(R):
    """Bytes 0 to 126: zero, the subnormal ones (1 to 7) and the largest, 448."""
    rng = np.random.default_rng(R)
    N, C = 140, 512
    xb = rng.integers(0, 127, (R, C // 16)).astype(np.uint8)
    xb[:8] = np.arange(8)[:, None]  # whole rows of zero and of subnormal scales
    wb = rng.integers(0, 127, (N, C // 16)).astype(np.uint8)
    wb[:8] = np.arange(8)[:, None]
    product_of(rng.integers(0, 16, (R, C)).astype(np.uint8), xb, rng.integers(0, 16, (N, C)).astype(np.uint8), wb, E4)


@pytest.mark.parametrize("xlo,wlo", [(0, 236), (60, 176), (176, 60), (236, 0)])
def test_product_of_every_e8m0_scale(xlo, wlo):
    """Bytes 0 to 254 (2^-127 to 2^127), those of w about as far above 127 as those of x are below."""
    rng = np.random.default_rng(xlo)
    R, N, C = 70, 140, 512
    xb, wb = (rng.integers(lo, lo + 19, (n, C // 32)).astype(np.uint8) for lo, n in ((xlo, R), (wlo, N)))
    product_of(rng.integers(0, 16, (R, C)).astype(np.uint8), xb, rng.integers(0, 16, (N, C)).astype(np.uint8), wb, E8)


# ---------------------------------------------------------------------------
# quantise and dequantise: rows of a small call, in a large one
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", [E8, E4])
@pytest.mark.parametrize("cols", [512, 300, 511])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("act", [moe.MOE_ACT_NONE, moe.MOE_ACT_SWIGLU])
@pytest.mark.parametrize("gather", [False, True])
def test_many_rows_are_as_few(fmt, cols, dtype, act, gather):
    rng = np.random.default_rng(cols)
    few, E = 96, 50
    base = torch.from_numpy(rng.normal(0, 1, (few, cols * (2 if act else 1))).astype(np.float32)).cuda().to(dtype)
    sizes = rng.integers(0, 1600, E)
    sizes[[3, 7]] = 0
    R = int(sizes.sum()) + 11  # the last rows belong to no group
    offsets = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    group = np.concatenate([np.repeat(np.arange(E), sizes), [-1] * 11]).astype(np.int32)
    assert R > 30000
    row = rng.integers(0, few, R).astype(np.int32)
    scales = rng.choice([0.5, 0.37], E).astype(np.float32)
    t = scales if fmt == E4 else None
    src_row = row.copy()
    left = (rng.random(R) < 0.02) & gather
    src_row[left] = -1
    m = moe.make_mx(fmt, R, cols, groups=E, ragged=True)
    m._data.fill_(0xEE)
    maps = dict(group_of_row=cuda(group), offsets=cuda(offsets), tensor_scale=None if t is None else cuda(t))
    moe.moe_mx_quantise(m, base if gather else base[cuda(row).long()].contiguous(), act,
                        src_row=cuda(src_row) if gather else None, **maps)
    # every row of `base` by a call of its own size, once for each tensor scale
    ref = {}
    for s in (0.5, 0.37):
        q = moe.make_mx(fmt, few, cols)
        ts = None if t is None else cuda(np.array([s], np.float32))
        moe.moe_mx_quantise(q, base, act, tensor_scale=ts)
        back = torch.empty((few, cols), device="cuda")
        moe.moe_mx_dequantise(q, back, tensor_scale=ts)
        ref[s] = (*mxo.read_tiles(q._data.cpu().numpy(), *mxo.uniform_place(1, few), cols, fmt), back)
    n = int(sizes.sum())
    code, byte = mxo.read_tiles(m._data.cpu().numpy(), *mxo.ragged_place(offsets, group[:n]), cols, fmt)
    second = scales[group[:n]] == np.float32(0.37)
    there = ~left[:n]
    for got, which in ((code, 0), (byte, 1)):
        want = np.where(second[:, None], ref[0.37][which][row[:n]], ref[0.5][which][row[:n]])
        assert np.array_equal(got[there], want[there]) and (got[~there] == (0xE if which == 0 else 0xEE)).all()
    for dt in (torch.float32, torch.bfloat16):
        out = torch.full((R, cols), 5.0, device="cuda", dtype=dt)
        moe.moe_mx_dequantise(m, out, **maps)
        want = torch.where(cuda(second)[:, None], ref[0.37][2][cuda(row[:n]).long()], ref[0.5][2][cuda(row[:n]).long()])
        assert torch.equal(out[:n][cuda(there)], want[cuda(there)].to(dt)) and (out[n:] == 5.0).all()


@pytest.mark.parametrize("cols", [512, 33])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gathered_swiglu_with_a_tensor_scale(cols, dtype):
    """As without one: nearly all values are the definition's, and each is within its block's rounding step."""
    rng = np.random.default_rng(cols)
    src = cuda(rng.normal(0, 2, (30, 2 * cols)).astype(np.float32)).to(dtype)
    row = rng.integers(0, 30, 70).astype(np.int32)
    t = np.float32(0.013)
    m = moe.make_mx(E4, 70, cols)
    ts = cuda(np.array([t], np.float32))
    moe.moe_mx_quantise(m, src, act=moe.MOE_ACT_SWIGLU, src_row=cuda(row), tensor_scale=ts)
    out = torch.empty((70, cols), device="cuda")
    moe.moe_mx_dequantise(m, out, tensor_scale=ts)
    s = src.double().cpu().numpy()[row]
    x = s[:, :cols] / (1 + np.exp(-s[:, :cols])) * s[:, cols:]
    code, byte = mxo.quantise(x.astype(np.float32), E4, np.full(70, t, np.float32))
    ref = (mxo.values(code, byte, E4)[:, :cols].astype(np.float32) * t).astype(np.float64)
    got = out.double().cpu().numpy()
    assert (got != ref).mean() < 1e-3
    a = np.zeros((70, -(-cols // 256) * 256))
    a[:, :cols] = np.abs(x)
    a = np.repeat(a.reshape(70, -1, 16).max(2), 16, 1)[:, :cols]
    # half a step of the codes 4 and 6 where a is 6 scales, the scale itself within 1/16, and blocks below the smallest scale
    assert (np.abs(got - x) <= a * 0.2 + 2.0 ** -8 * t).all()


# ---------------------------------------------------------------------------
# dispatch: more than 128 x 8192 pairs
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("T,k,E", [(150001, 8, 256), (262144, 5, 1000), (1048577, 1, 7)])
@pytest.mark.parametrize("dropped", [False, True])
def test_dispatch_of_more_than_a_million_pairs(T, k, E, dropped):
    rng = np.random.default_rng(T)
    idx = rng.integers(0, E, (T, k)).astype(np.int32)
    if dropped:
        idx[rng.random((T, k)) < 0.3] = -1
        idx[rng.random((T, k)) < 0.01] = E + 5
    for got, ref in zip(run_dispatch(idx, E), mxo.dispatch(idx, E)):
        assert np.array_equal(got, ref)


# ---------------------------------------------------------------------------
# several streams and host threads
# ---------------------------------------------------------------------------

def chain(seed, T, E, k, hidden, inter):
    """Inputs of a layer, and a function that runs it on a stream with buffers of its own."""
    from int4_expert_streaming_gb300 import mx_layer

    g = torch.Generator(device="cuda").manual_seed(seed)
    gate_up, down = (torch.randn(s, generator=g, device="cuda") * .05 for s in ((E, 2 * inter, hidden), (E, hidden, inter)))
    x, logits = torch.randn((T, hidden), generator=g, device="cuda"), torch.randn((T, E), generator=g, device="cuda")
    layer = mx_layer.MxLayer(gate_up, down, moe.make_route_config(E, k), T, x_scale=0.01, h_scale=0.02)
    return lambda y: layer.forward(x, logits, y), (T, hidden)


SHAPES = [(3, 64, 4, 512, 256), (700, 16, 3, 1024, 512), (40, 200, 8, 300, 160)]


def test_layers_on_several_streams_at_once():
    runs = [chain(i, *s) for i, s in enumerate(SHAPES)]
    want = []
    for run, shape in runs:
        want.append(run(torch.empty(shape, device="cuda")))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    got = [torch.empty((20, *shape), device="cuda") for _, shape in runs]
    torch.cuda.synchronize()
    for i in range(20):
        for s, (run, _), y in zip(streams, runs, got):
            with torch.cuda.stream(s):
                run(y[i])
    torch.cuda.synchronize()
    for y, w in zip(got, want):
        assert all(torch.equal(v, w) for v in y)


def test_layers_of_several_host_threads():
    runs = [chain(i, *s) for i, s in enumerate(SHAPES)]
    want = [run(torch.empty(shape, device="cuda")) for run, shape in runs]
    got = [torch.empty((20, *shape), device="cuda") for _, shape in runs]
    torch.cuda.synchronize()
    errors = []

    def work(run, y):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for v in y:
                    run(v)
                # a refusal of one thread's is no other's message
                with pytest.raises(moe.MoeError, match="score"):
                    cfg = moe.make_route_config(16, 2, score=9)
                    moe.moe_route(cfg, torch.zeros((1, 16), device="cuda"), None,
                                  torch.zeros((1, 2), dtype=torch.int32, device="cuda"), torch.zeros((1, 2), device="cuda"))
        except BaseException as e:  # noqa: BLE001 -- reported by the test's own thread
            errors.append(e)
    threads = [threading.Thread(target=work, args=(run, y)) for (run, _), y in zip(runs, got)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for y, w in zip(got, want):
        assert all(torch.equal(v, w) for v in y)
