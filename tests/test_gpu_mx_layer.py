"""A whole expert layer out of the operators without a context against its definition: the same roundings (codes of the
token rows, bf16 products, codes of the SwiGLU rows) with every sum in 64 bits.

A value of the SwiGLU rows that stands next to a boundary between two codes may fall on either side of it, because the
product before it and its exp are fp32; at most one in a thousand does.  Such a code is off by at most a third of its
value, so by their squares the rows are off by at most sqrt(1e-3) / 3 = 1.1e-2, and y as much: 1.5e-2 with y's other
roundings (bf16 rows, 2^-9 each)."""
import numpy as np
import pytest

import _mx_oracle as mxo

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

import int4_expert_streaming_gb300 as moe  # noqa: E402
from int4_expert_streaming_gb300 import mx_layer  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    moe.build()
    moe.load_library()


def dequantised_weights(w, fmt, t):
    """w [E, N, K] fp32 -> the numbers its matrix stands for, with the tensor scales t [E] the layer chose, fp64."""
    E, N, K = w.shape
    code, byte = mxo.quantise(w.reshape(E * N, K), fmt, None if t is None else np.repeat(t, N))
    v = mxo.values(code, byte, fmt)[:, :K].reshape(E, N, K)
    return v if t is None else v * t.astype(np.float64)[:, None, None]


def bf16(a):
    return torch.from_numpy(np.asarray(a, np.float64)).to(torch.bfloat16).double().numpy()


def definition(x, logits, gate_up, down, scales, cfg, bias, fmt):
    idx, w = mxo.route(logits, bias, cfg.top_k, cfg.n_groups, cfg.top_groups, cfg.group_best, cfg.score == 1, True,
                       cfg.scale)
    wu, wd = dequantised_weights(gate_up, fmt, scales[0]), dequantised_weights(down, fmt, scales[1])
    code, byte = mxo.quantise(x, fmt)
    xq = mxo.values(code, byte, fmt)[:, :x.shape[1]]
    inter = down.shape[2]
    y = np.zeros(x.shape)
    for t in range(x.shape[0]):
        for e, wt in zip(idx[t], w[t]):
            if e < 0:
                continue
            u = bf16(xq[t] @ wu[e].T)
            h = (u[:inter] / (1 + np.exp(-u[:inter])) * u[inter:]).astype(np.float32)
            c, b = mxo.quantise(h[None], fmt)
            y[t] += wt * bf16(mxo.values(c, b, fmt)[0, :inter] @ wd[e].T)
    return idx, y


@pytest.mark.parametrize("fmt", [moe.MOE_MX_E8M0, moe.MOE_MX_E4M3])
@pytest.mark.parametrize("T", [1, 7, 150])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_layer_matches_its_definition(fmt, T, dtype):
    rng = np.random.default_rng(T + fmt)
    E, k, hidden, inter = 24, 3, 320, 160
    gate_up = torch.from_numpy(rng.normal(0, .05, (E, 2 * inter, hidden)).astype(np.float32)).to(torch.bfloat16)
    down = torch.from_numpy(rng.normal(0, .05, (E, hidden, inter)).astype(np.float32)).to(torch.bfloat16)
    cfg = moe.make_route_config(E, k, n_groups=4, top_groups=2, group_best=1, score=moe.MOE_SCORE_SIGMOID, scale=1.5)
    logits = (rng.permutation(np.arange(T * E)).reshape(T, E) / (T * E) * 6 - 3).astype(np.float32)  # all different
    logits[T // 2, 5:] = -np.inf  # fewer experts than groups of a full choice
    if T > 2:
        logits[T - 1] = -np.inf  # a padding token: no expert at all
    x = torch.from_numpy(rng.normal(0, 1, (T, hidden)).astype(np.float32)).to(dtype)
    layer = mx_layer.MxLayer(gate_up.cuda(), down.cuda(), cfg, max_tokens=T + 3, fmt=fmt)
    y = torch.full((T, hidden), float("nan"), device="cuda")
    layer.forward(x.cuda(), torch.from_numpy(logits).cuda(), y)
    torch.cuda.synchronize()
    scales = [None if t is None else t.cpu().numpy() for t in (layer.alpha_up, layer.alpha_down)]
    idx, ref = definition(x.float().numpy(), logits, gate_up.float().numpy(), down.float().numpy(), scales, cfg, None, fmt)
    assert np.array_equal(layer.idx[:T].cpu().numpy(), idx)
    got = y.double().cpu().numpy()
    assert np.linalg.norm(got - ref) <= 1.5e-2 * np.linalg.norm(ref)
    if T > 2:
        assert (got[T - 1] == 0).all()


def test_layer_of_fewer_tokens_gives_the_same_rows():
    """A batch's rows do not depend on the batch: each token's result alone equals its row in the batch."""
    g = torch.Generator(device="cuda").manual_seed(2)
    E, k, hidden, inter, T = 64, 4, 512, 256, 40

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")
    layer = mx_layer.MxLayer(normal(E, 2 * inter, hidden) * .02, normal(E, hidden, inter) * .02,
                             moe.make_route_config(E, k), max_tokens=T)
    x, logits = normal(T, hidden), normal(T, E)
    y, one = torch.empty((T, hidden), device="cuda"), torch.empty((1, hidden), device="cuda")
    layer.forward(x, logits, y)
    for t in (0, 17, T - 1):
        layer.forward(x[t:t + 1], logits[t:t + 1], one)
        assert torch.equal(one[0], y[t])


def test_layer_refuses_what_does_not_fit():
    w = torch.zeros((8, 64, 128), device="cuda")
    with pytest.raises(ValueError):
        mx_layer.MxLayer(w, torch.zeros((8, 128, 64), device="cuda"), moe.make_route_config(8, 2), 4)
    layer = mx_layer.MxLayer(w, torch.zeros((8, 128, 32), device="cuda"), moe.make_route_config(8, 2), 4)
    x, logits, y = (torch.zeros((5, n), device="cuda") for n in (128, 8, 128))
    with pytest.raises(ValueError):
        layer.forward(x, logits, y)
    with pytest.raises(ValueError):
        layer.forward(x[:4], logits[:4, :7], y[:4])
