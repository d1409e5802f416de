"""The expert layer out of the operators without a context, against the layer of unquantised weights and values in 64
bits, at activations of any size.

An e2m1 code is off by 1/sqrt(12) of its step, 0.5 at 1 to 2: about 0.1 of the value (rms), for each of the four matrices
that are quantised.  Their errors are independent: gate and up rows sqrt(2) * 0.1, their product sqrt(2) times that, 0.2,
and with the two of the second product sqrt(0.2^2 + 2 * 0.1^2) = 0.245.  The bound is 0.3; a layer that drops blocks of
small values is off by about 1."""
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


E, K, HIDDEN, INTER = 16, 3, 320, 160


def inputs(T, sigma, seed=0):
    rng = np.random.default_rng(seed)
    gate_up = rng.normal(0, .05, (E, 2 * INTER, HIDDEN)).astype(np.float32)
    down = rng.normal(0, .05, (E, HIDDEN, INTER)).astype(np.float32)
    x = (rng.normal(0, 1, (T, HIDDEN)) * sigma).astype(np.float32)
    logits = (rng.permutation(np.arange(T * E)).reshape(T, E) / (T * E) * 6 - 3).astype(np.float32)
    return gate_up, down, x, logits


def definition(gate_up, down, x, logits):
    idx, w = mxo.route(logits, None, K, 1, 1, 1, False, True, 1.0)
    y = np.zeros(x.shape)
    for t in range(x.shape[0]):
        for e, wt in zip(idx[t], w[t]):
            if e >= 0:
                u = gate_up[e].astype(np.float64) @ x[t]
                y[t] += wt * (down[e].astype(np.float64) @ (u[:INTER] / (1 + np.exp(-u[:INTER])) * u[INTER:]))
    return y


def run(gate_up, down, x, logits, **scales):
    layer = mx_layer.MxLayer(torch.from_numpy(gate_up).cuda(), torch.from_numpy(down).cuda(),
                             moe.make_route_config(E, K), max_tokens=len(x), **scales)
    y = torch.full((len(x), HIDDEN), float("nan"), device="cuda")
    layer.forward(torch.from_numpy(x).cuda(), torch.from_numpy(logits).cuda(), y)
    return y.double().cpu().numpy()


@pytest.mark.parametrize("sigma", [100.0, 1.0, 0.03, 1e-3])
@pytest.mark.parametrize("T", [1, 40])
def test_layer_is_as_good_at_small_values_as_at_large_ones(T, sigma):
    a = inputs(T, sigma)
    ref = definition(*a)
    assert np.linalg.norm(run(*a) - ref) <= 0.3 * np.linalg.norm(ref)


@pytest.mark.parametrize("sigma", [100.0, 1e-3])
def test_layer_with_given_scales(sigma):
    """Scales found beforehand, with room: the SwiGLU rows reach about 0.5 * 4^2 * (0.05 * sqrt(320) * sigma)^2 where the
    gate is small, (4 * 0.9 * sigma)^2 where it is large."""
    a = inputs(40, sigma)
    y = run(*a, x_scale=mx_layer.tensor_scale(8 * sigma), h_scale=mx_layer.tensor_scale(16 * sigma ** 2))
    ref = definition(*a)
    assert np.linalg.norm(y - ref) <= 0.3 * np.linalg.norm(ref)


def test_measured_scales_leave_out_rows_without_an_expert_and_what_is_not_finite():
    gate_up, down, x, logits = inputs(40, 1e-3)
    ref = definition(gate_up, down, x, logits)
    logits[[3, 20]] = -np.inf
    x[3], x[20] = np.nan, 1e30
    x[7, 5] = np.inf
    y = run(gate_up, down, x, logits)
    there = np.isin(np.arange(40), [3, 7, 20], invert=True)
    assert (y[[3, 20]] == 0).all() and np.isnan(y[7]).all()
    assert np.linalg.norm((y - ref)[there]) <= 0.3 * np.linalg.norm(ref[there])


def test_layer_of_zeros_and_of_no_tokens():
    gate_up, down, x, logits = inputs(4, 1.0)
    assert (run(gate_up, down, x * 0, logits) == 0).all()
    assert (run(gate_up * 0, down, x, logits) == 0).all()
    layer = mx_layer.MxLayer(torch.from_numpy(gate_up).cuda(), torch.from_numpy(down).cuda(), moe.make_route_config(E, K), 4)
    none = torch.empty((0, HIDDEN), device="cuda")
    assert layer.forward(none, torch.empty((0, E), device="cuda"), none) is none


def test_scales_are_refused_where_they_cannot_be_used():
    w, d = torch.zeros((8, 64, 128), device="cuda"), torch.zeros((8, 128, 32), device="cuda")
    cfg = moe.make_route_config(8, 2)
    for kw in ({"x_scale": 0.0}, {"h_scale": float("nan")}, {"h_scale": -1.0}, {"x_scale": float("inf")},
               {"x_scale": 1.0, "fmt": moe.MOE_MX_E8M0}):
        with pytest.raises(ValueError):
            mx_layer.MxLayer(w, d, cfg, 4, **kw)
