"""SiLU of the convolution and of the head norms' gate where its values are small."""
import numpy as np
import pytest

import int4_expert_streaming_gb300 as moe

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    moe.build()
    moe.load_library()


def silu(x):
    return x / (1 + np.exp(-x))


POINTS = np.concatenate([np.linspace(-104, -79, 5000), -80 + np.linspace(-1e-4, 1e-4, 33), np.linspace(-79, 20, 2000),
                         [0.0, -0.0]]).astype(np.float32)


@pytest.mark.parametrize("op", ["conv", "gate"])
def test_fp32_down_to_the_smallest(op):
    """2^-21 of the value as the header says, and two steps of the smallest numbers, 2^-149."""
    x = torch.from_numpy(POINTS).cuda()
    y = torch.empty_like(x)
    if op == "conv":
        w = torch.tensor([[0.0, 1.0]], device="cuda")
        moe.moe_conv(x[:, None], w, y[:, None], stream=torch.cuda.current_stream())
    else:
        one = torch.ones((len(x), 1, 1), device="cuda")
        moe.moe_head_norm(moe.make_head_norm_config(moe.MOE_NORM_NONE), one, y.view(-1, 1, 1), gate=x.view(-1, 1, 1),
                          stream=torch.cuda.current_stream())
    want = silu(POINTS.astype(np.float64))
    off = np.abs(y.double().cpu().numpy() - want) / (2.0 ** -21 * np.abs(want) + 2.0 ** -148)
    assert off.max() <= 1, (POINTS[off.argmax()], off.max())


def test_bf16_as_the_header_says():
    """Rounded to bf16, 2^-21 + |x| 2^-24 before that; below 2^-126 it may be 0."""
    x = torch.from_numpy(POINTS).cuda().bfloat16()[:, None]
    y, w = torch.empty_like(x), torch.tensor([[0.0, 1.0]], device="cuda")
    moe.moe_conv(x, w, y, stream=torch.cuda.current_stream())
    v = x.double().cpu().numpy()
    want, got = silu(v), y.double().cpu().numpy()
    tol = np.abs(want) * (2.0 ** -8 + 2.0 ** -21 + np.abs(v) * 2.0 ** -24) + np.where(np.abs(want) < 2.0 ** -126, 2.0 ** -126, 0)
    assert (np.abs(got - want) <= tol).all()


def test_ends():
    """Infinities and NaN give what the formula gives."""
    x = torch.tensor([[float("inf")], [-float("inf")], [float("nan")], [3e38], [-3e38]], device="cuda")
    w = torch.tensor([[0.0, 1.0]], device="cuda")
    for dt in (torch.float32, torch.bfloat16):
        for i in range(5):
            y = torch.empty((1, 1), dtype=dt, device="cuda")
            moe.moe_conv(x[i:i + 1].to(dt), w.to(dt), y, stream=torch.cuda.current_stream())
            v = float(y)
            assert v == (float("inf"), None, None, float(x[3:4].to(dt)), 0)[i] if i not in (1, 2) else v != v
