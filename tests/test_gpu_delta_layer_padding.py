"""Rows of a batch that belong to no sequence, or to one without a slot: what the mixer and the decoder layer make of them."""
import numpy as np
import pytest

import int4_expert_streaming_gb300 as moe

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from int4_expert_streaming_gb300 import mx_layer  # noqa: E402
from test_gpu_delta_layer import BF, ints, mixer_of, weights_of  # noqa: E402

HEADS, HIDDEN = (2, 4, 64, 64), 128


def batch(kind):
    """seqs, rows of the batch, rows that are left out"""
    if kind == "padded decode":
        return moe.make_seqs(6, slot=ints([0, 3, -1, 1, 9, -1]), carry=ints([0] * 6)), 6, [2, 4, 5]
    return moe.make_seqs(3, ints([2, 40, 45, 75]), ints([1, -1, 0]), ints([0] * 3)), 80, [0, 1, *range(40, 45), *range(75, 80)]


def history(mixer, seed):
    """Calls that leave something in every row of the object's buffers."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((80, HIDDEN), generator=gen, device="cuda").to(BF)
    mixer.forward(x, moe.make_seqs(1, ints([0, 80])), torch.empty_like(x))
    mixer.forward(x[:4], moe.make_seqs(4), torch.empty_like(x[:4]))


@pytest.mark.parametrize("kind", ["padded decode", "ragged prompts"])
def test_rows_left_out_are_zeros(kind):
    w = weights_of(np.random.default_rng(61), HIDDEN, HEADS)
    mixer = mixer_of(w, HEADS, slots=4, max_tokens=80, max_seqs=8)
    seqs, T, out = batch(kind)
    history(mixer, 1)
    x = torch.randn((T, HIDDEN), generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").to(BF)
    y = torch.full_like(x, 7.0)
    mixer.forward(x, seqs, y)
    live = torch.ones(T, dtype=torch.bool, device="cuda")
    live[out] = False
    assert (y[~live] == 0).all() and (y[live].abs().amax(1) > 0).all()


@pytest.mark.parametrize("kind", ["padded decode", "ragged prompts"])
def test_rows_do_not_depend_on_earlier_calls(kind):
    """Through the experts too, whose scales are measured from the batch."""
    w = weights_of(np.random.default_rng(62), HIDDEN, HEADS)
    gen = torch.Generator(device="cuda").manual_seed(3)

    def normal(*shape, sigma=1.0):
        return torch.randn(shape, generator=gen, device="cuda") * sigma
    gate_up, down, router = normal(8, 128, HIDDEN, sigma=.05), normal(8, HIDDEN, 64, sigma=.05), normal(8, HIDDEN).to(BF)
    seqs, T, out = batch(kind)
    inputs = [normal(T, HIDDEN, sigma=0.1 + i).to(BF) for i in range(4)]
    for x in inputs:
        x[out] *= 1e-3  # of the rows left out little but what the mixer adds
    results = []
    for seed in (None, 4, 5):
        layer = mx_layer.DecoderLayer(mixer_of(w, HEADS, slots=4, max_tokens=80, max_seqs=8),
                                      mx_layer.MxLayer(gate_up, down, moe.make_route_config(8, 2), 80), router)
        if seed is not None:
            history(layer.mixer, seed)
        results.append(torch.stack([layer.forward(x, seqs) for x in inputs]))
    assert torch.equal(results[0], results[1]) and torch.equal(results[0], results[2])
