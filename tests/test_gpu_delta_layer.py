"""The delta rule's mixer as a layer, and the decoder layer that mx_layer's command times."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import _mix_oracle as ora  # noqa: E402
import int4_expert_streaming_gb300 as moe  # noqa: E402
from int4_expert_streaming_gb300 import delta_layer, mx_layer  # noqa: E402

BF = torch.bfloat16


def rounded(a):
    return torch.from_numpy(a).to(BF).double().numpy()


def weights_of(rng, hidden, heads, width=4):
    Hk, Hv, dk, dv = heads
    C, inner = 2 * Hk * dk + Hv * dv, Hv * dv
    n = rng.standard_normal
    return {"w_in": rounded(n((C + inner, hidden)) * hidden ** -0.5), "w_gates": rounded(n((2 * Hv, hidden)) * hidden ** -0.5),
            "conv": rounded(0.5 * n((C, width))), "a_log": np.float32(0.3 * n(Hv)).astype(np.float64),
            "dt_bias": np.float32(n(Hv) - 1).astype(np.float64), "norm": np.float32(1 + 0.1 * n(dv)).astype(np.float64),
            "w_out": rounded(n((hidden, inner)) * inner ** -0.5)}


def mixer_of(w, heads, **kw):
    t = {k: torch.from_numpy(v).cuda().to(torch.float32 if k in ("a_log", "dt_bias", "norm") else BF) for k, v in w.items()}
    return delta_layer.DeltaMixer(**t, heads=heads, **kw)


def plain(w, heads, x, seqs, conv_state, state, r):
    """The mixer by its formulas in 64 bits; r rounds where the layer does.  The states are replaced."""
    Hk, Hv, dk, dv = heads
    T, C = len(x), w["conv"].shape[0]
    p, gates = r(x @ w["w_in"].T), r(x @ w["w_gates"].T)
    m = np.zeros((T, C))
    ora.conv(p[:, :C], w["conv"], None, True, m, conv_state, seqs)
    m = r(m)
    q, k = (r(ora.head_norm(a.reshape(T, Hk, dk), "l2", 1e-6, None, 0, None, None, 0, True, None)[0])
            for a in (m[:, :Hk * dk], m[:, Hk * dk:2 * Hk * dk]))
    g = -np.exp(w["a_log"]) * np.logaddexp(0, gates[:, Hv:] + w["dt_bias"])
    o = np.zeros((T, Hv, dv))
    ora.delta(q, k, m[:, 2 * Hk * dk:].reshape(T, Hv, dv), g, 1 / (1 + np.exp(-gates[:, :Hv])), state, o, dk ** -0.5, seqs)
    gated = ora.head_norm(r(o), "rms", 1e-6, w["norm"], 0, None, None, 0, True, p[:, C:].reshape(T, Hv, dv))[0]
    return r(r(gated).reshape(T, -1) @ w["w_out"].T)


def ints(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("heads", [(2, 4, 64, 64), (1, 3, 128, 40)])
def test_prompts_then_single_tokens(heads):
    """The layer rounds where the rounding formulas do, from sums that differ in the last of 24 bits, so its own roundings
    are another draw of the same size: its distance from the exact formulas is that of the rounded ones, within the
    spread of a root mean square of thousands of values (a factor of two is far outside it)."""
    rng = np.random.default_rng(51)
    hidden, slots = 128, 3
    w = weights_of(rng, hidden, heads)
    mixer = mixer_of(w, heads, slots=slots, max_tokens=256, max_seqs=4)
    Hk, Hv, dk, dv = heads
    C = w["conv"].shape[0]
    exact, round_ = ((np.zeros((slots, 3, C)), np.zeros((slots, Hv, dv, dk))) for _ in range(2))
    for step in range(6):
        # a long prompt, a short one and one that is left out; then single tokens, the middle one going on with five
        lens = [150, 9, 20] if step == 0 else [1, 5, 1]
        slot = [2, 0, -1]
        off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        T = int(off[-1])
        x = rounded(rng.standard_normal((T, hidden)))
        seqs = moe.make_seqs(3, ints(off), ints(slot), ints([step > 0] * 3), max(lens) if step else 0)
        y = torch.full((T, hidden), 7.0, dtype=BF, device="cuda")
        mixer.forward(torch.from_numpy(x).cuda().to(BF), seqs, y)
        torch.cuda.synchronize()
        s = list(ora.sequences(T, off, slot, [step > 0] * 3))
        want, draw = plain(w, heads, x, s, *exact, lambda a: a), plain(w, heads, x, s, *round_, rounded)
        live = np.concatenate([np.arange(lo, hi) for lo, hi, _, _ in s])
        got = y.double().cpu().numpy()
        rms = lambda d: np.sqrt((d[live] ** 2).mean())  # noqa: E731
        assert 0 < rms(draw - want) and rms(got - want) <= 2 * rms(draw - want)
        state = mixer.state.double().cpu().numpy()
        assert np.abs(state[[0, 2]] - exact[1][[0, 2]]).max() <= 4 * np.abs(round_[1] - exact[1]).max()
        assert (state[1] == 0).all()


def test_refusals():
    rng = np.random.default_rng(52)
    heads = (1, 2, 64, 64)
    w = weights_of(rng, 64, heads)
    with pytest.raises(ValueError, match="w_out"):
        mixer_of({**w, "w_out": w["w_out"][:, :-1]}, heads, slots=1, max_tokens=8, max_seqs=1)
    mixer = mixer_of(w, heads, slots=1, max_tokens=8, max_seqs=1)
    x = torch.zeros((9, 64), dtype=BF, device="cuda")
    with pytest.raises(ValueError, match="room"):
        mixer.forward(x, moe.make_seqs(1, ints([0, 9])), torch.empty_like(x))
    with pytest.raises(ValueError, match="room"):
        mixer.forward(x[:2], moe.make_seqs(2), torch.empty_like(x[:2]))
    with pytest.raises(ValueError, match="width"):
        mixer.forward(x[:4, :32], moe.make_seqs(1, ints([0, 4])), torch.empty_like(x[:4]))
    two = mixer_of(w, heads, slots=2, max_tokens=8, max_seqs=2)
    with pytest.raises(moe.MoeError, match="n=2, T=1"):  # two sequences of single tokens, one row
        two.forward(x[:1], moe.make_seqs(2), torch.empty_like(x[:1]))
    assert mixer.forward(x[:0], moe.make_seqs(0), x[:0]).shape == (0, 64)


def test_a_decoder_layer_captured_and_replayed():
    """Prompts and a decode step of mixer and experts: replays of a captured step give what direct calls give."""
    gen = torch.Generator(device="cuda").manual_seed(3)

    def normal(*shape, sigma=1.0):
        return torch.randn(shape, generator=gen, device="cuda") * sigma
    heads, hidden, E, inter = (2, 4, 64, 64), 128, 8, 64
    w = weights_of(np.random.default_rng(53), hidden, heads)
    gate_up, down, router = normal(E, 2 * inter, hidden, sigma=.05), normal(E, hidden, inter, sigma=.05), normal(E, hidden).to(BF)
    prompt, tokens = normal(70, hidden).to(BF), normal(4, 2, hidden).to(BF)

    def layer_of():
        return mx_layer.DecoderLayer(mixer_of(w, heads, slots=2, max_tokens=80, max_seqs=2),
                                     mx_layer.MxLayer(gate_up, down, moe.make_route_config(E, 2), 80, x_scale=0.01, h_scale=0.02),
                                     router)
    first, decode = moe.make_seqs(2, ints([0, 30, 70]), carry=ints([0, 0])), moe.make_seqs(2)
    direct, captured = layer_of(), layer_of()
    results = [direct.forward(prompt, first).clone()]
    for t in tokens:
        results.append(direct.forward(t, decode).clone())
    assert torch.equal(captured.forward(prompt, first), results[0])
    # a capture needs a warm call, which must not touch the states: of sequences without slots
    x = tokens[0].clone()
    nowhere = moe.make_seqs(2, slot=ints([-1, -1]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        captured.forward(x, nowhere)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = captured.forward(x, decode)
    for t, want in zip(tokens, results[1:]):
        x.copy_(t)
        graph.replay()
        assert torch.equal(out, want)
    assert torch.isfinite(torch.stack([r.float().abs().max() for r in results])).all()
