"""The gated delta rule over long runs and changes of size, against its definition in 64 bits.

`size` is what tolerances go by: the largest magnitude of a head's state, an earlier one shrunk by the decays since."""
import math

import pytest

import int4_expert_streaming_gb300 as moe

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    moe.build()
    moe.load_library()


def definition(q, k, v, g, beta, S, scale):
    """Token by token; o [T, Hv, dv], the state after the last token, size [T, Hv] and o's state sums' magnitude."""
    share = v.shape[1] // k.shape[1]
    q, k = (t.double().repeat_interleave(share, 1)[..., None] for t in (q, k))
    v, g, beta, S = v.double()[..., None], g.double(), beta.double()[..., None, None], S[0].double()
    o, size, top = torch.empty(v.shape[:3], dtype=torch.float64, device="cuda"), [], S.abs().amax((1, 2))
    for t in range(len(v)):
        S = torch.where(torch.isneginf(g[t])[:, None, None], 0, S * torch.exp(g[t])[:, None, None])
        S = S + beta[t] * (v[t] - S @ k[t]) * k[t].transpose(1, 2)
        o[t] = scale * (S @ q[t])[..., 0]
        top = torch.maximum(torch.where(torch.isneginf(g[t]), 0, top * torch.exp(g[t])), S.abs().amax((1, 2)))
        size.append(top)
    return o, S[None], torch.stack(size)


def inputs(T, Hk, Hv, dk, dv, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")
    q, k = (t / t.norm(dim=2, keepdim=True) for t in (normal(T, Hk, dk), normal(T, Hk, dk)))
    return q.to(BF), k.to(BF), normal(T, Hv, dv).to(BF), torch.rand((T, Hv), generator=gen, device="cuda"), normal(1, Hv, dv, dk)


def run(q, k, v, g, beta, state, scale, piece=None):
    """One call, or one for each `piece` rows; o and the state after."""
    T, Hk, dk = q.shape
    Hv, dv = v.shape[1:]
    ws = torch.empty(max(1, moe.moe_delta_workspace(T, 1, Hk, Hv, dk, dv)), dtype=torch.uint8, device="cuda")
    o, state = torch.empty_like(v), state.clone()
    for lo in range(0, T, piece or T):
        at = slice(lo, lo + (piece or T))
        moe.moe_delta(q[at], k[at], v[at], g[at], beta[at], state, o[at], scale, workspace=ws, stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    return o.double(), state.double()


def check_state(got, want, size, bound, more=0.0):
    """Every value within bound of the size at the end."""
    off = (got - want).abs().amax((0, 2, 3)) / (bound * size[-1] + more)
    assert (off <= 1).all(), off


@pytest.mark.parametrize("g,beta", [(-1e-3, 0.5), (0.0, 0.5), (0.0, 0.01), (-1e-5, 0.001)])
def test_a_long_memory_in_chunks(g, beta):
    """16384 tokens, in whose 256 chunks little or nothing of the state is forgotten.  A chunk's sums of up to 16 steps of the
    tensor core lose up to 2^-24 of their size at each in the mean, if those round towards zero: 2^-20, of what the chunk adds
    to the state and not of the state, so it does not grow with the chunks; three sums follow each other, 2^-18.4.  One
    rounding a chunk of the state itself, without a bias: 5 sqrt(256) 2^-25.  Together below 2^-17."""
    q, k, v, r, start = inputs(16384, 1, 2, 128, 128, 1)
    decay, beta = torch.full_like(r, g), beta * (0.5 + 0.5 * r)
    o, state, size = definition(q, k, v, decay, beta, start, 0.1)
    got_o, got = run(q, k, v, decay, beta, start, 0.1)
    check_state(got, state, size, 2.0 ** -17)
    near = 2.0 ** -8 * 1.01 * o.abs() + 2.0 ** -9 * 0.1 * size[..., None]  # |q| is 1
    assert ((got_o - o).abs() <= near).all()


def test_constant_decays_in_chunks():
    """16384 tokens that only decay: what every chunk multiplies the state by must not be off by the same each time.  A
    chunk's rounding of a value goes one way while its decay does, up to 2^-24; what a head's 1024 values lose together spreads
    by 256 2^-24.8 sqrt(3 / 1024) = 2^-21, and 5 of that are 2^-18.7."""
    heads, T = 24, 16384
    q, k, v, r, start = inputs(T, 1, heads, 32, 32, 4)
    g = torch.logspace(-6, -3.4, heads, device="cuda").neg().expand(T, heads).contiguous()
    _, got = run(q, k, v, g, torch.zeros_like(g), start, 0.1)
    want = start.double() * torch.exp(g.double().sum(0))[None, :, None, None]
    lost = (got * want).sum((0, 2, 3)) / want.square().sum((0, 2, 3)) - 1
    assert (lost.abs() <= 2.0 ** -18.7).all(), lost


@pytest.mark.parametrize("piece", [24, 1])
@pytest.mark.parametrize("g", [-1e-5, -3e-4])
def test_a_long_memory_token_by_token(g, piece):
    """A state in fp32, rounded at each token by up to 2^-24 of a value.  Under a constant decay a value's roundings mostly go
    the same way, because what is taken from it hardly changes: T 2^-24.  But another value's go another way: what all N
    values have lost together, sum(got want) / sum(want^2) - 1, spreads by T 2^-24.8 sqrt(3 / N) where their magnitudes
    are normal, and 5 of that are T 2^-29.  A decay that is itself off by 2^-25 is T 2^-25 there."""
    T = 16384 if piece > 1 else 1024
    q, k, v, r, start = inputs(T, 1, 2, 128, 128, 2)
    decay, beta = torch.full_like(r, g), 0.001 + 0.0 * r
    o, state, size = definition(q, k, v, decay, beta, start, 0.1)
    got_o, got = run(q, k, v, decay, beta, start, 0.1, piece)
    check_state(got, state, size, T * 2.0 ** -24)
    assert abs((got * state).sum() / state.square().sum() - 1) <= T * 2.0 ** -29
    assert ((got_o - o).abs() <= 2.0 ** -8 * 1.01 * o.abs() + T * 2.0 ** -24 * 0.1 * size[..., None] * math.sqrt(128)).all()


@pytest.mark.parametrize("at", [20, 61, 64, 150])
@pytest.mark.parametrize("how", ["cleared", "shrunk"])
@pytest.mark.parametrize("times", [2.0 ** 10, 2.0 ** 20])
def test_a_large_state_is_cleared(times, how, at):
    """A state far above what is written later, cleared (or shrunk by e^-27 in three tokens) in the midst of a chunk, at its
    end, at its beginning, or in a later one.  The chunk with the clear has both sizes in its products, whose numbers are held
    in steps of 2^-37 of a bound: |k|_1 = 2^3.3 times the largest state, and for what goes into the state that times a row of
    T, of sums about 4.  Such a step's rounding has a spread of 2^-38.8 of the bound: 2^-33.5 of the largest state, and by
    up to 43 keys of values of 2^-3.5 into the state 2^-34.3; 5 spreads are below 2^-32.  Later chunks know the new size alone."""
    q, k, v, beta, start = inputs(266, 1, 2, 128, 128, 3)
    start = start * times
    g = -0.05 * beta.flip(0)
    g[at:at + 3] = -float("inf") if how == "cleared" else -9.0
    o, state, size = definition(q, k, v, g, beta, start, 0.1)
    got_o, got = run(q, k, v, g, beta, start, 0.1)
    left = 2.0 ** -32 * start.double().abs().amax((0, 2, 3))
    assert torch.isfinite(got).all()
    check_state(got, state, size, 2.0 ** -16, left)
    far = size.clone()
    far[at // 64 * 64:(at + 2) // 64 * 64 + 64] += 2.0 ** -9 * size[at // 64 * 64]  # beside the large ones in its chunk: 2^-20 of those
    near = 2.0 ** -8 * 1.01 * o.abs() + 0.1 * (2.0 ** -9 * far + left)[..., None]
    off = ((got_o - o).abs() / near).amax((1, 2))
    assert (off <= 1).all(), (off.argmax(), off.max())
