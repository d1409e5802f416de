"""Kernels of the operators between two expert layers that only some sizes and types reach, against the definitions in 64
bits, and what their Python calls refuse of real CUDA tensors."""
import numpy as np
import pytest

import _mix_oracle as ora
import int4_expert_streaming_gb300 as moe

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_mix import BF, F32, HALF, check_norm, cuda, delta_inputs, f64, ints, rng_of, run_delta, strided  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    moe.build()
    moe.load_library()


# ---------------------------------------------------------------------------
# convolution of single tokens
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("C,at", [(1, 0), (8, 0), (63, 0), (256, 0), (256, 1), (1027, 0)])
@pytest.mark.parametrize("bias,act", [(True, True), (False, False)])
def test_conv_of_single_tokens(dt, W, C, at, bias, act):
    """Tolerance: W products and a bias in fp32, silu to 2^-21 with a slope below 1.1, one rounding."""
    rng = rng_of(W, C, at)
    n, slots = 19, 21
    slot = rng.permutation(slots)[:n].astype(np.int32)
    slot[[2, 18]] = -1, slots  # no such slots
    carry = (rng.random(n) < 0.7).astype(np.int32)
    x = strided(cuda(rng.standard_normal((n, C)), dt), 8, at)
    y = strided(torch.full((n, C), 3.0, dtype=dt, device="cuda"), 16, at)
    w, b = cuda(rng.standard_normal((C, W)), F32 if W == 3 else BF), cuda(rng.standard_normal(C)) if bias else None
    st = cuda(rng.standard_normal((slots, W - 1, C)), dt)
    for s in range(n):
        if not carry[s] and 0 <= slot[s] < slots:
            st[int(slot[s])] = float("nan")  # not to be read
    want, ws = f64(y), f64(st)
    size = ora.conv(f64(x), f64(w), None if b is None else f64(b), act, want, ws, ora.sequences(n, None, slot, carry, slots))
    moe.moe_conv(x, w, y, bias=b, act=moe.MOE_ACT_SILU if act else moe.MOE_ACT_NONE,
                 seqs=moe.make_seqs(n, slot=ints(slot), carry=ints(carry)), state=st, stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    tol = HALF[dt] * np.abs(want) * 1.01 + (W + 1) * 2.0 ** -24 * size * 1.1 + (2.0 ** -21 * np.abs(want) if act else 0)
    assert (np.abs(f64(y) - want) <= tol + 1e-37).all()
    assert np.array_equal(f64(st), ws, equal_nan=True)


# ---------------------------------------------------------------------------
# head norms, two heads a group of threads
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,H,H2,D", [(401, 33, 0, 64), (401, 31, 3, 56), (211, 33, 2, 128), (701, 9, 1, 104), (103, 32, 5, 256),
                                      (467, 7, 7, 200)])
@pytest.mark.parametrize("rot", ["none", "halves", "adjacent"])
@pytest.mark.parametrize("gate", [False, True])
def test_norm_of_many_heads(dt, T, H, H2, D, rot, gate):
    check_norm(rng_of(T, D), dt, T, H, D, "rms", rot=0 if rot == "none" else D // 16 * 8, halves=rot == "halves", gate=gate, H2=H2)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_norm_of_many_heads_in_place_and_by_columns(dt, D):
    check_norm(rng_of(D), dt, 13000 // D * 64 // 8, 8, D, "l2", weight=False, H2=8, inplace=True)
    check_norm(rng_of(D), dt, 13000 // D * 64 // 8, 8, D, "rms", rot=D // 2, gate=True, H2=2, layout="columns")


# ---------------------------------------------------------------------------
# delta rule: what is written over
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("T", [20, 64, 190])
@pytest.mark.parametrize("Hv,dv", [(2, 128), (48, 64)])
def test_delta_keys_that_come_again(T, Hv, dv):
    """Every second token asks with the key that it has just written over, by zeros with beta 1: o is far smaller than what
    cancels in it.  In chunks three sums follow each other beside a fourth, each of up to 16 steps of the tensor core that
    may lose 2^-23 of sums below four times the size: 2^-17 each, 2^-15 of scale size |q| together.  Token by token: sums of
    128 in fp32, 2^-18."""
    rng = rng_of(T, Hv)
    k = rng.standard_normal((T, 1, 128))
    k[1::2] = k[0::2]
    k = cuda(k / np.linalg.norm(k, axis=2, keepdims=True), BF)
    v = rng.standard_normal((T, Hv, dv))
    v[1::2] = 0
    v, g, beta = cuda(v, BF), torch.zeros((T, Hv), device="cuda"), torch.ones((T, Hv), device="cuda")
    st, o = cuda(rng.standard_normal((1, Hv, dv, 128))), torch.empty((T, Hv, dv), dtype=BF, device="cuda")
    ws = torch.empty(max(1, moe.moe_delta_workspace(T, 1, 1, Hv, 128, dv)), dtype=torch.uint8, device="cuda")
    want, state = np.zeros((T, Hv, dv)), f64(st)
    top = ora.delta(f64(k), f64(k), f64(v), f64(g), f64(beta), state, want, 1.0, ora.sequences(T, [0, T]))
    moe.moe_delta(k, k, v, g, beta, st, o, 1.0, workspace=ws, stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    near = 2.0 ** -8 * 1.01 * np.abs(want) + (2.0 ** -18 if T <= 24 else 2.0 ** -15) * top[:, :, None] * 1.01
    assert (np.abs(f64(o) - want) <= near).all(), (np.abs(f64(o) - want) / near).max()
    assert (np.abs(f64(st) - state) <= 2.0 ** -16 * top[-1][None, :, None, None]).all()


@pytest.mark.parametrize("lens", [[24, 7], [64, 300], [90] * 40])
def test_delta_o_is_rounded_once(lens):
    """All but few values are the exact ones rounded.  The sums before are off by about 2^-20 of scale size |q|, a value of o
    is about half of that and bf16's steps are 2^-8 of it or more: one value in 2^10 is next to a border that near.  Numbers
    of 11 bits in the sums, 2^-13 in the mean, would make it one in ten."""
    rng = rng_of(len(lens), lens[0])
    T, n = sum(lens), len(lens)
    q, k, v, g, beta = delta_inputs(rng, T, 2, 4, 128, 64)
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    st, o = cuda(rng.standard_normal((n, 4, 64, 128))), torch.empty((T, 4, 64), dtype=BF, device="cuda")
    want, ws = np.zeros((T, 4, 64)), f64(st)
    ora.delta(f64(q), f64(k), f64(v), f64(g), f64(beta), ws, want, 0.1, ora.sequences(T, off))
    run_delta(q, k, v, g, beta, st, o, 0.1, moe.make_seqs(n, ints(off)), T, n)
    torch.cuda.synchronize()
    other = int((o != cuda(want, BF)).sum())
    assert other <= o.numel() // 100, other / o.numel()


# ---------------------------------------------------------------------------
# refusals of real tensors (stand-ins go another way through the module)
# ---------------------------------------------------------------------------

def refused(word, call):
    with pytest.raises(ValueError, match=word):
        call()


def bf(*shape):
    return torch.zeros(shape, dtype=BF, device="cuda")


def fp(*shape):
    return torch.zeros(shape, device="cuda")


def test_conv_refuses_tensors():
    x, w, y, st = bf(5, 64), bf(64, 4), bf(5, 64), bf(2, 3, 64)
    seqs = moe.make_seqs(1, ints([0, 5]))

    def call(x=x, w=w, y=y, state=st, **more):
        return lambda: moe.moe_conv(x, w, y, seqs=seqs, state=state, **more)
    for bad in (bf(64, 5).T, bf(5, 64, 1), x.half(), x.cpu(), fp(5, 64)[:, ::2]):
        refused("x: expected|w is|y is", call(x=bad))
    refused("w is", call(w=bf(4, 64)))
    refused("w is", call(w=bf(64, 8)[:, :4]))
    refused("w: expected", call(w=w.cpu()))
    refused("y is", call(y=fp(5, 64)))
    refused("y is", call(y=bf(4, 64)))
    for bad in (bf(2, 64, 3), bf(2, 64, 3).transpose(1, 2), bf(2, 192), fp(2, 3, 64), st.cpu(), bf(2, 3, 128)[:, :, :64], bf(2, 4, 64)):
        refused("state: expected", call(state=bad))
    for bad in (bf(64), fp(63), fp(128)[::2], fp(64).cpu()):
        refused("bias: expected", call(bias=bad))
    call()()
    torch.cuda.synchronize()


def test_norm_refuses_tensors():
    cfg = moe.make_head_norm_config(rot_dim=8)
    x, pos, freq = bf(5, 3, 16), ints([0] * 5), fp(4)

    def call(x=x, y=x, pos=pos, inv_freq=freq, **more):
        return lambda: moe.moe_head_norm(cfg, x, y, pos=pos, inv_freq=inv_freq, **more)
    for bad in (bf(5, 48), bf(5, 16, 3).transpose(1, 2), x.half(), x.cpu()):
        refused("x: expected", call(x=bad))
    refused("y is", call(y=bf(5, 3, 8)))
    refused("y is", call(y=fp(5, 3, 16)))
    refused("gate is", call(gate=bf(5, 2, 16)))
    refused("weight: expected", call(weight=bf(16)))
    refused("weight: expected", call(weight=fp(15)))
    refused("x2 is", call(x2=bf(5, 3, 8), y2=bf(5, 3, 8)))
    refused("y2", call(x2=bf(5, 1, 16)))
    refused("pos: expected", call(pos=pos.long()))
    refused("pos: expected", call(pos=pos[:4]))
    refused("inv_freq: expected", call(inv_freq=freq.double()))
    with pytest.raises(moe.MoeError, match="rotation"):
        call(pos=None)()
    call()()
    torch.cuda.synchronize()


def test_delta_refuses_tensors():
    q, v, g, st = bf(5, 2, 8), bf(5, 4, 16), fp(5, 4), fp(2, 4, 16, 8)
    seqs = moe.make_seqs(1, ints([0, 5]), max_len=5)

    def call(q=q, k=q, v=v, g=g, beta=g, state=st, o=None, **more):
        return lambda: moe.moe_delta(q, k, v, g, beta, state, bf(5, 4, 16) if o is None else o, seqs=seqs, **more)
    refused("bfloat16", call(q=fp(5, 2, 8)))
    refused("side by side", call(q=bf(5, 2, 16)[:, :, :8]))
    refused("q: expected", call(q=bf(5, 8, 2).transpose(1, 2)))
    refused("k 5 x 2 x 16", call(k=bf(5, 2, 16)))
    refused("o is", call(o=bf(5, 2, 16)))
    refused("o: expected", call(o=bf(5, 4, 16).cpu()))
    for bad in (fp(4, 5), fp(4, 5).T, fp(20), bf(5, 4), g.cpu(), g.double(), fp(4, 4)):
        refused("g: expected", call(g=bad))
        refused("beta: expected", call(beta=bad))
    for bad in (fp(2, 4, 8, 16), fp(2, 4, 8, 16).transpose(2, 3), fp(2, 512), fp(2, 8, 16, 8), bf(2, 4, 16, 8), st.cpu()):
        refused("state: expected", call(state=bad))
    with pytest.raises(moe.MoeError, match="heads must"):
        call(q=bf(5, 3, 8), k=bf(5, 3, 8))()
    call()()
    torch.cuda.synchronize()
