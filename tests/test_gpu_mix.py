"""Convolution, head norms and gated delta rule on the GPU against their plain definitions in 64 bits.

Tolerances.  A result is rounded once to its type (half a step: 2^-8 of the value for bf16, 2^-24 for fp32).  What comes
before is fp32: n operations leave at most n 2^-24 of the magnitudes that are added.  silu is good to 2^-21 (two units
good to 2^-22).  The delta rule in chunks: operands have 22 bits, and a value of the state or an update is a sum of 64 or
128 products whose roundings are independent, each 2^-23 of its column's largest; four such sums follow each other in a
chunk, so their spread is about 4 sqrt(128) 2^-23 / 2 = 2^-18.5 of the largest state, and 2^-16 stands 5 of that away.
Decays shrink a chunk's error with the state."""
import numpy as np
import pytest

import _mix_oracle as ora
import int4_expert_streaming_gb300 as moe

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
F32, BF = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    moe.build()
    moe.load_library()


def rng_of(*key):
    return np.random.default_rng(abs(hash(key)) % (1 << 32) if not all(isinstance(k, int) for k in key) else list(key))


def cuda(a, dtype=F32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).cuda()


def f64(t):
    return t.detach().double().cpu().numpy()


def strided(t, pad, at=0):
    """The same values as a view whose rows stand `pad` elements further apart, `at` elements into its memory."""
    room = torch.full((t.shape[0], int(np.prod(t.shape[1:])) + pad), 7.0, dtype=t.dtype, device="cuda")
    view = room[:, at:at + int(np.prod(t.shape[1:]))].view(t.shape) if t.dim() == 2 else \
        room[:, at:at + int(np.prod(t.shape[1:]))].unflatten(1, t.shape[1:])
    view.copy_(t)
    return view


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


# lengths of a batch's sequences: none, one, around the convolution's pieces, around the delta rule's chunks and its bound
LENGTHS = [0, 1, 2, 3, 31, 32, 33, 0, 65, 5]


def batch_of(rng, lens, slots, padded=()):
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    slot = rng.permutation(slots)[:len(lens)].astype(np.int32)
    for s in padded:
        slot[s] = -1
    return off, slot, (rng.random(len(lens)) < 0.6).astype(np.int32)


# ---------------------------------------------------------------------------
# convolution
# ---------------------------------------------------------------------------

def check_conv(rng, dt, C, W, bias, act, lens, w_type=None, pad=(0, 0), at=0, state=True, padded=(), tail=3):
    T, slots = int(np.sum(lens)) + tail, len(lens) + 2
    off, slot, carry = batch_of(rng, lens, slots, padded)
    x = strided(cuda(rng.standard_normal((T, C)), dt), pad[0], at)
    y = strided(torch.full((T, C), 3.0, dtype=dt, device="cuda"), pad[1], at)
    w = cuda(rng.standard_normal((C, W)), w_type or dt)
    b = cuda(rng.standard_normal(C)) if bias else None
    st = cuda(rng.standard_normal((slots, W - 1, C)), dt) if state else None
    want, want_state = f64(y), f64(st) if state else None
    with np.errstate(over="ignore"):
        size = ora.conv(f64(x), f64(w), None if b is None else f64(b), act, want, want_state,
                        ora.sequences(T, off, slot, carry, slots if state else None))
    q = moe.make_seqs(len(lens), ints(off), ints(slot), ints(carry))
    moe.moe_conv(x, w, y, bias=b, act=moe.MOE_ACT_SILU if act else moe.MOE_ACT_NONE, seqs=q, state=st,
                 stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    # W products and a bias in fp32; silu's slope is below 1.1
    tol = HALF[dt] * np.abs(want) * 1.01 + (W + 1) * 2.0 ** -24 * size * 1.1 + (2.0 ** -21 * np.abs(want) if act else 0)
    assert (np.abs(f64(y) - want) <= tol + 1e-37).all()
    if state:
        assert np.array_equal(f64(st), want_state)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("C", [1, 8, 100, 1027, 2048])
def test_conv_over_ragged_batches(dt, W, C):
    check_conv(rng_of(W, C), dt, C, W, bias=C != 100, act=C % 2 == 0, lens=LENGTHS, padded=(4,))


@pytest.mark.parametrize("dt", [BF, F32])
def test_conv_strides_alignment_and_weights(dt):
    for pad, at in (((8, 16), 0), ((5, 3), 0), ((9, 9), 1), ((8, 8), 8)):
        check_conv(rng_of(pad[0], at), dt, 64, 4, True, True, [7, 40], pad=pad, at=at)
    check_conv(rng_of(1), dt, 64, 4, False, True, [7, 40], w_type=F32 if dt is BF else BF)


@pytest.mark.parametrize("state", [True, False])
def test_conv_decode_batch(state):
    """Every row a sequence, some of them padding."""
    rng = rng_of(5)
    n, C, W = 37, 256, 4
    slot = rng.permutation(40)[:n].astype(np.int32)
    slot[[3, 36]] = -1, 40  # no such slots
    if not state:
        slot[36] = -5
    x, w = cuda(rng.standard_normal((n, C)), BF), cuda(rng.standard_normal((C, W)), BF)
    y = torch.full((n, C), 3.0, dtype=BF, device="cuda")
    st = cuda(rng.standard_normal((40, W - 1, C)), BF) if state else None
    want, ws = f64(y), f64(st) if state else None
    ora.conv(f64(x), f64(w), None, True, want, ws, ora.sequences(n, None, slot, None, 40 if state else None))
    moe.moe_conv(x, w, y, seqs=moe.make_seqs(n, slot=ints(slot), max_len=1), state=st)
    torch.cuda.synchronize()
    assert (np.abs(f64(y) - want) <= 2.0 ** -7 * np.abs(want) + 1e-5).all()
    if state:
        assert np.array_equal(f64(st), ws)


def test_conv_of_one_sequence_in_pieces_is_the_whole():
    rng = rng_of(6)
    x, w = cuda(rng.standard_normal((150, 72)), BF), cuda(rng.standard_normal((72, 4)), BF)
    whole, parts = torch.empty_like(x), torch.empty_like(x)
    moe.moe_conv(x, w, whole)
    st = torch.zeros((1, 3, 72), dtype=BF, device="cuda")
    for lo, hi in ((0, 1), (1, 3), (3, 70), (70, 150)):
        moe.moe_conv(x[lo:hi], w, parts[lo:hi], state=st)
    torch.cuda.synchronize()
    assert torch.equal(whole, parts) and torch.equal(st[0], x[-3:])


def test_conv_infinities_stay_in_their_channel_and_window():
    x = torch.ones((9, 16), dtype=F32, device="cuda")
    x[4, 3], x[2, 5] = float("nan"), float("inf")
    w, y = torch.ones((16, 3), device="cuda"), torch.empty_like(x)
    moe.moe_conv(x, w, y, act=moe.MOE_ACT_NONE)
    bad = ~torch.isfinite(y)
    assert bad[4:7, 3].all() and bad[2:5, 5].all() and int(bad.sum()) == 6


# ---------------------------------------------------------------------------
# head norms
# ---------------------------------------------------------------------------

def check_norm(rng, dt, T, H, D, norm="rms", weight=True, offset=1.0, rot=0, halves=True, gate=False, H2=0, far=0,
               inplace=False, layout="plain", eps=1e-6):
    def make(h):
        t = cuda(rng.standard_normal((T, h, D)) * np.exp(rng.standard_normal((T, h, 1))), dt)
        if layout == "heads first":
            return t.transpose(0, 1).contiguous().transpose(0, 1)
        if layout == "columns":  # of a wider matrix
            return strided(t, 24, 8)
        if layout == "odd":
            return strided(t, 3, 1)
        return t
    x, x2 = make(H), make(H2) if H2 else None
    g = make(H) if gate else None
    y, y2 = (x, x2) if inplace else (torch.empty_like(x), torch.empty_like(x2) if H2 else None)
    w, w2 = (cuda(rng.standard_normal(D)) if weight else None for _ in range(2))
    pos = ints(far + rng.integers(0, 5000, T)) if rot else None
    freq = cuda(1e4 ** (-np.arange(rot // 2) / max(1, rot // 2))) if rot else None
    cfg = moe.make_head_norm_config({"rms": moe.MOE_NORM_RMS, "l2": moe.MOE_NORM_L2, "none": moe.MOE_NORM_NONE}[norm],
                                    eps, offset, rot, moe.MOE_ROT_HALVES if halves else moe.MOE_ROT_ADJACENT)
    args = [(x, w, g)] + ([(x2, w2, None)] if H2 else [])
    want = [ora.head_norm(f64(a), norm, eps, None if b is None else f64(b), offset, None if pos is None else
                          pos.cpu().numpy(), None if freq is None else freq.cpu().numpy(), rot, halves,
                          None if c is None else f64(c)) for a, b, c in args]
    moe.moe_head_norm(cfg, x, y, weight=w, gate=g, x2=x2, y2=y2, weight2=w2 if H2 else None, pos=pos, inv_freq=freq,
                      stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    for got, (z, size) in zip((y, y2), want):
        # the sum: at most 16 terms a thread and 5 steps (its root halves that), ten operations after it; an angle is good
        # to 2^-22 of a turn's part; silu to 2^-21
        tol = HALF[dt] * np.abs(z) * 1.01 + (24 * 2.0 ** -24 + (2.0 ** -21 if rot else 0) + (2.0 ** -21 if gate else 0)) * size
        assert (np.abs(f64(got) - z) <= tol + 1e-37).all()


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("D", [1, 2, 7, 8, 40, 64, 72, 128, 130, 256, 264, 512])
def test_norm_dimensions(dt, D):
    rng = rng_of(D)
    check_norm(rng, dt, 5, 3, D, "rms", rot=D // 2 * 2, halves=True)
    check_norm(rng, dt, 5, 3, D, "l2", weight=False, rot=D // 4 * 2, halves=False, H2=1)
    check_norm(rng, dt, 5, 2, D, "rms", gate=True, offset=0.0)


@pytest.mark.parametrize("T,H,H2", [(1, 1, 0), (1, 16, 16), (1, 32, 2), (3, 1, 1), (70, 1, 0), (613, 18, 2), (33, 5, 7)])
def test_norm_tokens_and_heads(T, H, H2):
    rng = rng_of(T, H)
    check_norm(rng, BF, T, H, 128, "rms", rot=64, H2=H2)
    check_norm(rng, F32, T, H, 64, "l2", weight=False, H2=H2, inplace=True)


def test_norm_many_heads_go_round():
    """More heads than the CTAs of one pass hold."""
    check_norm(rng_of(9), BF, 9001, 4, 64, "rms", rot=32, halves=False, H2=1)


@pytest.mark.parametrize("layout", ["heads first", "columns", "odd"])
@pytest.mark.parametrize("dt", [BF, F32])
def test_norm_layouts(layout, dt):
    for halves in (True, False):
        check_norm(rng_of(3), dt, 11, 4, 80, "rms", rot=48, halves=halves, gate=True, H2=2, layout=layout)
        check_norm(rng_of(4), dt, 11, 4, 80, "none", weight=False, rot=80, halves=halves, layout=layout, inplace=True)


@pytest.mark.parametrize("far", [1 << 20, (1 << 31) - 6000])
def test_norm_far_positions(far):
    check_norm(rng_of(8), F32, 17, 2, 128, "none", weight=False, rot=128, far=far)


def test_norm_of_zeros_and_negative_positions():
    x = torch.zeros((2, 3, 64), device="cuda")
    y = torch.empty_like(x)
    moe.moe_head_norm(moe.make_head_norm_config(moe.MOE_NORM_L2, eps=1e-6), x, y)
    assert torch.equal(y, x)
    rng = rng_of(2)
    v = cuda(rng.standard_normal((2, 1, 8)))
    out = torch.empty_like(v)
    freq = cuda(np.array([1.0, 0.25, 0.1, 1e-3]))
    moe.moe_head_norm(moe.make_head_norm_config(moe.MOE_NORM_NONE, rot_dim=8), v, out, pos=ints([-3, 0]), inv_freq=freq)
    want, size = ora.head_norm(f64(v), "none", 0, None, 0, np.array([-3, 0]), freq.cpu().numpy(), 8, True, None)
    assert (np.abs(f64(out) - want) <= 2.0 ** -20 * size).all()
    assert torch.equal(out[1], v[1])


def test_norm_positions_at_the_ends():
    """Both ways of reducing an angle, and the ends of int32.  Good to 2^-22 of a turn, 2 pi 2^-22 = 2^-19.3 in what turns,
    and ten roundings."""
    at = [-1 << 31, (1 << 31) - 1, -(1 << 24), 1 << 24, (1 << 24) + 1, -(1 << 24) - 1, 0, -1]
    freq = np.array([1.0, 0.73, 1e-3, 1e-9], np.float32)
    rng = rng_of(31)
    x = cuda(rng.standard_normal((len(at), 2, 8)))
    y = torch.empty_like(x)
    moe.moe_head_norm(moe.make_head_norm_config(moe.MOE_NORM_NONE, rot_dim=8), x, y, pos=ints(at), inv_freq=cuda(freq),
                      stream=torch.cuda.current_stream())
    want, size = ora.head_norm(f64(x), "none", 0, None, 0, np.array(at), freq, 8, True, None)
    assert (np.abs(f64(y) - want) <= 2.0 ** -19 * size).all()
    wild = np.array([1.5, 40.0, -3.0, 1000.0], np.float32)  # angles up to 2^30
    at = [1000, -70000, 1 << 20, 5]
    moe.moe_head_norm(moe.make_head_norm_config(moe.MOE_NORM_NONE, rot_dim=8), x[:4], y[:4], pos=ints(at), inv_freq=cuda(wild),
                      stream=torch.cuda.current_stream())
    want, size = ora.head_norm(f64(x[:4]), "none", 0, None, 0, np.array(at), wild, 8, True, None)
    assert (np.abs(f64(y[:4]) - want) <= 2.0 ** -19 * size).all()


# ---------------------------------------------------------------------------
# gated delta rule
# ---------------------------------------------------------------------------

def delta_inputs(rng, T, Hk, Hv, dk, dv, layout="side by side"):
    a = rng.standard_normal((T, Hk, dk)) + rng.standard_normal((Hk, dk))
    b = rng.standard_normal((T, Hk, dk))
    q, k = (t / np.linalg.norm(t, axis=2, keepdims=True) for t in (b, a))
    v = rng.standard_normal((T, Hv, dv))
    g = -np.exp(rng.uniform(-6, 1, (T, Hv)))
    beta = rng.random((T, Hv))
    q, k, v = (cuda(t, BF) for t in (q, k, v))
    if layout == "odd":
        q, k, v = (strided(t, 3, 1) for t in (q, k, v))
    elif layout == "side by side":
        room = torch.cat([t.flatten(1) for t in (q, k, v)], 1)
        q, k, v = (t.unflatten(1, s) for t, s in zip(room.split([Hk * dk, Hk * dk, Hv * dv], 1),
                                                      ((Hk, dk), (Hk, dk), (Hv, dv))))
    return q, k, v, cuda(g), cuda(beta)


def run_delta(q, k, v, g, beta, state, o, scale, seqs, T, n, max_len=0, stream=None):
    Hk, dk, Hv, dv = q.shape[1], q.shape[2], v.shape[1], v.shape[2]
    ws = torch.empty(max(1, moe.moe_delta_workspace(T, n, Hk, Hv, dk, dv, max_len)), dtype=torch.uint8, device="cuda")
    moe.moe_delta(q, k, v, g, beta, state, o, scale=scale, seqs=seqs, workspace=ws,
                  stream=stream or torch.cuda.current_stream())
    return ws


def check_delta(rng, lens, Hk=2, Hv=4, dk=64, dv=64, layout="side by side", padded=(), change=None, state=True, tail=2,
                max_len=0, scale=0.3):
    T, slots, n = int(np.sum(lens)) + tail, len(lens) + 2, len(lens)
    off, slot, carry = batch_of(rng, lens, slots, padded)
    q, k, v, g, beta = delta_inputs(rng, T, Hk, Hv, dk, dv, layout)
    if change:
        change(q, k, v, g, beta)
    st = cuda(0.5 * rng.standard_normal((slots, Hv, dv, dk))) if state else None
    if state:
        st[slots - 1 if (slots - 1) not in slot else 0] = st[slots - 1 if (slots - 1) not in slot else 0]
        for s in range(n):
            if not carry[s] and slot[s] >= 0 and lens[s]:
                st[int(slot[s])] = float("nan")  # not to be read
    o = torch.full((T, Hv, dv), 3.0, dtype=BF, device="cuda")
    if layout == "odd":
        o = strided(o, 5, 1)
    want, ws = f64(o), f64(st) if state else None
    top = ora.delta(f64(q), f64(k), f64(v), f64(g), f64(beta), ws, want, scale,
                    ora.sequences(T, off, slot, carry, slots if state else None))
    seqs = moe.make_seqs(n, ints(off), ints(slot), ints(carry), max_len)
    run_delta(q, k, v, g, beta, st, o, scale, seqs, T, n, max_len)
    torch.cuda.synchronize()
    got = f64(o)
    qn = np.abs(f64(q)).sum(2).repeat(Hv // Hk, 1)
    # o: its rounding, and what enters by 11 bits: S, the updates and the products of q and k, each 2^-12 of its
    # column's or row's largest, over sums of 128 and 64 terms of which the roundings are independent: sqrt(128) 2^-12 / 2 of
    # scale max|S| |q|, of which 2^-8 is more than 5 times the spread
    near = 2.0 ** -8 * np.abs(want) * 1.01 + (2.0 ** -9 * scale * top * np.linalg.norm(f64(q), axis=2).repeat(Hv // Hk, 1))[:, :, None]
    assert np.isfinite(got).all() and qn.shape[1] == Hv
    assert (np.abs(got - want) <= near).all(), np.max(np.abs(got - want) / near)
    if state:
        gs = f64(st)
        for s, (lo, hi) in enumerate(zip(off[:-1], off[1:])):
            if slot[s] >= 0 and hi > lo:
                a, b = gs[slot[s]], ws[slot[s]]
                tol = 2.0 ** -16 * top[hi - 1][:, None, None]
                assert (np.abs(a - b) <= tol + 1e-30).all(), (s, hi - lo, np.max(np.abs(a - b) / tol))
        unused = [i for i in range(slots) if i not in slot[[j for j in range(n) if lens[j]]]]
        assert np.array_equal(gs[unused], ws[unused], equal_nan=True)
    return o, st


@pytest.mark.parametrize("dk,dv", [(8, 8), (64, 64), (64, 128), (128, 64), (128, 128), (96, 40), (72, 104)])
def test_delta_token_by_token(dk, dv):
    check_delta(rng_of(dk, dv), [1, 0, 2, 24, 5, 1], dk=dk, dv=dv, padded=(2,))
    check_delta(rng_of(dv, dk), [1, 3, 7], Hk=1, Hv=3, dk=dk, dv=dv, max_len=24)


@pytest.mark.parametrize("dk,dv", [(8, 8), (64, 64), (64, 128), (128, 64), (128, 128), (96, 40), (72, 104)])
def test_delta_in_chunks(dk, dv):
    check_delta(rng_of(dk, dv, 1), [25, 63, 0, 64, 3, 65, 200], dk=dk, dv=dv, padded=(4,))


@pytest.mark.parametrize("Hk,Hv", [(1, 1), (1, 4), (2, 2), (3, 9), (16, 32)])
def test_delta_shared_heads(Hk, Hv):
    check_delta(rng_of(Hk, Hv), [70, 2, 130], Hk=Hk, Hv=Hv, dk=64, dv=32)


@pytest.mark.parametrize("layout", ["plain", "odd"])
def test_delta_layouts(layout):
    check_delta(rng_of(4), [70, 2, 130, 1], dk=128, dv=72, layout=layout)


@pytest.mark.parametrize("dk,dv,Hk,Hv,layout", [(128, 128, 8, 16, "plain"), (72, 104, 8, 16, "odd"), (64, 40, 16, 32, "plain"),
                                                (64, 64, 16, 32, "odd")])
def test_delta_many_sequences_and_heads(dk, dv, Hk, Hv, layout):
    """More of both than there are SMs for blocks of 32 columns."""
    check_delta(rng_of(dk, Hv), [70, 2, 130, 64, 0, 29], Hk=Hk, Hv=Hv, dk=dk, dv=dv, layout=layout, padded=(3,))


def test_delta_without_state():
    check_delta(rng_of(5), [70, 2, 130, 1], dk=64, dv=72, state=False, padded=(2,))


def test_delta_long_run():
    """Many chunks: the state's rounding does not pile up."""
    check_delta(rng_of(6), [1500], Hk=1, Hv=2, dk=128, dv=128)


def gates(value, where):
    def change(q, k, v, g, beta):
        g[where] = value
    return change


@pytest.mark.parametrize("name", ["cleared", "no decay", "strong decay", "no update", "full update", "zero keys", "large v",
                                  "small v", "sizes"])
def test_delta_gates_and_sizes(name):
    def change(q, k, v, g, beta):
        if name == "cleared":
            g[5::31] = -float("inf")
        elif name == "no decay":
            g.zero_()
        elif name == "strong decay":
            g.fill_(-9.0)
        elif name == "no update":
            beta.zero_()
        elif name == "full update":
            beta.fill_(1.0)
        elif name == "zero keys":
            k[::3] = 0
            q[1::5] = 0
        elif name == "large v":
            v.mul_(2.0 ** 60)
        elif name == "small v":
            v.mul_(2.0 ** -60)
        elif name == "sizes":  # keys and queries of very different lengths
            k[::2].mul_(2.0 ** -20)
            q[::2].mul_(2.0 ** 20)
    check_delta(rng_of(7), [9, 150, 64], dk=128, dv=64, change=change)


def test_delta_does_not_depend_on_its_batch():
    rng = rng_of(11)
    lens = [150, 24, 1, 25, 700, 30, 64, 65, 2, 128, 40, 90]
    T, n = sum(lens), len(lens)
    q, k, v, g, beta = delta_inputs(rng, T, 2, 4, 128, 128)
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    st = cuda(rng.standard_normal((n, 4, 128, 128)))
    st1, o = st.clone(), torch.empty((T, 4, 128), dtype=BF, device="cuda")
    run_delta(q, k, v, g, beta, st, o, 0.1, moe.make_seqs(n, ints(off)), T, n)
    for s in range(n):
        lo, hi = int(off[s]), int(off[s + 1])
        o1 = torch.empty((hi - lo, 4, 128), dtype=BF, device="cuda")
        run_delta(q[lo:hi], k[lo:hi], v[lo:hi], g[lo:hi], beta[lo:hi], st1[s:s + 1], o1, 0.1,
                  None if s % 2 else moe.make_seqs(1, ints([0, hi - lo])), hi - lo, 1)
        torch.cuda.synchronize()
        assert torch.equal(o1, o[lo:hi]) and torch.equal(st1[s], st[s])


def test_delta_values_that_are_not_finite_stay_in_their_head():
    """NaN in v of one head, infinity in a key that two heads share: the other heads and sequences keep every bit."""
    rng = rng_of(15)
    lens = [100, 70, 10, 40]
    T, n = sum(lens), len(lens)
    q, k, v, g, beta = (t.contiguous() for t in delta_inputs(rng, T, 2, 4, 64, 64))
    seqs = moe.make_seqs(n, ints(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)))
    start = cuda(rng.standard_normal((n, 4, 64, 64)))
    results = []
    for spoilt in (False, True):
        if spoilt:
            v[50, 1, 3] = float("nan")
            k[120, 0, 5] = float("inf")
            g[185, 3] = float("nan")  # of the last sequence
        st, o = start.clone(), torch.zeros((T, 4, 64), dtype=BF, device="cuda")
        run_delta(q, k, v, g, beta, st, o, 0.1, seqs, T, n)
        torch.cuda.synchronize()
        results.append((o, st))
    (o, st), (o1, st1) = results
    for s, (lo, hi, heads) in enumerate([(0, 100, [0, 2, 3]), (100, 170, [2, 3]), (170, 180, [0, 1, 2, 3]), (180, 220, [0, 1, 2])]):
        assert torch.equal(o[lo:hi, heads], o1[lo:hi, heads]) and torch.equal(st[s, heads], st1[s, heads])
    assert o1[50:100, 1, 3].isnan().all() and st1[0, 1, 3].isnan().all()
    assert not o1[121:170, :2].isfinite().any() and not o1[185:220, 3].isfinite().any()


def test_delta_prefill_then_decode_is_the_whole():
    rng = rng_of(12)
    T = 200
    q, k, v, g, beta = delta_inputs(rng, T, 1, 2, 128, 128)
    whole, parts = (torch.empty((T, 2, 128), dtype=BF, device="cuda") for _ in range(2))
    st, st1 = (torch.zeros((1, 2, 128, 128), device="cuda") for _ in range(2))
    run_delta(q, k, v, g, beta, st, whole, 1.0, None, T, 1)
    for lo, hi in [(0, 130)] + [(t, t + 1) for t in range(130, 180)] + [(180, 184), (184, 200)]:
        run_delta(q[lo:hi], k[lo:hi], v[lo:hi], g[lo:hi], beta[lo:hi], st1, parts[lo:hi], 1.0, None, hi - lo, 1)
    torch.cuda.synchronize()
    want = np.full((T, 2, 128), 0.0)
    top = ora.delta(*(f64(t) for t in (q, k, v, g, beta)), None, want, 1.0, ora.sequences(T, [0, T]))
    assert np.abs(f64(st) - f64(st1)).max() <= 2.0 ** -15 * top.max()
    for got in (whole, parts):
        assert (np.abs(f64(got) - want) <= 2.0 ** -8 * np.abs(want) * 1.01 + 2.0 ** -9 * top.max()).all()


# ---------------------------------------------------------------------------
# streams, graphs, and all of it together
# ---------------------------------------------------------------------------

def test_graph_replays_with_new_lists():
    """One captured batch whose lists change between replays, as a server's decode and prefill steps do."""
    rng = rng_of(13)
    n, T, C = 4, 160, 2 * 2 * 64 + 4 * 64
    st = cuda(0.3 * rng.standard_normal((6, 4, 64, 64)))
    cs = cuda(rng.standard_normal((6, 3, C)), BF)
    x, w = cuda(rng.standard_normal((T, C)), BF), cuda(0.5 * rng.standard_normal((C, 4)), BF)
    g, beta = cuda(-rng.random((T, 4))), cuda(rng.random((T, 4)))
    off, slot, carry = ints([0, 20, 20, 90, 160]), ints([0, 1, 2, 3]), ints([1, 1, 0, 1])
    seqs = moe.make_seqs(n, off, slot, carry)
    ws = torch.empty(moe.moe_delta_workspace(T, n, 2, 4, 64, 64), dtype=torch.uint8, device="cuda")
    cfg = moe.make_head_norm_config(moe.MOE_NORM_L2)

    def step(y, o, cs, st, stream):
        q, k, v = y.split([128, 128, 256], 1)
        q, k, v = q.unflatten(1, (2, 64)), k.unflatten(1, (2, 64)), v.unflatten(1, (4, 64))
        moe.moe_conv(x, w, y, seqs=seqs, state=cs, stream=stream)
        moe.moe_head_norm(cfg, q, q, x2=k, y2=k, stream=stream)
        moe.moe_delta(q, k, v, g, beta, st, o, scale=0.1, seqs=seqs, workspace=ws, stream=stream)
        moe.moe_head_norm(moe.make_head_norm_config(moe.MOE_NORM_RMS), o, o, gate=v, stream=stream)

    def room():
        return torch.zeros((T, C), dtype=BF, device="cuda"), torch.zeros((T, 4, 64), dtype=BF, device="cuda")
    y, o = room()
    start = cs.clone(), st.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(y, o, cs, st, side)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(y, o, cs, st, torch.cuda.current_stream())
    for lists in (([0, 20, 20, 90, 160], [0, 1, 2, 3], [1, 1, 0, 1]), ([0, 1, 2, 3, 4], [5, 4, -1, 0], [1, 0, 1, 1]),
                  ([0, 100, 101, 118, 150], [3, 2, 1, 0], [0, 1, 1, 1])):
        for t, l in zip((off, slot, carry), lists):
            t.copy_(ints(l))
        cs.copy_(start[0])
        st.copy_(start[1])
        y.zero_()
        o.zero_()
        graph.replay()
        y1, o1 = room()
        cs1, st1 = start[0].clone(), start[1].clone()
        step(y1, o1, cs1, st1, torch.cuda.current_stream())
        torch.cuda.synchronize()
        for a, b in ((y, y1), (o, o1), (cs, cs1), (st, st1)):
            assert torch.equal(a, b)


def test_a_run_of_all_against_the_definitions():
    """Convolution, norms to unit length, delta rule, gated norm: two prompts and then five single tokens of each."""
    rng = rng_of(14)
    Hk, Hv, D = 2, 4, 64
    C = (2 * Hk + Hv) * D
    lens = [90, 21]
    w = cuda(0.5 * rng.standard_normal((C, 4)), BF)
    weight = cuda(1 + 0.1 * rng.standard_normal(D))
    cs, st = torch.zeros((2, 3, C), dtype=BF, device="cuda"), torch.zeros((2, Hv, D, D), device="cuda")
    cs64, st64 = f64(cs), f64(st)
    unit, gated = moe.make_head_norm_config(moe.MOE_NORM_L2), moe.make_head_norm_config(moe.MOE_NORM_RMS)
    stream = torch.cuda.current_stream()
    for step in range(6):
        n_tok = lens if step == 0 else [1, 1]
        T = sum(n_tok)
        off = np.concatenate([[0], np.cumsum(n_tok)]).astype(np.int32)
        x, z = cuda(rng.standard_normal((T, C)), BF), cuda(rng.standard_normal((T, Hv, D)), BF)
        g, beta = cuda(-0.3 * rng.random((T, Hv))), cuda(rng.random((T, Hv)))
        seqs = moe.make_seqs(2, ints(off), carry=ints([step > 0] * 2), max_len=max(n_tok))
        y, o = torch.empty_like(x), torch.empty((T, Hv, D), dtype=BF, device="cuda")
        moe.moe_conv(x, w, y, seqs=seqs, state=cs, stream=stream)
        q, k, v = (t.unflatten(1, (-1, D)) for t in y.split([Hk * D, Hk * D, Hv * D], 1))
        qn, kn = torch.empty_like(q), torch.empty_like(k)
        moe.moe_head_norm(unit, q, qn, x2=k, y2=kn, stream=stream)
        run_delta(qn, kn, v, g, beta, st, o, D ** -0.5, seqs, T, 2, max(n_tok))
        out = torch.empty_like(o)
        moe.moe_head_norm(gated, o, out, weight=weight, gate=z, stream=stream)
        torch.cuda.synchronize()
        # each operator against its definition on what it was given
        y64 = np.zeros((T, C))
        ora.conv(f64(x), f64(w), None, True, y64, cs64, ora.sequences(T, off, None, [step > 0] * 2))
        assert (np.abs(f64(y) - y64) <= 2.0 ** -7 * np.abs(y64) + 1e-5).all()
        for a, b in ((q, qn), (k, kn)):
            want, size = ora.head_norm(f64(a), "l2", 1e-6, None, 0, None, None, 0, True, None)
            assert (np.abs(f64(b) - want) <= 2.0 ** -8 * 1.01 * np.abs(want) + 2.0 ** -19 * size).all()
        o64 = np.zeros((T, Hv, D))
        top = ora.delta(f64(qn), f64(kn), f64(v), f64(g), f64(beta), st64, o64, D ** -0.5,
                        ora.sequences(T, off, None, [step > 0] * 2))
        assert (np.abs(f64(o) - o64) <= 2.0 ** -8 * 1.01 * np.abs(o64) + 2.0 ** -9 * D ** -0.5 * top[:, :, None]).all()
        assert np.abs(f64(st) - st64).max() <= 2.0 ** -15 * top.max()
        want, size = ora.head_norm(f64(o), "rms", 1e-6, f64(weight), 0, None, None, 0, True, f64(z))
        assert (np.abs(f64(out) - want) <= 2.0 ** -8 * 1.01 * np.abs(want) + 2.0 ** -18 * size).all()


# ---------------------------------------------------------------------------
# places beyond 2^31 elements; calls side by side
# ---------------------------------------------------------------------------

def test_states_and_rows_far_behind():
    """Slots and rows more than 2^31 elements from their tensor's start give what near ones give."""
    rng = rng_of(16)
    stream = torch.cuda.current_stream()
    q, k, v, g, beta = delta_inputs(rng, 72, 1, 1, 128, 128)
    big = torch.empty((132000, 1, 128, 128), device="cuda")  # 8.7 GB, of which two slots are touched
    small = cuda(rng.standard_normal((2, 1, 128, 128)))
    big[[131999, 131072]] = small
    off = ints([0, 70, 72])
    o, o1 = (torch.empty((72, 1, 128), dtype=BF, device="cuda") for _ in range(2))
    run_delta(q, k, v, g, beta, small, o, 0.1, moe.make_seqs(2, off), 72, 2)
    run_delta(q, k, v, g, beta, big, o1, 0.1, moe.make_seqs(2, off, ints([131999, 131072])), 72, 2)
    assert torch.equal(o, o1) and torch.equal(small, big[[131999, 131072]])
    del big

    w = cuda(rng.standard_normal((64, 4)), BF)
    room = torch.empty(2 * (1 << 31) + 4096, dtype=BF, device="cuda")  # two rows 2^31 elements from one another, and slots
    far = room.as_strided((3, 64), ((1 << 31), 1))
    x = cuda(rng.standard_normal((3, 64)), BF)
    far.copy_(x)
    slots = torch.empty((11200000, 3, 64), dtype=BF, device="cuda")  # 2^31 elements and more
    near = cuda(rng.standard_normal((1, 3, 64)), BF)
    slots[11199999:] = near
    y, y1 = torch.empty_like(x), torch.empty_like(x)
    moe.moe_conv(x, w, y, seqs=moe.make_seqs(1, ints([0, 3])), state=near, stream=stream)
    moe.moe_conv(far, w, y1, seqs=moe.make_seqs(1, ints([0, 3]), ints([11199999])), state=slots, stream=stream)
    assert torch.equal(y, y1) and torch.equal(near[0], slots[11199999])
    step, step1 = torch.empty_like(x), torch.empty_like(x)  # each row a sequence
    moe.moe_conv(x, w, step, seqs=moe.make_seqs(3), stream=stream)
    moe.moe_conv(far, w, step1, seqs=moe.make_seqs(3), stream=stream)
    assert torch.equal(step, step1)
    cfg = moe.make_head_norm_config(moe.MOE_NORM_RMS)
    n, n1 = (torch.empty((3, 1, 64), dtype=BF, device="cuda") for _ in range(2))
    moe.moe_head_norm(cfg, x[:, None], n, stream=stream)
    moe.moe_head_norm(cfg, far[:, None], n1, stream=stream)
    assert torch.equal(n, n1)
    moe.moe_head_norm(cfg, far[:, None], far[:, None], stream=stream)  # and written there
    assert torch.equal(far, n[:, 0])


def test_calls_side_by_side_on_two_streams():
    """Calls of two batches at once, each with its workspace, and two captured graphs at once: every bit as alone."""
    rng = rng_of(17)
    jobs = []
    for T, Hk, Hv, dk, dv in ((900, 4, 8, 128, 128), (700, 2, 8, 64, 96)):
        q, k, v, g, beta = delta_inputs(rng, T, Hk, Hv, dk, dv)
        ws = torch.empty(moe.moe_delta_workspace(T, 2, Hk, Hv, dk, dv), dtype=torch.uint8, device="cuda")
        st, o = torch.zeros((2, Hv, dv, dk), device="cuda"), torch.empty((T, Hv, dv), dtype=BF, device="cuda")
        seqs = moe.make_seqs(2, ints([0, T // 3, T]), carry=ints([0, 0]))

        def call(stream, a=(q, k, v, g, beta, st, o), kw={"scale": 0.1, "seqs": seqs, "workspace": ws}):
            moe.moe_delta(*a, **kw, stream=stream)
        call(torch.cuda.current_stream())
        torch.cuda.synchronize()
        jobs.append((call, torch.cuda.Stream(), o, st, o.clone(), st.clone()))
    graphs = []
    for call, stream, *_ in jobs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=stream):
            call(torch.cuda.current_stream())
    for replay in (False, True):
        for _, _, o, st, _, _ in jobs:
            o.zero_()
            st.zero_()
        torch.cuda.synchronize()
        for _ in range(5):
            for (call, stream, *_), graph in zip(jobs, graphs):
                with torch.cuda.stream(stream):
                    graph.replay() if replay else call(stream)
        torch.cuda.synchronize()
        for _, _, o, st, o0, st0 in jobs:
            assert torch.equal(o, o0) and torch.equal(st, st0)


def test_a_state_without_slots():
    """Every sequence is left out, and a batch without a slot list is refused as by the C call."""
    x, w = torch.ones((3, 8), dtype=BF, device="cuda"), torch.ones((8, 2), dtype=BF, device="cuda")
    y, none = torch.full_like(x, 5), torch.empty((0, 1, 8), dtype=BF, device="cuda")
    moe.moe_conv(x, w, y, seqs=moe.make_seqs(3, slot=ints([0, 1, -1])), state=none)
    moe.moe_conv(x, w, y, seqs=moe.make_seqs(1, ints([0, 3]), slot=ints([0])), state=none)
    torch.cuda.synchronize()
    assert (y == 5).all()
    with pytest.raises(moe.MoeError, match="0 slots"):
        moe.moe_conv(x, w, y, seqs=moe.make_seqs(3), state=none)
    q, g = torch.ones((30, 1, 8), dtype=BF, device="cuda"), torch.zeros((30, 1), device="cuda")
    o, none = torch.full_like(q, 5), torch.empty((0, 1, 8, 8), device="cuda")
    ws = torch.empty(moe.moe_delta_workspace(30, 1, 1, 1, 8, 8), dtype=torch.uint8, device="cuda")
    moe.moe_delta(q, q, q, g, g, none, o, seqs=moe.make_seqs(1, ints([0, 30]), slot=ints([0])), workspace=ws)
    torch.cuda.synchronize()
    assert (o == 5).all()
    with pytest.raises(moe.MoeError, match="0 slots"):
        moe.moe_delta(q, q, q, g, g, none, o, workspace=ws)
