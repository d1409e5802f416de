"""Convolution, head norms and gated delta rule as far as they go without a GPU: sizes, refusals (nothing is launched for
a bad argument), the Python module's checks on stand-ins for tensors, and the plain definitions' own properties."""
import ctypes

import numpy as np
import pytest

import _mix_oracle as ora
import int4_expert_streaming_gb300 as moe


@pytest.fixture(scope="module")
def lib():
    moe.build()
    return moe.load_library()


P = 1 << 20  # an address that is never read: every call here is refused before any GPU work


def refused(rc, word):
    assert rc == moe.MOE_EINVAL
    assert word in moe.moe_last_error(None), moe.moe_last_error(None)


def seqs(n, offsets=P, slot=None, carry=None, max_len=0):
    return ctypes.byref(moe.moe_seqs(offsets, slot, carry, n, max_len))


def test_conv_refuses_bad_arguments(lib):
    def call(q=None, x=P, kind=0, ld=64, T=4, C=64, w=P, w_kind=0, W=4, act=2, state=P, slots=8, y=2 * P, y_ld=64):
        return lib.moe_conv(q, x, kind, ld, T, C, w, w_kind, W, None, act, state, slots, y, y_ld, None)
    refused(call(kind=2), "type")
    refused(call(w_kind=-1), "type")
    refused(call(T=-1), "T=")
    refused(call(T=1 << 31), "T=")
    refused(call(C=0), "channels")
    refused(call(C=(1 << 22) + 1), "channels")
    refused(call(W=1), "width")
    refused(call(W=5), "width")
    refused(call(act=1), "activation")
    refused(call(ld=63), "stride")
    refused(call(y_ld=63), "stride")
    refused(call(x=None), "required")
    refused(call(w=None), "required")
    refused(call(y=None), "required")
    refused(call(y=P), "may not be x")
    refused(call(slots=0), "slots")
    refused(call(slots=-1), "slots")
    refused(call(q=seqs(-1)), "n=-1")
    refused(call(q=seqs((1 << 20) + 1)), "n=")
    refused(call(q=seqs(3, offsets=None)), "every row")
    refused(call(q=seqs(9), slots=8), "slots")
    refused(call(q=seqs(2, max_len=-1)), "max_len")
    assert call(T=0, x=None, w=None, y=None) == moe.MOE_OK
    assert call(q=seqs(0)) == moe.MOE_OK


def test_head_norm_refuses_bad_arguments(lib):
    def heads(x=P, y=P, ld=256, head=64, n=4, kind=0, **k):
        t = moe.moe_heads(x, y, k.get("gate"), None, ld, head, k.get("y_ld", ld), k.get("y_head", head), k.get("gate_ld", ld),
                          k.get("gate_head", head), n, kind)
        return ctypes.byref(t)

    def call(a=None, b=None, T=3, pos=P, freq=P, dim=64, norm=1, rot=32, pairs=0, eps=1e-6):
        cfg = moe.moe_head_norm_config(dim, norm, rot, pairs, eps, 0.0)
        return lib.moe_head_norm(ctypes.byref(cfg), a or heads(), b, pos, freq, T, None)
    refused(lib.moe_head_norm(None, heads(), None, P, P, 3, None), "required")
    refused(lib.moe_head_norm(ctypes.byref(moe.moe_head_norm_config(64, 1, 0, 0, 0, 0)), None, None, P, P, 3, None), "required")
    refused(call(dim=0), "dim")
    refused(call(dim=513), "dim")
    refused(call(norm=3), "norm")
    refused(call(rot=33), "rot_dim")
    refused(call(rot=66), "rot_dim")
    refused(call(rot=-2), "rot_dim")
    refused(call(pairs=2), "pairs")
    refused(call(eps=-1.0), "eps")
    refused(call(eps=float("nan")), "eps")
    refused(call(T=-1), "T=")
    refused(call(T=1 << 31), "T=")
    refused(call(pos=None), "rotation")
    refused(call(freq=None), "rotation")
    refused(call(a=heads(kind=2)), "type")
    refused(call(a=heads(n=0)), "heads")
    refused(call(a=heads(n=32769)), "heads")
    refused(call(a=heads(x=None)), "required")
    refused(call(a=heads(y=None)), "required")
    refused(call(a=heads(y=2 * P, y_head=63)), "shorter")
    refused(call(a=heads(y=2 * P, y_ld=63)), "shorter")
    refused(call(a=heads(head=-64)), "negative")
    refused(call(a=heads(gate=P, gate_ld=-1)), "negative")
    refused(call(a=heads(y_ld=512)), "other strides")
    refused(call(b=heads(kind=1, y=2 * P, x=2 * P)), "differ in type")
    refused(call(b=heads()), "same y")
    refused(call(a=heads(n=32768), T=(1 << 31) - 1), "2^33")
    assert call(a=heads(x=None, y=None), T=0, pos=None, freq=None) == moe.MOE_OK


def test_delta_refuses_bad_arguments(lib):
    def call(q=None, Hk=2, Hv=4, dk=64, dv=64, T=40, ld=(128, 128, 256, 256), ptr=(P, P, P, P, P), state=P, slots=4, o=P, ws=P,
             size=1 << 40):
        cfg = moe.moe_delta_config(Hk, Hv, dk, dv, 1.0)
        return lib.moe_delta(ctypes.byref(cfg), q, ptr[0], ld[0], ptr[1], ld[1], ptr[2], ld[2], ptr[3], ptr[4], state, slots, o,
                             ld[3], T, ws, size, None)
    for k in ({"Hk": 0}, {"Hv": 3}, {"Hv": 1}, {"Hk": 1, "Hv": 1025}, {"dk": 0}, {"dk": 68}, {"dk": 136}, {"dv": 4}, {"dv": 136}):
        refused(call(**k), "heads must")
    refused(lib.moe_delta(None, None, P, 1, P, 1, P, 1, P, P, P, 1, P, 1, 4, None, 0, None), "heads must")
    for i in range(4):
        refused(call(ld=tuple(v - (i == j) for j, v in enumerate((128, 128, 256, 256)))), "stride")
    refused(call(T=-1), "T=")
    refused(call(state=P + 8), "aligned")
    refused(call(slots=0), "slots")
    refused(call(slots=1 << 31), "slots")
    for i in range(5):
        refused(call(ptr=tuple(None if i == j else P for j in range(5))), "required")
    refused(call(o=None), "required")
    refused(call(q=seqs(5)), "slots")
    refused(call(q=seqs(5, offsets=None)), "every row")
    need = moe.moe_delta_workspace(40, 1, 2, 4, 64, 64)
    refused(call(size=need - 1), "workspace")
    refused(call(ws=None), "workspace")
    refused(call(ws=P + 64), "workspace")
    refused(call(q=seqs(2, max_len=25), size=0), "workspace")
    assert call(T=0, ptr=(None,) * 5, o=None, ws=None, size=0) == moe.MOE_OK
    assert call(q=seqs(0), ws=None, size=0) == moe.MOE_OK


def test_delta_workspace():
    w = moe.moe_delta_workspace
    assert w(24, 1, 16, 32, 128, 128) == 0 and w(4096, 4096, 16, 32, 128, 128, 1) == 0 and w(4096, 300, 16, 32, 128, 128, 24) == 0
    one = w(128, 1, 1, 1, 64, 64) - w(64, 1, 1, 1, 64, 64)
    assert 0 < one and one % 128 == 0
    more = w(25, 3, 1, 1, 64, 64) - w(25, 1, 1, 1, 64, 64)  # a chunk for each 64 rows, and one for each sequence
    assert 2 * one <= more <= 2 * (one + 64)
    assert one <= w(25, 1, 1, 1, 64, 64) <= one + 64
    assert w((1 << 31) - 1, 1, 16, 32, 128, 128) > 1 << 32
    for bad in ((-1, 1, 1, 1, 64, 64), (64, -1, 1, 1, 64, 64), (64, 1, 2, 3, 64, 64), (64, 1, 1, 1, 65, 64), (1 << 31, 1, 1, 1, 64, 64)):
        assert w(*bad) == 0


# ---------------------------------------------------------------------------
# the Python module, on stand-ins for CUDA tensors
# ---------------------------------------------------------------------------

class Tensor:
    is_cuda = True

    def __init__(self, dtype, *shape, device=0, stride=None):
        self.dtype, self.shape, self.at = dtype, shape, device
        self.steps = stride or tuple(int(np.prod(shape[i + 1:])) for i in range(len(shape)))

    def get_device(self):
        return self.at

    def stride(self):
        return self.steps

    def is_contiguous(self):
        return self.steps == tuple(int(np.prod(self.shape[i + 1:])) for i in range(len(self.shape)))

    def numel(self):
        return int(np.prod(self.shape))

    def data_ptr(self):
        return 1 << 20


def test_python_module_refuses_tensors_that_do_not_fit(lib):
    torch = pytest.importorskip("torch")
    F, B, I = torch.float32, torch.bfloat16, torch.int32
    x, w, y = Tensor(B, 5, 64), Tensor(B, 64, 4), Tensor(B, 5, 64)

    def no(call, word):
        with pytest.raises(ValueError, match=word):
            call()
    no(lambda: moe.moe_conv(x, Tensor(B, 65, 4), y), "w is")
    no(lambda: moe.moe_conv(x, Tensor(B, 64, 4, stride=(8, 1)), y), "w is")
    no(lambda: moe.moe_conv(x, w, Tensor(F, 5, 64)), "y is")
    no(lambda: moe.moe_conv(x, w, Tensor(B, 4, 64)), "y is")
    no(lambda: moe.moe_conv(x, w, y, bias=Tensor(F, 63)), "bias")
    no(lambda: moe.moe_conv(x, w, y, state=Tensor(F, 2, 3, 64)), "state")
    no(lambda: moe.moe_conv(x, w, y, state=Tensor(B, 2, 2, 64)), "state")
    no(lambda: moe.moe_conv(x, w, Tensor(B, 5, 64, device=1)), "GPU 1")
    no(lambda: moe.moe_conv(Tensor(I, 5, 64), w, y), "x")
    far = moe.moe_seqs(None, None, None, 5, 0)
    far.device = 1
    no(lambda: moe.moe_conv(x, w, y, seqs=far), "GPU 1")

    cfg = moe.make_head_norm_config(rot_dim=4)
    h = Tensor(B, 5, 3, 8)
    no(lambda: moe.moe_head_norm(cfg, Tensor(B, 5, 24), h), "x: expected a 3D")
    no(lambda: moe.moe_head_norm(cfg, h, Tensor(B, 5, 4, 8)), "y is")
    no(lambda: moe.moe_head_norm(cfg, h, h, weight=Tensor(F, 7)), "weight")
    no(lambda: moe.moe_head_norm(cfg, h, h, gate=Tensor(F, 5, 3, 8)), "gate is")
    no(lambda: moe.moe_head_norm(cfg, h, h, x2=Tensor(B, 4, 1, 8), y2=Tensor(B, 4, 1, 8)), "x2 is")
    no(lambda: moe.moe_head_norm(cfg, h, h, x2=Tensor(B, 5, 1, 8)), "y2")
    no(lambda: moe.moe_head_norm(cfg, h, h, y2=h), "y2 goes with x2")
    no(lambda: moe.moe_head_norm(cfg, h, h, weight2=Tensor(F, 8)), "weight2 goes with x2")
    no(lambda: moe.moe_head_norm(cfg, h, h, pos=Tensor(I, 4), inv_freq=Tensor(F, 2)), "pos")
    no(lambda: moe.moe_head_norm(cfg, h, h, pos=Tensor(I, 5), inv_freq=Tensor(F, 1)), "inv_freq")

    q, v, g = Tensor(B, 5, 2, 8), Tensor(B, 5, 4, 16), Tensor(F, 5, 4)

    def delta(q=q, k=q, v=v, g=g, beta=g, state=None, o=v, **more):
        return lambda: moe.moe_delta(q, k, v, g, beta, state, o, **more)
    no(delta(q=Tensor(F, 5, 2, 8)), "bfloat16")
    no(delta(k=Tensor(B, 5, 2, 16)), "k 5 x 2 x 16")
    no(delta(v=Tensor(B, 4, 4, 16)), "v has 4")
    no(delta(o=Tensor(B, 5, 2, 16)), "o is")
    no(delta(q=Tensor(B, 5, 2, 8, stride=(32, 16, 1))), "side by side")
    no(delta(g=Tensor(F, 5, 3)), "g")
    no(delta(beta=None), "required")
    no(delta(state=Tensor(F, 2, 4, 16, 7)), "state")
    no(delta(state=Tensor(F, 2, 4, 16, 8, device=1)), "GPU 1")
    q, v, g = Tensor(B, 50, 2, 8), Tensor(B, 50, 4, 16), Tensor(F, 50, 4)  # long enough for a workspace
    no(delta(q=q, k=q, v=v, g=g, beta=g, o=v, workspace=Tensor(F, 100)), "workspace")
    with pytest.raises(moe.MoeError, match="workspace"):  # the library's own refusal comes through
        moe.moe_delta(q, q, v, g, g, None, v)
    for call in (lambda: moe.moe_delta(q, q, v), lambda: moe.moe_delta(q, q, v, g, g, None, v, q=q),
                 lambda: moe.moe_delta(q, q, v, g, g, None, v, other=1), lambda: moe.moe_conv(*[x] * 9)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(AttributeError):
        moe.moe_nothing
    with pytest.raises(ValueError):
        moe.make_seqs(3, offsets=torch.zeros(4, dtype=torch.int32))


# ---------------------------------------------------------------------------
# the plain definitions
# ---------------------------------------------------------------------------

def test_definition_of_conv():
    x, w = np.arange(12.0).reshape(6, 2), np.array([[1.0, 10, 100], [0, 0, 1]])
    y, state = np.zeros((6, 2)), np.array([[[1.0, 5], [2, 6]]])
    ora.conv(x, w, None, False, y, state, ora.sequences(6, [0, 6]))
    assert y[0].tolist() == [1 + 20 + 0, 1] and y[1].tolist() == [2 + 0 + 200, 3] and y[5, 0] == 6 + 80 + 1000
    assert state[0].tolist() == x[4:].tolist()


def test_definition_of_rotation():
    x = np.zeros((1, 1, 6))
    x[0, 0] = [1, 2, 3, 4, 5, 6]
    quarter = np.array([np.pi / 2, 0])
    z, _ = ora.head_norm(x, "none", 0, None, 0, np.array([1]), quarter, 4, True, None)
    assert np.allclose(z[0, 0], [-3, 2, 1, 4, 5, 6])
    z, _ = ora.head_norm(x, "none", 0, None, 0, np.array([1]), quarter, 4, False, None)
    assert np.allclose(z[0, 0], [-2, 1, 3, 4, 5, 6])
    z, _ = ora.head_norm(x, "l2", 0, None, 0, None, None, 0, True, None)
    assert np.isclose((z * z).sum(), 1)


def test_definition_of_the_delta_rule():
    """With beta 1, no decay and orthonormal keys the state stores each value under its key, and a key seen again replaces
    its value."""
    k = np.eye(4)[[0, 1, 2, 0]][:, None]
    v = np.random.default_rng(1).standard_normal((4, 1, 3))
    o, state = np.zeros((4, 1, 3)), np.full((1, 1, 3, 4), 9.0)
    ora.delta(k, k, v, np.zeros((4, 1)), np.ones((4, 1)), state, o, 1.0, ora.sequences(4, [0, 4], None, [0]))
    assert np.allclose(o, v)
    assert np.allclose(state[0, 0], np.stack([v[3, 0], v[1, 0], v[2, 0], np.zeros(3)], 1))


def test_torch_tensors_that_do_not_fit_are_refused():
    """Real tensors (the stand-ins above go another way): of the host, without memory, without strides, of other types."""
    torch = pytest.importorskip("torch")
    w, y = torch.zeros(8, 4), torch.zeros(2, 8)
    host = torch.zeros(2, 8)
    for x in (host, torch.nn.Parameter(host), host.bfloat16(), host.to("meta"), host.double(), host[0], host.reshape(2, 2, 2, 2)):
        with pytest.raises(ValueError, match="x: expected a 2D CUDA tensor"):
            moe.moe_conv(x, w, y)
    with pytest.raises((ValueError, RuntimeError)):
        moe.moe_conv(host.to_sparse(), w, y)
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode() as mode:
        fake = mode.from_tensor(host)
    with pytest.raises((ValueError, RuntimeError)):
        moe.moe_conv(fake, w, y)
    for junk in (None, 3, "x", [[1.0]], np.zeros((2, 8), np.float32)):
        with pytest.raises(ValueError, match="x: expected a 2D CUDA tensor"):
            moe.moe_conv(junk, w, y)
    with pytest.raises(ValueError, match="q: expected a 3D CUDA tensor"):
        moe.moe_delta(host, host, host, host, host, None, host)
    with pytest.raises(ValueError, match="x: expected a 3D CUDA tensor"):
        moe.moe_head_norm(moe.make_head_norm_config(), host[None], host[None])
