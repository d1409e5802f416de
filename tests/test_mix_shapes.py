"""Shapes that the calls between two expert layers refuse: as many values as are expected, in another order.  On stand-ins
for CUDA tensors, whose addresses are never read: what passes the module's checks reaches a launch that fails without a GPU."""
import pytest

import int4_expert_streaming_gb300 as moe
from test_mix_host import Tensor

torch = pytest.importorskip("torch")
F, B = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    moe.build()
    moe.load_library()


def refused(word, call):
    with pytest.raises(ValueError, match=word):
        call()


@pytest.mark.parametrize("shape", [(2, 64, 3), (2, 3, 64, 1), (2, 192), (6, 64), (384,), (2, 6, 64), (2, 4, 64), (2, 3, 65)])
def test_conv_states_of_another_shape(shape):
    x, w = Tensor(B, 5, 64), Tensor(B, 64, 4)
    refused("state: expected .*slots, width - 1, channels", lambda: moe.moe_conv(x, w, Tensor(B, 5, 64), state=Tensor(B, *shape)))


@pytest.mark.parametrize("shape", [(2, 4, 8, 16), (2, 16, 8, 4), (2, 8, 16, 8), (2, 4, 128), (2, 4, 16, 8, 1), (8, 16, 8), (1024,),
                                   (2, 4, 16, 9), (2, 4, 17, 8), (2, 5, 16, 8)])
def test_delta_states_of_another_shape(shape):
    q, v, g = Tensor(B, 5, 2, 8), Tensor(B, 5, 4, 16), Tensor(F, 5, 4)
    refused("state: expected .*slots, v_heads, v_dim, k_dim",
            lambda: moe.moe_delta(q, q, v, g, g, Tensor(F, *shape), Tensor(B, 5, 4, 16)))


def test_states_that_are_not_contiguous():
    """A transposed view has the documented shape, and other values where the kernel reads."""
    q, v, g = Tensor(B, 5, 2, 8), Tensor(B, 5, 4, 16), Tensor(F, 5, 4)
    refused("state", lambda: moe.moe_delta(q, q, v, g, g, Tensor(F, 2, 4, 16, 8, stride=(512, 128, 1, 16)), v))
    refused("state", lambda: moe.moe_conv(Tensor(B, 5, 64), Tensor(B, 64, 4), Tensor(B, 5, 64),
                                          state=Tensor(B, 2, 3, 64, stride=(192, 1, 3))))


@pytest.mark.parametrize("shape", [(4, 5), (20,), (5, 4, 1), (10, 2), (4, 4), (5, 5), (1, 5, 4)])
def test_delta_gates_of_another_shape(shape):
    q, v, g, other = Tensor(B, 5, 2, 8), Tensor(B, 5, 4, 16), Tensor(F, 5, 4), Tensor(F, *shape)
    refused("g: expected .*T, v_heads", lambda: moe.moe_delta(q, q, v, other, g, None, v))
    refused("beta: expected .*T, v_heads", lambda: moe.moe_delta(q, q, v, g, other, None, v))
    refused("g: expected", lambda: moe.moe_delta(q, q, v, Tensor(F, 5, 4, stride=(1, 5)), g, None, v))


def test_shapes_that_fit_reach_the_library():
    """Its own refusal comes through, so nothing is launched: no workspace, and a stride shorter than a row."""
    q, v, g = Tensor(B, 50, 2, 8), Tensor(B, 50, 4, 16), Tensor(F, 60, 4)
    with pytest.raises(moe.MoeError, match="workspace"):
        moe.moe_delta(q, q, v, g, g, Tensor(F, 2, 4, 16, 8), v)
    x = Tensor(B, 5, 64, stride=(63, 1))
    with pytest.raises(moe.MoeError, match="stride"):
        moe.moe_conv(x, Tensor(B, 64, 4), Tensor(B, 5, 64), state=Tensor(B, 2, 3, 64))
