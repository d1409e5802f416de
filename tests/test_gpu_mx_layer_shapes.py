"""The expert layer refuses tensors that do not go together; a router row that is missing must not be made up of an
earlier call's choices."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

import int4_expert_streaming_gb300 as moe  # noqa: E402
from int4_expert_streaming_gb300 import mx_layer  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    moe.build()
    moe.load_library()


@pytest.mark.parametrize("xs,ls,ys", [((4, 128), (3, 8), (4, 128)), ((3, 128), (4, 8), (3, 128)),
                                      ((4, 128), (4, 8), (3, 128)), ((4, 128), (4, 8), (5, 128)),
                                      ((4, 96), (4, 8), (4, 96)), ((4, 128), (4, 8), (4, 96)), ((4, 128), (4, 9), (4, 128)),
                                      ((4, 128), (32,), (4, 128))])
def test_layer_refuses_tensors_that_do_not_go_together(xs, ls, ys):
    w, d = torch.zeros((8, 64, 128), device="cuda"), torch.zeros((8, 128, 32), device="cuda")
    layer = mx_layer.MxLayer(w, d, moe.make_route_config(8, 2), 4)
    layer.idx.fill_(-1)
    with pytest.raises(ValueError):
        layer.forward(*(torch.zeros(s, device="cuda") for s in (xs, ls, ys)))
    assert (layer.idx == -1).all()  # before anything ran
