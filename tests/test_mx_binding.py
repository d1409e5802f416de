"""The Python module that takes the tensors of the operators without a context apart, on stand-ins for CUDA tensors: what
is on another GPU than the rest of the call is refused before the library sees its address.  Every call here has one
argument that the library refuses as well, so nothing is ever launched."""
import pytest

import int4_expert_streaming_gb300 as moe

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _built():
    moe.build()
    moe.load_library()


class Tensor:
    """As much of a CUDA tensor as the module looks at."""
    is_cuda = True

    def __init__(self, dtype, *shape, device=0):
        self.dtype, self.shape, self._device = dtype, shape, device

    def get_device(self):
        return self._device

    def stride(self):
        return tuple(self.shape[1:]) + (1,)

    def is_contiguous(self):
        return True

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n

    def data_ptr(self):
        return 1 << 20


F, I, B = torch.float32, torch.int32, torch.uint8


def mx(fmt, rows, cols, groups=1, ragged=0, device=0):
    m = moe.moe_mx(1 << 20, rows, cols, groups, fmt, ragged)
    m.device = device
    return m


def bad_cfg():
    cfg = moe.make_route_config(16, 2)
    cfg.score = 9
    return cfg


# name: call of the tensors, their shapes, descriptors (made anew for each device)
CALLS = {
    "route": (lambda t, m: moe.moe_route(bad_cfg(), *t), [(F, 3, 16), (F, 16), (I, 3, 2), (F, 3, 2)], []),
    "dispatch": (lambda t, m: moe.moe_dispatch(t[0], 2000, *t[1:]),
                 [(I, 3, 2), (I, 2001), (I, 3, 2), (I, 6), (I, 6), (B, 64)], []),
    "quantise": (lambda t, m: moe.moe_mx_quantise(m[0], t[0], 7, *t[1:]), [(F, 4, 64), (I, 4), (I, 4), (I, 3), (F, 2)],
                 [(1, 4, 64, 2, 1)]),
    "dequantise": (lambda t, m: moe.moe_mx_dequantise(m[0], *t), [(F, 4, 64), (I, 4), (I, 3), (F, 2)], [(9, 4, 64, 2, 1)]),
    "product": (lambda t, m: moe.moe_mx_product(m[0], m[1], *t), [(F, 4, 32), (I, 3), (F, 2)],
                [(0, 4, 64, 2, 1), (1, 32, 64, 2, 0)]),
    "combine": (lambda t, m: moe.moe_combine(*t), [(F, 8, 16), (I, 3, 0), (F, 3, 0), (F, 3, 16)], []),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_tensors_of_one_gpu_reach_the_library(name):
    call, tensors, matrices = CALLS[name]
    with pytest.raises(moe.MoeError) as e:
        call([Tensor(*t) for t in tensors], [mx(*m) for m in matrices])
    assert e.value.code == moe.MOE_EINVAL


@pytest.mark.parametrize("name,at", [(n, i) for n, c in CALLS.items() for i in range(len(c[1]) + len(c[2]))])
def test_a_tensor_of_another_gpu_is_refused(name, at):
    call, tensors, matrices = CALLS[name]
    with pytest.raises(ValueError, match="GPU"):
        call([Tensor(*t, device=int(i == at)) for i, t in enumerate(tensors)],
             [mx(*m, device=int(len(tensors) + i == at)) for i, m in enumerate(matrices)])


def test_a_tensor_of_the_host_is_refused():
    call, tensors, matrices = CALLS["route"]
    for at in range(len(tensors)):
        with pytest.raises(ValueError, match="expected"):
            call([Tensor(*t, device=-int(i == at)) for i, t in enumerate(tensors)], [])


def test_a_descriptor_without_a_device_is_taken_as_it_is():
    call, tensors, matrices = CALLS["product"]
    with pytest.raises(moe.MoeError):
        call([Tensor(*t) for t in tensors], [mx(*m, device=-1) for m in matrices])


def test_counts_and_faults_refuse_what_they_do_not_know():
    lib = moe.load_library()
    assert lib.moe_mx_timeouts(None) == moe.MOE_EINVAL
    assert lib.moe_mx_set_fault(1) == moe.MOE_EINVAL and lib.moe_mx_set_fault(0) == moe.MOE_OK


def test_row_counts_below_zero_are_refused():
    lib, P = moe.load_library(), 1 << 20
    m = moe.moe_mx(P, 4, 64, 1, moe.MOE_MX_E8M0, 0)
    assert lib.moe_mx_quantise_rows(m, P, -1, 0, 64, 0, P, None, None, None, None) == moe.MOE_EINVAL
    assert "src_rows" in moe.moe_last_error(None)
    assert lib.moe_combine_rows(P, -1, 0, 8, P, P, 2, 2, 8, P, 0, 8, None) == moe.MOE_EINVAL
    assert "n_rows" in moe.moe_last_error(None)
