"""A product whose wait runs out: the kernel ends by itself, the count of the device says so once the stream has been
synchronised, in a call or in a graph's replay, and no other call is refused or wrong because of it.

The wait is one that nothing ends (moe_mx_set_fault), bounded by 1 ms; every other wait of the kernel ends as ever."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

import int4_expert_streaming_gb300 as moe  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    moe.build()
    moe.load_library()


@pytest.fixture(autouse=True)
def _no_fault_stays():
    yield
    moe.moe_mx_set_fault(0)


# the one-CTA forms with 64 and 128 rows a tile, the pair, and a tile split over a cluster; several tiles a CTA and one
FORMS = {"64": ([5], 1024, 1024), "128": ([90] * 3, 1024, 2048), "128 many": ([70, 1, 60] * 30, 640, 512),
         "pair": ([1300], 4000, 1100), "pair many": ([300] * 40, 1024, 1024), "split": ([1], 1024, 8192),
         "split rows": ([100], 300, 6400)}


def problem(sizes, N, K, fmt):
    g = torch.Generator(device="cuda").manual_seed(0)
    E, R = len(sizes), sum(sizes)
    group = torch.from_numpy(np.repeat(np.arange(E, dtype=np.int32), sizes)).cuda()
    offsets = torch.from_numpy(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)).cuda()
    w = moe.make_mx(fmt, N, K, groups=E)
    moe.moe_mx_quantise(w, torch.randn((E * N, K), generator=g, device="cuda"))
    x = moe.make_mx(fmt, R, K, groups=E, ragged=True)
    moe.moe_mx_quantise(x, torch.randn((R, K), generator=g, device="cuda"), group_of_row=group, offsets=offsets)
    return x, w, offsets


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("fmt", [moe.MOE_MX_E8M0, moe.MOE_MX_E4M3])
def test_a_wait_that_runs_out_is_counted_and_nothing_else_suffers(form, fmt):
    x, w, offsets = problem(*FORMS[form], fmt)
    want, y = (torch.empty((x.rows, w.rows), device="cuda") for _ in range(2))
    moe.moe_mx_product(x, w, want, offsets=offsets)
    torch.cuda.synchronize()
    before = moe.moe_mx_timeouts()
    moe.moe_mx_set_fault(moe.MOE_FAULT_DEVICE_WAIT)
    moe.moe_mx_product(x, w, y, offsets=offsets)
    torch.cuda.synchronize()
    after = moe.moe_mx_timeouts()
    assert after > before
    moe.moe_mx_set_fault(0)
    y.fill_(float("nan"))
    moe.moe_mx_product(x, w, y, offsets=offsets)  # the next call on the device: not refused, and right
    torch.cuda.synchronize()
    assert torch.equal(y, want) and moe.moe_mx_timeouts() == after


def test_replays_of_a_graph_are_counted():
    x, w, offsets = problem([5, 3], 512, 1024, moe.MOE_MX_E8M0)
    y = torch.empty((8, 512), device="cuda")
    moe.moe_mx_product(x, w, y, offsets=offsets)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    moe.moe_mx_set_fault(moe.MOE_FAULT_DEVICE_WAIT)
    with torch.cuda.graph(graph):
        moe.moe_mx_product(x, w, y, offsets=offsets, stream=torch.cuda.current_stream())
    moe.moe_mx_set_fault(0)
    for _ in range(2):
        before = moe.moe_mx_timeouts()
        graph.replay()
        torch.cuda.synchronize()
        assert moe.moe_mx_timeouts() > before


def test_unknown_faults_are_refused():
    with pytest.raises(moe.MoeError):
        moe.moe_mx_set_fault(1)
