"""Row indices that lead out of the tensor they go with count as none: quantisation leaves such rows unwritten, the
combine skips such pairs.  (The rows past the end stand in the same allocation here, so nothing is read out of range
whatever happens; they hold numbers that would show.)"""
import numpy as np
import pytest

import _mx_oracle as mxo

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

import int4_expert_streaming_gb300 as moe  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    moe.build()
    moe.load_library()


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


OUT = [-2 ** 31, -1, 6, 7, 2 ** 31 - 1]  # of six rows


@pytest.mark.parametrize("cols", [64, 300, 31])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("act", [moe.MOE_ACT_NONE, moe.MOE_ACT_SWIGLU])
def test_quantise_leaves_rows_without_a_source_unwritten(cols, dtype, act):
    width = 2 * cols if act else cols
    big = torch.full((9, width), 500.0, device="cuda", dtype=dtype)
    big[:6] = torch.randn((6, width), device="cuda")
    row = np.array([0, 5, 3] + OUT + [1], np.int32)
    m, ref = moe.make_mx(moe.MOE_MX_E8M0, len(row), cols), moe.make_mx(moe.MOE_MX_E8M0, 6, cols)
    m._data.fill_(0xEE)
    moe.moe_mx_quantise(m, big[:6], act, src_row=cuda(row))
    moe.moe_mx_quantise(ref, big[:6], act)
    code, byte = mxo.read_tiles(m._data.cpu().numpy(), *mxo.uniform_place(1, len(row)), cols, 0)
    rcode, rbyte = mxo.read_tiles(ref._data.cpu().numpy(), *mxo.uniform_place(1, 6), cols, 0)
    there = (row >= 0) & (row < 6)
    assert np.array_equal(code[there], rcode[row[there]]) and np.array_equal(byte[there], rbyte[row[there]])
    assert (code[~there] == 0xE).all() and (byte[~there] == 0xEE).all()


@pytest.mark.parametrize("cols", [64, 62, 31])
@pytest.mark.parametrize("tin", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tout", [torch.float32, torch.bfloat16])
def test_combine_skips_pairs_without_a_row(cols, tin, tout):
    big = torch.full((9, cols), 500.0, device="cuda", dtype=tin)
    big[:6] = torch.randn((6, cols), device="cuda")
    row = cuda(np.array([[0, 5, -1, 3, 2, 1], OUT + [4], OUT + [-7]], np.int32))
    kept = torch.where((row >= 0) & (row < 6), row, -1)
    w = torch.rand((3, 6), device="cuda")
    y, want = (torch.full((3, cols), 7.0, device="cuda", dtype=tout) for _ in range(2))
    moe.moe_combine(big[:6], row, w, y)
    moe.moe_combine(big, kept, w, want)
    assert torch.equal(y, want) and (y[2] == 0).all() and y.abs().max() < 100


def test_no_rows_at_all():
    y = torch.full((2, 16), 7.0, device="cuda")
    moe.moe_combine(torch.empty((0, 16), device="cuda"), torch.zeros((2, 3), dtype=torch.int32, device="cuda"),
                    torch.ones((2, 3), device="cuda"), y)
    assert (y == 0).all()
    m = moe.make_mx(moe.MOE_MX_E8M0, 3, 64)
    m._data.fill_(0xEE)
    moe.moe_mx_quantise(m, torch.empty((0, 64), device="cuda"), src_row=torch.zeros(3, dtype=torch.int32, device="cuda"))
    assert (m._data == 0xEE).all()
