"""The operators without a context at the edges of what they take: tensor scales of zero and next to zero."""
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


def rows_of(m, groups, rows, cols):
    place = mxo.uniform_place(groups, rows)
    return mxo.read_tiles(m._data.cpu().numpy(), *place, cols, m.format)


@pytest.mark.parametrize("cols", [32, 300])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_tensor_scale_of_zero_gives_no_nan(cols, dtype):
    """An expert without weights: largest value 0, so tensor scale 0.  Its scales are 0, as of any block of zeros; what is
    not zero takes the largest scale and stands for 0 all the same."""
    rng = np.random.default_rng(0)
    src = np.zeros((3, 5, cols), np.float32)
    src[1] = np.round(rng.normal(0, 1, (5, cols)) * 8) / 8 + 0.0625  # no zeros
    src[2] = 1.0
    m = moe.make_mx(moe.MOE_MX_E4M3, 5, cols, groups=3)
    t = cuda(np.array([0, 0.01, 0], np.float32))
    moe.moe_mx_quantise(m, cuda(src.reshape(15, cols)).to(dtype), tensor_scale=t)
    code, byte = (v.reshape(3, 5, -1) for v in rows_of(m, 3, 5, cols))
    used = -(-cols // 16)
    assert (byte[0] == 0).all() and (code[0] & 7 == 0).all()
    assert (byte[1, :, :used] > 0).all() and (byte[1] < 127).all() and (byte[1, :, used:] == 0).all()
    assert (byte[2, :, :used] == 126).all() and (byte[2, :, used:] == 0).all() and (code[2] & 7 == 0).all()
    out = torch.full((15, cols), 5.0, device="cuda")
    moe.moe_mx_dequantise(m, out, tensor_scale=t)
    out = out.view(3, 5, cols).cpu()
    assert (out[0] == 0).all() and (out[2] == 0).all() and out[1].isfinite().all() and (out[1] != 0).any()
    x = moe.make_mx(moe.MOE_MX_E4M3, 3, cols, groups=3, ragged=True)
    moe.moe_mx_quantise(x, torch.ones((3, cols), device="cuda"), group_of_row=cuda(np.arange(3, dtype=np.int32)),
                        offsets=cuda(np.arange(4, dtype=np.int32)))
    y = torch.full((3, 5), 7.0, device="cuda")
    moe.moe_mx_product(x, m, y, offsets=cuda(np.arange(4, dtype=np.int32)), alpha=t)
    assert (y[0] == 0).all() and (y[2] == 0).all() and y.isfinite().all()

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_swiglu_zeros_stay_zeros_at_the_smallest_scales(dtype):
    """A block whose scale times the tensor scale has no reciprocal in fp32."""
    cols, t = 48, 2.0 ** -120
    src = np.zeros((1, 2 * cols), np.float32)
    src[0, :cols] = 2.0 ** -63
    src[0, cols:] = np.where(np.arange(cols) % 3 == 0, 2.0 ** -63, 0)  # silu(g) u = 2^-127, or 0
    m = moe.make_mx(moe.MOE_MX_E4M3, 1, cols)
    moe.moe_mx_quantise(m, cuda(src).to(dtype), act=moe.MOE_ACT_SWIGLU, tensor_scale=cuda(np.array([t], np.float32)))
    code, byte = rows_of(m, 1, 1, cols)
    # a / (6 t) = 2^-7 / 6, two thirds of the smallest scale 2^-9: the scale is 2^-9, the values 2^-127 / 2^-129 = 4
    assert (byte[0, :3] == 1).all()
    assert np.array_equal(code[0, :cols] & 7, np.where(np.arange(cols) % 3 == 0, 6, 0))
