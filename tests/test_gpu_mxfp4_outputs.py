"""Where the MXFP4 operators write on the GPU: outputs in the middle of larger buffers."""
import numpy as np
import pytest
import torch

from gpu_util import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    import nvfp4_block_scaled_quantize_amd as nv
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    nv.load_library()
    return nv


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("lead", [(5, 1), (2, 3, 1), (1, 1), (3, 4)])
def test_decode_of_a_stack_into_its_middle(nv, dtype, lead):
    """A stack decoded into a contiguous out whose one-row matrices have a row stride of their own:
    the values, and nothing beside them (the buffer around holds any row at that stride)."""
    k = 130
    n = int(np.prod(lead))
    x = torch.randn(n, k, device=dev()).to(dtype)
    row = nv.MXTensor.empty(lead, k, dev())
    flat, _ = nv.mxfp4_quantize(x, nv.mxfp4_quant_params())
    row.codes.copy_(flat.codes.view_as(row.codes))
    row.scales.copy_(flat.scales.view_as(row.scales))
    buf = torch.full((40 * n * k,), 7.0, dtype=dtype, device=dev())
    first = 13 * n * k
    stride = [1]
    for d in reversed((*lead[1:], k)):
        stride.insert(0, stride[0] * d)
    if lead[-1] == 1:
        stride[-2] = 2 * n * k // max(n - 1, 1)      # of an axis of length 1: any
    out = buf.as_strided((*lead, k), stride, first)
    assert out.is_contiguous()
    print(f"decode of a stack {lead} {dtype}", flush=True)
    assert nv.mxfp4_dequantize(row, out=out) is out
    want = nv.mxfp4_dequantize(flat, dtype)
    assert torch.equal(out, want.view(*lead, k))
    buf[first:first + n * k] = 7.0
    assert (buf == 7.0).all()
