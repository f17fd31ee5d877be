"""A checkpoint's codes and scales can be replaced, as a copy's can."""
import pytest
import torch

import nvfp4_block_scaled_quantize_amd as nv
from nvfp4_block_scaled_quantize_amd import mxffn, mxfp4


@pytest.mark.parametrize("kind,width", [("MXTensor", 64), ("MX8Tensor", 128)])
def test_codes_and_scales_are_replaced(kind, width):
    t = getattr(nv, kind).empty((2, 3), 40, "cpu")
    codes, scales = torch.ones(2, 3, width, dtype=torch.uint8), torch.full((2, 3, 4), 7, dtype=torch.uint8)
    t.scales.fill_(5)
    t.codes = codes
    assert t.codes is codes and (t.scales == 5).all() and t.shape == (2, 3, 40)
    t.scales = scales
    assert t.codes is codes and t.scales is scales and "shape=(2, 3, 40)" in repr(t)
    t = getattr(nv, kind).empty(4, 40, "cpu")
    t.codes.fill_(9)
    t.scales = scales[0, :1].repeat(4, 1)
    assert (t.codes == 9).all() and (t.scales == 7).all() and t.shape == (4, 40)


def test_replaced_ones_are_what_a_call_takes(monkeypatch):
    """The buffer that both lay in is no longer looked at."""
    for module, operand in ((mxfp4, mxfp4._operand), (mxffn, mxffn._operand8)):
        t = (nv.MXTensor if module is mxfp4 else nv.MX8Tensor).empty(3, 40, "cpu")
        t.codes = t.codes.clone()
        c, lead = operand(t, "t", -1)
        assert (c.codes, c.scales) == (t.codes.data_ptr(), t.scales.data_ptr()) and lead == (3,)
        t.scales = torch.zeros(3, 5, dtype=torch.uint8)
        with pytest.raises(nv.Nvfp4Error, match="do not"):
            operand(t, "t", -1)
