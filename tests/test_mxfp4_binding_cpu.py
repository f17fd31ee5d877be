"""What the MXFP4 binding hands to the C calls, on the CPU: the calls themselves are stubbed, so
that no kernel runs."""
import pytest
import torch


@pytest.fixture
def calls(monkeypatch):
    """Arguments of the stubbed C calls, with CPU tensors let through."""
    from nvfp4_block_scaled_quantize_amd import mxfp4
    seen = []

    class Lib:
        def __getattr__(self, name):
            return name

    monkeypatch.setattr(mxfp4, "_lib", Lib)
    monkeypatch.setattr(mxfp4, "_device", lambda t: t.get_device())
    monkeypatch.setattr(mxfp4, "_call", lambda f, device, *args: seen.append((f, args)))
    return seen


def one_row_stacks(k):
    """Stacks whose contiguity says nothing of the row stride: their matrices have one row, or
    there is one matrix of one row."""
    return [torch.empty(1, 5, k).transpose(0, 1), torch.empty(5 * k).as_strided((5, 1, k), (k, 7 * k, 1)),
            torch.empty(5 * k).as_strided((5, 1, k), (k, k + 3, 1)), torch.empty(k).as_strided((1, 1, k), (9, 5 * k, 1)),
            torch.empty(6 * k).as_strided((2, 3, 1, k), (3 * k, k, 11 * k, 1)), torch.empty(4, 3, k)]


@pytest.mark.parametrize("k", [1, 64, 130])
@pytest.mark.parametrize("case", range(6))
def test_decode_of_a_stack_writes_its_own_rows(calls, case, k):
    import nvfp4_block_scaled_quantize_amd as nv
    out = one_row_stacks(k)[case]
    assert out.is_contiguous()
    q = nv.MXTensor.empty(tuple(out.shape[:-1]), k, "cpu")
    assert nv.mxfp4_dequantize(q, out=out) is out
    (f, (_, n, got_k, _, _, _, at, pitch)), = calls
    assert f == "mxfp4_dequantize" and got_k == k
    rows = out.reshape(-1, k)       # of a contiguous tensor: a view
    assert n == rows.shape[0]
    assert [at + i * pitch * out.element_size() for i in range(n)] == [r.data_ptr() for r in rows]
