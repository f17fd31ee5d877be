"""The activations' slopes on the GPU at every 8-bit gate, to a few roundings of binary32: with dH = 1 and U = 1
the gradient of G is a'(g) itself, exactly rounded products apart."""
import numpy as np
import pytest
import torch

import mxffn_reference as ref
from gpu_util import dev
from mxffn_reference import EPS

pytestmark = pytest.mark.gpu
SCALES = list(range(118, 130))      # 2^-9 .. 2^2: gates from 2^-18 to 1792


@pytest.fixture(scope="module")
def nv():
    import nvfp4_block_scaled_quantize_amd as nv
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    nv.load_library()
    return nv


def slope_error(x, act):
    """Bound on the error of a'(x) = S + a T y', S = 1 / (1 + e^-y) and T = e^-y S, in binary32 with exponential and
    reciprocal good to 2 EPS each (EPS: half a step, relative).  y takes up to five roundings, so e^-y is off by
    d = (5 |y| + 2) EPS relative.  S takes the part 1 - S of that, and an addition and a reciprocal: rho = ((1 - S) d +
    3) EPS; T the part S, and those and a product: ((S d) + 4) EPS.  a = x S: rho and a rounding; y': three roundings;
    the two products one each; the sum one of its own.  Where S is below 2^-126 it is 0, and so is T where e^-y is: less
    than 2^-126 (1 + |x| |y'|)."""
    y, dy = ref.exponent(x, act)
    with np.errstate(over="ignore"):
        s, t = 1 / (1 + np.exp(-y)), 1 / (1 + np.exp(y))
    d = 5 * np.abs(y) + 2
    rho, rho_t = (t * d + 3) * EPS, (s * d + 4) * EPS
    part = np.abs(x * s * t * dy)
    return s * rho + part * (rho + rho_t + 6 * EPS) + (s + part) * EPS + 2.0 ** -126 * (1 + np.abs(x)) * (1 + np.abs(dy))


@pytest.mark.parametrize("act", [ref.SILU, ref.GELU])
def test_slope_of_every_gate(nv, act):
    codes = torch.arange(256, dtype=torch.uint8)
    codes[[127, 255]] = 0
    gate = codes.repeat(len(SCALES), 1)
    scales = torch.tensor(SCALES, dtype=torch.uint8)[:, None].repeat(1, 8)
    g = ref.decode(gate.numpy(), scales.numpy())
    want = torch.from_numpy(ref.activation(g, act)[1]).to(dev())
    bound = torch.from_numpy(slope_error(g, act)).to(dev())
    # from dH, by the kernel for few rows, by tiles
    for name, rows, cols in (("from dH", 1, 1), ("few rows", 1, 1), ("tiles", 86, 4)):
        M, N = len(SCALES) * rows, 256 * cols
        one, unit = torch.full((M, N), 0x38, dtype=torch.uint8), torch.full((M, N // 32), 127, dtype=torch.uint8)
        kept = nv.MX8Tensor(torch.stack([gate.repeat(rows, cols), one]).to(dev()),
                            torch.stack([scales.repeat(rows, cols), unit]).to(dev()), N)
        if name == "from dH":
            dgu = nv.mxfp8_gated_backward(torch.ones(M, N, device=dev()), kept, activation=act)[0]
        else:
            a, w = (nv.MXTensor(torch.zeros(n, 64, dtype=torch.uint8, device=dev()),
                                torch.full((n, 4), 127, dtype=torch.uint8, device=dev()), 128) for n in (M, N))
            a.codes[:, 0], w.codes[:, 0] = 2, 2       # 1 x 1
            dgu = nv.mxfp4_gated_backward(a, w, kept, activation=act, out_dtype=torch.float32)[0]
        err = (dgu[:, :N].double() - want.repeat(rows, cols)).abs()
        worst = (err / bound.repeat(rows, cols)).max().item()
        print(f"{name}: {err.max().item():.3g}, {worst:.2f} of the bound", flush=True)
        assert worst <= 1, name
