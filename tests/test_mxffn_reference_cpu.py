"""Pins of the tests' own reference of MXFP8 and of the gated block, and the block's gradient formulas
against differences."""
import numpy as np
import pytest
import torch

import mxffn_reference as ref


def test_e4m3_table_is_torchs():
    got = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(got, ref.VALUES, equal_nan=True)


def test_quantize_is_nearest_and_never_saturates():
    r = np.random.RandomState(0)
    x = r.standard_normal((50, 300)) * np.exp(r.standard_normal((50, 1)) * 5)
    codes, scales = ref.quantize_rows(x)
    v = ref.decode(codes, scales)
    assert v.shape == (50, 384) and (v[:, 300:] == 0).all() and (scales[:, 10:] == 0).all()
    s = np.repeat(np.ldexp(1.0, scales.astype(int) - 127), 32, axis=1)[:, :300]
    step = np.maximum(np.abs(v[:, :300]) * 2.0 ** -4, s * 2.0 ** -10)      # half a step of the upper neighbour
    assert (np.abs(v[:, :300] - x) <= step).all()
    amax = np.abs(np.pad(x, ((0, 0), (0, 20)))).reshape(50, 10, 32).max(-1)
    s = np.ldexp(1.0, scales[:, :10].astype(int) - 127)
    assert (amax <= 448 * s).all() and (amax > 224 * s).all()


def test_quantize_borders():
    x = np.zeros((6, 32))
    x[0, 0], x[1, 0], x[2, 0] = 448, np.nextafter(448, 500), 2.0 ** -140
    x[3, 5], x[4, 5] = np.inf, np.nan
    x[5, :4] = [448, 17 * 2.0 ** -9 / 2, -0.0, 2.0 ** -10]       # ties: 8.5 steps to 8, half a step to 0
    codes, scales = ref.quantize_rows(x)
    assert scales[:, 0].tolist() == [127, 128, 0, 255, 255, 127] and (codes[3:5] == 0).all()
    assert codes[0, 0] == 0x7E and codes[5, :4].tolist() == [0x7E, 8, 128, 0]


@pytest.mark.parametrize("act", [ref.SILU, ref.GELU])
def test_activation_is_torchs_and_its_slope_a_difference(act):
    x = np.linspace(-12, 12, 2001)
    a, slope = ref.activation(x, act)
    t = torch.from_numpy(x)
    want = torch.nn.functional.silu(t) if act == ref.SILU else torch.nn.functional.gelu(t, approximate="tanh")
    assert np.abs(a - want.numpy()).max() < 1e-14 * 12
    d = 1e-5
    diff = (ref.activation(x + d, act)[0] - ref.activation(x - d, act)[0]) / (2 * d)
    assert np.abs(diff - slope).max() < 1e-9       # d^2 / 6 times a third derivative below 2, and 1e-15 / d


@pytest.mark.parametrize("act", [ref.SILU, ref.GELU])
def test_gradients_of_the_product_are_differences(act):
    r = np.random.RandomState(1)
    g, u, dh = r.standard_normal((3, 40)) * 2
    a, slope = ref.activation(g, act)
    d = 1e-5

    def loss(g, u):
        return dh * ref.activation(g, act)[0] * u

    assert np.abs((loss(g + d, u) - loss(g - d, u)) / (2 * d) - dh * u * slope).max() < 1e-8
    assert np.abs((loss(g, u + d) - loss(g, u - d)) / (2 * d) - dh * a).max() < 1e-8
