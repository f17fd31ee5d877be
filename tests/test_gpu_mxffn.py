"""The gated feed-forward block on the GPU against float64: forward (a tensor, the packed copy, the
checkpoint of G and U), backward, grouped by expert, the one-call layer; over sizes around every tile
edge."""
import numpy as np
import pytest
import torch

import mxffn_reference as ref
import mxfp4_reference as ref4
from gpu_util import GEMM_TOL, dev
from test_gpu_mx8 import DTYPES, close, gradients, on_gpu, values_of
from test_gpu_mxfp4_gemm import copy_of, many_offsets, product, spread_offsets, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    import nvfp4_block_scaled_quantize_amd as nv
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    nv.load_library()
    return nv


def weights(nv, lead, k, seed):
    """A random copy whose products with copy_of's are of the size of activations: a few units."""
    w = copy_of(nv, lead, k, seed, spread=1)
    w.scales[..., :-(-k // 32)] -= 8
    return w


def gate(p, e, act):
    """a(p) and the bound of its error, p being off by e: the slope stays below 1.13."""
    a, _ = ref.activation(p, act)
    return a, ref.activation_error(p, act)[0] * (1 + 1e-3) + 1.13 * e


def forward(a, w, n, act):
    """(H, bound of its error), (G, bound), (U, bound) in float64 of values a [M][K], w [2n][K]."""
    (g, eg), (u, eu) = ((p, GEMM_TOL * t) for p, t in (product(a, w[:n]), product(a, w[n:])))
    x, ex = (torch.from_numpy(v).to(dev()) for v in gate(g.cpu().numpy(), eg.cpu().numpy(), act))
    h = x * u
    return (h, ex * (u.abs() + eu) + x.abs() * eu + 2 * ref.EPS * h.abs() + 1e-45), (g, eg), (u, eu)


def blocks(v):
    """[n][k] -> [n][blocks][32], padded with zeros to whole units of 128."""
    return torch.nn.functional.pad(v, (0, -v.shape[1] % 128)).unflatten(1, (-1, 32))


def check_copy(got, scales, want, tol, expo, low_step, n, what):
    """A quantized copy's values [M][kp] against those quantized, known up to tol: the scale is that of a
    largest magnitude within tol, and a value within half a step of its binade (or of the lowest one), or
    of where the format ends."""
    v, x, t = blocks(got[:, :n]), blocks(want), blocks(tol)
    s = torch.ldexp(torch.ones_like(v[..., :1]), scales.double().unsqueeze(-1) - 127)
    lo, hi = ((x.abs() + sign * t).clamp(min=0).amax(-1, keepdim=True) for sign in (-1, 1))
    assert ((expo(lo) <= s) & (s <= expo(hi))).all(), f"{what}: scales"
    step = torch.maximum(torch.maximum(v.abs(), x.abs()) * low_step[0], s * low_step[1])
    bad = ~((v - x).abs() <= t + step)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} values"


def power(p, amax):
    """2^p, 2^-127 at least and where the largest magnitude is 0."""
    return torch.ldexp(torch.ones_like(amax), p.clamp(min=-127)).where(amax > 0, torch.full_like(amax, 2.0 ** -127))


def scale8(amax):
    """The checkpoint's scale of a largest magnitude."""
    m, e = torch.frexp(amax)
    return power(torch.where(m <= 0.875, e - 9, e - 8), amax)


def scale4(rule):
    def of(amax):
        m, e = torch.frexp(amax)
        p = e - 3 if rule == ref4.FLOOR else torch.where(m <= 0.75, e - 3, e - 2)
        return power(p, amax)
    return of


def check_forward(nv, a, w, n, got, act, rule, what):
    """got: (h in float32 or bfloat16, copy, checkpoint), each of them or None."""
    h, copy, kept = got
    (x, ex), (g, eg), (u, eu) = forward(values(a), values(w), n, act)
    if h is not None:
        close(h, x, ex, f"{what} H")
    if copy is not None:
        v = values(copy)
        assert (v[:, n:] == 0).all() and (copy.scales[:, -(-n // 32):] == 0).all()
        # half a step is at most a quarter of the value's magnitude (1 of 4 from 5 on, saturating at 6
        # from below 8: a quarter); a quarter of the scale below 1
        check_copy(v, copy.scales, x, ex, scale4(rule), (0.25, 0.25), n, f"{what} copy")
    if kept is not None:
        for i, (p, e) in enumerate(((g, eg), (u, eu))):
            v = torch.from_numpy(ref.decode(kept.codes[i].cpu().numpy(), kept.scales[i].cpu().numpy())).to(dev())
            assert (v[:, n:] == 0).all() and (kept.scales[i][:, -(-n // 32):] == 0).all()
            check_copy(v, kept.scales[i], p, e, scale8, (2.0 ** -4, 2.0 ** -10), n, f"{what} checkpoint {i}")


SIZES = [(1, 1, 1), (1, 2048, 128), (1, 33, 4096), (2, 150, 2080), (7, 65, 31), (16, 16, 32), (17, 500, 1000), (31, 32, 257),
         (32, 256, 512), (33, 129, 640), (64, 1025, 384), (65, 64, 129), (100, 100, 100), (128, 128, 256), (129, 127, 384),
         (200, 350, 1500), (255, 130, 512), (256, 255, 1024), (257, 511, 130), (300, 1, 700), (513, 257, 2500),
         (1024, 1024, 896), (2000, 65, 4097), (2304, 1280, 1152), (3000, 1501, 200), (2, 7200, 128), (33, 1800, 128)]


@pytest.mark.parametrize("M,N,K", SIZES)
def test_forward(nv, M, N, K):
    print(f"gated {M}x{N}x{K}", flush=True)
    act, rule = (ref.SILU, ref4.FLOOR) if (M + N) % 2 else (ref.GELU, ref4.CEIL)
    a, w = copy_of(nv, (M,), K, 1, spread=1), weights(nv, (2 * N,), K, 2)
    copy, kept = nv.MXTensor.empty(M, N, dev()), nv.MX8Tensor.empty((2, M), N, dev())
    for t in (copy, kept):
        t.codes.fill_(0x55), t.scales.fill_(0x55)
    for dt in DTYPES:
        got = nv.mxfp4_gated(a, w, activation=act, out_dtype=dt, packed=copy, scale_rule=rule, checkpoint=kept)
        assert got[1] is copy and got[2] is kept and got[0].dtype == dt
        check_forward(nv, a, w, N, got, act, rule, f"{dt}")
        # a tensor alone, into a view with a wider pitch: nothing written beside it
        buf = torch.full((M + 2, N + 5), 3.0, dtype=dt, device=dev())
        alone = nv.mxfp4_gated(a, w, activation=act, out=buf[1:-1, 2:2 + N])
        assert alone[1] is None and alone[2] is None
        check_forward(nv, a, w, N, alone, act, rule, f"{dt} alone")
        buf[1:-1, 2:2 + N] = 3.0
        assert (buf == 3.0).all()
    # the results do not depend on which of them are asked for beside the copy
    for more in (dict(checkpoint=True), dict()):
        none, only, other = nv.mxfp4_gated(a, w, activation=act, out_dtype=None, packed=True, scale_rule=rule, **more)
        assert none is None and torch.equal(only.codes, copy.codes) and torch.equal(only.scales, copy.scales)
        if more:
            assert torch.equal(other.codes, kept.codes) and torch.equal(other.scales, kept.scales)


@pytest.mark.parametrize("M,N,K", [(6144, 2500, 640), (6100, 2495, 130), (5000, 2050, 1500), (6144, 2560, 257)])
def test_forward_more_tiles_than_compute_units(nv, M, N, K):
    test_forward(nv, M, N, K)


def exact_copies(nv, lead_a, lead_w, k, seed):
    """Copies whose products are sums of multiples of 1/4 below 2^22: exact in binary32 in any order."""
    return copy_of(nv, lead_a, k, seed, spread=0), copy_of(nv, lead_w, k, seed + 1, spread=0)


@pytest.mark.parametrize("M,N,K", [(1, 40, 70), (33, 129, 300), (130, 250, 1000), (300, 1000, 513), (2100, 1100, 256)])
def test_checkpoint_bit_for_bit(nv, M, N, K):
    a, w = exact_copies(nv, (M,), (2 * N,), K, 21)
    kept = nv.mxfp4_gated(a, w, out_dtype=None, checkpoint=True)[2]
    want = product(values(a), values(w))[0]
    for i in range(2):
        codes, scales = ref.quantize_rows(want[:, i * N:(i + 1) * N].cpu().numpy())
        assert torch.equal(kept.scales[i].cpu(), torch.from_numpy(scales))
        assert torch.equal(kept.codes[i].cpu(), torch.from_numpy(codes))


GROUPED = [(1, 3, 40, 96, [0, 0, 1, 1]), (24, 8, 150, 500, spread_offsets(24, 8, 0)), (100, 3, 129, 130, [0, 33, 33, 100]),
           (600, 5, 128, 384, [0, 256, 257, 300, 600, 600]), (900, 70, 48, 160, spread_offsets(900, 70, 1)),
           (1500, 4, 260, 1000, spread_offsets(1500, 4, 2, tail=300)), (64, 2, 33, 64, [0, 0, 0]), (300, 3, 50, 64, [5, 900, 2, 300]),
           (6000, 5, 2300, 300, [0, 2000, 2000, 2600, 2601, 5500]), (20000, 70, 1050, 200, many_offsets(20000, 70, 7, 100)),
           # few groups of many rows: the forward's large tiles, one round of them and two, with rows in no group
           (2048, 1, 3584, 200, [0, 2000]), (3840, 2, 4096, 130, [0, 1000, 3000]), (400, 17, 1024, 256, spread_offsets(400, 17, 3))]


@pytest.mark.parametrize("case", range(len(GROUPED)))
def test_forward_grouped(nv, case):
    M, G, N, K, off = GROUPED[case]
    print(f"gated grouped {case}", flush=True)
    act, rule = (ref.SILU, ref4.CEIL) if case % 2 else (ref.GELU, ref4.FLOOR)
    a, w = copy_of(nv, (M,), K, 5, spread=1), weights(nv, (G, 2 * N), K, 6)
    offsets = torch.tensor(off, dtype=torch.int32, device=dev())
    spans = ref4.spans(off, M)
    end = spans[-1][1]
    for dt in DTYPES:
        copy, kept = nv.MXTensor.empty(M, N, dev()), nv.MX8Tensor.empty((2, M), N, dev())
        for t in (copy, kept):
            t.codes.fill_(0x55), t.scales.fill_(0x55)
        buf = torch.full((M + 2, N + 3), float("nan"), dtype=dt, device=dev())
        h = buf[1:-1, :N]
        nv.mxfp4_gated(a, w, offsets, act, h, packed=copy, scale_rule=rule, checkpoint=kept)
        alone = nv.mxfp4_gated(a, w, offsets, act, out_dtype=dt)[0]
        for e, (i, j) in enumerate(spans):
            if j > i:
                part = lambda t: nv.MXTensor(t.codes[i:j].contiguous(), t.scales[i:j].contiguous(), t.k)
                pa, pw = part(a), nv.MXTensor(w.codes[e], w.scales[e], K)
                pk = nv.MX8Tensor(kept.codes[:, i:j].contiguous(), kept.scales[:, i:j].contiguous(), N)
                check_forward(nv, pa, pw, N, (h[i:j], part(copy), pk), act, rule, f"group {e}")
                check_forward(nv, pa, pw, N, (alone[i:j], None, None), act, rule, f"group {e} alone")
        for t in (h[end:], alone[end:], copy.codes[end:], copy.scales[end:], kept.codes[:, end:], kept.scales[:, end:]):
            assert (t == 0).all()       # rows in no group
        assert torch.isnan(buf[0]).all() and torch.isnan(buf[-1]).all() and torch.isnan(buf[:, N:]).all()


def backward64(dy, w, v, act=ref.SILU):
    """gradients() of dH = dy w^T, known up to the product's tolerance."""
    d, t = product(dy, w)
    return gradients(*v.cpu().numpy(), d.cpu().numpy(), act, (GEMM_TOL * t).cpu().numpy())


def check_backward(nv, dy, w, kept, got, act, what):
    n = w.codes.shape[0]
    v = torch.from_numpy(ref.decode(kept.codes.cpu().numpy(), kept.scales.cpu().numpy())[..., :n])
    pairs = on_gpu(backward64(values(dy), values(w), v, act))
    for x, pair, name in zip((got[0][:, :n], got[0][:, n:], got[1]), pairs, ("dG", "dU", "H")):
        close(x, *pair, f"{what} {name}")


def kept_of(nv, M, N, seed):
    return nv.mxfp8_quantize(2 * values_of((2, M, N), seed, torch.float32).clamp_(-10, 10))


@pytest.mark.parametrize("M,N,K", SIZES + [(6144, 5000, 640), (6100, 4990, 130)])
def test_backward(nv, M, N, K):
    print(f"gated backward {M}x{N}x{K}", flush=True)
    act = ref.SILU if (M + N) % 2 else ref.GELU
    dy, w, kept = copy_of(nv, (M,), K, 31), copy_of(nv, (N,), K, 32), kept_of(nv, M, N, 33)
    kept.codes[..., N:] = 0x70      # what lies behind a row's end does not matter
    for dt in DTYPES:
        got = nv.mxfp4_gated_backward(dy, w, kept, activation=act, out_dtype=dt, h=True)
        check_backward(nv, dy, w, kept, got, act, f"{dt}")
        for pad in (3, 4):
            buf = torch.full((M + 2, 2 * N + 2 * pad), 3.0, dtype=dt, device=dev())
            hbuf = torch.full((M + 2, N + pad), 3.0, dtype=dt, device=dev())
            nv.mxfp4_gated_backward(dy, w, kept, activation=act, out=buf[1:-1, pad:pad + 2 * N], h=hbuf[1:-1, :N])
            assert torch.equal(buf[1:-1, pad:pad + 2 * N], got[0]) and torch.equal(hbuf[1:-1, :N], got[1])
            buf[1:-1, pad:pad + 2 * N], hbuf[1:-1, :N] = 3.0, 3.0
            assert (buf == 3.0).all() and (hbuf == 3.0).all()
        only, none = nv.mxfp4_gated_backward(dy, w, kept, activation=act, out_dtype=dt)
        assert none is None and torch.equal(only, got[0])


@pytest.mark.parametrize("case", range(len(GROUPED)))
def test_backward_grouped(nv, case):
    M, G, N, K, off = GROUPED[case]
    print(f"gated backward grouped {case}", flush=True)
    act = ref.SILU if case % 2 else ref.GELU
    dy, w, kept = copy_of(nv, (M,), K, 35), copy_of(nv, (G, N), K, 36), kept_of(nv, M, N, 37)
    offsets = torch.tensor(off, dtype=torch.int32, device=dev())
    spans = ref4.spans(off, M)
    end = spans[-1][1]
    kept.scales[:, end:] = 255      # the checkpoint of rows in no group is not looked at
    for dt in DTYPES:
        buf = torch.full((M + 2, 2 * N + 3), float("nan"), dtype=dt, device=dev())
        dgu = buf[1:-1, :2 * N]
        got = nv.mxfp4_gated_backward(dy, w, kept, offsets, act, dgu, h=True)
        assert got[0] is dgu
        for e, (i, j) in enumerate(spans):
            if j > i:
                pa = nv.MXTensor(dy.codes[i:j].contiguous(), dy.scales[i:j].contiguous(), K)
                pk = nv.MX8Tensor(kept.codes[:, i:j].contiguous(), kept.scales[:, i:j].contiguous(), N)
                check_backward(nv, pa, nv.MXTensor(w.codes[e], w.scales[e], K), pk, (dgu[i:j], got[1][i:j]), act, f"group {e}")
        assert (dgu[end:] == 0).all() and (got[1][end:] == 0).all()
        assert torch.isnan(buf[0]).all() and torch.isnan(buf[-1]).all() and torch.isnan(buf[:, 2 * N:]).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rule", [ref4.FLOOR, ref4.CEIL])
def test_linear_is_quantize_then_gated(nv, dtype, rule):
    for M, N, K in [(1, 2500, 1024), (1, 31, 70), (3, 513, 3000), (16, 320, 513), (33, 350, 260), (70, 129, 128), (300, 257, 777),
                    (2100, 150, 512), (12, 2048, 4096), (40, 96, 300), (33, 1800, 128), (64, 2200, 256), (3, 4000, 256)]:
        print(f"gated linear {M}x{N}x{K} {dtype} {rule}", flush=True)
        x = torch.randn(M, K + 3, device=dev()).to(dtype)[:, 1:1 + K]
        w = weights(nv, (2 * N,), K, 7)
        a = nv.mxfp4_quantize(x, nv.mxfp4_quant_params(scale_rule=rule))[0]
        for act in (ref.SILU, ref.GELU):
            h = nv.mxfp4_gated_linear(x, w, activation=act, scale_rule=rule)
            assert h.dtype == dtype and torch.equal(h, nv.mxfp4_gated(a, w, activation=act, out_dtype=dtype)[0])
            check_forward(nv, a, w, N, (h, None, None), act, rule, "linear")


@pytest.mark.parametrize("M,G,N,K,off", [(1, 4, 100, 300, [0, 0, 0, 1, 1]), (24, 8, 150, 500, spread_offsets(24, 8, 0)),
                                         (40, 3, 512, 2048, [0, 13, 13, 40]), (100, 6, 640, 512, [0, 5, 40, 40, 90, 95, 97]),
                                         (400, 17, 1024, 256, spread_offsets(400, 17, 3)),
                                         (30, 6, 1500, 500, [0, 3, 3, 11, 18, 24, 29]), (1500, 4, 260, 1000, [0, 7, 700, 1300, 1500])])
def test_linear_grouped(nv, M, G, N, K, off):
    print(f"gated linear grouped {M} {G} {N} {K}", flush=True)
    offsets = torch.tensor(off, dtype=torch.int32, device=dev())
    w = weights(nv, (G, 2 * N), K, 8)
    for dtype in DTYPES:
        x = torch.randn(M, K, device=dev()).to(dtype)
        a = nv.mxfp4_quantize(x, nv.mxfp4_quant_params())[0]
        h = nv.mxfp4_gated_linear(x, w, offsets)
        assert torch.equal(h, nv.mxfp4_gated(a, w, offsets, out_dtype=dtype)[0])
        for e, (i, j) in enumerate(ref4.spans(off, M)):
            if j > i:
                pa = nv.MXTensor(a.codes[i:j].contiguous(), a.scales[i:j].contiguous(), K)
                check_forward(nv, pa, nv.MXTensor(w.codes[e], w.scales[e], K), N, (h[i:j], None, None), ref.SILU, 0, f"group {e}")
        assert (h[ref4.spans(off, M)[-1][1]:] == 0).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_weights_past_two_gigabytes(nv, dtype):
    """A token through 65536 rows of W of 32 KiB each: the kernel for few rows reads the two halves as two buffers."""
    N, K = 32768, 65536
    g = torch.Generator(device=dev()).manual_seed(51)
    w = nv.MXTensor(torch.randint(0, 256, (2 * N, K // 2), generator=g, device=dev(), dtype=torch.uint8),
                    torch.randint(114, 117, (2 * N, K // 32), generator=g, device=dev(), dtype=torch.uint8), K)
    x = torch.randn(1, K, generator=g, device=dev()).to(dtype)
    a = nv.mxfp4_quantize(x, nv.mxfp4_quant_params())[0]
    h = nv.mxfp4_gated_linear(x, w)
    assert torch.equal(h, nv.mxfp4_gated(a, w, out_dtype=dtype)[0])
    some = torch.cat([torch.arange(0, 40), torch.randint(0, N, (50,)), torch.arange(N - 40, N)]).to(dev())
    rows = torch.cat([some, some + N])
    part = nv.MXTensor(w.codes[rows], w.scales[rows], K)
    check_forward(nv, a, part, some.numel(), (h[:, some], None, None), ref.SILU, 0, "two gigabytes")


@pytest.mark.parametrize("M,N,K", [(0, 5, 40), (5, 0, 40), (5, 40, 0), (300, 200, 0)])
def test_empty(nv, M, N, K):
    a, w = nv.MXTensor.empty(M, K, dev()), nv.MXTensor.empty(2 * N, K, dev())
    h, copy, kept = nv.mxfp4_gated(a, w, packed=True, checkpoint=True)
    assert h.shape == (M, N) and (h == 0).all() and (copy.codes == 0).all() and (kept.codes == 0).all()
    assert (copy.scales == 0).all() and (kept.scales == 0).all()
    kept = nv.mxfp8_quantize(torch.ones(2, M, N, device=dev()))
    dgu, h = nv.mxfp4_gated_backward(a, nv.MXTensor.empty(N, K, dev()), kept, h=True)
    assert dgu.shape == (M, 2 * N) and (dgu == 0).all() and (h > 0).all()
    assert (nv.mxfp4_gated_linear(torch.ones(M, K, device=dev()), w) == 0).all()


@pytest.mark.parametrize("M", [7, 40, 300])
def test_nan_and_infinities_reach_their_rows(nv, M):
    """A token with a NaN or an infinity: its own row of H only; a row of W: its own column, and there a
    block of the copies."""
    N, K = 200, 300
    x = torch.randn(M, K, device=dev())
    x[3, 200], x[6, 0] = float("nan"), float("inf")
    w = nv.mxfp4_quantize(0.05 * torch.randn(2 * N, K, device=dev()), nv.mxfp4_quant_params())[0]
    h = nv.mxfp4_gated_linear(x, w)
    assert torch.isnan(h).any(1).nonzero().flatten().tolist() == [3, 6] and torch.isnan(h[[3, 6]]).all()
    a = nv.mxfp4_quantize(x.nan_to_num(0, 1, -1), nv.mxfp4_quant_params())[0]
    w.scales[N + 70, 2] = 255
    h, copy, kept = nv.mxfp4_gated(a, w, packed=True, checkpoint=True)
    assert torch.isnan(h).any(0).nonzero().flatten().tolist() == [70]
    assert torch.isnan(nv.mxfp4_dequantize(copy)).all(0).nonzero().flatten().tolist() == list(range(64, 96))
    v = nv.mxfp8_dequantize(kept)
    assert torch.isfinite(v[0]).all() and torch.isnan(v[1]).any(0).nonzero().flatten().tolist() == list(range(64, 96))
    a.scales[5, 1] = 255
    h, copy, kept = nv.mxfp4_gated(a, w, packed=True, checkpoint=True)
    assert torch.isnan(h[5]).all() and not torch.isnan(h[4, :70]).any()
    assert (copy.scales[5, :7] == 255).all() and (copy.scales[5, 7:] == 0).all() and (copy.codes[5] == 0).all()
    assert (kept.scales[:, 5, :7] == 255).all() and (kept.scales[:, 5, 7:] == 0).all() and (kept.codes[:, 5] == 0).all()


def test_a_step_as_it_is_used(nv):
    """Forward and backward of a block, dense and of experts, as training runs them: every gradient against
    the same step in float64 on the operands that the calls quantized."""
    for G, off in ((0, None), (4, [0, 100, 100, 333, 500])):
        M, D, N = 500, 320, 288
        offsets = None if off is None else torch.tensor(off, dtype=torch.int32, device=dev())
        lead = (G,) if G else ()
        gen = torch.Generator(device=dev()).manual_seed(3)
        rand = lambda *s: torch.randn(*s, generator=gen, device=dev())
        x, dy = rand(M, D).bfloat16(), (1e-3 * rand(M, D)).bfloat16()
        w1, w2 = 0.05 * rand(*lead, 2 * N, D), 0.05 * rand(*lead, D, N)
        both = nv.mxfp4_quant_params(True, True, nv.MXFP4_SCALE_CEIL)
        gemm = lambda a, b, **k: nv.mxfp4_gemm_grouped(a, b, offsets, **k) if G else nv.mxfp4_gemm(a, b, **k)
        wgrad = lambda a, b: nv.mxfp4_gemm_grouped_wgrad(a, b, offsets) if G else nv.mxfp4_gemm(a, b)
        x8 = nv.mxfp8_quantize(x)
        (w1r, w1c), (w2r, w2c) = nv.mxfp4_quantize(w1, both), nv.mxfp4_quantize(w2, both)
        xr, _ = nv.mxfp8_to_mxfp4(x8, nv.mxfp4_quant_params(scale_rule=nv.MXFP4_SCALE_CEIL))
        _, hq, kept = nv.mxfp4_gated(xr, w1r, offsets, out_dtype=None, packed=True, scale_rule=nv.MXFP4_SCALE_CEIL, checkpoint=True)
        y = gemm(hq, w2r)
        dyr, dyc = nv.mxfp4_quantize(dy, both, offsets=offsets)
        dgu, h = nv.mxfp4_gated_backward(dyr, w2c, kept, offsets, out_dtype=torch.float32, h=True)
        _, hc = nv.mxfp4_quantize(h, both, offsets=offsets)
        dr, dc = nv.mxfp4_quantize(dgu, both, offsets=offsets)
        _, xc = nv.mxfp8_to_mxfp4(x8, both, offsets=offsets)
        dx, dw1, dw2 = gemm(dr, w1c), wgrad(dc, xc), wgrad(dyc, hc)
        assert dw1.shape == w1.shape and dw2.shape == w2.shape

        D64 = lambda q, **k: nv.mxfp4_dequantize(q, **k).double()
        spans = [(0, M)] if off is None else ref4.spans(off, M)
        pick = lambda t, e: t[e] if G else t
        x4, h4, dy4, dr4 = (D64(q) for q in (xr, hq, dyr, dr))
        cols = {n: D64(q, offsets=offsets) for n, q in (("x", xc), ("h", hc), ("dy", dyc), ("d", dc))}
        ws = {n: D64(q) for n, q in (("w1r", w1r), ("w1c", w1c), ("w2r", w2r), ("w2c", w2c))}
        k8 = nv.mxfp8_dequantize(kept).double()
        def near(got, a, b, what):
            want, absdot = product(a, b)
            assert ((got.double() - want).abs() <= GEMM_TOL * absdot).all(), what
        for e, (i, j) in enumerate(spans):
            if j == i:
                continue
            (hx, hex_), _, _ = forward(x4[i:j], pick(ws["w1r"], e), N, ref.SILU)
            # H's copy to nearest of 6 s >= amax: half a step is at most an amax / 6 (s < amax / 3, steps of up to 2 s)
            amax = blocks(hx.abs() + hex_).amax(-1).repeat_interleave(32, -1)[:, :N]
            assert ((h4[i:j] - hx).abs() <= hex_ + amax / 3).all()
            near(y[i:j], h4[i:j], pick(ws["w2r"], e), "Y")
            pairs = on_gpu(backward64(dy4[i:j], pick(ws["w2c"], e), k8[:, i:j]))
            for got, pair, name in zip((dgu[i:j, :N], dgu[i:j, N:], h[i:j]), pairs, ("dG", "dU", "H")):
                close(got, *pair, name)
            near(dx[i:j], dr4[i:j], pick(ws["w1c"], e), "dX")
            near(pick(dw1, e), cols["d"][:, i:j], cols["x"][:, i:j], "dW1")
            near(pick(dw2, e), cols["dy"][:, i:j], cols["h"][:, i:j], "dW2")
        if G:
            assert (dw1[1] == 0).all() and (dw2[1] == 0).all()


def test_streams_and_graphs(nv):
    """Calls on a stream of their own, two at once on the same inputs, and captured: every replay gives the
    eager results on the inputs of the moment."""
    M, N, K = 96, 200, 512
    w, w2 = weights(nv, (2 * N,), K, 41), copy_of(nv, (N,), K, 42)
    x, dy = torch.randn(M, K, device=dev()).bfloat16(), torch.randn(M, K, device=dev()).bfloat16()
    p = nv.mxfp4_quant_params(True, True)

    def step():
        h = nv.mxfp4_gated_linear(x, w)
        x8 = nv.mxfp8_quantize(x)
        xr, xc = nv.mxfp8_to_mxfp4(x8, p)
        _, hq, kept = nv.mxfp4_gated(xr, w, out_dtype=None, packed=True, checkpoint=True)
        dgu, hb = nv.mxfp4_gated_backward(nv.mxfp4_quantize(dy, p)[0], w2, kept, h=True)
        back, _ = nv.mxfp8_gated_backward(hb, kept)
        return [h, xc.codes, xc.scales, hq.codes, hq.scales, kept.codes, kept.scales, dgu, hb, back, nv.mxfp8_dequantize(x8)]

    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    results = []
    for s in streams:
        with torch.cuda.stream(s):
            results.append(step())
    torch.cuda.synchronize()
    for got in results:
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in range(4):
        torch.manual_seed(seed)
        x.copy_(torch.randn(M, K, device=dev())), dy.copy_(torch.randn(M, K, device=dev()))
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), seed


def test_refusals(nv):
    """What does not fit is refused before anything runs."""
    a, w, w2 = copy_of(nv, (5,), 64, 1), copy_of(nv, (40,), 64, 2), copy_of(nv, (20,), 64, 3)
    kept = nv.mxfp8_quantize(torch.randn(2, 5, 20, device=dev()))
    off = torch.tensor([0, 2, 5], dtype=torch.int32, device=dev())
    stack = copy_of(nv, (2, 40), 64, 4)
    E = nv.Nvfp4Error
    x = torch.randn(5, 64, device=dev())
    for call in (lambda: nv.mxfp4_gated(a, w, activation=2), lambda: nv.mxfp4_gated(a, copy_of(nv, (41,), 64, 2)),
                 lambda: nv.mxfp4_gated(a, copy_of(nv, (40,), 65, 2)), lambda: nv.mxfp4_gated(a, w, out_dtype=None),
                 lambda: nv.mxfp4_gated(a, w, scale_rule=2), lambda: nv.mxfp4_gated(a, stack), lambda: nv.mxfp4_gated(a, w, off),
                 lambda: nv.mxfp4_gated(a, w, out=torch.empty(5, 21, device=dev())), lambda: nv.mxfp4_gated(a, w, out_dtype=torch.half),
                 lambda: nv.mxfp4_gated(a, w, packed=nv.MXTensor.empty(5, 21, dev())), lambda: nv.mxfp4_gated(a, w, packed=kept),
                 lambda: nv.mxfp4_gated(a, w, checkpoint=nv.MX8Tensor.empty((2, 5), 19, dev())), lambda: nv.mxfp4_gated(kept, w),
                 lambda: nv.mxfp4_gated(a, w, checkpoint=a), lambda: nv.mxfp4_gated(stack, w),
                 lambda: nv.mxfp4_gated(a, stack, torch.tensor([0, 5], device=dev())),
                 lambda: nv.mxfp4_gated_linear(x, copy_of(nv, (40,), 128, 2)), lambda: nv.mxfp4_gated_linear(x[:, ::2], w),
                 lambda: nv.mxfp4_gated_linear(x, w, scale_rule=7), lambda: nv.mxfp4_gated_linear(x.half(), w),
                 lambda: nv.mxfp4_gated_linear(x.cpu(), w), lambda: nv.mxfp4_gated_linear(x, w, activation=-1),
                 lambda: nv.mxfp4_gated_backward(a, w2, nv.mxfp8_quantize(torch.randn(5, 20, device=dev()))),
                 lambda: nv.mxfp4_gated_backward(a, w, kept), lambda: nv.mxfp4_gated_backward(a, w2, kept, off),
                 lambda: nv.mxfp4_gated_backward(a, w2, kept, activation=9), lambda: nv.mxfp4_gated_backward(a, w2, a),
                 lambda: nv.mxfp4_gated_backward(a, w2, kept, h=torch.empty(5, 20, device=dev())),
                 lambda: nv.mxfp4_gated_backward(a, w2, kept, out=torch.empty(5, 20, device=dev())),
                 lambda: nv.mxfp8_gated_backward(torch.randn(5, 21, device=dev()), kept),
                 lambda: nv.mxfp8_gated_backward(torch.randn(5, 20), kept), lambda: nv.mxfp8_gated_backward(torch.randn(5, 20, device=dev()).half(), kept),
                 lambda: nv.mxfp8_quantize(torch.randn(2, 2, 2, 2, device=dev())), lambda: nv.mxfp8_quantize(x.half()),
                 lambda: nv.mxfp8_quantize(x, out=kept), lambda: nv.mxfp8_dequantize(kept, out=torch.empty(2, 5, 21, device=dev())),
                 lambda: nv.mxfp8_dequantize(a), lambda: nv.mxfp8_to_mxfp4(kept, nv.mxfp4_quant_params(), off),
                 lambda: nv.mxfp8_to_mxfp4(kept, nv.mxfp4_quant_params(), row_out=nv.MXTensor.empty(5, 20, dev())),
                 lambda: nv.mxfp8_to_mxfp4(kept, nv.mxfp4_quant_params(False, False)),
                 lambda: nv.mxfp8_to_mxfp4(nv.MX8Tensor(kept.codes[..., :64], kept.scales, 20), nv.mxfp4_quant_params())):
        with pytest.raises(E):
            call()
