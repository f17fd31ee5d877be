"""The packed copy of H that the gated product makes from its accumulators is the copy that mxfp4_quantize makes of H in
float32, bit for bit: rounded once, to nearest even, by either rule, whatever else the call writes."""
import pytest
import torch

import mxfp4_reference as ref4
from gpu_util import dev
from test_gpu_mxffn import GROUPED, SIZES, exact_copies, nv, weights  # noqa: F401  (nv: fixture)
from test_gpu_mxfp4_gemm import copy_of

pytestmark = pytest.mark.gpu
# over 64 groups, most of them empty, a few with most of the rows, some rows in none: large tiles, one round of them, two
MANY = [(12500, 70, 328, 200, {3: 5000, 20: 1, 41: 4000, 69: 2000}), (34000, 70, 328, 130, {0: 300, 1: 17000, 33: 9000, 64: 7000})]


def same_copies(nv, a, w, offsets=None):  # noqa: F811
    for act in (nv.MXFP4_SILU, nv.MXFP4_GELU):
        for rule in (nv.MXFP4_SCALE_FLOOR, nv.MXFP4_SCALE_CEIL):
            h, copy, _ = nv.mxfp4_gated(a, w, offsets, act, out_dtype=torch.float32, packed=True, scale_rule=rule)
            want = nv.mxfp4_quantize(h, nv.mxfp4_quant_params(scale_rule=rule))[0]
            others = [nv.mxfp4_gated(a, w, offsets, act, out_dtype=dt, packed=True, scale_rule=rule, checkpoint=kept)[1]
                      for dt, kept in ((torch.bfloat16, False), (None, True), (torch.bfloat16, True))]
            for c in (copy, *others):
                assert torch.equal(c.scales, want.scales) and torch.equal(c.codes, want.codes)


@pytest.mark.parametrize("M,N,K", SIZES + [(6144, 2500, 640)])
def test_copy_is_quantize_of_h(nv, M, N, K):  # noqa: F811
    print(f"copy {M}x{N}x{K}", flush=True)
    a = copy_of(nv, (M,), K, 61, spread=1)
    same_copies(nv, a, weights(nv, (2 * N,), K, 62))
    # values over many binades, and sums that are multiples of 1/4: ties
    same_copies(nv, copy_of(nv, (M,), K, 63), copy_of(nv, (2 * N,), K, 64))
    a, w = exact_copies(nv, (M,), (2 * N,), K, 65)
    same_copies(nv, a, w)
    # a NaN in a row of A and in one of W
    a.scales[M // 2, 0], w.scales[N + N // 3, 0] = 255, 255
    same_copies(nv, a, w)


@pytest.mark.parametrize("case", range(len(GROUPED)))
def test_copy_by_expert(nv, case):  # noqa: F811
    M, G, N, K, off = GROUPED[case]
    same_copies(nv, copy_of(nv, (M,), K, 66, spread=1), weights(nv, (G, 2 * N), K, 67),
                torch.tensor(off, dtype=torch.int32, device=dev()))


@pytest.mark.parametrize("M,G,N,K,counts", MANY)
def test_more_than_64_experts_on_large_tiles(nv, M, G, N, K, counts):  # noqa: F811
    """Each expert's rows as in a call of their own, which the other tests check; the others 0."""
    off = [0]
    for e in range(G):
        off.append(off[-1] + counts.get(e, 0))
    offsets = torch.tensor(off, dtype=torch.int32, device=dev())
    a, w = copy_of(nv, (M,), K, 68, spread=1), weights(nv, (G, 2 * N), K, 69)
    copy, kept = nv.MXTensor.empty(M, N, dev()), nv.MX8Tensor.empty((2, M), N, dev())
    for t in (copy, kept):
        t.codes.fill_(0x55), t.scales.fill_(0x55)
    h = torch.full((M + 2, N + 3), float("nan"), dtype=torch.bfloat16, device=dev())
    nv.mxfp4_gated(a, w, offsets, out=h[1:-1, :N], packed=copy, checkpoint=kept)
    assert torch.isnan(h[0]).all() and torch.isnan(h[-1]).all() and torch.isnan(h[:, N:]).all()
    h = h[1:-1, :N]
    for e, (i, j) in enumerate(ref4.spans(off, M)):
        if j == i:
            continue
        part = nv.MXTensor(a.codes[i:j].contiguous(), a.scales[i:j].contiguous(), K)
        x, c, k = nv.mxfp4_gated(part, nv.MXTensor(w.codes[e], w.scales[e], K), packed=True, checkpoint=True)
        print(f"expert {e}: {j - i} rows", flush=True)
        assert torch.equal(h[i:j], x)
        assert torch.equal(copy.codes[i:j], c.codes) and torch.equal(copy.scales[i:j], c.scales)
        assert torch.equal(kept.codes[:, i:j], k.codes) and torch.equal(kept.scales[:, i:j], k.scales)
    end = off[-1]
    for t in (h[end:], copy.codes[end:], copy.scales[end:], kept.codes[:, end:], kept.scales[:, end:]):
        assert t.numel() and (t == 0).all()
    same_copies(nv, a, w, offsets)
