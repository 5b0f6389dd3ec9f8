"""The int8 product at scales from the smallest to the largest that fp32 holds, of either
sign, zeros among them: the logit is right wherever it lies in the output's range,
although the product of its two scales may not.

Tolerance: three fp32 roundings (3 u, u = 2^-24) and the output's (half a step), relative
in the normal range; below it half a step of the subnormals, 2^-150 (fp32), once for the
last product and once for the output, 2^-134 (bf16).
"""
import numpy as np
import pytest
import torch

import draft_step_ref as ref
from speculative_decoding_verification_84_b200 import binding

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24


def _run(sa, sw, dtype, K=100, zeros=True):
    """Rows and channels of these scales: small and large sums, and sums of 0."""
    M, V = len(sa), len(sw)
    g = torch.Generator().manual_seed(M + V)
    ld = (K + 15) // 16 * 16
    a = torch.randint(-128, 128, (M, ld), generator=g, dtype=torch.int8)
    w = torch.randint(-128, 128, (V, ld), generator=g, dtype=torch.int8)
    a[::3], w[::2] = 127, 127
    if zeros:
        w[::5] = 0
    a, w = a.to(DEV)[:, :K], w.to(DEV)[:, :K]
    z = binding.q8_matmul(a, sa.to(DEV), w, sw.to(DEV), dtype)
    with np.errstate(invalid="ignore"):  # 0 times an infinite scale
        want = ref.q8_matmul(a.cpu().numpy(), ref.f64(sa), w.cpu().numpy(), ref.f64(sw))
    return ref.f64(z), want


def _check(got, want, dtype):
    h = torch.finfo(dtype).eps / 2
    rel = (3 * U + h) * (1 + h)
    least = 2.0 ** -150 * (1 + h) + (2.0 ** -150 if dtype == torch.float32 else 2.0 ** -134)
    top = float(torch.finfo(dtype).max) * (1 + h)  # from here on the output's type has only inf
    with np.errstate(all="ignore"):
        near = np.abs(np.abs(want) / top - 1) <= rel
        over = (np.abs(want) >= top) & ~near
        fine = ~over & ~near
        off = np.abs(got - want)
    assert (got[over] == np.sign(want[over]) * np.inf).all()
    assert (off[fine] <= rel * np.abs(want[fine]) + least).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [270, 271])
def test_scales_of_any_size(V, dtype):
    """From 2^-149 to 2^128, each against each, some with their sign turned."""
    g = torch.Generator().manual_seed(V)
    e = torch.linspace(-149, 127, V)
    sw = torch.exp2(e.double()).float() * (1 + torch.rand(V, generator=g) * 0.99)
    sa = sw[::2].flip(0).contiguous()
    sw[::7] *= -1
    sa[::9] *= -1
    sa[4], sw[9] = 0.0, 0.0
    got, want = _run(sa, sw, dtype)
    _check(got, want, dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_one_scale_out_of_range_beside_ordinary_ones(dtype):
    """A token or a channel at an end of the range leaves its neighbours' logits as they are."""
    g = torch.Generator().manual_seed(1)
    sa, sw = 0.5 + torch.rand(50, generator=g), (0.5 + torch.rand(300, generator=g)) / 64
    plain, _ = _run(sa, sw, dtype)
    sa2, sw2 = sa.clone(), sw.clone()
    sa2[[0, 17, 33]] = torch.tensor([1e-38, 3e38, 2.0 ** -140])
    sw2[[0, 101, 299]] = torch.tensor([2.0 ** -149, 3e38, 1e-30])
    got, want = _run(sa2, sw2, dtype)
    _check(got, want, dtype)
    rows, cols = np.ones(50, bool), np.ones(300, bool)
    rows[[0, 17, 33]], cols[[0, 101, 299]] = False, False
    np.testing.assert_array_equal(got[np.ix_(rows, cols)], plain[np.ix_(rows, cols)])


def test_scales_that_are_not_finite():
    """Infinite scales: infinite logits, NaN where the sum or the other scale is 0; NaN stays
    in its row or channel, whatever the other scale."""
    sa = torch.tensor([1.0, float("inf"), float("nan"), 1e-40, 0.0, 3e38])
    sw = torch.tensor([1.0, 1e-40, float("inf"), 0.0, float("nan"), 3e38, -float("inf"), 1e-20])
    got, want = _run(sa, sw, torch.float32, K=16)
    assert (np.isnan(got) == np.isnan(want)).all()
    with np.errstate(all="ignore"):
        inf = np.isinf(want) | (np.abs(want) > 3.5e38)
    assert (got[inf] == np.sign(want[inf]) * np.inf).all()
