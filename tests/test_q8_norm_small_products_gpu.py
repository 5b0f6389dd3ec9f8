"""The normed rows of the 8-bit norm where a product x w is below fp32's normal range and
the quotient by a small rms is not: the quotient is right to its own precision.

Tolerance as in test_draft_step_gpu: 18 u (u = 2^-24) and the output's half step, relative,
and half the least subnormal of the output twice (an fp32 subnormal rounded to bf16).
"""
import numpy as np
import pytest
import torch

import draft_step_ref as ref
from speculative_decoding_verification_84_b200 import binding

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,d", [(3, 64), (40, 512), (5, 1001), (7, 4096), (3, 16384)])
def test_small_products(M, d, dtype):
    g = torch.Generator().manual_seed(M + d)
    x = torch.randn((M, d), generator=g)
    x[0] *= 1e-20
    x[1] *= 1e-6
    x[2, ::3] = 0.0
    x[2] *= 1e-12
    r = 0.5 * x * torch.rand((M, d), generator=g)
    w = torch.ones(d)
    w[1::4] = 10.0 ** (-20 - 15 * torch.rand(len(w[1::4]), generator=g))
    w[2::4] = 10.0 ** (-30 - 8 * torch.rand(len(w[2::4]), generator=g)) * -1
    x, r, w = x.to(dtype), r.to(dtype), w.to(dtype)
    h = torch.finfo(dtype).eps / 2
    least = 2.0 ** -150 + (2.0 ** -134 if dtype == torch.bfloat16 else 2.0 ** -150)
    for res in (None, r):
        for eps in (0.0, 1e-12):
            out = binding.q8_norm(x.to(DEV), w.to(DEV), eps, residual=res.to(DEV) if res is not None else None, with_normed=True)
            q, scale, s, normed = ref.q8_rows(ref.f64(x), ref.f64(res) if res is not None else None, ref.f64(w), float(np.float32(eps)))
            np.testing.assert_array_equal(out[0].cpu().numpy(), q)
            off = np.abs(ref.f64(out[-1]) - normed)
            assert (off <= (h + 18 * U) * (1 + h) * np.abs(normed) + least).all(), (eps, (off / np.abs(normed).clip(2.0 ** -126)).max())
