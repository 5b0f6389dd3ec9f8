"""8-bit rows of zeros, as the padding of a batch has them, beside rows whose products are
zero in fp32 only: integers and scales are what fp64 gives (tolerances as in
test_draft_step_gpu), and padding costs no more than other rows do."""
import numpy as np
import pytest
import torch

import draft_step_ref as ref
from speculative_decoding_verification_84_b200 import binding

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24


def _check(x, r, w, eps):
    dev = [t.to(DEV) if t is not None else None for t in (x, r, w)]
    got = binding.q8_norm(dev[0], dev[2], eps, residual=dev[1], with_normed=True)
    q, scale, s, normed = ref.q8_rows(*[ref.f64(t) if t is not None else None for t in (x, r, w)], float(np.float32(eps)))
    np.testing.assert_array_equal(got[0].cpu().numpy(), q)
    assert (np.abs(ref.f64(got[1]) - scale) <= 16 * U * scale + 2.0 ** -149).all()
    h = torch.finfo(x.dtype).eps / 2
    least = 2.0 ** -150 + (2.0 ** -134 if x.dtype == torch.bfloat16 else 2.0 ** -150)
    assert (np.abs(ref.f64(got[-1]) - normed) <= (h + 18 * U) * (1 + h) * np.abs(normed) + least).all()
    if w is None and r is None:
        q2, scale2 = binding.q8_quantize(dev[0])
        want = ref.q8_rows(ref.f64(x))
        np.testing.assert_array_equal(q2.cpu().numpy(), want[0])
        assert (np.abs(ref.f64(scale2) - want[1]) <= 16 * U * want[1] + 2.0 ** -149).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [1, 40, 75, 512, 1001, 2048, 4096, 4100, 8200, 20001])
def test_zero_rows(d, dtype):
    g = torch.Generator().manual_seed(d)
    x = torch.randn((9, d), generator=g)
    x[1] = 0.0
    x[2] = -0.0
    x[3] = 0.0
    x[3, d - 1] = 1e-25       # the one product of the row: zero in fp32 with the weight below
    x[4] = 0.0
    x[4, 0] = -1e-25
    x[5] *= 1e-24
    x[6, : d // 2] = 0.0
    w = 1e-25 * (1 + torch.rand(d, generator=g))
    x, w = x.to(dtype), w.to(dtype)
    r = torch.randn((9, d), generator=g).to(dtype)
    r[1:6] = 0
    r[2] = -x[2]
    for eps in (1e-6, 0.0):
        for weight in (None, w, torch.zeros_like(w)):
            _check(x, None, weight, eps)
            _check(x, r, weight, eps)
        _check(x, -x, None, eps)  # sums of zero


@pytest.mark.parametrize("normed", [False, True])
def test_padding_costs_no_more_than_rows_do(normed):
    """A batch of padding within four times the time of a batch of rows."""
    M, d = 8192, 4096
    w = torch.ones(d, dtype=torch.bfloat16, device=DEV)

    def time(x):
        graph = torch.cuda.CUDAGraph()
        binding.q8_norm(x, w, 1e-6, residual=x, with_normed=normed)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            for _ in range(8):
                binding.q8_norm(x, w, 1e-6, residual=x, with_normed=normed)
        best = float("inf")
        for _ in range(5):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            graph.replay()
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        return best

    rows = torch.randn((M, d), device=DEV).to(torch.bfloat16)
    assert time(torch.zeros_like(rows)) <= 4 * time(rows)
