"""Selection over beams at logits far from a softmax's usual range: whole stretches of the
vocabulary at a finite mask value, logits / T up to fp32's largest, greedy rows of any
finite logits.

Tolerance of a key: 2^-19 on the normaliser (derived in test_draft_step_gpu), plus
2^-24 |key| for the fp32 result and 2^-51 |key| for the fp64 steps.  The reference takes
(l - max) / T, whose roundings are relative to the difference.
"""
import numpy as np
import pytest
import torch

import draft_step_ref as ref
from speculative_decoding_verification_84_b200 import binding

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
LSE = 2.0 ** -19
MAX = float(torch.finfo(torch.float32).max)


def _keys(logits, scores, temperature):
    """[B, W, V] keys and [B, W] whether a row is at fault, in fp64."""
    keys = np.full(logits.shape, -np.inf)
    bad = np.zeros(logits.shape[:2], bool)
    for b, w in np.ndindex(bad.shape):
        row, T = logits[b, w], float(temperature[b])
        top = row.max()
        bad[b, w] = not np.isfinite(top) or (T > 0 and abs(top / T) > MAX)
        if bad[b, w]:
            continue
        if T == 0:
            keys[b, w, int(np.argmax(row))] = scores[b, w]
        else:
            d = (row - top) / T
            keys[b, w] = scores[b, w] + (d - np.log(np.exp(d).sum()))
    return keys, bad


def _select(keys, logits, K):
    """(parent, token, key): decreasing key, then the lower beam, the larger logit (two
    logits of a beam may have one fp64 key) and the lower token."""
    B, W, V = keys.shape
    parent, token, key = np.full((B, K), -1), np.full((B, K), -1), np.full((B, K), -np.inf)
    for b in range(B):
        flat = keys[b].reshape(-1)
        order = np.lexsort((-logits[b].reshape(-1), np.arange(W * V) // V, -flat))[:K]
        order = order[flat[order] > -np.inf]
        n = len(order)
        parent[b, :n], token[b, :n], key[b, :n] = order // V, order % V, flat[order]
    return parent, token, key


def _check(logits, scores, temperature, K):
    got = binding.beam_select(logits.to(DEV), scores.to(DEV), temperature.to(DEV), K, return_row_status=True)
    keys, bad = _keys(ref.f64(logits), ref.f64(scores), ref.f64(temperature))
    wp, wt, wk = _select(keys, ref.f64(logits), K + 1)
    gp, gt, gs, status = got[0].cpu().numpy(), got[1].cpu().numpy(), ref.f64(got[2]), got[3].cpu().numpy()
    np.testing.assert_array_equal(status, 2 * bad.any(axis=1))
    for b in range(keys.shape[0]):
        n = int((wk[b, :K] > -np.inf).sum())
        assert (gp[b, n:] == -1).all() and (gt[b, n:] == -1).all()
        for k in range(n):
            tol = LSE + (2.0 ** -24 + 2.0 ** -51) * abs(wk[b, k])
            assert abs(gs[b, k] - wk[b, k]) <= tol, (b, k, gs[b, k], wk[b, k])
            near = (k > 0 and wk[b, k - 1] != wk[b, k] and wk[b, k - 1] - wk[b, k] <= 2 * tol) or \
                   (wk[b, k + 1] > -np.inf and wk[b, k] != wk[b, k + 1] and wk[b, k] - wk[b, k + 1] <= 2 * tol)
            assert near or (gp[b, k], gt[b, k]) == (wp[b, k], wt[b, k]), (b, k)


def _rows(seed, B, W, V):
    return 3 * torch.randn((B, W, V), generator=torch.Generator().manual_seed(seed))


# V: rows of one batch, of several, off and on a 16-byte boundary
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [700, 6000, 12001])
@pytest.mark.parametrize("mask", [-1e4, -1e9, -3e9, -1e10, -7e20, -1e30, -2.2e38])
def test_masked_stretches(V, mask, dtype):
    """A mask value over all tokens but a few hundred, at either end, and noise on it: the
    masked tokens have no weight, and the row is as good as any other."""
    B, W, K = 4, 3, 6
    logits = _rows(V, B, W, V)
    logits[0, :, 200:] = mask
    logits[1, :, : V - 200] = mask
    logits[2, :, 100 : V - 100] = mask * (1 + 0.2 * torch.rand(W, V - 200, generator=torch.Generator().manual_seed(1)))
    scores = -torch.rand((B, W), generator=torch.Generator().manual_seed(2))
    _check(logits.to(dtype), scores, torch.tensor([1.0, 0.7, 1.0, 1.3]), K)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [700, 6000, 12001])
@pytest.mark.parametrize("size", [1e6, 3e8, 1e9, 7e10, 2.5e21, 1e30, 1.1e38])
def test_large_logits(V, size, dtype):
    """Rows of that size, of either sign, with a few equal best tokens far apart and some
    near them, at temperatures from 0 up."""
    W, K = 2, 5
    temps = torch.tensor([1.0, 0.0, 0.5, 1.7, 1.0, 0.0])
    B = len(temps)
    logits = _rows(V + 1, B, W, V) * (size / 30)
    best = torch.tensor(size).to(dtype).float()
    step = best * 2.0 ** -7  # the next value of either type
    for i in (3, V // 3, V - 2):
        logits[:, :, i] = best
    logits[:, 1, V // 2] = best - step
    logits[4:] -= 2 * best  # all negative
    if size == 1e6:
        temps[3] = 1e-6
    scores = -torch.rand((B, W), generator=torch.Generator().manual_seed(3))
    _check(logits.to(dtype), scores, temps, K)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_greedy_rows_of_any_size(dtype):
    """T = 0: the first argmax, with maxima of different sizes in different stretches."""
    V = 9000
    logits = _rows(5, 5, 1, V)
    logits[0, 0, 10], logits[0, 0, V - 10] = 1e21, 2e21
    logits[1, 0, 10], logits[1, 0, V - 10] = 3e38, 1e19
    logits[2, 0, 5000] = 2.0 ** 68
    logits[3] = -3e38
    logits[3, 0, 4000] = -1e38
    logits[4] = torch.finfo(dtype).min
    _check(logits.to(dtype), torch.zeros(5, 1), torch.zeros(5), 3)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_the_end_of_the_range(dtype):
    """logits / T up to fp32's largest are taken; beyond it, above or with all below, the
    row is at fault, and NaN is found beside values of any size."""
    V = 5000
    logits = _rows(6, 9, 1, V)
    temps = torch.ones(9)
    logits[0, 0, 77] = 3e38
    logits[1, 0, 77], temps[1] = 2.6e38, 0.8   # 3.25e38, though log2(e) times it is beyond
    logits[2, 0, 77], temps[2] = 3e38, 0.5     # 6e38
    logits[3] = -3e38
    logits[4], temps[4] = -3e38, 0.5
    logits[5, 0, 77], logits[5, 0, 78] = 3e38, float("nan")
    logits[6, 0, 77], logits[6, 0, 4000], temps[6] = 1e20, float("nan"), 0.0
    logits[7, 0, 2048:], logits[7, 0, 4999] = -1e30, float("nan")
    logits[8, 0, 77] = float("inf")
    _check(logits.to(dtype), torch.zeros(9, 1), temps, 4)
