"""GPU parity of the draft step's operators with their fp64 forms (draft_step_ref).

Tolerances, from the arithmetic (u = 2^-24, half(t) = finfo(t).eps / 2):

* 8-bit rows: the integers equal the fp64 formula's.  scale: the sum of squares adds at
  most 16 terms a thread (fp32, each fma u) and 10 tree levels, of squares of a sum
  rounded once: (16 + 10 + 2) u on the mean, half of that on the root, and the final
  rounding: 16 u.  normed: two roundings of p, the factor's, the root's 14 u and the
  product's: 18 u, plus half(t).  sum: u + half(t).
* product: float(acc), the scales' product and theirs: 3 u, plus half(t).
* beam keys: the exponents x * khi - mk are rounded to u |y|; terms of |y| <= 16 move by
  16 u ln 2, the others are below 2^-16 each of the largest and move by at most
  |y| 2^-|y| u; ex2.approx has 2^-22; a thread adds at most 8 x 8 / 8 terms into each of
  8 accumulators, 3 + 5 tree levels: 16 u.  Together below 12 u + 4 u + 16 u < 2^-19 on
  the sum, so on lse: 2^-19, plus u |key| for the fp32 result.
"""
import numpy as np
import pytest
import torch

import draft_step_ref as ref
import oracle
from speculative_decoding_verification_84_b200 import binding

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
LSE = 2.0 ** -19


def half(dtype):
    return torch.finfo(dtype).eps / 2


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape):
    return torch.randn(shape, generator=g)


# ----------------------------------------------------------------------------- 8-bit rows


def _check_rows(q, scale, want_q, want_scale):
    np.testing.assert_array_equal(q.cpu().numpy(), want_q)
    s = ref.f64(scale)
    assert (np.isnan(s) == np.isnan(want_scale)).all()
    fin = ~np.isnan(want_scale)
    assert (np.abs(s - want_scale)[fin] <= 16 * U * want_scale[fin] + 2.0 ** -149).all()


def _norm_case(x, r, w, eps, with_normed=True):
    dev = [t.to(DEV) if t is not None else None for t in (x, r, w)]
    out = binding.q8_norm(dev[0], dev[2], eps, residual=dev[1], with_normed=with_normed)
    f = [ref.f64(t) if t is not None else None for t in (x, r, w)]
    q, scale, s, normed = ref.q8_rows(f[0], f[1], f[2], float(np.float32(eps)))
    _check_rows(out[0], out[1], q, scale)
    h = half(x.dtype)
    tiny = 2.0 ** -133 if x.dtype == torch.bfloat16 else 2.0 ** -149
    if r is not None:
        got = ref.f64(out[2])
        assert (np.abs(got - s) <= (h + 2 * U) * np.abs(s) + tiny).all()
    if with_normed:
        got = ref.f64(out[-1])
        assert (np.isnan(got) == np.isnan(normed)).all()
        fin = ~np.isnan(normed)
        assert (np.abs(got - normed)[fin] <= (h + 18 * U) * (1 + h) * np.abs(normed)[fin] + tiny).all()
    return out


# one element, one warp, several rows a CTA, whole vectors, rows off a vector boundary,
# each register shape, and rows beyond the registers
SHAPES = [(1, 1), (3, 7), (9, 64), (17, 512), (5, 513), (2, 1000), (33, 1001), (320, 4096), (3, 4100), (4, 8192),
          (2, 16384), (1, 16400), (1, 20001), (2, 40000)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,d", SHAPES)
def test_norm_shapes(M, d, dtype):
    g = gen(M * 131 + d)
    x, r = randn(g, M, d).to(dtype), (0.3 * randn(g, M, d)).to(dtype)
    w = (1 + 0.1 * randn(g, d)).to(dtype)
    _norm_case(x, r, w, 1e-6)
    _norm_case(x, None, w, 1e-5)
    _norm_case(x, r, None, 0.0, with_normed=False)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,d", [(2500, 4096), (2500, 1001), (12001, 72), (12001, 75), (900, 8200), (700, 16383)])
def test_norm_many_rows(M, d, dtype):
    """More rows than are worked on at once, out of place and in place."""
    g = gen(M + d)
    x, r = randn(g, M, d).to(dtype), (0.3 * randn(g, M, d)).to(dtype)
    w = (1 + 0.1 * randn(g, d)).to(dtype)
    q, scale, total, normed = _norm_case(x, r, w, 1e-6)
    lib = binding.load_library()
    for where in (0, 1):
        xd, rd, wd = x.to(DEV), r.to(DEV), w.to(DEV)
        q2 = torch.empty_strided(q.shape, q.stride(), dtype=q.dtype, device=DEV)
        scale2 = torch.empty_like(scale)
        to = (xd, rd)[where]
        st = lib.spec_verify_q8_norm(xd.data_ptr(), rd.data_ptr(), wd.data_ptr(), 0 if dtype == torch.float32 else 1, 1e-6, M, d,
                                     q2.data_ptr(), q2.stride(0), scale2.data_ptr(), to.data_ptr(), None,
                                     torch.cuda.current_stream().cuda_stream)
        assert st == 0
        assert torch.equal(q2, q) and torch.equal(scale2, scale) and torch.equal(to, total)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,d", [(1, 1), (5, 96), (3, 1001), (2, 4096), (1, 131056)])
def test_quantize_shapes(M, d, dtype):
    x = (randn(gen(d), M, d) * 0.02).to(dtype)
    q, scale = binding.q8_quantize(x.to(DEV))
    want = ref.q8_rows(ref.f64(x))
    _check_rows(q, scale, want[0], want[1])
    assert q.stride(0) % 16 == 0 and q.shape == (M, d)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_halves_and_borders(dtype):
    """Values that fall on the integers' borders exactly (odd multiples of max / 254), of
    both signs: ties to even, as the formula in fp64 gives."""
    top = 127 * 2.0 ** -3
    row = torch.arange(-254, 255, dtype=torch.float64) / 254 * top  # k / 2 in units of the scale
    x = torch.stack([row, row.flip(0), row * 2, -row / 4]).to(dtype)
    for w in (None, torch.full((x.shape[1],), 0.5).to(dtype)):
        _norm_case(x, None, w, 1e-6)
        _norm_case(x, x, w, 0.0)


@pytest.mark.parametrize("d", [64, 1001, 4096, 20001])
def test_norm_extremes(d):
    """Rows of zeros, of one large channel, of values whose squares leave fp32 from above
    and below, denormals, and rows with NaN or inf."""
    g = gen(d)
    x = randn(g, 10, d)
    x[0] = 0
    x[1] = 0
    x[1, d // 2] = -3.0
    x[2] *= 1e25
    x[3] *= 1e-30
    x[4] = 1e-42
    x[5, d - 1] = float("nan")
    x[6, 0] = float("inf")
    x[7, d // 3] = float("-inf")
    x[8] *= 1e-38
    for eps in (1e-6, 0.0):
        out = _norm_case(x, None, None, eps)
        assert torch.isnan(out[1][5:8]).all() and (out[0][5:8] == 0).all() and out[1][0] == 0
    q, scale = binding.q8_quantize(x.to(DEV))
    want = ref.q8_rows(ref.f64(x))
    _check_rows(q, scale, want[0], want[1])


def test_norm_residual_in_place_and_padding():
    """out_sum over x or over the residual (the C ABI allows both), and the bytes between
    rows left as they were."""
    lib = binding.load_library()
    M, d, ld = 5, 1001, 1024
    for dtype, dt in ((torch.float32, 0), (torch.bfloat16, 1)):
        for where in ("x", "r"):
            g = gen(7)
            x, r = randn(g, M, d).to(dtype).to(DEV), randn(g, M, d).to(dtype).to(DEV)
            want = ref.q8_rows(ref.f64(x), ref.f64(r), None, 1e-6)
            q = torch.full((M, ld), 77, dtype=torch.int8, device=DEV)
            scale = torch.empty(M, device=DEV)
            to = x if where == "x" else r
            st = lib.spec_verify_q8_norm(x.data_ptr(), r.data_ptr(), None, dt, 1e-6, M, d, q.data_ptr(), ld,
                                         scale.data_ptr(), to.data_ptr(), None, torch.cuda.current_stream().cuda_stream)
            assert st == 0
            assert (q[:, d:] == 77).all()
            np.testing.assert_array_equal(q[:, :d].cpu().numpy(), want[0])
            assert (np.abs(ref.f64(to) - want[2]) <= (half(dtype) + 2 * U) * np.abs(want[2])).all()


# ----------------------------------------------------------------------------- the product


def _q8(g, rows, K, lo=-128, hi=128):
    ld = (K + 15) // 16 * 16
    buf = torch.randint(-128, 128, (rows, ld), generator=g, dtype=torch.int8)  # the padding holds anything
    buf[:, :K] = torch.randint(lo, hi, (rows, K), generator=g, dtype=torch.int8)
    return buf.to(DEV)[:, :K]


def _check_product(z, a, sa, w, sw):
    want = ref.q8_matmul(a.cpu().numpy(), ref.f64(sa), w.cpu().numpy(), ref.f64(sw))
    got = ref.f64(z)
    h = half(z.dtype)
    assert (np.abs(got - want) <= (3 * U + h) * (1 + h) * np.abs(want) + 2.0 ** -130).all()


PRODUCTS = [(1, 16, 1), (1, 1, 1), (1, 4096, 300), (2, 100, 129), (15, 128, 128), (16, 129, 127), (17, 640, 1000),
            (37, 1001, 3001), (128, 256, 512), (200, 96, 2000), (255, 512, 640), (256, 512, 641), (257, 512, 640),
            (320, 4096, 2048), (513, 300, 1030), (700, 64, 19000)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K,V", PRODUCTS)
def test_product_shapes(M, K, V, dtype):
    g = gen(M + K + V)
    a, w = _q8(g, M, K), _q8(g, V, K)
    sa = (0.5 + torch.rand(M, generator=g)).to(DEV)
    sw = (0.5 + torch.rand(V, generator=g)).to(DEV) / 64
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    z = binding.q8_matmul(a, sa, w, sw, dtype, error=err)
    assert int(err) == 0
    _check_product(z, a, sa, w, sw)


def test_product_many_rounds():
    """More tiles than SMs, several rounds of the ring and of both accumulators, the
    longest K, and the largest sums."""
    g = gen(3)
    a, w = _q8(g, 40, 2048), _q8(g, 128 * 148 * 3 + 5, 2048)
    sa, sw = torch.ones(40, device=DEV), torch.full((w.shape[0],), 2.0 ** -12, device=DEV)
    _check_product(binding.q8_matmul(a, sa, w, sw, torch.float32), a, sa, w, sw)
    K = binding.Q8_MAX_K
    a = torch.full((3, K), -128, dtype=torch.int8, device=DEV)
    w = torch.full((130, K), -128, dtype=torch.int8, device=DEV)
    w[1] = 127
    sa, sw = torch.ones(3, device=DEV), torch.ones(130, device=DEV)
    z = binding.q8_matmul(a, sa, w, sw, torch.float32)
    want = np.full((3, 130), 128.0 * 128 * K)
    want[:, 1] = -128.0 * 127 * K
    assert (np.abs(ref.f64(z) - want) <= 3 * U * np.abs(want)).all()


def test_product_scales_that_are_not_finite():
    """A token whose scale is NaN has NaN logits, which the verifier reports; the other
    tokens keep theirs."""
    g = gen(5)
    a, w = _q8(g, 4, 64), _q8(g, 200, 64)
    sa, sw = torch.ones(4, device=DEV), torch.ones(200, device=DEV)
    sa[2] = float("nan")
    z = binding.q8_matmul(a, sa, w, sw, torch.float32)
    assert torch.isnan(z[2]).all() and torch.isfinite(z[[0, 1, 3]]).all()


@pytest.mark.parametrize("xdt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,d,V", [(1, 512, 1000), (5, 1001, 640), (320, 256, 3001)])
def test_head_is_norm_then_product(M, d, V, xdt):
    g = gen(M + d)
    x, r = randn(g, M, d).to(xdt).to(DEV), randn(g, M, d).to(xdt).to(DEV)
    w = (1 + 0.1 * randn(g, d)).to(xdt).to(DEV)
    wq, ws = binding.q8_quantize((randn(g, V, d) / 16).to(DEV))
    q, scale, total = binding.q8_norm(x, w, 1e-6, residual=r)
    z = binding.q8_matmul(q, scale, wq, ws)
    z2, total2 = binding.q8_head(x, w, 1e-6, wq, ws, residual=r)
    assert torch.equal(z, z2) and torch.equal(total, total2)
    z3 = binding.q8_head(total, w, 1e-6, wq, ws, torch.float32)
    q, scale = binding.q8_norm(total, w, 1e-6)
    assert torch.equal(z3, binding.q8_matmul(q, scale, wq, ws, torch.float32))


# ----------------------------------------------------------------------------- beams


def _check_select(logits, scores, temperature, K, frozen=None, pad=0, exact=False):
    """Against the fp64 keys: each slot's key within the tolerance of the reference's, every
    pick a different candidate, and the picks equal wherever the keys are further apart
    than twice the tolerance (everywhere with ``exact``)."""
    dev = [t.to(DEV) if t is not None else None for t in (logits, scores, temperature, frozen)]
    parent, token, score, status = binding.beam_select(dev[0], dev[1], dev[2], K, frozen=dev[3], pad_token=pad,
                                                       return_row_status=True)
    keys, st = ref.beam_keys(ref.f64(logits), ref.f64(scores), ref.f64(temperature),
                             frozen.numpy() if frozen is not None else None, pad)
    wp, wt, wk = ref.beam_select(keys, K + 1)
    gp, gt, gs = parent.cpu().numpy(), token.cpu().numpy(), ref.f64(score)
    np.testing.assert_array_equal(status.cpu().numpy(), st)
    for b in range(keys.shape[0]):
        n = int((wk[b, :K] > -np.inf).sum())
        assert (gp[b, n:] == -1).all() and (gt[b, n:] == -1).all() and (gs[b, n:] == -np.inf).all()
        assert len(set(zip(gp[b, :n].tolist(), gt[b, :n].tolist()))) == n
        for k in range(n):
            tol = LSE + U * abs(wk[b, k])
            assert abs(gs[b, k] - wk[b, k]) <= tol, (b, k)
            assert abs(keys[b, gp[b, k], gt[b, k]] - wk[b, k]) <= 2 * tol, (b, k)
            near = not exact and ((k > 0 and wk[b, k - 1] - wk[b, k] <= 2 * tol) or
                                  (wk[b, k + 1] > -np.inf and wk[b, k] - wk[b, k + 1] <= 2 * tol))
            assert near or (gp[b, k], gt[b, k]) == (wp[b, k], wt[b, k]), (b, k)
    return parent, token, score


def _temps(B):
    return torch.tensor([1.0, 0.7, 1.5, 0.6])[torch.arange(B) % 4]


BEAMS = [(1, 1, 1, 1), (2, 2, 2, 5), (3, 1, 7, 32), (2, 4, 64, 4), (5, 3, 257, 8), (1, 4, 3001, 4), (4, 8, 1000, 8),
         (3, 32, 999, 32), (1, 16, 32000, 31), (2, 5, 32001, 7), (1, 2, 128256, 16), (1, 3, 128257, 8), (40, 8, 4099, 6)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,W,V,K", BEAMS)
def test_select_shapes(B, W, V, K, dtype):
    g = gen(B + W + V + K)
    logits = (3 * randn(g, B, W, V)).to(dtype)
    _check_select(logits, -5 * torch.rand(B, W, generator=g), _temps(B), K)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_select_long_vocabulary(dtype):
    """Several segments of the largest size, and the largest vocabulary."""
    g = gen(11)
    V = 1 << 20
    logits = (3 * randn(g, 1, 2, V)).to(dtype)
    _check_select(logits, -torch.rand(1, 2, generator=g), _temps(1), 32)
    # many rows: segments of 8 vectors a thread
    logits = (3 * randn(g, 20, 16, 20011)).to(dtype)
    _check_select(logits, -torch.rand(20, 16, generator=g), _temps(20), 9)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [5, 300, 3001, 40000])
def test_select_ties(V, dtype):
    """Equal logits, equal rows (wherever they lie in memory) and equal scores: the lower
    beam, then the lower token."""
    W = 4
    flat = torch.zeros(2, W, V).to(dtype)
    flat[1] = -2.5
    _check_select(flat, torch.zeros(2, W), torch.ones(2), 32, exact=True)
    g = gen(V)
    row = torch.randint(-3, 4, (V,), generator=g).float()  # seven values: ties everywhere
    same = row.expand(1, W, V).contiguous().to(dtype)
    _check_select(same, torch.zeros(1, W), torch.ones(1), 32, exact=True)
    _check_select(same, torch.tensor([[-1.0, 0.0, -1.0, 0.0]]), torch.ones(1), 32, exact=True)
    # +0 and -0 are equal
    z = torch.zeros(1, 1, V)
    z[0, 0, ::2] = -0.0
    _check_select(z.to(dtype), torch.zeros(1, 1), torch.ones(1), 7, exact=True)


@pytest.mark.parametrize("W,K", [(8, 32), (32, 32), (32, 5), (17, 31)])
def test_select_ties_over_many_beams(W, K):
    """More candidates than the last step ranks at once, all keys equal, or two values of
    them, or none at all but a few."""
    V = 300
    flat = torch.zeros(3, W, V)
    flat[1, :, ::2] = 1.0
    flat[2] = float("-inf")
    flat[2, :, 7] = 0.5
    scores = torch.zeros(3, W)
    scores[2, 1:] = float("-inf")
    scores[2, W - 1] = 0.0
    _check_select(flat, scores, torch.ones(3), K, exact=True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [700, 40000, 128256])
def test_select_sorted_logits(V, dtype):
    """The best logits side by side at one end of the row, at the other, and in one place."""
    up = torch.linspace(-8, 8, V)
    bump = torch.full((V,), -5.0)
    bump[V // 2 : V // 2 + 40] = torch.linspace(1, 5, 40)
    rows = torch.stack([up, up.flip(0), bump]).to(dtype)
    scores = torch.tensor([[0.0, -0.125, -0.25]])
    for K in (1, 9, 32):
        _check_select(rows[None], scores, torch.ones(1), K)
    one = rows[:1].expand(1, 2, V).contiguous()
    _check_select(one, torch.zeros(1, 2), torch.ones(1), 32, exact=True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [40, 3001, 33000])
def test_select_masks(V, dtype):
    g = gen(V)
    B, W, K = 5, 3, 6
    logits = (3 * randn(g, B, W, V)).to(dtype)
    low = torch.finfo(dtype).min
    logits[0, :, 3:] = float("-inf")                # three tokens a beam
    logits[1, 1] = float("-inf")                    # a beam without any: status 2
    logits[1, 0, : V // 2] = low                    # masked by the type's lowest value
    logits[2, :, 2:] = low                          # two tokens a beam above it
    logits[3] = float("-inf")
    logits[3, 2, V - 1] = 1.0                       # one token in all
    scores = -torch.rand(B, W, generator=g)
    dev = [t.to(DEV) for t in (logits, scores)]
    parent, token, score, status = binding.beam_select(dev[0], dev[1], torch.ones(B, device=DEV), K, return_row_status=True)
    keys, st = ref.beam_keys(ref.f64(logits), ref.f64(scores), np.ones(B))
    wp, wt, wk = ref.beam_select(keys, K)
    np.testing.assert_array_equal(status.cpu().numpy(), st)
    np.testing.assert_array_equal(parent.cpu().numpy(), wp)
    np.testing.assert_array_equal(token.cpu().numpy(), wt)
    got = ref.f64(score)
    fin = wk > -1e38
    with np.errstate(invalid="ignore"):
        off = np.abs(got - wk)
    assert (off[fin] <= LSE + U * np.abs(wk[fin])).all()
    assert (got[wk == -np.inf] == -np.inf).all() and (got[~fin] < -1e38).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_select_first_level_frozen_and_greedy(dtype):
    g = gen(21)
    B, W, V, K = 6, 4, 2050, 5
    logits = (3 * randn(g, B, W, V)).to(dtype)
    scores = -torch.rand(B, W, generator=g)
    scores[0] = torch.tensor([0.0] + [float("-inf")] * 3)
    scores[1] = float("-inf")                       # nothing at all
    logits[0, 1:] = float("nan")                    # beams that are out are not read
    logits[1] = float("nan")
    frozen = torch.zeros(B, W, dtype=torch.int32)
    frozen[2] = 1
    frozen[3, 1] = 1
    frozen[4, 2] = -7
    logits[2] = float("nan")                        # nor are frozen ones
    temp = torch.tensor([1.0, 1.0, 1.0, 0.0, 0.7, 0.0])
    _check_select(logits, scores, temp, K, frozen=frozen, pad=9)
    _check_select(logits[3:], scores[3:], temp[3:], K)


def test_select_faults():
    """Bad temperatures, scores and rows: reported, and only the beam at fault is out."""
    g = gen(22)
    B, W, V = 9, 3, 700
    logits = 3 * randn(g, B, W, V)
    scores = -torch.rand(B, W, generator=g)
    temp = torch.ones(B)
    temp[0], temp[1], temp[2], temp[3] = -1.0, float("nan"), float("inf"), 1e-7
    scores[4, 1] = float("nan")
    scores[5, 0] = float("inf")
    logits[6, 2, 13] = float("nan")
    logits[7, 0, 699] = float("inf")
    logits[8, 1] = float("nan")
    frozen = torch.zeros(B, W, dtype=torch.int32)
    frozen[0, 1] = 1                                # counts whatever the temperature
    _check_select(logits, scores, temp, 4, frozen=frozen, pad=3)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.uint8])
@pytest.mark.parametrize("shape", [(1, 1, 1, 1, 1, 1, 1), (2, 3, 4, 5, 2, 7, 8), (1, 2, 3, 3, 1, 1, 33),
                                   (3, 2, 8, 8, 4, 100, 64), (1, 5, 32, 32, 2, 3, 10), (2, 1, 1, 6, 3, 513, 24)])
def test_reorder(shape, dtype):
    L, B, W, K, H, S, D = shape
    g = gen(sum(shape))
    src = torch.randint(0, 256, (L, B, W, H, S, D), generator=g).to(dtype)
    parent = torch.randint(0, W, (B, K), generator=g, dtype=torch.int32)
    got = binding.beam_reorder(src.to(DEV), parent.to(DEV))
    assert torch.equal(got.cpu(), ref.reorder(src, parent, torch.zeros((L, B, K, H, S, D), dtype=dtype)))
    # lengths from none to more than there is, parents that are none: the rest stays
    lengths = torch.randint(-1, S + 2, (B,), generator=g, dtype=torch.int32)
    parent[torch.rand(B, K, generator=g) < 0.3] = -1
    parent[0, 0] = W
    out = torch.randint(0, 256, (L, B, K, H, S, D), generator=g).to(dtype)
    got = binding.beam_reorder(src.to(DEV), parent.to(DEV), out=out.to(DEV), lengths=lengths.to(DEV))
    assert torch.equal(got.cpu(), ref.reorder(src, parent, out, lengths))


def test_reorder_refuses_overlap():
    src = torch.zeros(1, 1, 2, 1, 4, 8, device=DEV)
    parent = torch.zeros(1, 2, dtype=torch.int32, device=DEV)
    with pytest.raises(binding.SpecVerifyError):
        binding.beam_reorder(src, parent, out=src)


# ----------------------------------------------------------------------------- together


class _Draft:
    """A small recurrent draft: state s, hidden x = s, residual r = embedding of the token."""

    def __init__(self, B, d, V, seed):
        g = gen(seed)
        self.d, self.V = d, V
        self.emb = randn(g, V, d).to(torch.bfloat16).to(DEV)
        self.norm = (1 + 0.1 * randn(g, d)).to(torch.bfloat16).to(DEV)
        self.wq, self.ws = binding.q8_quantize((randn(g, V, d) * 3 / d ** 0.5).to(torch.bfloat16).to(DEV))
        self.state = randn(g, 1, B, 1, 1, 1, d).to(torch.bfloat16).to(DEV)

    def step(self, state, token):
        """state [1, B, W, 1, 1, d], token [B, W]: logits [B, W, V] and the next state."""
        B, W = token.shape
        z, s = binding.q8_head(state.reshape(B * W, self.d), self.norm, 1e-6, self.wq, self.ws,
                               residual=self.emb[token.long().clamp(min=0)].reshape(B * W, self.d))
        return z.reshape(B, W, self.V), s.reshape(1, B, W, 1, 1, self.d)


def _grow(m, B, K, depth, first):
    """A tree of ``depth`` levels of K nodes under the root: (parent, token [B, N], rows
    [B, N, V] of draft logits at each node, the calls' inputs and outputs)."""
    temp = torch.ones(B, device=DEV)
    logits, state = m.step(m.state, first)
    scores = torch.zeros(B, 1, device=DEV)
    parent, token, rows, calls, base = [torch.full((B, 1), -1, dtype=torch.int32, device=DEV)], [first], [logits], [], 0
    for level in range(depth):
        p, t, s = binding.beam_select(logits, scores, temp, K)
        calls.append((logits, scores, p, t, s))
        state = binding.beam_reorder(state, p)
        parent.append(p + base)
        token.append(t)
        base += 1 if level == 0 else K
        logits, state = m.step(state, t)
        rows.append(logits)
        scores = s
    return torch.cat(parent, 1), torch.cat(token, 1), torch.cat(rows, 1), calls


def test_grown_tree_is_verified():
    """Hidden states to logits to the chosen level to the reordered states, three levels:
    every level the fp64 selection's, every node's row the draft's at the node's path; then
    the tree to the verifier, against the oracle."""
    B, d, V, K, depth = 3, 64, 500, 4, 3
    m = _Draft(B, d, V, 1)
    first = torch.tensor([[1], [2], [3]], dtype=torch.int32, device=DEV)
    parent, token, rows, calls = _grow(m, B, K, depth, first)
    for logits, scores, p, t, s in calls:
        keys, _ = ref.beam_keys(ref.f64(logits), ref.f64(scores), np.ones(B))
        wk = ref.beam_select(keys, K)[2]
        assert (np.abs(ref.f64(s) - wk) <= LSE + U * np.abs(wk)).all()
    # every node's row is the draft's at its path: the states followed their parents
    par, tok = parent.cpu().numpy(), token.cpu().numpy()
    for b in range(B):
        for n in (1, K, K + 1, 2 * K, 3 * K):
            path, at = [], n
            while at >= 0:
                path.append(int(tok[b, at]))
                at = int(par[b, at])
            state = m.state[:, b:b + 1]
            for x in reversed(path):
                z, state = m.step(state, torch.tensor([[x]], dtype=torch.int32, device=DEV))
            assert torch.equal(z[0, 0], rows[b, n])
    N = parent.shape[1]
    uni = torch.full((B, N), 0.5, device=DEV)
    nodes, toks, n, st = binding.tree_verify(rows.contiguous(), rows.contiguous(), parent.contiguous(), token.contiguous(),
                                             torch.zeros(B, device=DEV), uni, uni[:, 0].contiguous(), return_row_status=True)
    assert (st == 0).all()
    want = oracle.tree_verify(rows.cpu().view(torch.int16).numpy().view(np.uint16), rows.cpu().view(torch.int16).numpy().view(np.uint16),
                              par, tok, np.zeros(B, np.float32), uni.cpu().numpy(), uni[:, 0].cpu().numpy())
    np.testing.assert_array_equal(toks.cpu().numpy(), want.out_tokens)
    np.testing.assert_array_equal(n.cpu().numpy(), want.n_accepted)


def test_captured_step_replays_with_new_inputs():
    """Head, selection and reordering captured into two graphs that live at once, replayed
    with other inputs: the results of the eager calls."""
    B, W, d, V, K = 2, 3, 128, 1000, 4
    m = _Draft(B, d, V, 2)
    g = gen(9)
    graphs = []
    for _ in range(2):
        state = randn(g, 1, B, W, 1, 1, d).to(torch.bfloat16).to(DEV)
        token = torch.randint(0, V, (B, W), generator=g, dtype=torch.int32).to(DEV)
        scores = -torch.rand(B, W, generator=g).to(DEV)
        temp = torch.ones(B, device=DEV)

        def step(state=state, token=token, scores=scores, temp=temp):
            z, s = m.step(state, token)
            out = binding.beam_select(z, scores, temp, K)
            return (*out, binding.beam_reorder(s, out[0]), z)

        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = step()
        graphs.append((graph, outs, step, state, token, scores))
    for round_ in range(3):
        for graph, outs, step, state, token, scores in graphs:
            state.copy_(randn(g, *state.shape))
            token.copy_(torch.randint(0, V, token.shape, generator=g, dtype=torch.int32))
            scores.copy_(-torch.rand(scores.shape, generator=g))
        for graph, *_ in graphs:
            graph.replay()
        for graph, outs, step, *_ in graphs:
            for x, y in zip(outs, step()):
                assert torch.equal(x, y)


def test_two_streams_at_once():
    """The same calls on two streams that overlap, with the library's own workspaces."""
    g = gen(12)
    B, W, V, K, d = 8, 4, 32000, 4, 512
    x = [randn(g, B * W, d).to(torch.bfloat16).to(DEV) for _ in range(2)]
    wq, ws = binding.q8_quantize((randn(g, V, d) / 8).to(DEV))
    scores = [-torch.rand(B, W, generator=g).to(DEV) for _ in range(2)]
    temp = torch.ones(B, device=DEV)

    def step(i, stream):
        z = binding.q8_head(x[i], None, 1e-6, wq, ws, stream=stream)
        return (z, *binding.beam_select(z.view(B, W, V), scores[i], temp, K, stream=stream))

    want = [step(i, None) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        got = [step(i, streams[i]) for i in range(2)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        for u, v in zip(a, b):
            assert torch.equal(u, v)


def test_results_do_not_depend_on_the_run():
    g = gen(13)
    logits = (3 * randn(g, 4, 8, 32000)).to(torch.bfloat16).to(DEV)
    scores = -torch.rand(4, 8, generator=g).to(DEV)
    first = binding.beam_select(logits, scores, torch.ones(4, device=DEV), 16)
    for _ in range(20):
        for u, v in zip(first, binding.beam_select(logits, scores, torch.ones(4, device=DEV), 16)):
            assert torch.equal(u, v)


def test_refusals_on_the_gpu():
    q = torch.zeros(4, 40, dtype=torch.int8, device=DEV)  # a pitch of 40
    one = torch.ones(4, device=DEV)
    good, gs = binding.q8_quantize(torch.ones(4, 40, device=DEV))
    x = torch.ones(4, 40, device=DEV)
    logits = torch.zeros(2, 3, 50, device=DEV)
    for call, error in ((lambda: binding.q8_matmul(q, one, good, gs), ValueError),
                        (lambda: binding.q8_matmul(good, gs, good.t(), gs), ValueError),
                        (lambda: binding.q8_matmul(good, gs, good, gs, torch.float16), TypeError),
                        (lambda: binding.q8_matmul(good, gs.double(), good, gs), TypeError),
                        (lambda: binding.q8_norm(x.half(), None, 1e-6), TypeError),
                        (lambda: binding.q8_norm(x, one, 1e-6), ValueError),
                        (lambda: binding.q8_norm(x, None, -1.0), binding.SpecVerifyError),
                        (lambda: binding.q8_norm(x[:, ::2], None, 1e-6), ValueError),
                        (lambda: binding.beam_select(logits, one.view(2, 2), one[:2], 3), ValueError),
                        (lambda: binding.beam_select(logits, torch.zeros(2, 3, device=DEV), one[:2], 33), binding.SpecVerifyError),
                        (lambda: binding.beam_select(logits, torch.zeros(2, 3, device=DEV), one[:2], 0), binding.SpecVerifyError)):
        with pytest.raises(error):
            call()
