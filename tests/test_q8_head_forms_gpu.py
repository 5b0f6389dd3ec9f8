"""The int8 product and the 8-bit head in each form that the product takes: single SMs or
pairs, one accumulator a tile or two, one or two K blocks a stage.  ``_cut`` restates the
rule by which a call gets its form, so that each case here names the form it reaches.

Tolerance: the sum, the scales' product and theirs are each rounded to fp32 (3 u, u =
2^-24), then to the output's type (half a step, finfo.eps / 2).
"""
import pytest
import torch

from speculative_decoding_verification_84_b200 import binding

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
RING = 227 * 1024 - 2048  # bytes of a ring of stages


def _cdiv(a, b):
    return -(-a // b)


def _cut(M, K, V, pairs_at_once):
    """(pairs, tokens of an accumulator, accumulators of a tile, K blocks of a stage, tiles
    that a CTA walks at most)."""
    kbs, accs = _cdiv(K, 128), _cdiv(M, 256)
    pairs = _cdiv(accs * _cdiv(V, 256), pairs_at_once) * kbs >= 32
    unit = 32 if pairs else 16
    units = pairs_at_once if pairs else torch.cuda.get_device_properties(0).multi_processor_count
    v_tiles, parts = _cdiv(V, 256 if pairs else 128), accs
    if parts * v_tiles < units:
        parts = min(units // v_tiles, max(accs, _cdiv(M, 32)))
    nt = _cdiv(_cdiv(M, parts), unit) * unit
    parts = _cdiv(M, nt)
    groups = 2 if pairs and parts == 2 and nt <= 160 and 9 * _cdiv(v_tiles, units) < 5 * _cdiv(2 * v_tiles, units) else 1
    block = 128 * 128 + groups * (nt // 2 if pairs else nt) * 128
    return pairs, nt, groups, 2 if 4 * 2 * block <= RING else 1, _cdiv(_cdiv(parts, groups) * v_tiles, units)


def _form(M, K, V):
    # pairs of SMs that are resident at once: 74 where every SM has a partner, fewer where
    # some have none; a case here has one form for all of them
    forms = {_cut(M, K, V, n)[:4] for n in (70, 72, 74)}
    assert len(forms) == 1, forms
    return forms.pop(), min(_cut(M, K, V, n)[4] for n in (70, 72, 74))


def _gen(*sizes):
    return torch.Generator().manual_seed(sum(sizes))


def _q8(g, rows, K):
    ld = (K + 15) // 16 * 16
    return torch.randint(-128, 128, (rows, ld), generator=g, dtype=torch.int8).to(DEV)[:, :K]


def _check(z, a, sa, w, sw):
    # the exact sums on the GPU, in fp64 a stretch of channels at a time
    h = torch.finfo(z.dtype).eps / 2
    for v in range(0, w.shape[0], 8192):
        want = (a.double() @ w[v : v + 8192].double().T) * sa.double()[:, None] * sw[v : v + 8192].double()
        off = (z[:, v : v + 8192].double() - want).abs()
        assert (off <= (3 * U + h) * (1 + h) * want.abs() + 2.0 ** -130).all(), (v, off.max())


# (M, K, V): pairs, tokens of an accumulator, accumulators of a tile, K blocks of a stage
FORMS = {
    (257, 1024, 35000): (True, 160, 2, 1),   # 97 tokens in the second accumulator
    (320, 1100, 51177): (True, 160, 2, 1),   # three tiles a CTA; K and V off every boundary
    (300, 768, 69001): (True, 160, 2, 1),    # four, of as many K blocks as the ring has stages
    (300, 200, 152000): (True, 160, 2, 1),   # many, shorter than the ring
    (256, 2000, 38000): (True, 256, 1, 1),
    (1000, 1152, 15000): (True, 256, 1, 1),
    (2048, 640, 25000): (True, 256, 1, 1),
    (2048, 100, 76001): (True, 256, 1, 1),   # one K block
    (5, 4096, 20001): (True, 32, 1, 2),
    (320, 1024, 56833): (True, 160, 1, 2),
    (700, 1025, 12000): (False, 240, 1, 1),
}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K,V", FORMS)
def test_product_forms(M, K, V, dtype):
    form, rounds = _form(M, K, V)
    assert form == FORMS[M, K, V] and rounds > 1
    g = _gen(M, K, V)
    a, w = _q8(g, M, K), _q8(g, V, K)
    sa = (0.5 + torch.rand(M, generator=g)).to(DEV)
    sw = (0.5 + torch.rand(V, generator=g)).to(DEV) / 64
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    z = binding.q8_matmul(a, sa, w, sw, dtype, error=err)
    assert int(err) == 0
    _check(z, a, sa, w, sw)


@pytest.mark.parametrize("xdt,dtype", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("M,d,V", [(5, 4096, 20001), (300, 768, 69001), (257, 1024, 35000), (1000, 1152, 15000)])
def test_head_forms(M, d, V, xdt, dtype):
    """The norm and the product that overlaps it, several times in a row: the halves' results
    to the bit, and the product of the norm's integers."""
    form, _ = _form(M, d, V)
    assert form == FORMS[M, d, V]
    g = _gen(M, d, V)
    w, ws = binding.q8_quantize((torch.randn((V, d), generator=g) / 16).to(torch.bfloat16).to(DEV))
    norm = (1 + 0.1 * torch.randn(d, generator=g)).to(xdt).to(DEV)
    for _ in range(3):
        x, r = [torch.randn((M, d), generator=g).to(xdt).to(DEV) for _ in range(2)]
        z, total = binding.q8_head(x, norm, 1e-6, w, ws, dtype, residual=r)
        q, scale, total2 = binding.q8_norm(x, norm, 1e-6, residual=r)
        assert torch.equal(total, total2)
        assert torch.equal(z, binding.q8_matmul(q, scale, w, ws, dtype))
    _check(z, q, scale, w, ws)


@pytest.mark.parametrize("xdt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,d,V", [(1, 512, 1000), (64, 1024, 2001)])
def test_heads_in_a_row_share_a_workspace(M, d, V, xdt):
    """Calls one after the other, each with other hidden states, in one workspace: the
    product of each reads the integers and scales that its own norm left there."""
    g = _gen(M, d, V)
    wq, ws = binding.q8_quantize((torch.randn((V, d), generator=g) / 16).to(DEV))
    lib = binding.load_library()
    work = torch.empty(lib.spec_verify_q8_head_workspace_size(M, d), dtype=torch.uint8, device=DEV)
    xs = [(torch.randn((M, d), generator=g) * 4.0 ** (i % 5 - 2)).to(xdt).to(DEV) for i in range(16)]
    want = []
    for x in xs:
        q, scale = binding.q8_norm(x, None, 1e-6)
        want.append(binding.q8_matmul(q, scale, wq, ws))
    torch.cuda.synchronize()
    for _ in range(4):
        got = [binding.q8_head(x, None, 1e-6, wq, ws, workspace=work) for x in xs]
        for a, b in zip(got, want):
            assert torch.equal(a, b)
