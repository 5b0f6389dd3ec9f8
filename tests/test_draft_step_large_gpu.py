"""The draft step's operators on arrays of more than 2^31 elements (2^32 bytes): the last
rows, and some from the middle, are those that a call on them alone gives, to the bit."""
import pytest
import torch

from speculative_decoding_verification_84_b200 import binding

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
PAST = (1 << 31) + 12345


@pytest.fixture(autouse=True)
def _give_back():
    yield
    torch.cuda.empty_cache()


def _rows(M, d, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.empty((M, d), dtype=torch.bfloat16, device=DEV)
    for i in range(0, M, 1 << 16):
        x[i : i + (1 << 16)] = torch.randn(x[i : i + (1 << 16)].shape, generator=g, device=DEV)
    return x


@pytest.mark.parametrize("d", [4096, 4001])
def test_norm(d):
    M = PAST // d + 3
    x = _rows(M, d, d)
    w = (1 + 0.1 * torch.randn(d, device=DEV)).to(torch.bfloat16)
    q, scale, total, normed = binding.q8_norm(x, w, 1e-6, residual=x, with_normed=True)
    for rows in (slice(0, 5), slice(M // 2, M // 2 + 7), slice(M - 16, M)):
        part = x[rows].clone()
        want = binding.q8_norm(part, w, 1e-6, residual=part, with_normed=True)
        for a, b in zip((q, scale, total, normed), want):
            assert torch.equal(a[rows], b)


@pytest.mark.parametrize("V", [128256, 128257])
def test_product(V):
    M, K = PAST // V + 3, 256
    g = torch.Generator(device=DEV).manual_seed(1)
    a, w = [torch.randint(-128, 128, (n, K), generator=g, device=DEV, dtype=torch.int8) for n in (M, V)]
    sa, sw = torch.rand(M, generator=g, device=DEV), torch.rand(V, generator=g, device=DEV)
    z = binding.q8_matmul(a, sa, w, sw)
    for rows in (slice(0, 5), slice(M // 2, M // 2 + 7), slice(M - 16, M)):
        assert torch.equal(z[rows], binding.q8_matmul(a[rows].clone(), sa[rows].clone(), w, sw))


@pytest.mark.parametrize("V", [128256, 128257])
def test_select(V):
    W, K = 8, 8
    B = PAST // (W * V) + 2
    logits = _rows(B * W, V, 2).view(B, W, V)
    scores = -torch.rand((B, W), device=DEV)
    temp = torch.ones(B, device=DEV)
    got = binding.beam_select(logits, scores, temp, K)
    for rows in (slice(0, 2), slice(B // 2, B // 2 + 3), slice(B - 4, B)):
        want = binding.beam_select(logits[rows].clone(), scores[rows].clone(), temp[rows].clone(), K)
        for a, b in zip(got, want):
            assert torch.equal(a[rows], b)


@pytest.mark.parametrize("D,dtype", [(128, torch.bfloat16), (3, torch.uint8)])
def test_reorder(D, dtype):
    L, W, K, H = 3, 3, 4, 2
    S = (1 << 32) // (L * W * H * D * torch.empty(0, dtype=dtype).element_size()) + 7
    src = torch.empty((L, 1, W, H, S, D), dtype=dtype, device=DEV)
    for l in range(L):
        for w in range(W):
            at = torch.arange(S, device=DEV)[None, :, None] * 7 + l * 3 + w * 5 + torch.arange(H, device=DEV)[:, None, None]
            src[l, 0, w] = (at % 251).to(dtype)
    parent = torch.tensor([[2, 0, -1, 2]], dtype=torch.int32, device=DEV)
    lengths = torch.tensor([S - 2], dtype=torch.int32, device=DEV)
    out = torch.full((L, 1, K, H, S, D), 9, dtype=dtype, device=DEV)
    binding.beam_reorder(src, parent, out=out, lengths=lengths)
    for k, p in enumerate((2, 0, -1, 2)):
        for l in range(L):
            assert (out[l, 0, k, :, S - 2 :] == 9).all()
            if p < 0:
                assert (out[l, 0, k] == 9).all()
            else:
                assert torch.equal(out[l, 0, k, :, : S - 2], src[l, 0, p, :, : S - 2])
