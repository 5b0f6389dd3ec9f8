"""Host-side checks of the draft step's entry points: sizes, and every refusal, before
any CUDA call (no GPU needed)."""
import ctypes

import pytest
import torch

from speculative_decoding_verification_84_b200 import binding, build

OK, INVALID, DTYPE, MISALIGNED, SMALL = 0, 1, 2, 3, 4
vp = ctypes.c_void_p
GOOD = vp(1 << 20)
OTHER = vp(1 << 40)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load_library()


def _each(fn, good, cases):
    for at, value, want in cases:
        args = list(good)
        args[at] = value
        assert fn(*args) == want, (at, value)


def test_quantize_refusals(lib):
    good = [GOOD, 1, 4, 40, GOOD, 48, GOOD, None]
    _each(lib.spec_verify_q8_quantize, good, [
        (0, None, INVALID), (4, None, INVALID), (6, None, INVALID), (1, 2, DTYPE), (2, 0, INVALID), (2, -1, INVALID), (2, (1 << 30) + 1, INVALID),
        (3, 0, INVALID), (3, binding.Q8_MAX_K + 1, INVALID), (5, 32, INVALID), (5, 47, INVALID), (5, 0, INVALID),
        (0, vp((1 << 20) + 8), MISALIGNED), (4, vp((1 << 20) + 8), MISALIGNED), (6, vp((1 << 20) + 2), MISALIGNED)])


def test_norm_refusals(lib):
    good = [GOOD, None, None, 0, 1e-6, 4, 40, GOOD, 48, GOOD, None, None, None]
    _each(lib.spec_verify_q8_norm, good, [
        (0, None, INVALID), (7, None, INVALID), (9, None, INVALID), (3, 7, DTYPE), (4, -1e-6, INVALID),
        (4, float("nan"), INVALID), (4, float("inf"), INVALID), (5, 0, INVALID), (6, 0, INVALID), (8, 32, INVALID),
        (8, 50, INVALID), (1, vp(8), MISALIGNED), (2, vp(8), MISALIGNED), (10, vp(8), MISALIGNED), (11, vp(8), MISALIGNED)])


def test_matmul_refusals(lib):
    good = [GOOD, 48, GOOD, GOOD, 48, GOOD, 4, 40, 100, GOOD, 1, None, None]
    _each(lib.spec_verify_q8_matmul, good, [
        *[(i, None, INVALID) for i in (0, 2, 3, 5, 9)], (1, 32, INVALID), (1, 47, INVALID), (4, 32, INVALID),
        (4, 56, INVALID), (6, 0, INVALID), (7, 0, INVALID), (7, binding.Q8_MAX_K + 1, INVALID), (8, 0, INVALID),
        (8, (1 << 30) + 1, INVALID), (6, (1 << 30) + 1, INVALID), (10, 5, DTYPE), (0, vp(8), MISALIGNED), (3, vp(8), MISALIGNED), (9, vp(8), MISALIGNED), (2, vp(2), MISALIGNED),
        (5, vp(2), MISALIGNED), (11, vp(2), MISALIGNED)])


def test_matmul_refuses_more_tiles_than_it_counts(lib):
    args = [GOOD, 48, GOOD, GOOD, 48, GOOD, 1 << 30, 40, 1 << 30, GOOD, 1, None, None]
    assert lib.spec_verify_q8_matmul(*args) == INVALID


def test_head_refusals(lib):
    need = lib.spec_verify_q8_head_workspace_size(4, 40)
    assert need >= 4 * 48 + 16 and need % 256 == 0
    assert lib.spec_verify_q8_head_workspace_size(0, 40) == 0 and lib.spec_verify_q8_head_workspace_size(4, 0) == 0
    assert lib.spec_verify_q8_head_workspace_size(4, binding.Q8_MAX_K + 1) == 0
    good = [GOOD, None, None, 1, 1e-6, GOOD, 48, GOOD, 4, 40, 100, None, GOOD, 1, GOOD, need, None, None]
    _each(lib.spec_verify_q8_head, good, [
        (0, None, INVALID), (5, None, INVALID), (7, None, INVALID), (12, None, INVALID), (14, None, INVALID),
        (3, 4, DTYPE), (13, 4, DTYPE), (4, -1.0, INVALID), (6, 40, INVALID), (8, 0, INVALID), (9, 0, INVALID),
        (10, 0, INVALID), (14, vp((1 << 20) + 128), MISALIGNED), (15, need - 1, SMALL), (11, vp(8), MISALIGNED)])


def test_select_refusals(lib):
    need = lib.spec_verify_beam_workspace_size(2, 3, 100, 4, 1)
    assert need > 0 and need % 256 == 0
    for bad in ((0, 3, 100, 4, 1), (2, 0, 100, 4, 1), (2, 33, 100, 4, 1), (2, 3, 0, 4, 1), (2, 3, (1 << 20) + 1, 4, 1),
                (2, 3, 100, 0, 1), (2, 3, 100, 33, 1), (2, 3, 100, 4, 2)):
        assert lib.spec_verify_beam_workspace_size(*bad) == 0, bad
    good = [GOOD, 1, GOOD, GOOD, None, 0, 2, 3, 100, 4, GOOD, GOOD, GOOD, None, GOOD, need, None]
    _each(lib.spec_verify_beam_select, good, [
        *[(i, None, INVALID) for i in (0, 2, 3, 10, 11, 12, 14)], (1, 3, DTYPE), (6, 0, INVALID), (7, 33, INVALID),
        (8, 0, INVALID), (8, (1 << 20) + 1, INVALID), (9, 0, INVALID), (9, 33, INVALID), (0, vp(8), MISALIGNED),
        (2, vp(2), MISALIGNED), (14, vp(128), MISALIGNED), (15, need - 1, SMALL)])
    for pad in (-1, 100):
        args = list(good)
        args[4], args[5] = GOOD, pad
        assert lib.spec_verify_beam_select(*args) == INVALID


def test_reorder_refusals(lib):
    good = [GOOD, OTHER, GOOD, None, 2, 3, 4, 5, 2, 8, 64, None]
    _each(lib.spec_verify_beam_reorder, good, [
        (0, None, INVALID), (1, None, INVALID), (2, None, INVALID), *[(i, 0, INVALID) for i in range(4, 11)],
        (6, 33, INVALID), (7, 33, INVALID), (2, vp((1 << 20) + 2), MISALIGNED), (3, vp(2), MISALIGNED),
        (9, 1 << 62, INVALID), (10, 1 << 60, INVALID),
        (1, GOOD, INVALID),                                                   # in place
        (1, vp((1 << 20) + 2 * 3 * 4 * 2 * 8 * 64 - 1), INVALID),             # the last byte of src
        (1, vp((1 << 20) - 2 * 3 * 5 * 2 * 8 * 64 + 1), INVALID)])            # dst's last byte on src's first


def test_binding_refuses_before_the_library():
    x = torch.zeros(2, 32)
    q = torch.zeros(2, 32, dtype=torch.int8)
    for call in (lambda: binding.q8_quantize(x), lambda: binding.q8_norm(x, None, 1e-6),
                 lambda: binding.q8_matmul(q, torch.ones(2), q, torch.ones(2)),
                 lambda: binding.q8_head(x, None, 1e-6, q, torch.ones(2)),
                 lambda: binding.beam_select(torch.zeros(1, 2, 8), torch.zeros(1, 2), torch.ones(1), 2),
                 lambda: binding.beam_reorder(torch.zeros(1, 1, 2, 1, 1, 4), torch.zeros(1, 2, dtype=torch.int32))):
        with pytest.raises(ValueError):
            call()
