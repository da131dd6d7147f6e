"""The router and the orthogonalised updates of include/zc_experts.h without a
GPU: sizes, refusals before any HIP call, and the 64-bit definitions that the
GPU is held to."""
import pytest
import torch

import lossless_bf16_exponent_zc_amd as zc
import router_plain as plain
from lossless_bf16_exponent_zc_amd import binding, experts

BAD, CAP, UNSUP = binding.ZC_ERR_INVALID_ARG, binding.ZC_ERR_CAPACITY, binding.ZC_ERR_UNSUPPORTED
P = 0x10000  # an aligned address that is never followed: each call is refused first


@pytest.fixture(scope="module")
def L():
    return experts.lib()


def rc(f, base, i, v):
    a = list(base)
    a[i] = v
    return f(*a)


def test_choose_refusals(L):
    good = [P, 16, 2, 8, 2, 16, 0, 0, 1.0, 0.0, None, None, P, P, P, P, P, P, P, 1 << 20, None]
    for i, v in ((0, None), (0, P + 2), (1, 15), (2, 3), (6, 2), (10, P + 1), (12, None), (13, P + 2), (14, None),
                 (15, P + 1), (16, None), (17, None), (18, None), (18, P + 64)):
        assert rc(L.zc_choose, good, i, v) == BAD, (i, v)
    for i, v in ((3, 1 << 31), (4, 0), (4, 65), (5, 0), (5, 1025)):
        assert rc(L.zc_choose, good, i, v) == UNSUP, (i, v)
    need = L.zc_choose_workspace_bytes(8, 2, 16)
    assert need > 0 and need % 256 == 0 and rc(L.zc_choose, good, 19, need - 1) == CAP
    for args in ((8, 0, 16), (8, 65, 16), (8, 2, 0), (8, 2, 1025), (1 << 31, 1, 4)):
        assert L.zc_choose_workspace_bytes(*args) == 0


def test_choose_backward_refusals(L):
    good = [P, 16, 2, 8, 2, 16, 0, 0, 1.0, 0.0, None, P, P, P, P, None, P, 16, None]
    for i, v in ((0, None), (1, 15), (2, 3), (6, 2), (11, None), (12, None), (12, P + 1), (13, None), (14, P + 2),
                 (15, P + 1), (16, None), (17, 15)):
        assert rc(L.zc_choose_backward, good, i, v) == BAD, (i, v)
    for i, v in ((3, 1 << 31), (4, 65), (5, 1025)):
        assert rc(L.zc_choose_backward, good, i, v) == UNSUP, (i, v)
    assert rc(L.zc_choose_backward, good, 3, 0) == binding.ZC_OK


@pytest.mark.parametrize("args", [(8, 2**32 + 2, 4), (8, 2, 2**32 + 4), (2**64 + 8, 2, 4)])
def test_sizes_past_the_librarys_types_are_refused(args):
    with pytest.raises(zc.ZcError) as e:
        zc.Router(*args)
    assert e.value.code == UNSUP


def test_host_tensors_are_refused():
    router = zc.Router(4, 2, 3)
    c, ws, x = router.empty_choice("cpu"), router.empty_workspace("cpu"), torch.zeros(4, 3)
    for call in (lambda: router.choose(x, c, ws), lambda: router.choose_backward(x, c, None, None, x)):
        with pytest.raises(zc.ZcError) as e:
            call()
        assert e.value.code == BAD


def test_definitions_by_hand():
    x = torch.tensor([[0.0, 0.0, 0.0], [2.0, 1.0, -float("inf")]], dtype=torch.float64)
    ids, w, counts, sums, n, loss = plain.choose(x, 2, normalize=True, balance=1.0)
    assert ids.tolist() == [[0, 1], [0, 1]] and counts.tolist() == [2, 2, 0] and n == 2
    e = float(torch.sigmoid(torch.tensor(1.0, dtype=torch.float64)))
    assert torch.allclose(w, torch.tensor([[0.5, 0.5], [e, 1 - e]], dtype=torch.float64), rtol=1e-15)
    want = torch.tensor([1 / 3 + e, 1 / 3 + 1 - e, 1 / 3], dtype=torch.float64)
    assert torch.allclose(sums, want, rtol=1e-15)
    assert abs(float(loss) - 3 * (0.5 * (1 / 3 + e) / 2 + 0.5 * (1 / 3 + 1 - e) / 2)) < 1e-15
    even = torch.zeros(6, 3, dtype=torch.float64)
    assert abs(float(plain.loss_of(torch.tensor([4, 4, 4]), plain.shares(even + 1).sum(0), 6, 2, 1.0)) - 1) < 1e-15


def test_orthogonalize_refusals(L):
    good = [P, 2, 2, 8, 12, 5, 3.0, -4.0, 2.0, 0.0, P, P, 1 << 24, None]
    for i, v in ((0, None), (0, P + 2), (1, 3), (3, 0), (4, 0), (5, 0), (10, None), (10, P + 1), (11, None), (11, P + 64)):
        assert rc(L.zc_orthogonalize, good, i, v) == BAD, (i, v)
    for i, v in ((2, 65536), (3, 65537), (4, 65537), (5, 65)):
        assert rc(L.zc_orthogonalize, good, i, v) == UNSUP, (i, v)
    need = zc.orthogonalize_workspace_bytes(2, 8, 12)
    assert need > 0 and rc(L.zc_orthogonalize, good, 12, need - 1) == CAP
    assert rc(L.zc_orthogonalize, good, 2, 0) == binding.ZC_OK
    for args in ((0, 8, 8), (1, 0, 8), (1, 8, 65537), (65536, 8, 8), (2**32 + 1, 8, 8), (1, 2**32 + 8, 8), (-1, 8, 8)):
        assert zc.orthogonalize_workspace_bytes(*args) == 0


def test_updates_in_place_are_of_16_bits(L):
    need = zc.orthogonalize_workspace_bytes(2, 8, 12)
    size = 2 * 8 * 12
    for dtype, out in ((2, P), (2, P + size * 4 - 2), (0, P + 2), (1, P + size * 2 - 2), (0, P - size * 2 + 2), (2, P - 2)):
        args = [P, dtype, 2, 8, 12, 5, 3.0, -4.0, 2.0, 0.0, out, P + (1 << 20), need, None]
        assert rc(L.zc_orthogonalize, args, 1, dtype) == BAD, (dtype, out)


def test_a_product_of_almost_too_many_tiles_is_refused(L):
    """Workgroups are launched in eights: 61,455 matrices of 273 tiles of 64 are
    2^24 - 1, one more than the last multiple of eight that a launch may have."""
    batch, n = 61455, 273 * 64
    need = zc.orthogonalize_workspace_bytes(batch, n, 1)
    far = 1 << 45  # addresses that do not overlap and are never followed
    assert batch * 273 == 2**24 - 1
    assert L.zc_orthogonalize(P, 0, batch, n, 1, 5, 3.0, -4.0, 2.0, 0.0, far, 2 * far, need, None) == UNSUP


@pytest.mark.parametrize("coefficients", [3.0, None])
def test_coefficients_that_are_not_three_numbers_are_refused(coefficients):
    x = torch.zeros(1, 2, 3)
    with pytest.raises(zc.ZcError, match="coefficients") as e:
        zc.orthogonalize(x, x.bfloat16(), coefficients=coefficients)
    assert e.value.code == BAD
