"""include/zc_experts.h without a GPU: every symbol is exported, sizes are
what the header says, and bad arguments are refused before any HIP call."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import experts_plain as plain
import lossless_bf16_exponent_zc_amd as zc
from lossless_bf16_exponent_zc_amd import binding, experts

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BAD, CAP, UNSUP = binding.ZC_ERR_INVALID_ARG, binding.ZC_ERR_CAPACITY, binding.ZC_ERR_UNSUPPORTED
P = 0x10000  # an aligned address that is never followed: each call is refused first


@pytest.fixture(scope="module")
def L():
    return experts.lib()


def test_exports_every_declared_symbol(L):
    src = open(os.path.join(ROOT, "include", "zc_experts.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    assert sorted(zc.EXPERT_EXPORTS) == sorted(set(re.findall(r"\b(zc_\w+)\s*\(", src)))
    for n in zc.EXPERT_EXPORTS:
        assert hasattr(L, n), n


@pytest.mark.parametrize("tokens,topk,experts_,align", [
    (0, 1, 1, 1), (1, 1, 1, 1), (8, 8, 256, 1), (8, 8, 256, 16), (8192, 8, 256, 128), (1021, 3, 37, 8)])
def test_row_capacity_holds_every_routing(L, tokens, topk, experts_, align):
    slots = tokens * topk
    want = plain.up(slots + min(experts_, slots) * (align - 1), align)
    assert L.zc_route_rows(tokens, topk, experts_, align) == want
    assert zc.ExpertPlan(tokens, topk, experts_, align).rows == want


@pytest.mark.parametrize("args", [(1, 0, 1, 1), (1, 65, 1, 1), (1, 1, 0, 1), (1, 1, 1025, 1), (1, 1, 1, 0),
                                  (1, 1, 1, 3), (1, 1, 1, 2048), (1 << 31, 1, 1, 1), (1 << 30, 8, 1, 1)])
def test_plan_limits(L, args):
    assert L.zc_route_rows(*args) == 0
    with pytest.raises(zc.ZcError) as e:
        zc.ExpertPlan(*args)
    assert e.value.code == UNSUP


@pytest.mark.parametrize("args", [(8, 2**32 + 2, 4, 1), (8, 2, 2**32 + 4, 1), (8, 2, 4, 2**32 + 1), (2**64 + 8, 2, 4, 1)])
def test_sizes_past_the_librarys_types_are_refused(args):
    with pytest.raises(zc.ZcError) as e:
        zc.ExpertPlan(*args)
    assert e.value.code == UNSUP


def test_weight_gradient_workspace_of_sizes_past_the_librarys_types():
    assert zc.expert_weight_grad_workspace_bytes(32768, 1, 60, 300) > 0
    for args in ((32768, 2**32 + 1, 60, 300), (32768, 1, 2**32 + 60, 300), (32768, 1, 60, 2**32 + 300),
                 (2**64 + 32768, 1, 60, 300), (-1, 1, 60, 300)):
        assert zc.expert_weight_grad_workspace_bytes(*args) == 0


def test_rows_of_columns_blocks_stay_below_their_limit(L):
    """2^24, where rows of every other call go to 2^31."""
    q = [P, 64, 0, 1 << 24, 64, None, P, P, None]
    assert L.zc_quantize_columns(*q) == UNSUP
    assert L.zc_expert_weight_grad_workspace_bytes((1 << 24) - 1, 1, 60, 300) > 0
    assert L.zc_expert_weight_grad_workspace_bytes(1 << 24, 1, 60, 300) == 0
    header = open(os.path.join(ROOT, "include", "zc_experts.h")).read()
    assert "below 2^24 in blocks of 128 rows" in header


def test_route_refusals(L):
    ok = [P, 8, 2, 4, 1, P, P, P, P, 16, P, 256, None]

    def rc(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return L.zc_route(*a)

    for i in (0, 5, 6, 7, 8, 10):
        assert rc(**{f"_{i}": None}) == BAD, i
        assert rc(**{f"_{i}": P + 2}) == BAD, i
    assert rc(_9=15) == CAP and rc(_11=255) == CAP
    assert rc(_2=0) == UNSUP and rc(_3=1025) == UNSUP and rc(_4=3) == UNSUP and rc(_9=1 << 31) == UNSUP


def test_row_call_refusals(L):
    d = L.zc_dispatch
    good = [P, 64, 0, 8, 2, 4, 64, P, P, P, P, 64, 16, None]

    def rc(f, base, i, v):
        a = list(base)
        a[i] = v
        return f(*a)

    for i in (0, 7, 9, 10):  # counts may be null: no padding rows
        assert rc(d, good, i, None) == BAD, i
    assert rc(d, good, 8, P + 1) == BAD
    assert rc(d, good, 0, P + 1) == BAD
    assert rc(d, good, 1, 63) == BAD and rc(d, good, 11, 63) == BAD   # strides shorter than a row
    assert rc(d, good, 2, 3) == BAD and rc(d, good, 6, 0) == BAD
    assert rc(d, good, 4, 65) == UNSUP and rc(d, good, 5, 1025) == UNSUP and rc(d, good, 6, 1 << 24) == UNSUP
    assert rc(d, good, 12, 1 << 31) == UNSUP
    assert rc(d, good, 3, 0) == binding.ZC_OK  # no tokens: nothing to do
    f = [P, 64, 0, 8, 2, 4, 64, P, P, P, P, P, 16, None]
    for i in (10, 11):
        assert rc(L.zc_dispatch_fp8, f, i, P + 8) == BAD
    c = [P, 64, None, 0, 8, 2, 64, P, 16, P, 64, None]
    for i, v in ((0, None), (1, 8), (2, P + 1), (3, 9), (7, None), (9, None), (10, 8)):
        assert rc(L.zc_combine, c, i, v) == BAD, (i, v)
    g = [P, 64, P, 64, None, 0, 8, 2, 4, 64, P, P, P, 16, P, 64, P, None]
    for i, v in ((0, None), (2, None), (3, 1), (10, None), (11, P + 1), (12, None), (15, 1), (16, P + 2)):
        assert rc(L.zc_combine_backward, g, i, v) == BAD, (i, v)
    neither = list(g)
    neither[14] = neither[16] = None
    assert L.zc_combine_backward(*neither) == BAD


def test_cast_and_product_refusals(L):
    def rc(f, base, i, v):
        a = list(base)
        a[i] = v
        return f(*a)

    for f in (L.zc_quantize_rows, L.zc_quantize_columns):
        q = [P, 64, 0, 8, 64, None, P, P, None]
        for i, v in ((0, None), (1, 8), (2, 3), (4, 0), (5, P + 1), (6, P + 4), (7, None)):
            assert rc(f, q, i, v) == BAD, (i, v)
        assert rc(f, q, 4, 1 << 24) == UNSUP
    w = [P, 0, 2, 64, 64, 0, P, P, None]
    for i, v in ((0, None), (1, 3), (2, 0), (3, 0), (4, 0), (6, P + 8), (7, None)):
        assert rc(L.zc_quantize_weights, w, i, v) == BAD, (i, v)
    assert rc(L.zc_quantize_weights, w, 2, 1025) == UNSUP
    p = [P, P, 8, P, P, 4, 64, 128, P, P, P, 64, 0, None]
    for i, v in ((0, None), (1, P + 8), (3, None), (4, None), (5, 0), (6, 0), (7, 0), (8, None), (9, P + 1),
                 (10, None), (11, 8), (12, 3)):
        assert rc(L.zc_expert_product, p, i, v) == BAD, (i, v)
    assert rc(L.zc_expert_product, p, 2, 1 << 31) == UNSUP and rc(L.zc_expert_product, p, 2, 0) == binding.ZC_OK
    g = [P, P, P, P, 256, 4, 64, 64, P, P, 0, None, 0, None]
    for i, v in ((0, None), (1, P + 8), (2, P + 1), (3, None), (5, 0), (6, 0), (7, 0), (8, None), (9, None), (10, 3),
                 (11, P + 64)):
        assert rc(L.zc_expert_weight_grad, g, i, v) == BAD, (i, v)
    assert rc(L.zc_expert_weight_grad, g, 4, 1 << 24) == UNSUP


def test_binding_refuses_host_tensors_and_shapes():
    plan = zc.ExpertPlan(4, 2, 3)
    r = plan.empty_routing(device="cpu")
    for call in (lambda: plan.route(torch.zeros(4, 2, dtype=torch.int32), r, plan.empty_workspace("cpu")),
                 lambda: plan.dispatch(torch.zeros(4, 8), r, plan.empty_rows(8, torch.float32, "cpu")),
                 lambda: plan.combine(plan.empty_rows(8, torch.float32, "cpu"), None, r, torch.zeros(4, 8)),
                 lambda: zc.quantize_rows(torch.zeros(4, 8), zc.empty_fp8_rows(4, 8, "cpu")),
                 lambda: zc.quantize_weights(torch.zeros(4, 8), zc.empty_fp8_weights(1, 4, 8, "cpu")),
                 lambda: zc.expert_product(zc.empty_fp8_rows(4, 8, "cpu"), zc.empty_fp8_rows(4, 8, "cpu"),
                                           torch.zeros(4, 4))):
        with pytest.raises(zc.ZcError) as e:
            call()
        assert e.value.code == BAD


def test_blocks_stand_for_their_values():
    x = np.random.default_rng(0).standard_normal((5, 200)).astype(np.float32)
    data, scale = plain.cast(x)
    f = zc.Fp8Blocks(torch.from_numpy(data).view(torch.float8_e4m3fn),
                     torch.from_numpy(scale).view(torch.float8_e8m0fnu), 200)
    v = f.float().numpy()
    assert v.shape == (5, 200)
    assert np.array_equal(v, plain.values(data, scale)[:, :200])
    # a value is off by at most half a step: 2^-4 of itself, or 2^-10 scales
    s = np.repeat(2.0 ** (scale[:, :2].astype(float) - 127), 128, 1)[:, :200]
    assert (np.abs(v - x) <= np.maximum(np.abs(x) * 2.0 ** -4, s * 2.0 ** -10)).all()


def test_plain_cast_agrees_with_torch():
    """The oracle's rounding against torch's cast, on the CPU."""
    x = np.random.default_rng(1).standard_normal(4096) * 2.0 ** np.random.default_rng(2).integers(-12, 6, 4096)
    x = np.clip(x, -448, 448).astype(np.float32)
    got = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(got, plain.e4m3_bytes(x.astype(np.float64)))
