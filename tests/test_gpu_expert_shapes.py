"""The expert products and casts in the forms that large and decoding calls
take, exactly.

Values are whole numbers in -3..3 times a power of two that differs from block
to block, so that a scale taken from the wrong row, column or block shows.
All sums of their products are whole numbers below 2^24, which every kernel
has to give exactly: products of 8 neighbours lie within a factor of 9, far
inside what the 8-bit unit keeps.  Results are compared with products in 64
bits, rounded once to the result's type.

Each case says which kernel the library takes for it.
"""
import pytest
import torch

import lossless_bf16_exponent_zc_amd as zc
from experts_plain import up

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def generator(seed):
    return torch.Generator("cuda").manual_seed(seed)


def blocks_of(g, rows, cols, block_rows, block_cols):
    """[rows, cols] whole numbers, each block_rows x block_cols of them times
    1, 2, 4 or 8."""
    x = torch.randint(-3, 4, (rows, cols), generator=g, device="cuda").float()
    e = torch.randint(0, 4, (-(-rows // block_rows), -(-cols // block_cols)), generator=g, device="cuda").float()
    return x * torch.exp2(e).repeat_interleave(block_rows, 0)[:rows].repeat_interleave(block_cols, 1)[:, :cols]


def int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def segments(counts, align):
    off = [0]
    for c in counts:
        off.append(off[-1] + up(c, align))
    return off


def check_product(counts, align, n, k, dense=False):
    g, experts, off = generator(len(counts) + n + k), len(counts), segments(counts, align)
    rows = off[-1]
    a = blocks_of(g, rows, k, 1, 128)
    w = torch.stack([blocks_of(g, n, k, 128, 128) for _ in range(experts)])
    fa, fw = zc.empty_fp8_rows(rows, k), zc.empty_fp8_weights(experts, n, k)
    zc.quantize_rows(a, fa)
    zc.quantize_weights(w, fw)
    want = torch.zeros(rows, n, dtype=torch.float64, device="cuda")
    for e, c in enumerate(counts):
        if c:
            want[off[e]:off[e] + c] = a[off[e]:off[e] + c].double() @ w[e].double().t().contiguous()
    for dtype in DT.values():
        for beside in (0, 3):
            whole = torch.full((rows + 1, n + beside), float("nan"), dtype=dtype, device="cuda")
            out = whole[:rows, :n]
            if dense:
                zc.expert_product(fa, fw, out)
            else:
                zc.expert_product(fa, fw, out, int32(off), int32(counts))
            assert torch.equal(out, want.to(dtype)), (dtype, beside)
            assert bool(torch.isnan(whole[rows]).all()) and bool(torch.isnan(whole[:, n:]).all())


@pytest.mark.parametrize("counts,align,n,k", [
    ([0, 1, 16, 17, 33, 64] + [0] * 34, 1, 130, 1300),   # every number of row tiles, each with rows of others around it
    ([70, 1, 0, 48] + [0] * 36 + [3], 1, 33, 7168),      # a second slot of one segment; a last expert with rows
    ([1, 0, 9, 17, 40, 130] + [0] * 60, 8, 97, 129),     # padding rows after one, two and three slots
    ([2] * 32, 1, 4096, 640),                            # a decoding step
    ([1] * 60, 1, 40, 100), ([5, 0, 20], 4, 31, 2304),
])
def test_product_of_few_rows(counts, align, n, k):
    assert segments(counts, align)[-1] <= 4 * len(counts) + 32  # product_few
    check_product(counts, align, n, k)


@pytest.mark.parametrize("rows", [1, 16, 17, 32, 36])
def test_dense_product_of_few_rows(rows):
    check_product([rows], 1, 300, 1400, dense=True)


@pytest.mark.parametrize("counts,align,n,k", [
    ([3000, 1000, 300, 40], 1, 2050, 1300),        # 256 wide in order: tiles of 256, 128, 64 and 32 rows
    ([3000, 1000, 300, 40], 32, 7000, 1300),       # the same in runs, with padding rows
    ([2100, 90, 1111, 3], 1, 7001, 1930),          # in runs, rows of 16-bit results at odd addresses
    ([700, 1, 650], 8, 3001, 1500),                # 128 wide, two workgroups on a CU
    ([1000, 900], 1, 3000, 2300),                  # the same, for its rows
    ([20] * 20, 1, 2000, 2100),                    # 128 wide, one workgroup on a CU
    ([500, 100, 60], 64, 2050, 2400),              # the same, tiles of 64 and 128 rows
    ([600], 1, 70, 2100), ([130, 7, 0, 90], 16, 200, 1700), ([1, 0, 9, 17, 40] + [0] * 30 + [130] + [2] * 9, 8, 97, 129),  # 64 wide
])
def test_product_of_differing_scales(counts, align, n, k):
    check_product(counts, align, n, k)


def test_dense_product_of_differing_scales():
    check_product([4100], 1, 4097, 1500, dense=True)


def check_weight_grad(counts, n, k):
    g, experts, off = generator(len(counts) + n + k), len(counts), segments(counts, 128)
    rows = off[-1]
    x, y = blocks_of(g, rows, k, 128, 1), blocks_of(g, rows, n, 128, 1)
    for e, c in enumerate(counts):
        x[off[e] + c:off[e + 1]] = 0
    fx, fy = zc.empty_fp8_columns(rows, k), zc.empty_fp8_columns(rows, n)
    zc.quantize_columns(x, fx)
    zc.quantize_columns(y, fy)
    want = torch.zeros(experts, n, k, dtype=torch.float64, device="cuda")
    for e in range(experts):
        if counts[e]:
            want[e] = y[off[e]:off[e + 1]].double().t().contiguous() @ x[off[e]:off[e + 1]].double()
    need, offsets = zc.expert_weight_grad_workspace_bytes(rows, experts, n, k), int32(off)
    for dtype in DT.values():
        whole = torch.full((experts + 1, n, k), float("nan"), dtype=dtype, device="cuda")
        zc.expert_weight_grad(fy, fx, whole[:experts], offsets)
        assert torch.equal(whole[:experts], want.to(dtype)), dtype
        assert bool(torch.isnan(whole[experts]).all())
        if not need:
            continue
        whole[:experts] = float("nan")
        ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")
        zc.expert_weight_grad(fy, fx, whole[:experts], offsets, ws=ws[:need])
        assert torch.equal(whole[:experts], want.to(dtype)) and bool((ws[need:] == 0xFF).all()), dtype
        whole[:experts] = float("nan")
        rc = zc.lib().zc_expert_weight_grad(fy.data.data_ptr(), fy.scale.data_ptr(), fx.data.data_ptr(), fx.scale.data_ptr(),
                                            rows, experts, n, k, offsets.data_ptr(), whole.data_ptr(),
                                            list(DT.values()).index(dtype), None, 0, torch.cuda.current_stream().cuda_stream)
        assert rc == 0 and torch.equal(whole[:experts], want.to(dtype)), dtype


@pytest.mark.parametrize("counts,n,k", [
    ([700, 300, 400], 3300, 3830),      # 256 wide in runs, row tiles no multiple of 4
    ([500, 200], 3040, 3039),           # 256 wide in order
    ([700, 300, 400], 1700, 2000),      # 128 wide in runs, two workgroups on a CU
    ([130] * 3, 1300, 1301),            # the same in order
    ([700, 0, 260], 900, 1001),         # 128 wide, one workgroup on a CU
    ([400, 0, 129, 1], 130, 140),       # 64 wide
    ([300, 40, 200] * 7, 60, 2000),     # 64 wide in runs, four workgroups on a CU
    ([16900, 100, 0], 300, 333),        # one long segment, summed whole
])
def test_weight_gradient_of_differing_scales(counts, n, k):
    check_weight_grad(counts, n, k)


@pytest.mark.parametrize("counts,n,k,side", [
    ([9000], 700, 650, 128), ([9000, 8000], 300, 500, 128), ([25300, 100, 0], 300, 333, 128), ([9000], 60, 130, 64),
])
def test_weight_gradient_in_parts_of_differing_scales(counts, n, k, side):
    """Joined into every type; with the caller's workspace, and without one
    summed whole, the same."""
    experts, rows = len(counts), segments(counts, 128)[-1]
    tiles = lambda s: experts * -(-n // s) * -(-k // s)
    parts = min(16, 256 // tiles(side))
    assert (tiles(64) <= 32) == (side == 64)
    assert zc.expert_weight_grad_workspace_bytes(rows, experts, n, k) == up(parts * experts * n * k * 4, 256)
    check_weight_grad(counts, n, k)


@pytest.mark.parametrize("hidden", [100, 250, 500, 1100])
def test_casts_past_the_caches(hidden):
    """Rows of more than 64 MB, whose stores go around the caches, for 8, 16,
    32 and 64 lanes a row: the bytes of the same tokens cast by themselves."""
    topk, experts, align = 6, 19, 4
    tokens = (64 << 20) // (topk * up(hidden, 128)) + 77
    g = generator(hidden)
    x = torch.randn(tokens, hidden, generator=g, device="cuda") * torch.exp(torch.randn(tokens, 1, generator=g, device="cuda"))
    x[5, :3] = torch.tensor([float("nan"), float("inf"), 0.0])
    x = x.to(torch.bfloat16)
    once = zc.empty_fp8_rows(tokens, hidden)
    zc.quantize_rows(x, once)  # below 64 MB
    data, scale = once.data.view(torch.uint8), once.scale.view(torch.uint8)

    ids = torch.randint(-1, experts + 1, (tokens, topk), generator=g, device="cuda", dtype=torch.int32)
    plan = zc.ExpertPlan(tokens, topk, experts, align)
    r, out = plan.empty_routing(), plan.empty_fp8(hidden)
    out.data.view(torch.uint8).fill_(0xA5)
    out.scale.view(torch.uint8).fill_(0xA5)
    plan.route(ids, r, plan.empty_workspace())
    plan.dispatch_fp8(x, r, out)
    used = int(r.offsets[-1])
    live, token = (r.slot[:used] >= 0)[:, None], r.slot[:used].clamp(min=0).long() // topk
    got, got_scale = out.data.view(torch.uint8), out.scale.view(torch.uint8)
    assert 0 < used < plan.rows and not bool(live.all())
    assert torch.equal(got[:used], torch.where(live, data[token], 0))
    assert torch.equal(got_scale[:used], torch.where(live, scale[token], 127))
    assert bool((got[used:] == 0xA5).all()) and bool((got_scale[used:] == 0xA5).all())

    many = torch.cat([x] * topk)
    whole = zc.empty_fp8_rows(len(many), hidden)
    zc.quantize_rows(many, whole)
    assert torch.equal(whole.data.view(torch.uint8), data.repeat(topk, 1))
    assert torch.equal(whole.scale.view(torch.uint8), scale.repeat(topk, 1))


def test_products_of_clamped_segments():
    """Offsets and counts that leave the rows are cut to them, and what is
    left is multiplied as ever."""
    rows, n, k, g = 100, 64, 256, generator(1)
    a, w = blocks_of(g, rows, k, 1, 128), torch.stack([blocks_of(g, n, k, 128, 128) for _ in range(3)])
    fa, fw = zc.empty_fp8_rows(rows, k), zc.empty_fp8_weights(3, n, k)
    zc.quantize_rows(a, fa)
    zc.quantize_weights(w, fw)
    want = torch.zeros(rows, n, device="cuda")
    want[:60], want[80:] = a[:60] @ w[0].t(), a[80:] @ w[2].t()
    whole = torch.full((rows + 64, n), float("nan"), device="cuda")
    zc.expert_product(fa, fw, whole[:rows], int32([-5, 60, 80, 1 << 30]), int32([1 << 30, -3, 1 << 30]))
    assert torch.equal(whole[:rows], want) and bool(torch.isnan(whole[rows:]).all())

    x, y = blocks_of(g, 384, k, 128, 1), blocks_of(g, 384, n, 128, 1)
    fx, fy = zc.empty_fp8_columns(384, k), zc.empty_fp8_columns(384, n)
    zc.quantize_columns(x, fx)
    zc.quantize_columns(y, fy)
    whole = torch.full((4, n, k), float("nan"), device="cuda")
    zc.expert_weight_grad(fy, fx, whole[:3], int32([-128, 128, 256, 1 << 30]))
    for e in range(3):
        at = slice(128 * e, 128 * e + 128)
        assert torch.equal(whole[e], y[at].t() @ x[at]), e
    assert bool(torch.isnan(whole[3]).all())


@pytest.mark.parametrize("tokens,topk,experts,align", [(1000, 2, 1024, 128), (2048, 1, 1024, 1), (31, 64, 1000, 1024)])
def test_route_by_one_workgroup_of_all_its_waves(tokens, topk, experts, align):
    g = generator(tokens)
    ids = torch.randint(-1, experts + 1, (tokens, topk), generator=g, device="cuda", dtype=torch.int32)
    plan = zc.ExpertPlan(tokens, topk, experts, align)
    r = plan.empty_routing()
    plan.route(ids, r, plan.empty_workspace())
    flat, row, slot = ids.flatten().tolist(), [-1] * (tokens * topk), []
    for e in range(experts):
        mine = [i for i, v in enumerate(flat) if v == e]
        assert int(r.offsets[e]) == len(slot) and int(r.counts[e]) == len(mine)
        for i in mine:
            row[i] = len(slot)
            slot.append(i)
        slot += [-1] * (-len(slot) % align)
    assert int(r.offsets[-1]) == len(slot)
    assert r.row.flatten().tolist() == row
    assert r.slot.tolist() == slot + [-1] * (plan.rows - len(slot))
