"""The expert operators on the GPU against plain 64-bit numpy (experts_plain).

Row buffers are filled with NaN (8-bit data with 0xA5) before each call, with
guard columns beside strided rows, so what a call forgets or overruns shows.

Tolerances.  Copies, routing and 8-bit casts: equal.  Sums of n products in
32 bits: n 2^-24 times the sum of magnitudes, plus the output's own rounding.
Products of 8-bit blocks: exact where all partial sums are small whole
numbers; else the bound that follows from how the matrix unit adds
(experts_plain.unit_bound).
"""
import types

import numpy as np
import pytest
import torch

import experts_plain as plain
import lossless_bf16_exponent_zc_amd as zc
from gpu_util import say

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def gen(seed):
    return torch.Generator(device="cpu").manual_seed(seed)


def strided(rows, cols, dtype, pad, fill=float("nan")):
    """A [rows, cols] view of a wider buffer, and the buffer."""
    whole = torch.full((rows, cols + pad), fill, dtype=dtype, device="cuda")
    return whole[:, :cols], whole


def guard_intact(whole, cols):
    return bool(torch.isnan(whole[:, cols:]).all())


def routed(tokens, topk, experts, align, seed, drop=0.3):
    g = gen(seed)
    ids = torch.randint(0, experts, (tokens, topk), generator=g, dtype=torch.int32)
    out = torch.rand(tokens, topk, generator=g) < drop
    other = torch.tensor([-1, experts, 2**31 - 1, -2**31], dtype=torch.int64)[torch.randint(0, 4, (tokens, topk), generator=g)]
    ids = torch.where(out, other.to(torch.int32), ids)
    plan = zc.ExpertPlan(tokens, topk, experts, align)
    r = plan.empty_routing()
    for t in r:
        t.fill_(-77)
    plan.route(ids.cuda(), r, plan.empty_workspace())
    return plan, ids, r


ROUTES = [
    (1, 1, 1, 1, 0.0), (1, 1, 1, 128, 1.0), (0, 2, 3, 8, 0.0), (3, 2, 5, 1, 0.3), (64, 8, 256, 1, 0.0),
    (65, 1, 2, 16, 0.5), (1000, 64, 3, 1024, 0.9), (1021, 3, 37, 16, 0.5), (1024, 8, 1024, 1, 0.1),
    (1025, 8, 1000, 4, 0.1), (1024, 8, 5, 1, 0.2), (8195, 1, 1024, 8, 0.2), (3001, 7, 255, 128, 0.3), (4096, 9, 1, 1, 0.0), (5000, 2, 1024, 2, 1.0),
]


@pytest.mark.parametrize("tokens,topk,experts,align,drop", ROUTES)
def test_route(tokens, topk, experts, align, drop):
    plan, ids, r = routed(tokens, topk, experts, align, seed=tokens + topk, drop=drop)
    off, cnt, row, slot = plain.route(ids.numpy(), experts, align)
    assert np.array_equal(r.offsets.cpu().numpy(), off)
    assert np.array_equal(r.counts.cpu().numpy(), cnt)
    assert np.array_equal(r.row.cpu().numpy(), row)
    got = r.slot.cpu().numpy()
    assert np.array_equal(got[:off[-1]], slot) and (got[off[-1]:] == -1).all()


def test_route_of_many_tiles():
    """Past the tiles that a workgroup adds up by itself: against a stable
    sort on the GPU (the plain form goes slot by slot)."""
    tokens, topk, experts, align = 262145, 5, 300, 64
    plan, ids, r = routed(tokens, topk, experts, align, seed=11)
    flat = ids.cuda().reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < experts), flat, experts)
    order = torch.argsort(key, stable=True)
    count = torch.bincount(key, minlength=experts + 1)
    padded = (count[:experts] + align - 1) // align * align
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), padded.cumsum(0)])
    assert torch.equal(r.counts.long(), count[:experts]) and torch.equal(r.offsets.long(), offsets)
    n = int(count[:experts].sum())
    live = order[:n]
    want = offsets[key[live]] + torch.arange(n, device="cuda") - (count.cumsum(0) - count)[key[live]]
    row = torch.full_like(flat, -1)
    row[live] = want
    assert torch.equal(r.row.reshape(-1).long(), row)
    slot = torch.full((plan.rows,), -1, dtype=torch.int64, device="cuda")
    slot[want] = live
    assert torch.equal(r.slot.long(), slot)


ROWS = [  # tokens, topk, experts, align, hidden, dtype, columns beside x's and the rows'
    (1, 1, 1, 1, 1, "bf16", 0), (3, 2, 5, 8, 7, "fp16", 0), (5, 9, 4, 1, 64, "fp32", 3), (17, 8, 256, 1, 7168, "bf16", 0),
    (33, 3, 7, 16, 1001, "bf16", 1), (33, 3, 7, 16, 1000, "fp16", 4), (40, 64, 6, 128, 129, "fp32", 0),
    (257, 2, 3, 1, 66, "bf16", 0), (1500, 8, 37, 4, 40, "bf16", 8), (9, 4, 2, 1, 8200, "fp32", 0),
]


def row_case(tokens, topk, experts, align, hidden, dtype, pad):
    plan, ids, r = routed(tokens, topk, experts, align, seed=hidden + tokens)
    off, cnt, row, slot = plain.route(ids.numpy(), experts, align)
    return plan, r, off, row, slot


@pytest.mark.parametrize("tokens,topk,experts,align,hidden,dtype,pad", ROWS)
def test_dispatch(tokens, topk, experts, align, hidden, dtype, pad):
    plan, r, off, row, slot = row_case(tokens, topk, experts, align, hidden, dtype, pad)
    x, _ = strided(tokens, hidden, DT[dtype], pad)
    x.copy_(torch.randn(tokens, hidden, generator=gen(1)))
    rows, whole = strided(plan.rows, hidden, DT[dtype], 2 * pad)
    plan.dispatch(x, r, rows)
    got = rows.float().cpu().numpy()
    want = np.where((slot >= 0)[:, None], x.float().cpu().numpy()[np.maximum(slot, 0) // topk], 0)
    assert np.array_equal(got[:off[-1]], want)
    assert np.isnan(got[off[-1]:]).all() and guard_intact(whole, hidden)


@pytest.mark.parametrize("tokens,topk,experts,align,hidden,dtype,pad", ROWS)
def test_dispatch_fp8(tokens, topk, experts, align, hidden, dtype, pad):
    plan, r, off, row, slot = row_case(tokens, topk, experts, align, hidden, dtype, pad)
    x, _ = strided(tokens, hidden, DT[dtype], pad)
    x.copy_(torch.randn(tokens, hidden, generator=gen(2)) * torch.exp(torch.randn(tokens, 1, generator=gen(3))))
    out = plan.empty_fp8(hidden)
    out.data.view(torch.uint8).fill_(0xA5)
    out.scale.view(torch.uint8).fill_(0xA5)
    plan.dispatch_fp8(x, r, out)
    data, scale = plain.cast(x.double().cpu().numpy())
    live, at = (slot >= 0)[:, None], np.maximum(slot, 0) // topk
    d, s = out.data.view(torch.uint8).cpu().numpy(), out.scale.view(torch.uint8).cpu().numpy()
    assert np.array_equal(d[:off[-1]], np.where(live, data[at], 0))
    assert np.array_equal(s[:off[-1]], np.where(live, scale[at], 127))
    assert (d[off[-1]:] == 0xA5).all() and (s[off[-1]:] == 0xA5).all()


def rows_with_garbage(plan, off, slot, hidden, dtype, pad, seed):
    """Rows whose padding and tail hold NaN: nothing may read them."""
    rows, whole = strided(plan.rows, hidden, DT[dtype], pad)
    rows[:off[-1]] = torch.where(torch.from_numpy(slot >= 0)[:, None].cuda(),
                                 torch.randn(int(off[-1]), hidden, generator=gen(seed)).cuda().to(DT[dtype]),
                                 torch.tensor(float("nan"), dtype=DT[dtype], device="cuda"))
    return rows


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("tokens,topk,experts,align,hidden,dtype,pad", ROWS)
def test_combine(tokens, topk, experts, align, hidden, dtype, pad, weighted):
    plan, r, off, row, slot = row_case(tokens, topk, experts, align, hidden, dtype, pad)
    rows = rows_with_garbage(plan, off, slot, hidden, dtype, pad, 4)
    w = torch.randn(tokens, topk, generator=gen(5))
    y, whole = strided(tokens, hidden, DT[dtype], pad)
    plan.combine(rows, w.cuda() if weighted else None, r, y)
    x = rows.double().cpu().numpy()
    part = np.where((row >= 0)[..., None], x[np.maximum(row, 0)], 0)
    if weighted:
        part = part * w.double().numpy()[..., None]
    part = np.where((row >= 0)[..., None], part, 0)
    want, mag = part.sum(1), np.abs(part).sum(1)
    got = y.double().cpu().numpy()
    assert (np.abs(got - want) <= plain.U[dtype] * np.abs(want) * 1.01 + (topk + 1) * 2.0 ** -24 * mag + 2.0 ** -25).all()
    assert (got[(row < 0).all(1)] == 0).all() and guard_intact(whole, hidden)


@pytest.mark.parametrize("want_rows,want_weights", [(True, True), (True, False), (False, True)])
@pytest.mark.parametrize("tokens,topk,experts,align,hidden,dtype,pad", ROWS)
def test_combine_backward(tokens, topk, experts, align, hidden, dtype, pad, want_rows, want_weights):
    plan, r, off, row, slot = row_case(tokens, topk, experts, align, hidden, dtype, pad)
    rows = rows_with_garbage(plan, off, slot, hidden, dtype, 0, 6)
    w = torch.randn(tokens, topk, generator=gen(7))
    dy, _ = strided(tokens, hidden, DT[dtype], pad)
    dy.copy_(torch.randn(tokens, hidden, generator=gen(8)))
    drows, whole = strided(plan.rows, hidden, DT[dtype], pad)
    dw = torch.full((tokens, topk), float("nan"), device="cuda")
    plan.combine_backward(dy, rows if want_weights else None, w.cuda(), r, drows if want_rows else None,
                          dw if want_weights else None)
    d, x = dy.double().cpu().numpy(), rows.double().cpu().numpy()
    if want_rows:
        got = drows.double().cpu().numpy()
        want = np.where((slot >= 0)[:, None], w.double().numpy().reshape(-1)[np.maximum(slot, 0)][:, None]
                        * d[np.maximum(slot, 0) // topk], 0)
        assert (np.abs(got[:off[-1]] - want) <= (plain.U[dtype] * 1.01 + 2.0 ** -24) * np.abs(want) + 2.0 ** -25).all()
        assert np.isnan(got[off[-1]:]).all() and guard_intact(whole, hidden)
    if want_weights:
        part = np.where((row >= 0)[..., None], x[np.maximum(row, 0)] * d[:, None], 0)
        got = dw.double().cpu().numpy()
        assert (np.abs(got - part.sum(-1)) <= hidden * 2.0 ** -24 * np.abs(part).sum(-1)).all()
        assert (got[row < 0] == 0).all()


@pytest.mark.parametrize("hidden,dtype,pad", [(2048, "bf16", 0), (2049, "bf16", 0), (2053, "fp16", 1), (1100, "fp32", 1),
                                              (2056, "bf16", 64), (4120, "fp16", 0), (1024, "bf16", 9)])
def test_rows_past_the_caches(hidden, dtype, pad):
    """Row buffers past 256 MB, whose stores go around the caches, at every
    kind of row start: multiples of 64 bytes, of 16, of 4 and of 2."""
    topk, experts, align = 6, 19, 4
    tokens = (256 << 20) // (topk * hidden * DT[dtype].itemsize) + 77
    plan, ids, r = routed(tokens, topk, experts, align, seed=hidden, drop=0.1)
    x, _ = strided(tokens, hidden, DT[dtype], 0)
    g = torch.Generator("cuda").manual_seed(hidden)
    x.normal_(generator=g)
    weights = torch.rand(tokens, topk, device="cuda", generator=g)
    rows, whole = strided(plan.rows, hidden, DT[dtype], pad)
    plan.dispatch(x, r, rows)
    used = int(r.offsets[-1])
    slot = r.slot[:used].long()
    token = slot.clamp(min=0) // topk
    assert torch.equal(rows[:used], torch.where((slot >= 0)[:, None], x[token], 0))
    assert torch.isnan(rows[used:]).all() and torch.isnan(whole[:, hidden:]).all()
    live = rows.clone()  # dispatched rows, as an expert's outputs
    want = torch.where((slot >= 0)[:, None], weights.reshape(-1)[slot.clamp(min=0)][:, None] * x[token].double(), 0)
    for with_weights in (False, True):
        whole.fill_(float("nan"))
        dw = torch.full((tokens, topk), float("nan"), device="cuda") if with_weights else None
        plan.combine_backward(x, live if with_weights else None, weights, r, rows, dw)
        assert ((rows[:used].double() - want).abs() <= (plain.U[dtype] * 1.01 + 2.0 ** -24) * want.abs() + 2.0 ** -25).all()
        assert torch.isnan(rows[used:]).all() and torch.isnan(whole[:, hidden:]).all()
    size = x.double().square().sum(1)[:, None]  # <dy, R>: rows are the tokens' own
    assert ((dw - torch.where(r.row >= 0, size, 0)).abs() <= size * (hidden * 2.0**-24)).all()


def test_gradients_are_those_of_differences():
    """<dispatch(x), g> and combine are linear in each argument, so a
    difference of any step is the derivative up to 32-bit rounding."""
    tokens, topk, experts, hidden = 50, 3, 7, 129
    plan, ids, r = routed(tokens, topk, experts, 8, seed=9)
    live = (r.slot >= 0)[:, None]
    f32 = torch.float32
    x, h = torch.randn(2, tokens, hidden, generator=gen(1)).cuda()
    g = torch.randn(plan.rows, hidden, generator=gen(2)).cuda() * live
    rows = plan.empty_rows(hidden, f32)

    def inner(a):
        plan.dispatch(a, r, rows)
        return float((rows.double() * g.double()).sum())

    dx = torch.empty(tokens, hidden, device="cuda")
    plan.combine(g, None, r, dx)
    want = inner(x + h) - inner(x)
    assert abs(float((dx.double() * h.double()).sum()) - want) <= 1e-4 * hidden ** 0.5 * tokens ** 0.5

    w, dwt = torch.randn(2, tokens, topk, generator=gen(3)).cuda()
    rr, dr = torch.randn(2, plan.rows, hidden, generator=gen(4)).cuda() * live
    gy = torch.randn(tokens, hidden, generator=gen(5)).cuda()
    y = torch.empty(tokens, hidden, device="cuda")

    def loss(a, b):
        plan.combine(a, b, r, y)
        return float((y.double() * gy.double()).sum())

    drows, dw = plan.empty_rows(hidden, f32), torch.empty(tokens, topk, device="cuda")
    plan.combine_backward(gy, rr, w, r, drows, dw)
    tol = 1e-4 * hidden ** 0.5 * tokens ** 0.5
    assert abs(float((drows.double() * dr.double()).sum()) - (loss(rr + dr, w) - loss(rr, w))) <= tol
    assert abs(float((dw.double() * dwt.double()).sum()) - (loss(rr, w + dwt) - loss(rr, w))) <= tol


# ------------------------------------------------------------------- casts

def special(x):
    """Infinities, NaN, signed zeros, subnormals, whole-block zeros, the
    largest value and exact scale boundaries (448 * 2^k)."""
    x = x.clone()
    top = torch.finfo(x.dtype).max
    vals = torch.tensor([float("inf"), float("-inf"), float("nan"), 0.0, -0.0, 448.0, 7.0, 3.5, 1e-7, -6e-8])
    n = min(len(vals), x.shape[-1])
    x.view(-1, x.shape[-1])[0, :n] = vals[:n].to(x.dtype)
    x.view(-1, x.shape[-1])[-1] = 0
    if x.view(-1, x.shape[-1]).shape[0] > 2:
        x.view(-1, x.shape[-1])[1, -1] = top
        x.view(-1, x.shape[-1])[2] = torch.finfo(x.dtype).smallest_normal / 4
    return x


CASTS = [(1, 1, "bf16", 0), (3, 128, "fp16", 0), (130, 200, "bf16", 0), (5, 1024, "fp32", 0), (9, 2047, "fp16", 1),
         (257, 1100, "bf16", 4), (64, 7168, "bf16", 0), (300, 130, "fp32", 2), (77, 400, "bf16", 3), (50, 512, "fp32", 0),
         (1001, 98, "fp16", 0)]


def as_bytes(f):
    return f.data.view(torch.uint8).cpu().numpy(), f.scale.view(torch.uint8).cpu().numpy()


def dirty(f):
    f.data.view(torch.uint8).fill_(0xA5)
    f.scale.view(torch.uint8).fill_(0xA5)
    return f


@pytest.mark.parametrize("rows,cols,dtype,pad", CASTS)
@pytest.mark.parametrize("used", [None, 0.6])
def test_quantize_rows(rows, cols, dtype, pad, used):
    x, _ = strided(rows, cols, DT[dtype], pad)
    x.copy_(special(torch.randn(rows, cols, generator=gen(1)).to(DT[dtype])))
    out = dirty(zc.empty_fp8_rows(rows, cols))
    n = rows if used is None else int(rows * used)
    zc.quantize_rows(x, out, None if used is None else torch.tensor([n], dtype=torch.int32, device="cuda"))
    want, got = plain.cast(x.double().cpu().numpy()), as_bytes(out)
    for a, b in zip(got, want):
        assert np.array_equal(a[:n], b[:n]) and (a[n:] == 0xA5).all()


@pytest.mark.parametrize("experts,n,k,dtype", [(1, 1, 1, "bf16"), (2, 128, 256, "bf16"), (3, 200, 130, "fp16"),
                                               (2, 130, 200, "fp32"), (1, 257, 1032, "bf16")])
@pytest.mark.parametrize("transpose", [False, True])
def test_quantize_weights(experts, n, k, dtype, transpose):
    w = special(torch.randn(experts, n, k, generator=gen(2)).to(DT[dtype]))
    out = dirty(zc.empty_fp8_weights(experts, n, k))
    zc.quantize_weights((w.transpose(1, 2) if transpose else w).contiguous().cuda(), out, transpose=transpose)
    got = as_bytes(out)
    for e in range(experts):
        want = plain.cast(w[e].double().numpy(), 128)
        assert np.array_equal(got[0][e], want[0]) and np.array_equal(got[1][e], want[1])


@pytest.mark.parametrize("rows,cols,dtype,pad", CASTS)
@pytest.mark.parametrize("used", [None, 0.6])
def test_quantize_columns(rows, cols, dtype, pad, used):
    x, _ = strided(rows, cols, DT[dtype], pad)
    x.copy_(special(torch.randn(rows, cols, generator=gen(3)).to(DT[dtype])))
    out = dirty(zc.empty_fp8_columns(rows, cols))
    n = rows if used is None else int(rows * used)
    zc.quantize_columns(x, out, None if used is None else torch.tensor([n], dtype=torch.int32, device="cuda"))
    v = x.double().cpu().numpy().copy()
    v[n:] = 0
    data, scale = plain.cast(np.ascontiguousarray(v.T))  # rows of x along the blocks
    got, blocks, done = as_bytes(out), plain.up(rows, 128) // 128, plain.up(n, 128) // 128
    assert np.array_equal(got[0][:done], data.reshape(cols, blocks, 128).transpose(1, 0, 2)[:done])
    assert np.array_equal(got[1][:done, :cols], scale[:, :blocks].T[:done]) and (got[1][:done, cols:] == 127).all()
    assert (got[0][done:] == 0xA5).all() and (got[1][done:] == 0xA5).all()
    if done == blocks:
        # on the CPU: torch's products on the GPU flush 32-bit subnormals; what
        # rounds up to 2^128 is infinity in 32 bits
        back = zc.Fp8Columns(out.data.cpu(), out.scale.cpu(), rows, cols).float().numpy()
        with np.errstate(over="ignore"):
            want = plain.values(data, scale)[:, :rows].T.astype(np.float32)
        assert np.array_equal(back, want, equal_nan=True)


# ---------------------------------------------------------------- products

def whole_numbers(g, *shape):
    """Small whole numbers: casts to 8 bits and sums of products are exact."""
    return torch.randint(-3, 4, shape, generator=g).float()


def segments(counts, align):
    off = [0]
    for c in counts:
        off.append(off[-1] + plain.up(c, align))
    return off


PRODUCTS = [  # rows of each expert, align, n, k
    ([1], 1, 1, 1), ([5], 1, 130, 128), ([0, 3, 0, 17, 64, 1], 1, 200, 300), ([129, 0, 70], 128, 64, 1000),
    ([16] * 20, 16, 260, 520), ([300, 2, 515], 8, 300, 260), ([1000], 1, 1030, 384), ([0, 0, 0], 1, 64, 64),
    ([33, 250, 256, 257], 32, 514, 640), ([7] * 70, 1, 17, 129), ([513], 1, 512, 2048),
]


@pytest.mark.parametrize("out_dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("counts,align,n,k", PRODUCTS)
def test_product_of_whole_numbers_is_exact(counts, align, n, k, out_dtype):
    g, E, off = gen(1), len(counts), segments(counts, align)
    rows = off[-1] + 5  # rows past the segments stay as they are
    a, w = whole_numbers(g, rows, k), whole_numbers(g, E, n, k)
    fa, fw = zc.empty_fp8_rows(rows, k), zc.empty_fp8_weights(E, n, k)
    zc.quantize_rows(a.cuda(), fa)
    zc.quantize_weights(w.cuda(), fw)
    out, whole = strided(rows, n, DT[out_dtype], 3)
    zc.expert_product(fa, fw, out, torch.tensor(off, dtype=torch.int32, device="cuda"),
                      torch.tensor(counts, dtype=torch.int32, device="cuda"))
    got = out.cpu()
    want = torch.zeros(rows, n, dtype=torch.float64)
    for e, c in enumerate(counts):
        want[off[e]:off[e] + c] = a[off[e]:off[e] + c].double() @ w[e].double().T
    assert torch.equal(got[:off[-1]], want[:off[-1]].to(DT[out_dtype]))
    assert bool(torch.isnan(got[off[-1]:]).all()) and guard_intact(whole, n)


SHAPES = [  # sizes that reach every shape of tile, in order and in runs, at ragged ends
    ([3000, 1000, 257, 130, 100, 40, 20], 1, 2000, 300), ([3000, 1000, 257, 130, 100, 40, 20], 32, 6001, 140),
    ([700, 1, 650], 8, 3001, 200), ([20] * 20, 1, 2000, 2100), ([500, 100, 60], 64, 2050, 2100), ([600], 1, 70, 2100),
]


@pytest.mark.parametrize("out_dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("counts,align,n,k", SHAPES)
def test_product_in_every_shape_of_tile_is_exact(counts, align, n, k, out_dtype):
    """Sums of whole numbers below 2^24, against a product in 64 bits."""
    g = torch.Generator("cuda").manual_seed(len(counts) + n)
    E, off = len(counts), segments(counts, align)
    a = torch.randint(-3, 4, (off[-1], k), generator=g, device="cuda").float()
    w = torch.randint(-3, 4, (E, n, k), generator=g, device="cuda").float()
    fa, fw = zc.empty_fp8_rows(off[-1], k), zc.empty_fp8_weights(E, n, k)
    zc.quantize_rows(a, fa)
    zc.quantize_weights(w, fw)
    for pad in (0, 3):
        out, whole = strided(off[-1], n, DT[out_dtype], pad)
        zc.expert_product(fa, fw, out, torch.tensor(off, dtype=torch.int32, device="cuda"),
                          torch.tensor(counts, dtype=torch.int32, device="cuda"))
        for e, c in enumerate(counts):
            want = a[off[e]:off[e] + c].double() @ w[e].double().T
            assert torch.equal(out[off[e]:off[e] + c], want.to(DT[out_dtype])), e
            assert (out[off[e] + c:off[e + 1]] == 0).all(), e
        assert guard_intact(whole, n)


@pytest.mark.parametrize("counts,align,n,k", PRODUCTS)
def test_product_of_any_numbers(counts, align, n, k):
    g, E, off = gen(2), len(counts), segments(counts, align)
    rows = max(off[-1], 1)
    a = torch.randn(rows, k, generator=g) * torch.exp(torch.randn(rows, 1, generator=g))
    w = torch.randn(E, n, k, generator=g) * torch.exp(torch.randn(E, n, 1, generator=g))
    fa, fw = zc.empty_fp8_rows(rows, k), zc.empty_fp8_weights(E, n, k)
    zc.quantize_rows(a.cuda(), fa)
    zc.quantize_weights(w.cuda(), fw)
    out = torch.full((rows, n), float("nan"), device="cuda")
    zc.expert_product(fa, fw, out, torch.tensor(off, dtype=torch.int32, device="cuda"),
                      torch.tensor(counts, dtype=torch.int32, device="cuda"))
    got = out.double().cpu().numpy()
    A = plain.values(*as_bytes(fa))
    for e, c in enumerate(counts):
        W = plain.values(as_bytes(fw)[0][e], as_bytes(fw)[1][e], 128)
        seg = A[off[e]:off[e] + c]
        assert (np.abs(got[off[e]:off[e] + c] - seg @ W.T) <= plain.unit_bound(seg, W)).all()
        assert (got[off[e] + c:off[e + 1]] == 0).all()


@pytest.mark.parametrize("rows,n,k", [(1, 512, 1024), (70, 100, 100), (700, 1024, 512)])
def test_dense_product_and_transposed_weights(rows, n, k):
    """One expert without offsets; the input's gradient from the transpose."""
    g = gen(3)
    x, w, dy = whole_numbers(g, rows, k), whole_numbers(g, n, k), whole_numbers(g, rows, n)
    fx, fw, fwt = zc.empty_fp8_rows(rows, k), zc.empty_fp8_weights(1, n, k), zc.empty_fp8_weights(1, k, n)
    fdy = zc.empty_fp8_rows(rows, n)
    zc.quantize_rows(x.cuda(), fx)
    zc.quantize_rows(dy.cuda(), fdy)
    zc.quantize_weights(w[None].cuda(), fw)
    zc.quantize_weights(w[None].cuda(), fwt, transpose=True)
    y, dx = torch.empty(rows, n, device="cuda"), torch.empty(rows, k, device="cuda")
    zc.expert_product(fx, fw, y)
    zc.expert_product(fdy, fwt, dx)
    assert torch.equal(y.cpu(), x @ w.T) and torch.equal(dx.cpu(), dy @ w)


GRADS = [([128], 128, 1, 1), ([5, 0, 200], 128, 70, 130), ([0, 0], 128, 64, 64), ([300, 1, 128, 0, 129], 128, 260, 300),
         ([40] * 9, 128, 257, 140), ([1000, 30], 256, 520, 512)]


@pytest.mark.parametrize("out_dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("counts,align,n,k", GRADS)
def test_weight_gradient_of_whole_numbers_is_exact(counts, align, n, k, out_dtype):
    g, E, off = gen(4), len(counts), segments(counts, align)
    rows = off[-1] + 128
    live = torch.zeros(rows, 1)
    for e, c in enumerate(counts):
        live[off[e]:off[e] + c] = 1
    x, dy = whole_numbers(g, rows, k) * live, whole_numbers(g, rows, n) * live
    fx, fy = dirty(zc.empty_fp8_columns(rows, k)), dirty(zc.empty_fp8_columns(rows, n))
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    zc.quantize_columns(x.cuda(), fx, offsets[-1:])
    zc.quantize_columns(dy.cuda(), fy, offsets[-1:])
    dw = torch.full((E, n, k), float("nan"), dtype=DT[out_dtype], device="cuda")
    zc.expert_weight_grad(fy, fx, dw, offsets)
    for e, c in enumerate(counts):
        a, b = off[e], off[e] + c
        assert torch.equal(dw[e].cpu(), (dy[a:b].T @ x[a:b]).to(DT[out_dtype])), e


@pytest.mark.parametrize("out_dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("counts,n,k", [([300, 200], 3040, 3039), ([130] * 3, 1300, 1301), ([700, 0], 1200, 1401),
                                        ([40] * 20, 60, 2000), ([300, 5000, 0, 60], 130, 71)])
def test_weight_gradient_in_every_shape_of_tile_is_exact(counts, n, k, out_dtype):
    g = torch.Generator("cuda").manual_seed(n + k)
    E, off = len(counts), segments(counts, 128)
    rows = off[-1]
    x = torch.randint(-3, 4, (rows, k), generator=g, device="cuda").float()
    dy = torch.randint(-3, 4, (rows, n), generator=g, device="cuda").float()
    for e, c in enumerate(counts):
        x[off[e] + c:off[e + 1]] = 0
    fx, fy = zc.empty_fp8_columns(rows, k), zc.empty_fp8_columns(rows, n)
    zc.quantize_columns(x, fx)
    zc.quantize_columns(dy, fy)
    dw = torch.full((E, n, k), float("nan"), dtype=DT[out_dtype], device="cuda")
    zc.expert_weight_grad(fy, fx, dw, torch.tensor(off, dtype=torch.int32, device="cuda"))
    for e in range(E):
        y64, x64 = dy[off[e]:off[e + 1]].double().t().contiguous(), x[off[e]:off[e + 1]].double()
        assert torch.equal(dw[e], (y64 @ x64).to(DT[out_dtype])), e


@pytest.mark.parametrize("counts,n,k", [([9000], 60, 130), ([17000, 0], 200, 70), ([40, 33000], 1, 129)])
def test_weight_gradient_of_long_segments_in_parts(counts, n, k):
    """Segments long enough to be summed in parts: with the caller's
    workspace, with torch's, on another stream, and whole, all exact."""
    E, off, g = len(counts), segments(counts, 128), gen(8)
    rows = off[-1]
    need = zc.expert_weight_grad_workspace_bytes(rows, E, n, k)
    assert need >= 2 * E * n * k * 4
    x, dy = torch.zeros(rows, k), torch.zeros(rows, n)
    for e, c in enumerate(counts):
        x[off[e]:off[e] + c], dy[off[e]:off[e] + c] = whole_numbers(g, c, k), whole_numbers(g, c, n)
    fx, fy = zc.empty_fp8_columns(rows, k), zc.empty_fp8_columns(rows, n)
    zc.quantize_columns(x.cuda(), fx)
    zc.quantize_columns(dy.cuda(), fy)
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    want = torch.stack([dy[off[e]:off[e + 1]].double().T @ x[off[e]:off[e + 1]].double() for e in range(E)]).float()
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for kw in ({}, {"ws": ws[:need]}, {"stream": side}):
        dw = torch.full((E, n, k), float("nan"), device="cuda")
        torch.cuda.synchronize()
        zc.expert_weight_grad(fy, fx, dw, offsets, **kw)
        torch.cuda.synchronize()
        assert torch.equal(dw.cpu(), want), kw
    assert (ws[need:] == 0xFF).all()
    dw = torch.full((E, n, k), float("nan"), device="cuda")
    L = zc.lib()
    rc = L.zc_expert_weight_grad(fy.data.data_ptr(), fy.scale.data_ptr(), fx.data.data_ptr(), fx.scale.data_ptr(), rows, E,
                                 n, k, offsets.data_ptr(), dw.data_ptr(), 2, None, 0, torch.cuda.current_stream().cuda_stream)
    assert rc == 0 and torch.equal(dw.cpu(), want)
    with pytest.raises(zc.ZcError) as e:
        zc.expert_weight_grad(fy, fx, dw, offsets, ws=ws[:need - 1])
    assert e.value.code == 2


@pytest.mark.parametrize("rows,parts", [(1024, False), (65536, True)])
def test_weight_gradient_of_segments_that_share_a_block_is_nan(rows, parts):
    """Rows of segments that begin inside a block of 128 cannot be told apart;
    the segments around them, the last one's end, and empty ones wherever they
    begin are as ever."""
    n, k = 60, 130
    off = [0, 128, 200, 200, 384, 512, rows - 60, rows - 60]
    want = [128, None, 0, None, 128, rows - 60 - 512, 0]
    assert (zc.expert_weight_grad_workspace_bytes(rows, len(want), n, k) > 0) == parts
    x, y = torch.ones(rows, k, device="cuda"), torch.ones(rows, n, device="cuda")
    x[rows - 60:] = 0
    fx, fy = zc.empty_fp8_columns(rows, k), zc.empty_fp8_columns(rows, n)
    zc.quantize_columns(x, fx)
    zc.quantize_columns(y, fy)
    for dt in DT.values():
        dw = torch.zeros(len(want), n, k, dtype=dt, device="cuda")
        zc.expert_weight_grad(fy, fx, dw, torch.tensor(off, dtype=torch.int32, device="cuda"))
        for e, v in enumerate(want):
            got = dw[e].cpu()
            assert bool((torch.isnan(got) if v is None else got == torch.tensor(float(v)).to(dt)).all()), e


def test_weight_gradient_of_any_numbers():
    counts, n, k = [200, 0, 513], 300, 260
    off = segments(counts, 128)
    g = gen(5)
    x, dy = torch.randn(off[-1], k, generator=g), torch.randn(off[-1], n, generator=g)
    for e, c in enumerate(counts):
        x[off[e] + c:off[e + 1]] = 0
        dy[off[e] + c:off[e + 1]] = 0
    fx, fy = zc.empty_fp8_columns(off[-1], k), zc.empty_fp8_columns(off[-1], n)
    zc.quantize_columns(x.cuda(), fx)
    zc.quantize_columns(dy.cuda(), fy)
    dw = torch.empty(3, n, k, device="cuda")
    zc.expert_weight_grad(fy, fx, dw, torch.tensor(off, dtype=torch.int32, device="cuda"))
    X, Y = fx.float().double().cpu().numpy().T, fy.float().double().cpu().numpy().T
    for e in range(3):
        a, b = Y[:, off[e]:off[e + 1]], X[:, off[e]:off[e + 1]]
        assert (np.abs(dw[e].double().cpu().numpy() - a @ b.T) <= plain.unit_bound(a, b)).all()


def test_product_gradients_are_those_of_differences():
    """L(A, W) = <A W^T, G> with whole numbers: both gradients, exactly."""
    rows, n, k = 256, 96, 130
    g = gen(6)
    a, da = whole_numbers(g, 2, rows, k)
    w, dw = whole_numbers(g, 2, n, k)
    G = whole_numbers(g, rows, n)

    def loss(x, m):
        fx, fm = zc.empty_fp8_rows(rows, k), zc.empty_fp8_weights(1, n, k)
        zc.quantize_rows(x.cuda(), fx)
        zc.quantize_weights(m[None].cuda(), fm)
        y = torch.empty(rows, n, device="cuda")
        zc.expert_product(fx, fm, y)
        return float((y.double().cpu() * G.double()).sum())

    fx, fg = zc.empty_fp8_columns(rows, k), zc.empty_fp8_columns(rows, n)
    zc.quantize_columns(a.cuda(), fx)
    zc.quantize_columns(G.cuda(), fg)
    gw = torch.empty(1, n, k, device="cuda")
    zc.expert_weight_grad(fg, fx, gw)
    fgr, fwt, ga = zc.empty_fp8_rows(rows, n), zc.empty_fp8_weights(1, k, n), torch.empty(rows, k, device="cuda")
    zc.quantize_rows(G.cuda(), fgr)
    zc.quantize_weights(w[None].cuda(), fwt, transpose=True)
    zc.expert_product(fgr, fwt, ga)
    assert float((gw[0].cpu().double() * dw.double()).sum()) == loss(a, w + dw) - loss(a, w)
    assert float((ga.cpu().double() * da.double()).sum()) == loss(a + da, w) - loss(a, w)


def test_nan_stays_in_its_row():
    """A NaN or infinity spoils its own row (or column), no other; the rows of
    other experts and padding rows that hold NaN spoil nothing."""
    counts, n, k = [40, 300], 270, 256
    off, g = segments(counts, 64), gen(7)
    a, w = whole_numbers(g, off[-1], k), whole_numbers(g, 2, n, k)
    a[3, 5], a[off[1] + 299, 255] = float("nan"), float("inf")
    for e, c in enumerate(counts):
        a[off[e] + c:off[e + 1]] = float("nan")
    w[1, 17, 200] = float("-inf")
    fa, fw = zc.empty_fp8_rows(off[-1], k), zc.empty_fp8_weights(2, n, k)
    zc.quantize_rows(a.cuda(), fa)
    zc.quantize_weights(w.cuda(), fw)
    out = torch.empty(off[-1], n, device="cuda")
    zc.expert_product(fa, fw, out, torch.tensor(off, dtype=torch.int32, device="cuda"),
                      torch.tensor(counts, dtype=torch.int32, device="cuda"))
    bad = torch.zeros(off[-1], n, dtype=torch.bool)
    bad[3], bad[off[1] + 299], bad[off[1]:off[1] + 300, 17] = True, True, True
    assert torch.equal(torch.isnan(out.cpu()), bad)
    assert (out[40:64] == 0).all() and (out[off[1] + 300:] == 0).all()


# ------------------------------------------------- streams, graphs, refusals

def test_other_stream_and_graph_replays():
    """The whole path on a stream of its own and in a graph that is replayed
    with new inputs, between eager calls: the same as eager every time."""
    tokens, topk, experts, hidden, n = 70, 4, 9, 256, 192
    plan = zc.ExpertPlan(tokens, topk, experts, 128)
    r, ws = plan.empty_routing(), plan.empty_workspace()
    ids = torch.zeros(tokens, topk, dtype=torch.int32, device="cuda")
    x, w = torch.zeros(tokens, hidden, device="cuda"), torch.zeros(tokens, topk, device="cuda")
    fa, fw = plan.empty_fp8(hidden), zc.empty_fp8_weights(experts, n, hidden)
    zc.quantize_weights(torch.randn(experts, n, hidden, generator=gen(1)).cuda(), fw)
    out, y = plan.empty_rows(n, torch.float32), torch.zeros(tokens, n, device="cuda")

    def path(y):
        plan.route(ids, r, ws)
        plan.dispatch_fp8(x, r, fa)
        zc.expert_product(fa, fw, out, r.offsets, r.counts)
        plan.combine(out, w, r, y)

    def load(seed):
        g = gen(seed)
        ids.copy_(torch.randint(-1, experts, (tokens, topk), generator=g, dtype=torch.int32))
        x.copy_(torch.randn(tokens, hidden, generator=g))
        w.copy_(torch.rand(tokens, topk, generator=g))

    load(0)
    path(y)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        path(y)
    want = torch.zeros_like(y)
    for seed in range(1, 6):
        load(seed)
        y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        path(want)
        torch.cuda.synchronize()
        assert torch.equal(got, want), seed
    load(9)
    path(want)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        y.fill_(float("nan"))
        path(y)
    side.synchronize()
    assert torch.equal(y, want)


def test_rows_past_32_bit_offsets():
    """Row buffers of more than 2^32 bytes and 2^31 elements."""
    tokens, topk, experts, hidden = 40000, 8, 16, 8192
    say("  rows: 320,000 x 8192 BF16 (5.2 GB)")
    plan = zc.ExpertPlan(tokens, topk, experts)
    r = plan.empty_routing()
    ids = (torch.arange(tokens * topk, dtype=torch.int32) % experts).reshape(tokens, topk).cuda()
    plan.route(ids, r, plan.empty_workspace())
    x = (torch.arange(tokens, device="cuda", dtype=torch.int32)[:, None] % 251 + torch.arange(hidden, device="cuda") % 5).to(torch.bfloat16)
    rows = plan.empty_rows(hidden)
    plan.dispatch(x, r, rows)
    token = (r.slot // topk).long()
    for lo in range(0, plan.rows, 40000):
        assert torch.equal(rows[lo:lo + 40000], x[token[lo:lo + 40000]]), lo
    y = torch.empty_like(x)
    plan.combine(rows, torch.full((tokens, topk), 0.125, device="cuda"), r, y)
    assert torch.equal(y, x)


def test_refusals():
    plan = zc.ExpertPlan(8, 2, 4)
    r, ws = plan.empty_routing(), plan.empty_workspace()
    x, rows = torch.zeros(8, 64, device="cuda"), plan.empty_rows(64, torch.float32)
    ids = torch.zeros(8, 2, dtype=torch.int32, device="cuda")
    fa, fw = zc.empty_fp8_rows(8, 128), zc.empty_fp8_weights(4, 64, 128)
    out = torch.zeros(8, 64, device="cuda")
    off = torch.zeros(5, dtype=torch.int32, device="cuda")
    for call, code in [
        (lambda: plan.route(ids.long(), r, ws), 1), (lambda: plan.route(ids[:4].contiguous(), r, ws), 2),
        (lambda: plan.route(ids, r, ws[:16]), 2), (lambda: plan.route(ids, r._replace(slot=r.slot[:3]), ws), 2),
        (lambda: plan.dispatch(x.double(), r, rows), 1), (lambda: plan.dispatch(x, r, rows.half()), 1),
        (lambda: plan.dispatch(x[:5], r, rows), 2), (lambda: plan.dispatch(x.t(), r, rows), 1),
        (lambda: plan.dispatch(x, r, rows[:10]), 2), (lambda: plan.dispatch(x[:, ::2], r, plan.empty_rows(32, torch.float32)), 1),
        (lambda: plan.dispatch_fp8(x, r, zc.empty_fp8_rows(plan.rows, 65)), 1),
        (lambda: plan.combine(rows, torch.zeros(3, device="cuda"), r, x), 2),
        (lambda: plan.combine_backward(x, rows, None, r, None, None), 1),
        (lambda: plan.combine_backward(x, None, None, r, None, torch.zeros(8, 2, device="cuda")), 1),
        (lambda: zc.quantize_rows(x, zc.empty_fp8_rows(7, 64)), 2),
        (lambda: zc.quantize_weights(torch.zeros(4, 64, 100, device="cuda"), fw), 1),
        (lambda: zc.expert_product(fa, fw, out), 1),                       # four experts need offsets
        (lambda: zc.expert_product(fa, fw, out, off[:4].contiguous()), 2),
        (lambda: zc.expert_product(fa, fw, out[:, :63], off), 1),
        (lambda: zc.expert_product(zc.empty_fp8_rows(8, 256), fw, out, off), 1),
        (lambda: zc.expert_weight_grad(zc.empty_fp8_columns(128, 8), zc.empty_fp8_columns(256, 8),
                                       torch.zeros(1, 8, 8, device="cuda")), 1),
    ]:
        with pytest.raises(zc.ZcError) as e:
            call()
        assert e.value.code == code


def test_a_stream_of_another_gpu_is_refused():
    plan = zc.ExpertPlan(8, 2, 4)
    r, ws, ids = plan.empty_routing(), plan.empty_workspace(), torch.zeros(8, 2, dtype=torch.int32, device="cuda")
    own = torch.cuda.Stream()
    other = types.SimpleNamespace(cuda_stream=own.cuda_stream, device_index=own.device_index + 1)
    with pytest.raises(zc.ZcError) as e:
        plan.route(ids, r, ws, stream=other)
    assert e.value.code == 1
    torch.cuda.synchronize()
    plan.route(ids, r, ws, stream=own)
    own.synchronize()
    assert r.counts.tolist() == [16, 0, 0, 0]


def test_widths_past_32_bits_are_refused():
    """8.6 GB that no call may take for rows of 64 values."""
    plan = zc.ExpertPlan(1, 1, 1)
    r, wide = plan.empty_routing(), torch.empty(1, 2**32 + 64, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: plan.dispatch(wide, r, wide), lambda: plan.combine(wide, None, r, wide),
                 lambda: plan.combine_backward(wide, wide, None, r, wide, None),
                 lambda: zc.quantize_weights(wide[None], zc.empty_fp8_weights(1, 1, 64))):
        with pytest.raises(zc.ZcError) as e:
            call()
        assert e.value.code == 3


def test_offsets_and_counts_out_of_range_are_clamped():
    """Segments that leave the buffers are cut to them; nothing is read or
    written outside."""
    rows, n, k = 100, 64, 128
    fa, fw = zc.empty_fp8_rows(rows, k), zc.empty_fp8_weights(2, n, k)
    whole = torch.full((rows + 64, n), float("nan"), device="cuda")
    off = torch.tensor([-5, 60, 1 << 30], dtype=torch.int32, device="cuda")
    cnt = torch.tensor([1 << 30, -3], dtype=torch.int32, device="cuda")
    zc.expert_product(fa, fw, whole[:rows], off, cnt)
    assert (whole[:rows] == 0).all() and torch.isnan(whole[rows:]).all()
    fy, fx = zc.empty_fp8_columns(256, 64), zc.empty_fp8_columns(256, 64)
    dw = torch.full((2, 64, 64), float("nan"), device="cuda")
    zc.expert_weight_grad(fy, fx, dw, torch.tensor([-128, 128, 1 << 30], dtype=torch.int32, device="cuda"))
    assert (dw == 0).all()
