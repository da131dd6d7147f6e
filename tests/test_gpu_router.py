"""The router on the GPU against its definitions in 64 bits (router_plain):
choices, weights, balance loss and their gradient.

Tolerances.  A score is e^(x - m) over a sum: x - m is rounded once, 2^-24 of
its size R, which the exponential turns into R 2^-24 of its result; the
exponentials, the sum over up to 1024 experts in lanes and trees of at most 16
+ 6 additions, the quotients and products add fewer than 32 roundings of 2^-23
or less.  So (R + 32) 2^-23 of a weight, 16 more for the sums over tokens (at
most 16 tokens a lane, then 64-bit), and (R + 64) 2^-23 of the terms that a
gradient is added up from, with the rounding to its type."""
import math

import pytest
import torch

import lossless_bf16_exponent_zc_amd as zc
import router_plain as plain

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
INF = math.inf


def logits_of(tokens, experts, dtype, seed, closed=0.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(tokens, experts, generator=g) * 2
    x[torch.rand(tokens, experts, generator=g) < closed] = -INF
    return x.to(dtype), g


def spread(x):
    """R: the largest |x| or difference to the row's largest, of open experts."""
    v = x.double()
    v = torch.where(torch.isfinite(v), v, 0.0)
    return float((v.amax() - v.amin()) + v.abs().amax()) if v.numel() else 0.0


def run(x, router, bias=None, mask=None, ws=None, choice=None):
    c = choice or router.empty_choice()
    router.choose(x.cuda(), c, ws if ws is not None else router.empty_workspace(),
                  bias=None if bias is None else bias.cuda(), mask=None if mask is None else mask.cuda())
    return c


def check_choice(c, x, router, bias=None, mask=None):
    opt = dict(score=router.score, normalize=router.normalize, scale=router.scale, balance=router.balance)
    ids, w, counts, sums, counted, loss = plain.choose(x.double(), router.topk, bias=bias, mask=mask, **opt)
    assert torch.equal(c.ids.cpu().long(), ids)
    assert torch.equal(c.counts.cpu().long(), counts) and int(c.counted) == counted
    R = spread(x)
    assert ((c.weights.cpu().double() - w).abs() <= w.abs() * (R + 32) * 2.0 ** -23 + 1e-38).all()
    assert ((c.sums.cpu().double() - sums).abs() <= sums * (R + 48) * 2.0 ** -23 + 1e-38).all()
    assert abs(float(c.loss) - float(loss)) <= abs(float(loss)) * (R + 64) * 2.0 ** -23 + 1e-38
    return ids, counts, counted


SIZES = [(1, 1, 1), (1, 8, 256), (3, 2, 5), (8, 8, 256), (17, 6, 64), (33, 3, 65), (100, 4, 128), (65, 7, 129),
         (300, 8, 257), (40, 16, 512), (21, 9, 513), (50, 64, 1024), (1021, 3, 37), (2049, 1, 2), (70, 20, 13)]


@pytest.mark.parametrize("tokens,topk,experts", SIZES)
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("score,normalize,biased", [("softmax", False, False), ("softmax", True, True),
                                                    ("sigmoid", True, False), ("sigmoid", False, True)])
def test_choice(tokens, topk, experts, dtype, score, normalize, biased):
    x, g = logits_of(tokens, experts, TYPES[dtype], tokens * 31 + experts, closed=0.1)
    bias = torch.randn(experts, generator=g) * 0.1 if biased else None
    mask = torch.rand(tokens, generator=g) < 0.8
    router = zc.Router(tokens, topk, experts, score=score, normalize=normalize, scale=1.5, balance=0.01)
    for m in (None, mask):
        check_choice(run(x, router, bias, m), x, router, bias, m)


@pytest.mark.parametrize("tokens,topk,experts", SIZES)
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("score,normalize", [("softmax", False), ("softmax", True), ("sigmoid", True), ("sigmoid", False)])
def test_gradient(tokens, topk, experts, dtype, score, normalize):
    x, g = logits_of(tokens, experts, TYPES[dtype], tokens * 37 + experts, closed=0.1)
    mask = torch.rand(tokens, generator=g) < 0.8
    opt = dict(score=score, normalize=normalize, scale=1.5, balance=0.5)
    router = zc.Router(tokens, topk, experts, **opt)
    for m in (None, mask):
        c = run(x, router, None, m)
        for dw, dl in ((torch.randn(tokens, topk, generator=g), None), (None, 2.0), (torch.randn(tokens, topk, generator=g), -0.5)):
            out = torch.full((tokens, experts), 7.0, dtype=x.dtype, device="cuda")
            router.choose_backward(x.cuda(), c, None if dw is None else dw.cuda(),
                                   None if dl is None else torch.tensor([dl], device="cuda"), out,
                                   mask=None if m is None else m.cuda())
            want, size = plain.gradient(x.double(), c.ids.cpu().long(), c.counts.cpu(), int(c.counted),
                                        None if dw is None else dw.double(), 1.0 if dl is None else dl, topk, mask=m, **opt)
            tiny = 2.0 ** -24 if x.dtype == torch.float16 else 1e-37  # below the type's normal numbers
            bound = want.abs() * HALF[x.dtype] + size * (spread(x) + 64) * 2.0 ** -23 + tiny
            assert ((out.cpu().double() - want).abs() <= bound).all()


@pytest.mark.parametrize("score,normalize", [("softmax", False), ("softmax", True), ("sigmoid", True), ("sigmoid", False)])
def test_gradient_against_differences(score, normalize):
    """Central differences of the 64-bit definitions with steps of h = 2^-13:
    off by h^2 / 6 of a third derivative of terms of order 10, below 1e-7,
    and by the gradient's own 32 bits."""
    tokens, topk, experts = 6, 2, 7
    x, g = logits_of(tokens, experts, torch.float32, 5)
    opt = dict(score=score, normalize=normalize, scale=1.0, balance=0.3)
    router = zc.Router(tokens, topk, experts, **opt)
    c = run(x, router)
    ids, counts, n = c.ids.cpu().long(), c.counts.cpu(), int(c.counted)
    dw = torch.randn(tokens, topk, generator=g)
    out = torch.empty(tokens, experts, device="cuda")
    router.choose_backward(x.cuda(), c, dw.cuda(), None, out)

    def value(v):
        w = plain.weights_of(v, ids, score, normalize, 1.0)
        s = plain.shares(plain.scores(v, score)).sum(0)
        return float((w * dw.double()).sum() + plain.loss_of(counts, s, n, topk, 0.3))

    h = 2.0 ** -13
    for t in range(tokens):
        for e in range(experts):
            up, down = x.double(), x.double()
            up[t, e] += h
            down[t, e] -= h
            assert abs(float(out[t, e]) - (value(up) - value(down)) / (2 * h)) < 1e-5


@pytest.mark.parametrize("topk", [5, 8, 12])
@pytest.mark.parametrize("bias", [None, 0.0, 0.25])
def test_ties_go_to_the_lower_index(bias, topk):
    x = torch.zeros(9, 300)
    x[3, 7::11] = 1.0
    x[4] = -0.0
    x[5, ::2] = -0.0
    x[6] = torch.finfo(torch.float32).min
    x[6, 250] = -INF
    x[7] = torch.arange(300) // 4 * 0.125
    x[8] = x[7].flip(0)
    bias = None if bias is None else torch.full((300,), bias)
    for score in zc.Router.SCORES:
        router = zc.Router(9, topk, 300, score=score)
        ids, *_ = check_choice(run(x, router, bias), x, router, bias)
        assert ids[0].tolist() == list(range(topk)) == ids[4].tolist() == ids[6].tolist()


def test_infinite_logits_and_biases():
    """+inf is above every number, for logits and for biases, ties by index."""
    x = torch.zeros(4, 70)
    x[0, 40] = x[0, 20] = INF
    x[1, 5] = torch.finfo(torch.float32).max
    x[1, 6] = INF
    bias = torch.zeros(70)
    for topk in (3, 20):
        router = zc.Router(4, topk, 70, score="sigmoid")
        c = run(x, router)
        assert c.ids[0, :2].tolist() == [20, 40] and c.ids[1, :2].tolist() == [6, 5]
        assert c.weights[0, :2].tolist() == [1.0, 1.0]
        bias[33] = bias[9] = INF
        c = run(x, router, bias)
        assert (c.ids[:, :2].cpu() == torch.tensor([9, 33])).all() and torch.isfinite(c.weights).all()


def test_neighbouring_biased_scores_are_told_apart():
    """Scores that 32 bits hold alike, in an order that 64 bits know: sigmoid
    near its end, where a step of the logit changes it by less than 2^-24."""
    experts = 64
    x = torch.full((4, experts), -3.0)
    x[:, 20:28] = 12.0 + torch.arange(8) * 2.0 ** -10
    x[1] = x[0].flip(0)
    bias = torch.linspace(-1e-3, 1e-3, experts)[torch.randperm(experts, generator=torch.Generator().manual_seed(1))]
    for b in (torch.zeros(experts), bias, torch.full((experts,), 0.25)):
        for topk in (1, 6, 8, 30):
            router = zc.Router(4, topk, experts, score="sigmoid", normalize=True)
            check_choice(run(x, router, b), x, router, b)


@pytest.mark.parametrize("experts", [64, 128, 256, 500, 1000])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_order_of_biased_scores_that_nearly_meet(score, experts):
    """Biases that undo the scores' differences up to some 2^-22, so that every
    comparison is between sums that 32 bits put in another order."""
    g = torch.Generator().manual_seed(experts)
    x = torch.randn(1, experts, generator=g) * 2
    s = plain.scores(x.double(), score)[0]
    bias = (0.5 - s + torch.randn(experts, generator=g).double() * 2.0 ** -22).float()
    x = x.expand(6, -1).contiguous()
    for topk in (4, 8, 17):
        router = zc.Router(6, topk, experts, score=score)
        c = run(x, router, bias)
        want = plain.choose(x.double(), topk, score=score, bias=bias)[0]
        assert torch.equal(c.ids.cpu().long(), want)


@pytest.mark.parametrize("experts", [66, 200, 400, 1000])
@pytest.mark.parametrize("topk", [8, 33, 64])
def test_last_choice_and_the_first_one_left_out_nearly_meet(topk, experts):
    """All choices far apart but the last, whose biased score and that of the
    next expert differ by about 2^-25: 64 bits know which one is chosen."""
    tokens, last = 100, topk - 1
    g = torch.Generator().manual_seed(topk)
    x = torch.full((tokens, experts), -8.0)
    x[:, :last] = torch.linspace(8.0, 2.0, last)
    x[:, last] = torch.rand(tokens, generator=g) * 2 - 1
    x[:, topk] = torch.logit(torch.sigmoid(x[:, last].double()) - 0.125).float()
    bias = torch.zeros(experts)
    bias[topk] = 0.125
    router = zc.Router(tokens, topk, experts, score="sigmoid", normalize=True)
    ids, _, _ = check_choice(run(x, router, bias), x, router, bias)
    assert 10 < int((ids[:, last] == topk).sum()) < 90


@pytest.mark.parametrize("experts", [20, 100, 256, 500, 1000])
@pytest.mark.parametrize("more", [-1, 0, 1, 2])
def test_order_of_a_choice_whose_scores_nearly_meet(more, experts):
    """topk + more scores that nearly meet: fewer than are chosen (the others
    closed), just those, and some that are left out, at places in any lane."""
    for topk in (2, 5, 8):
        for seed in range(20):
            g = torch.Generator().manual_seed(seed)
            x = torch.full((3, experts), -INF if more < 0 else -8.0)
            near = torch.randperm(experts, generator=g)[:topk + more]
            x[:, near] = torch.randn(topk + more, generator=g) * 2
            bias = torch.zeros(experts)
            s = plain.scores(x.double(), "sigmoid")[0]
            bias[near] = (0.5 - s[near] + torch.randn(topk + more, generator=g).double() * 2.0 ** -23).float()
            bias[near[0]] = bias[near[-1]]
            x[:, near[0]] = x[:, near[-1]]
            x[2] = x[2].flip(0)
            router = zc.Router(3, topk, experts, score="sigmoid", normalize=True)
            want = plain.choose(x.double(), topk, score="sigmoid", bias=bias)[0]
            assert torch.equal(run(x, router, bias).ids.cpu().long(), want), (topk, seed)


def test_tokens_with_few_open_experts():
    x = torch.full((6, 40), -INF)
    x[1, 39] = -5.0
    x[2, 3], x[2, 30] = torch.finfo(torch.float32).min, 2.0
    x[3] = torch.linspace(-90, -700, 40)
    x[5, :3] = 100.0
    for score in zc.Router.SCORES:
        for normalize in (False, True):
            router = zc.Router(6, 4, 40, score=score, normalize=normalize, balance=0.1)
            c = run(x, router)
            assert c.ids[0].tolist() == [-1] * 4 and c.ids[1].tolist() == [39, -1, -1, -1]
            assert not torch.isnan(c.weights).any() and not c.weights[0].any()
            want = plain.choose(x.double(), 4, score=score, normalize=normalize, balance=0.1)
            assert torch.equal(c.ids.cpu().long(), want[0])
            # e^(x - m) of x - m up to 610: 610 2^-23 of it, below 1e-4
            assert torch.allclose(c.weights.cpu().double(), want[1], rtol=1e-4, atol=1e-38)
            assert torch.allclose(c.sums.cpu().double(), want[3], rtol=1e-4, atol=1e-38)
            out = torch.full((6, 40), 7.0, device="cuda")
            router.choose_backward(x.cuda(), c, torch.ones(6, 4, device="cuda"), None, out)
            assert torch.isfinite(out).all() and not out[0].any()


def test_a_bias_of_minus_infinity_closes_an_expert():
    x, _ = logits_of(20, 9, torch.float32, 3)
    bias = torch.zeros(9)
    bias[4] = -INF
    router = zc.Router(20, 9, 9)
    c = run(x, router, bias)
    assert not (c.ids == 4).any() and (c.ids[:, 8] == -1).all()
    check_choice(c, x, router, bias)


def test_what_is_not_finite_stays_with_its_token():
    x, _ = logits_of(5, 33, torch.float32, 4)
    clean = x.clone()
    x[1, 5], x[3, 6] = math.nan, INF
    for score in zc.Router.SCORES:
        router = zc.Router(5, 3, 33, score=score, normalize=True, balance=0.1)
        c, d = run(x, router), run(clean, router)
        rows = [0, 2, 4]
        assert torch.equal(c.ids[rows], d.ids[rows]) and torch.equal(c.weights[rows], d.weights[rows])
        assert not (c.ids[1] == 5).any() and c.ids[3, 0] == 6
        assert ((c.ids >= -1) & (c.ids < 33)).all()
        assert torch.isnan(c.loss).all()  # a NaN is not lost
        if score == "softmax":
            assert torch.isnan(c.weights[1]).all() and torch.isnan(c.weights[3]).all()
        out = torch.zeros(5, 33, device="cuda")
        router.choose_backward(x.cuda(), d, torch.ones(5, 3, device="cuda"), None, out)
        assert torch.isfinite(out[rows]).all() and torch.isnan(out[1]).any()


def test_all_masked_and_no_tokens():
    x, _ = logits_of(50, 30, torch.bfloat16, 6)
    router = zc.Router(50, 4, 30, balance=0.1)
    mask = torch.zeros(50, dtype=torch.bool)
    x[:] = math.nan  # masked logits are not looked at
    c = run(x, router, mask=mask)
    assert (c.ids == -1).all() and not c.weights.any() and not c.counts.any() and not c.sums.any()
    assert int(c.counted) == 0 and float(c.loss) == 0
    out = torch.full((50, 30), 7.0, dtype=torch.bfloat16, device="cuda")
    router.choose_backward(x.cuda(), c, torch.ones(50, 4, device="cuda"), None, out, mask=mask.cuda())
    assert not out.any()
    router = zc.Router(0, 4, 30, balance=0.1)
    c = router.empty_choice()
    c.counts.fill_(5), c.sums.fill_(5), c.counted.fill_(5), c.loss.fill_(5)
    x = torch.empty(0, 30)
    run(x, router, choice=c)
    assert not c.counts.any() and not c.sums.any() and int(c.counted) == 0 and float(c.loss) == 0
    router.choose_backward(x.cuda(), c, None, None, x.cuda())


@pytest.mark.parametrize("offset,pad", [(0, 0), (1, 0), (0, 3), (1, 5), (3, 2)])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_rows_at_any_address(offset, pad, dtype):
    tokens, experts = 37, 61
    x, g = logits_of(tokens, experts, TYPES[dtype], 8)
    router = zc.Router(tokens, 5, experts, normalize=True, balance=0.1)
    room = torch.full((offset + tokens * (experts + pad) + 8,), math.nan, dtype=x.dtype, device="cuda")
    view = room[offset:offset + tokens * (experts + pad)].view(tokens, experts + pad)[:, :experts]
    view.copy_(x)
    c = router.empty_choice()
    router.choose(view, c, router.empty_workspace())
    check_choice(c, x, router)
    dw = torch.randn(tokens, 5, generator=g).cuda()
    a, b = torch.empty(tokens, experts, dtype=x.dtype, device="cuda"), room.clone()
    vb = b[offset:offset + tokens * (experts + pad)].view(tokens, experts + pad)[:, :experts]
    router.choose_backward(x.cuda(), c, dw, None, a)
    router.choose_backward(view, c, dw, None, vb)
    assert torch.equal(a, vb)
    outside = torch.ones_like(room, dtype=torch.bool)
    outside[offset:offset + tokens * (experts + pad)].view(tokens, experts + pad)[:, :experts] = False
    assert torch.isnan(b[outside]).all()  # nothing written between the rows


def test_longer_buffers_keep_their_ends():
    x, _ = logits_of(40, 20, torch.float32, 9)
    router = zc.Router(33, 3, 20)
    c = zc.Choice(*(torch.full((v.numel() + 9,), 77, dtype=v.dtype, device="cuda") for v in router.empty_choice()))
    dx = torch.full((40, 20), 77.0, device="cuda")
    router.choose(x.cuda(), c, router.empty_workspace())
    router.choose_backward(x.cuda(), c, c.weights, None, dx)
    want = plain.choose(x[:33].double(), 3)
    assert torch.equal(c.ids[:99].cpu().long().view(33, 3), want[0])
    for v, n in zip(c, (99, 99, 20, 20, 1, 1)):
        assert (v[n:] == 77).all()
    assert (dx[33:] == 77).all()


def test_the_same_call_gives_the_same_bits_whatever_the_workspace_held():
    x, g = logits_of(5000, 256, torch.bfloat16, 10)
    bias = torch.randn(256, generator=g) * 0.1
    router = zc.Router(5000, 8, 256, score="sigmoid", normalize=True, balance=0.1)
    ws = router.empty_workspace()
    first = None
    for fill in (0, 255, 1):
        ws.fill_(fill)
        c = run(x, router, bias, ws=ws)
        first = first or c
        assert all(torch.equal(a, b) for a, b in zip(c, first))


def test_many_tokens():
    """More tokens than the workgroups take at once, and a launch that goes
    round several times, in parts whose sums add up."""
    x, g = logits_of(30000, 8, torch.float32, 11)
    router = zc.Router(30000, 2, 8, balance=0.1)
    c = run(x, router)
    top = x.double().topk(2, 1).indices
    assert torch.equal(c.ids.cpu().long(), top)
    p = torch.softmax(x.double(), 1)
    # at most 4 tokens a lane and 16 lanes in 32 bits
    assert ((c.sums.cpu().double() - p.sum(0)).abs() <= p.sum(0) * (spread(x) + 48) * 2.0 ** -23).all()
    assert int(c.counts.sum()) == 60000 and int(c.counted) == 30000


def test_another_stream_and_a_captured_graph():
    x, g = logits_of(700, 130, torch.bfloat16, 12)
    x2, _ = logits_of(700, 130, torch.bfloat16, 13)
    router = zc.Router(700, 4, 130, normalize=True, balance=0.1)
    dw = torch.randn(700, 4, generator=g).cuda()
    want = []
    for v in (x, x2):
        c = run(v, router)
        out = torch.empty(700, 130, dtype=v.dtype, device="cuda")
        router.choose_backward(v.cuda(), c, dw, None, out)
        want.append((c, out))
    static, c, out, ws = x.cuda(), router.empty_choice(), torch.empty_like(want[0][1]), router.empty_workspace()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    router.choose(static, c, ws, stream=side)
    router.choose_backward(static, c, dw, None, out, stream=side)
    side.synchronize()
    assert torch.equal(out, want[0][1]) and all(torch.equal(a, b) for a, b in zip(c, want[0][0]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        router.choose(static, c, ws)
        router.choose_backward(static, c, dw, None, out)
    for i in (1, 0, 1, 1, 0):
        static.copy_((x, x2)[i])
        for v in (*c, out):
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i][1]) and all(torch.equal(a, b) for a, b in zip(c, want[i][0]))


@pytest.mark.parametrize("tokens,topk,experts,hidden", [(100, 3, 9, 64), (1, 2, 4, 32), (257, 8, 64, 128)])
def test_with_the_routing_it_feeds(tokens, topk, experts, hidden):
    """Choice, sorting, an elementwise expert, combination and the gradient
    back to the logits, against torch's derivative of the whole in 64 bits.
    The chain's values are in 32 bits: sums over hidden and topk terms, fewer
    than 2^8 + 64 roundings of 2^-23 of terms that add up to `size`."""
    x, g = logits_of(tokens, experts, torch.float32, 14)
    h = torch.randn(tokens, hidden, generator=g)
    factor = torch.randn(experts, hidden, generator=g)
    dy = torch.randn(tokens, hidden, generator=g)
    opt = dict(score="softmax", normalize=True, scale=1.0, balance=0.01)
    router, p = zc.Router(tokens, topk, experts, **opt), zc.ExpertPlan(tokens, topk, experts)
    c, r = router.empty_choice(), p.empty_routing()
    router.choose(x.cuda(), c, router.empty_workspace())
    p.route(c.ids, r, p.empty_workspace())
    assert torch.equal(r.counts, c.counts)
    rows, y = p.empty_rows(hidden, torch.float32), torch.empty(tokens, hidden, device="cuda")
    p.dispatch(h.cuda(), r, rows)
    rows *= torch.repeat_interleave(factor.cuda(), c.counts.long(), 0)
    p.combine(rows, c.weights, r, y)
    dweights, dx = torch.empty_like(c.weights), torch.empty(tokens, experts, device="cuda")
    p.combine_backward(dy.cuda(), rows, c.weights, r, None, dweights)
    router.choose_backward(x.cuda(), c, dweights, None, dx)
    ids = c.ids.cpu().long()
    v = x.double().requires_grad_()
    w = plain.weights_of(v, ids, "softmax", True, 1.0)
    parts = h.double()[:, None] * factor.double()[ids]
    want_y = (w[..., None] * parts).sum(1)
    sums = plain.shares(plain.scores(v, "softmax")).sum(0)
    loss = plain.loss_of(c.counts.cpu(), sums, tokens, topk, 0.01)
    (want,) = torch.autograd.grad((want_y * dy.double()).sum() + loss, v)
    eps = (spread(x) + 64 + 256) * 2.0 ** -23
    size_y = (w[..., None].detach() * parts.abs()).sum(1)
    assert ((y.cpu().double() - want_y.detach()).abs() <= size_y * eps).all()
    each = (parts.abs() * dy.double().abs()[:, None]).sum(2)
    _, size = plain.gradient(x.double(), ids, c.counts.cpu(), tokens, each, 1.0, topk, **opt)
    assert ((dx.cpu().double() - want).abs() <= size * eps + 1e-37).all()
    assert abs(float(c.loss) - float(loss.detach())) <= float(loss.detach()) * eps


@pytest.mark.parametrize("experts", [20, 100, 256, 500, 1000])
@pytest.mark.parametrize("topk", [1, 2, 5, 8, 12])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_equal_scores_at_the_border_hide_no_larger_one(score, topk, experts):
    """The last choice and the first one left out have the same logit and bias,
    and a later expert is larger by less than 32 bits tell (sigmoids of 20 and
    21; softmax scores 2^-14 apart beside biases of 1024), behind clearly larger
    choices, between others, and twice."""
    level = 1024.0 if score == "softmax" else 0.0
    equal, larger = (0.0, 2.0 ** -13) if score == "softmax" else (20.0, 21.0)
    g = torch.Generator().manual_seed(experts + topk)
    x, bias = torch.full((8, experts), equal - 8.0), torch.full((experts,), level)
    place = torch.randperm(experts, generator=g)
    bias[place[:topk - 1]] += torch.arange(topk - 1) * 0.5 + 1  # chosen first
    at = place[topk - 1:topk + 4].sort().values
    for t, values in enumerate([(equal, equal, larger), (equal, equal, larger, larger), (equal, equal, equal, larger),
                                (equal, equal), (equal, larger, equal), (larger, equal, equal), (equal, larger, equal, larger),
                                (equal, equal, equal, equal, larger)]):
        x[t, place[:topk - 1]] = equal
        x[t, at[:len(values)]] = torch.tensor(values)
    router = zc.Router(8, topk, experts, score=score, normalize=True, balance=0.1)
    ids, *_ = check_choice(run(x, router, bias), x, router, bias)
    assert ids[0, -1] == at[2] and ids[3, -1] == at[0]


@pytest.mark.parametrize("topk", [1, 2, 8, 9])
@pytest.mark.parametrize("experts", [64, 256, 600])
def test_scores_that_saturate(experts, topk):
    """16-bit logits so large that many sigmoids are 1, or nearly, in 32 bits:
    without differences in the bias the order is that of 64 bits."""
    g = torch.Generator().manual_seed(experts)
    x = (torch.randn(3000, experts, generator=g) * 16).bfloat16()
    for bias in (torch.zeros(experts), torch.full((experts,), 0.3)):
        router = zc.Router(3000, topk, experts, score="sigmoid")
        want = plain.choose(x.double(), topk, score="sigmoid", bias=bias)[0]
        assert torch.equal(run(x, router, bias).ids.cpu().long(), want)


@pytest.mark.parametrize("gap", [10, 20, 60, 83, 87, 100, 1000])
@pytest.mark.parametrize("experts,topk", [(3, 2), (40, 8), (130, 1), (300, 12), (1000, 64)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_weights_of_choices_far_below_the_largest_logit(score, experts, topk, gap):
    """A bias that keeps the largest logits from being chosen: weights over their
    sum, and their gradient, are those of the chosen ones alone.  Differences
    between the chosen are below 24 and so is what their exponents are rounded by."""
    tokens = 9
    x, g = logits_of(tokens, experts, torch.float32, gap + experts)
    x -= gap
    x[4] += gap  # nothing far below in one
    bias = torch.randn(experts, generator=g) * 0.1
    top = torch.randperm(experts, generator=g)[:max(1, (experts - topk) // 2)]
    x[:, top] = 5.0 - torch.rand(tokens, len(top), generator=g)
    bias[top] = -INF
    opt = dict(score=score, normalize=True, scale=1.5, balance=0.5)
    router = zc.Router(tokens, topk, experts, **opt)
    c = run(x, router, bias)
    ids, w, counts, _, counted, _ = plain.choose(x.double(), topk, bias=bias, **opt)
    assert torch.equal(c.ids.cpu().long(), ids)
    assert ((c.weights.cpu().double() - w).abs() <= w * (24 + 32) * 2.0 ** -23 + 1e-38).all()
    dw = torch.randn(tokens, topk, generator=g)
    for dtype in TYPES.values():
        out = torch.full((tokens, experts), 7.0, dtype=dtype, device="cuda")
        router.choose_backward(x.to(dtype).cuda(), c, dw.cuda(), None, out)
        want, size = plain.gradient(x.to(dtype).double(), ids, counts, counted, dw.double(), 1.0, topk, **opt)
        # shares further than 120 below the largest are below the smallest number
        tiny = 2.0 ** -24 if dtype == torch.float16 else 1e-37
        bound = want.abs() * HALF[dtype] + size * (min(spread(x), 120) + 64) * 2.0 ** -23 + tiny
        assert ((out.cpu().double() - want).abs() <= bound).all()


def test_sums_over_millions_of_tokens():
    """Equal tokens, whose shares 32-bit sums of thousands would all round to one
    side: a part is 16 tokens a lane at most, whatever their number."""
    tokens, experts = 1 << 25, 8
    row = torch.tensor([0.3, -0.7, 0.1, 0.9, -0.2, 0.55, -0.35, 0.0]).bfloat16()
    x = row.cuda().expand(tokens, experts).contiguous()
    router = zc.Router(tokens, 1, experts, balance=0.5)
    c = router.empty_choice()
    router.choose(x, c, router.empty_workspace())
    p = torch.softmax(row.double(), 0)
    assert (c.ids == 3).all() and int(c.counted) == tokens and c.counts.tolist() == [0, 0, 0, tokens, 0, 0, 0, 0]
    R = spread(row)
    assert ((c.sums.cpu().double() - p * tokens).abs() <= p * tokens * (R + 48) * 2.0 ** -23).all()
    assert abs(float(c.loss) - 0.5 * experts * float(p[3])) <= 0.5 * experts * float(p[3]) * (R + 64) * 2.0 ** -23


@pytest.mark.parametrize("score,biased", [("softmax", False), ("sigmoid", True)])
def test_more_workgroups_than_the_cus_hold(score, biased):
    """Tokens past 16 of 4 at a time in 768 workgroups, some masked."""
    tokens, topk, experts = 50_001, 3, 520
    x, g = logits_of(tokens, experts, torch.float32, 21)
    mask = torch.rand(tokens, generator=g) < 0.8
    bias = torch.randn(experts, generator=g) * 0.1 if biased else None
    router = zc.Router(tokens, topk, experts, score=score, normalize=True, balance=0.1)
    assert router.workspace_bytes > 768 * experts * 8 + 768 * 4 + 1280
    c = run(x, router, bias, mask)
    s = plain.scores(x.double(), score)
    key = x.double() if bias is None else s + bias.double()
    ids = torch.where(mask[:, None], torch.sort(key, dim=1, descending=True, stable=True).indices[:, :topk], -1)
    counts = torch.bincount(ids[ids >= 0], minlength=experts)
    sums = plain.shares(s)[mask].sum(0)
    assert torch.equal(c.ids.cpu().long(), ids) and torch.equal(c.counts.cpu().long(), counts)
    assert int(c.counted) == int(mask.sum())
    assert ((c.sums.cpu().double() - sums).abs() <= sums * (spread(x) + 48) * 2.0 ** -23).all()
    loss = float(plain.loss_of(counts, sums, int(mask.sum()), topk, 0.1))
    assert abs(float(c.loss) - loss) <= loss * (spread(x) + 64) * 2.0 ** -23


def test_refusals():
    from lossless_bf16_exponent_zc_amd.binding import ZC_ERR_CAPACITY, ZC_ERR_INVALID_ARG, ZC_ERR_UNSUPPORTED
    router = zc.Router(8, 2, 16)
    x, c, ws = torch.zeros(8, 16, device="cuda"), router.empty_choice(), router.empty_workspace()
    good = dict(logits=x, choice=c, ws=ws)
    wrong = [
        (ZC_ERR_INVALID_ARG, dict(logits=x[:, :15])), (ZC_ERR_INVALID_ARG, dict(logits=x.double())),
        (ZC_ERR_INVALID_ARG, dict(logits=x.t())), (ZC_ERR_CAPACITY, dict(logits=x[:7])),
        (ZC_ERR_INVALID_ARG, dict(logits=x.cpu())), (ZC_ERR_INVALID_ARG, dict(choice=c._replace(ids=c.ids.long()))),
        (ZC_ERR_CAPACITY, dict(choice=c._replace(weights=c.weights[:7]))),
        (ZC_ERR_CAPACITY, dict(choice=c._replace(counts=c.counts[:15]))),
        (ZC_ERR_INVALID_ARG, dict(choice=c[:5])), (ZC_ERR_CAPACITY, dict(ws=ws[:-1])),
        (ZC_ERR_INVALID_ARG, dict(bias=torch.zeros(16, device="cuda", dtype=torch.bfloat16))),
        (ZC_ERR_CAPACITY, dict(bias=torch.zeros(15, device="cuda"))),
        (ZC_ERR_INVALID_ARG, dict(mask=torch.zeros(8, device="cuda"))),
        (ZC_ERR_CAPACITY, dict(mask=torch.zeros(7, device="cuda", dtype=torch.bool))),
    ]
    for code, change in wrong:
        with pytest.raises(zc.ZcError) as e:
            router.choose(**{**good, **change})
        assert e.value.code == code, change
    back = dict(logits=x, choice=c, dweights=c.weights, dloss=c.loss, dlogits=torch.zeros_like(x))
    for code, change in [(ZC_ERR_INVALID_ARG, dict(dlogits=x.bfloat16())), (ZC_ERR_INVALID_ARG, dict(dlogits=x[:, 1:])),
                         (ZC_ERR_CAPACITY, dict(dweights=c.weights[:5])), (ZC_ERR_INVALID_ARG, dict(dloss=c.counted)),
                         (ZC_ERR_CAPACITY, dict(dlogits=x[:7]))]:
        with pytest.raises(zc.ZcError) as e:
            router.choose_backward(**{**back, **change})
        assert e.value.code == code, change
    for args, kw, code in [((8, 65, 16), {}, ZC_ERR_UNSUPPORTED), ((8, 0, 16), {}, ZC_ERR_UNSUPPORTED),
                           ((8, 2, 1025), {}, ZC_ERR_UNSUPPORTED), ((1 << 31, 1, 2), {}, ZC_ERR_UNSUPPORTED),
                           ((8, 2, 16), dict(score="relu"), ZC_ERR_INVALID_ARG), ((-1, 2, 16), {}, ZC_ERR_INVALID_ARG)]:
        with pytest.raises(zc.ZcError) as e:
            zc.Router(*args, **kw)
        assert e.value.code == code
