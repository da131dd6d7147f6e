"""Orthogonalised updates on the GPU against the iteration in 64 bits.

Tolerance.  `model` is the iteration in 64 bits with the roundings that the
operator documents (fp16 factors, X in 22 bits, the diagonals' remainders put
back), so |model - exact| is what those choices cost for an input, computed
without the GPU's code.  What is left are 32-bit sums, which turn a rounding of
a factor the other way where they fall next to a border (2^-24 times the sum's
length against steps of 2^-11, a few in a hundred), and the rounding to bf16, at
most 2^-8 of an element.  So
  |out - exact| <= 2^-8 |exact| + 1.5 |model - exact|   (root of the sum of squares)
for every input; and for matrices of 4096 values or more, whose roundings
average out, the error is within a fifth of the model's, rounded to bf16."""
import math

import pytest
import torch

import lossless_bf16_exponent_zc_amd as zc

pytestmark = pytest.mark.gpu

MUON = (3.4445, -4.7750, 2.0315)
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def steps_of(x, steps, coefficients, rounded, eps=1e-7):
    a, b, c = coefficients
    x = x.double()
    size = x.norm() + eps
    X = x / size if size else x
    if x.shape[0] > x.shape[1]:
        return steps_wide(X.t(), steps, a, b, c, rounded).t()
    return steps_wide(X, steps, a, b, c, rounded)


def steps_wide(X, steps, a, b, c, rounded):
    if not rounded:
        for _ in range(steps):
            A = X @ X.t()
            X = a * X + (b * A + c * (A @ A)) @ X
        return X
    scale = 2.0 ** math.floor(math.log2(X.shape[1]) / 2)
    half = lambda v: v.to(torch.float16).double()

    def kept(m):  # a matrix in fp16, and what its diagonal was rounded by
        h = half(m)
        return h, (m - h).diagonal()

    def whole(m):
        return m[0] + torch.diag(m[1])

    def times(m, n):
        return m[0] @ n[0] + m[1][:, None] * n[0] + m[0] * n[1]

    side, length = (-(-v // 64) * 64 for v in X.shape)
    done = 0
    while done < steps:
        hi = half(X * scale) / scale
        X = hi + half((X - hi) * scale) / scale
        two = side >= 512 and 8 * length >= 11 * side and done + 2 < steps
        A = kept(hi @ hi.t())
        B = kept(b * whole(A) + c * times(A, A))
        factor = a
        if two:
            T = kept(a * whole(A) + times(B, A))
            A = kept(a * whole(T) + times(T, B))
            D = kept(b * whole(A) + c * times(A, A))
            B = kept(a * whole(D) + a * whole(B) + times(D, B))
            factor = a * a
        X = (factor + B[1])[:, None] * X + B[0] @ hi
        done += 2 if two else 1
    return X


def matrices(batch, n, k, kind="plain", seed=0, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed * 1000 + n * 7 + k)
    z = torch.randn(batch, n, k, generator=g)
    if kind == "rows":
        z *= torch.exp(torch.randn(batch, n, 1, generator=g))
    elif kind == "few":  # rank one and noise
        z = 0.01 * z + torch.randn(batch, n, 1, generator=g) * torch.randn(batch, 1, k, generator=g)
    elif kind == "steep":
        u, _, v = torch.linalg.svd(z.double(), full_matrices=False)
        z = (u * (torch.arange(1, u.shape[-1] + 1.0).double() ** -2)) @ v
    return (z * 1e-3).to(dtype)


def check(x, out, steps=5, coefficients=MUON, eps=1e-7):
    assert out.shape == x.shape and out.dtype == torch.bfloat16
    for m, o in zip(x.cpu(), out.cpu().double()):
        exact = steps_of(m, steps, coefficients, False, eps)
        model = steps_of(m, steps, coefficients, True, eps)
        off, whole, cost = (o - exact).norm(), exact.norm(), (model - exact).norm()
        assert off <= 2.0 ** -8 * whole + 1.5 * cost, (float(off / whole), float(cost / whole))
        if m.numel() >= 4096:
            assert off <= 1.2 * (model.to(torch.bfloat16).double() - exact).norm(), (float(off / whole), float(cost / whole))


SIZES = [(300, 33, 20), (5, 64, 512), (2, 512, 63), (2, 64, 513), (1, 512, 704), (1, 512, 705), (1, 1, 1), (3, 1, 7), (2, 7, 1), (2, 5, 3), (1, 16, 16), (2, 63, 65), (2, 65, 63), (1, 64, 64), (1, 64, 256),
         (20, 64, 48), (1, 100, 1000), (1, 1000, 100), (3, 129, 257), (3, 257, 129), (1, 300, 300), (2, 512, 640),
         (1, 640, 512), (1, 577, 1100), (1, 1025, 514), (1, 1, 2000), (1, 2000, 1), (1, 40, 4100)]


@pytest.mark.parametrize("batch,n,k", SIZES)
@pytest.mark.parametrize("dtype", list(TYPES))
def test_sizes(batch, n, k, dtype):
    x = matrices(batch, n, k, "rows", dtype=TYPES[dtype]).cuda()
    out = torch.full((batch, n, k), 7.0, dtype=torch.bfloat16, device="cuda")
    zc.orthogonalize(x, out)
    check(x, out)


@pytest.mark.parametrize("kind", ["plain", "few", "steep"])
@pytest.mark.parametrize("n,k", [(64, 64), (300, 200), (200, 900), (512, 512)])
def test_spectra(kind, n, k):
    x = matrices(1, n, k, kind, dtype=torch.float32).cuda()
    out = torch.empty(1, n, k, dtype=torch.bfloat16, device="cuda")
    zc.orthogonalize(x, out)
    check(x, out)


@pytest.mark.parametrize("steps,coefficients", [(1, MUON), (2, MUON), (3, MUON), (10, MUON), (20, (1.5, -0.5, 0.0)),
                                                (12, (15 / 8, -10 / 8, 3 / 8))])
def test_steps_and_coefficients(steps, coefficients):
    for n, k in ((96, 200), (200, 96)):
        x = matrices(2, n, k, dtype=torch.float32).cuda()
        out = torch.empty(2, n, k, dtype=torch.bfloat16, device="cuda")
        zc.orthogonalize(x, out, steps=steps, coefficients=coefficients)
        check(x, out, steps, coefficients)
        if steps >= 12:  # these converge: rows (or columns) are orthonormal
            o = out[0].double() if n < k else out[0].double().t()
            gram = o @ o.t()
            # elements of 1 / sqrt(200) off by up to 2^-8 and the factors' errors, 96 or 200 to a sum
            assert (gram - torch.eye(96, device="cuda", dtype=torch.float64)).abs().amax() < 2.0 ** -6


def test_zeros_and_what_is_not_finite():
    for n, k in ((70, 130), (130, 70), (40, 61), (500, 64), (600, 530)):
        x = matrices(6, n, k, dtype=torch.float32)
        x[1] = 0
        x[3, 5, 60], x[5, 0, 0] = math.nan, -math.inf
        out = torch.full((6, n, k), 7.0, dtype=torch.bfloat16, device="cuda")
        zc.orthogonalize(x.cuda(), out)
        assert not out[1].any() and torch.isnan(out[3]).all() and torch.isnan(out[5]).all()
        check(x[[0, 2, 4]], out[[0, 2, 4]])
        zc.orthogonalize(x.cuda(), out, eps=0.0)
        assert not out[1].any()


@pytest.mark.parametrize("size", [1e-38, 1e-30, 1e-9, 1.0, 1e30, 3e38])
def test_values_of_any_size(size):
    """The sum of squares leaves neither end of its range; eps counts against
    the small ones as the definition has it."""
    g = torch.Generator().manual_seed(2)
    x = ((torch.rand(1, 90, 120, generator=g) * 2 - 1) * size).float()
    for eps in (0.0, 1e-7):
        out = torch.empty(1, 90, 120, dtype=torch.bfloat16, device="cuda")
        zc.orthogonalize(x.cuda(), out, eps=eps)
        if eps == 0.0 or size >= 1e-9:
            check(x, out, eps=eps)
        else:  # X and all that follows next to nothing
            assert out.abs().amax() < 1e-15


def test_smallest_elements_of_each_type():
    x = torch.zeros(3, 4, 4)
    x[0, 1, 2] = 2.0 ** -149
    x[1, 3, 0] = -(2.0 ** -126)
    x[2] = torch.eye(4) * torch.finfo(torch.float32).max
    out = torch.empty(3, 4, 4, dtype=torch.bfloat16, device="cuda")
    zc.orthogonalize(x.cuda(), out, eps=0.0)
    check(x, out, eps=0.0)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("offset", [1, 2, 3])
@pytest.mark.parametrize("n,k", [(67, 81), (81, 67), (33, 45), (520, 719)])
def test_any_address_and_nothing_beside_it(dtype, offset, n, k):
    batch = 3
    x = matrices(batch, n, k, dtype=TYPES[dtype])
    room = torch.full((offset + batch * n * k + 9,), math.nan, dtype=x.dtype, device="cuda")
    view = room[offset:offset + batch * n * k].view(batch, n, k)
    view.copy_(x)
    target = torch.full((offset + batch * n * k + 9,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = target[offset:offset + batch * n * k].view(batch, n, k)
    zc.orthogonalize(view, out)
    check(x, out)
    assert (target[:offset] == 7).all() and (target[offset + batch * n * k:] == 7).all()


@pytest.mark.parametrize("n,k", [(130, 190), (60, 50), (512, 800)])
def test_in_place(n, k):
    x = matrices(4, n, k)
    apart, own = torch.empty_like(x, device="cuda"), x.cuda()
    zc.orthogonalize(x.cuda(), apart)
    zc.orthogonalize(own, own)
    assert torch.equal(apart, own)


@pytest.mark.parametrize("n,k", [(200, 333), (30, 70), (900, 600)])
def test_a_matrix_does_not_depend_on_its_neighbours_or_the_workspace(n, k):
    x = matrices(9, n, k, dtype=torch.float32).cuda()
    x[4] = x[8] = x[0]
    out = torch.empty(9, n, k, dtype=torch.bfloat16, device="cuda")
    one = torch.empty(1, n, k, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(zc.orthogonalize_workspace_bytes(9, n, k), dtype=torch.uint8, device="cuda")
    for fill in (0, 255, 0x7B):  # NaN and large numbers among them
        ws.fill_(fill)
        zc.orthogonalize(x, out, ws)
        assert torch.equal(out[4], out[0]) and torch.equal(out[8], out[0])
    for i in (0, 5):
        zc.orthogonalize(x[i:i + 1], one)
        assert torch.equal(one[0], out[i])


def test_no_matrices():
    x = torch.empty(0, 5, 6, device="cuda")
    zc.orthogonalize(x, x.bfloat16())


def test_offsets_past_32_bits():
    """600 matrices of 2^22 values: the last ones lie past 2^31 elements."""
    x = torch.randn(4, 2048, 2048, device="cuda").to(torch.bfloat16)
    big = torch.empty(600, 2048, 2048, dtype=torch.bfloat16, device="cuda")
    big.copy_(x[:1].expand(600, -1, -1))
    big[597:600] = x[1:]
    zc.orthogonalize(big, big)
    want = torch.empty_like(x)
    zc.orthogonalize(x, want)
    assert torch.equal(big[596], want[0]) and torch.equal(big[597:], want[1:]) and torch.equal(big[511], want[0])


@pytest.mark.parametrize("n,k", [(150, 260), (48, 64), (520, 800)])
def test_another_stream_and_a_captured_graph(n, k):
    inputs = [matrices(3, n, k, seed=s).cuda() for s in range(2)]
    want = [torch.empty_like(v) for v in inputs]
    for v, w in zip(inputs, want):
        zc.orthogonalize(v, w)
    static, out = inputs[0].clone(), torch.empty_like(want[0])
    ws = torch.empty(zc.orthogonalize_workspace_bytes(3, n, k), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    zc.orthogonalize(static, out, ws, stream=side)
    zc.orthogonalize(static, out, stream=side)
    side.synchronize()
    assert torch.equal(out, want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        zc.orthogonalize(static, out, ws)
    for i in (1, 0, 0, 1):
        static.copy_(inputs[i])
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i])
        zc.orthogonalize(inputs[1 - i], out)
        assert torch.equal(out, want[1 - i])


def test_after_the_weight_gradient():
    """One expert's gradient of whole numbers, exact in 8-bit blocks, then its
    update."""
    rows, n, k = 256, 96, 200
    g = torch.Generator().manual_seed(3)
    y = torch.randint(-2, 3, (rows, n), generator=g).to(torch.bfloat16).cuda()
    x = torch.randint(-2, 3, (rows, k), generator=g).to(torch.bfloat16).cuda()
    fy, fx = zc.empty_fp8_columns(rows, n), zc.empty_fp8_columns(rows, k)
    zc.quantize_columns(y, fy)
    zc.quantize_columns(x, fx)
    dw = torch.empty(1, n, k, device="cuda")
    zc.expert_weight_grad(fy, fx, dw)
    assert torch.equal(dw[0], y.float().t() @ x.float())
    out = torch.empty(1, n, k, dtype=torch.bfloat16, device="cuda")
    zc.orthogonalize(dw, out)
    check(dw, out)


def limit(steps):
    """What include/zc_experts.h has for the default coefficients, relative to
    the result's root mean square: of matrices of 4096 unlike elements or more."""
    return 5e-4 * steps + 2.0 ** -22 * MUON[0] ** steps


SPECTRA = ["plain", "rows", "few", "one", "rank8", "one16", "zero rows", "steep"]


def spectrum(kind, n, k):
    g = torch.Generator().manual_seed(n + k)
    if kind in ("plain", "rows", "few", "steep"):
        return matrices(1, n, k, kind, dtype=torch.float32)
    if kind == "rank8":
        x = torch.randn(n, 8, generator=g) @ torch.randn(8, k, generator=g)
    elif kind == "zero rows":
        x = torch.randn(n, k, generator=g)
        x[16:] = 0
    else:
        x = torch.randn(n, 1, generator=g) * torch.randn(1, k, generator=g)
        if kind == "one16":
            x = x.bfloat16().float()
    return x[None]


@pytest.mark.parametrize("kind", SPECTRA)
@pytest.mark.parametrize("n,k", [(64, 64), (64, 300), (70, 2000), (300, 200), (512, 512), (512, 1024), (1100, 520)])
def test_documented_error(n, k, kind):
    """Against the iteration in 64 bits alone, whatever the roundings were: the
    documented limit, with the result's own rounding to bf16 of 2^-8 at most."""
    x = spectrum(kind, n, k).cuda()
    out = torch.empty(1, n, k, dtype=torch.bfloat16, device="cuda")
    for steps in (1, 2, 3, 5, 8, 10, 12):
        zc.orthogonalize(x, out, steps=steps)
        exact = steps_of(x[0].cpu(), steps, MUON, False)
        off = float((out[0].cpu().double() - exact).norm() / exact.norm())
        assert off <= 2.0 ** -8 + limit(steps), (steps, off, limit(steps))


@pytest.mark.parametrize("n,k", [(1, 1), (1, 7), (2, 2), (3, 5), (8, 8), (64, 64), (64, 3000), (300, 300), (640, 1280)])
def test_documented_error_of_like_elements(n, k):
    """Equal elements, or few: ten times the limit's first part, as roundings
    of factors that are all alike do not average out."""
    g = torch.Generator().manual_seed(n + k)
    for x in (torch.ones(n, k), torch.eye(n, k), torch.randn(n, k, generator=g) * torch.exp(torch.randn(1, k, generator=g))):
        out = torch.empty(1, n, k, dtype=torch.bfloat16, device="cuda")
        for steps in (1, 2, 3, 5, 8, 10):
            zc.orthogonalize(x[None].cuda(), out, steps=steps)
            exact = steps_of(x, steps, MUON, False)
            off = float((out[0].cpu().double() - exact).norm() / exact.norm())
            assert off <= 2.0 ** -8 + 5e-3 * steps + 2.0 ** -22 * MUON[0] ** steps, (steps, off)


@pytest.mark.parametrize("size", [2.0 ** -7, 2.0 ** -11, 2.0 ** -13])
def test_small_elements_of_a_step_keep_their_digits(size):
    """One element carries the norm, the others lie where a remainder of fp16
    without a factor would have no digits.  Steps of X <- 0.5 X (b = c = 0) pass
    X on as it is held: hi + lo, 2^-22 of an element and 2^-36 of the norm,
    halved with it, which leave the bf16 result the rounding of the exact one or
    the next (2^-7 of an element between them) in those few that lie so near
    the border: 2^-13 of all by the same count, 1 in 200 allowed."""
    n, k = 130, 256
    g = torch.Generator().manual_seed(5)
    x = (torch.rand(1, n, k, generator=g) + 1) * size / 16  # Y is held times 16
    x[0, 0, 0] = 1.0
    out = torch.empty(1, n, k, dtype=torch.bfloat16, device="cuda")
    for steps in (1, 2, 4):
        zc.orthogonalize(x.cuda(), out, steps=steps, coefficients=(0.5, 0.0, 0.0), eps=0.0)
        want = (x[0].double() / x[0].double().norm() * 0.5 ** steps)
        got = out[0].cpu()
        assert ((got.double() - want).abs() <= want * (2.0 ** -8 + 2.0 ** -16) + 2.0 ** -40).all()
        assert int((got != want.to(torch.bfloat16)).sum()) <= n * k // 200


@pytest.mark.parametrize("kind", ["plain", "rows", "few", "steep", "zero rows"])
@pytest.mark.parametrize("n,k", [(64, 1024), (128, 1000), (200, 900), (512, 704), (512, 1024), (640, 2000), (1024, 1401)])
def test_five_steps_are_near_those_in_32_bits(n, k, kind):
    """A result in bf16 is off by its rounding whatever the arithmetic, 1.66e-3 of
    its root mean square.  Factors in fp16, with the diagonal's product with what
    they leave out added in the last two steps, cost up to 9e-4 more in 64-bit
    arithmetic with those roundings (without that product 1.1e-3 to 2.4e-3 where
    nothing is small), 1e-3 with the 32-bit sums', so 1.17 times as much at most."""
    x = spectrum(kind, n, k).cuda()
    out = torch.empty(1, n, k, dtype=torch.bfloat16, device="cuda")
    zc.orthogonalize(x, out)
    exact = steps_of(x[0].cpu(), 5, MUON, False)
    off, rounding = ((v.double() - exact).norm() for v in (out[0].cpu(), exact.to(torch.bfloat16)))
    assert off <= 1.17 * rounding, float(off / rounding)


def test_refusals():
    from lossless_bf16_exponent_zc_amd.binding import ZC_ERR_CAPACITY, ZC_ERR_INVALID_ARG, ZC_ERR_UNSUPPORTED
    x = torch.zeros(2, 8, 12, device="cuda")
    out = torch.zeros(2, 8, 12, device="cuda", dtype=torch.bfloat16)
    ws = torch.empty(zc.orthogonalize_workspace_bytes(2, 8, 12), dtype=torch.uint8, device="cuda")
    good = dict(x=x, out=out, ws=ws)
    for code, change in [(ZC_ERR_INVALID_ARG, dict(x=x[0])), (ZC_ERR_INVALID_ARG, dict(x=x.double())),
                         (ZC_ERR_INVALID_ARG, dict(x=x.transpose(1, 2))), (ZC_ERR_INVALID_ARG, dict(x=x.cpu())),
                         (ZC_ERR_INVALID_ARG, dict(out=x)), (ZC_ERR_INVALID_ARG, dict(out=out[:1])),
                         (ZC_ERR_INVALID_ARG, dict(out=out.half())), (ZC_ERR_CAPACITY, dict(ws=ws[:-1])),
                         (ZC_ERR_INVALID_ARG, dict(ws=ws.view(torch.int8))), (ZC_ERR_INVALID_ARG, dict(steps=0)),
                         (ZC_ERR_UNSUPPORTED, dict(steps=65)), (ZC_ERR_INVALID_ARG, dict(steps=-1)),
                         (ZC_ERR_INVALID_ARG, dict(coefficients=(1.0, 2.0))), (ZC_ERR_INVALID_ARG, dict(eps="small")),
                         (ZC_ERR_INVALID_ARG, dict(x=x[:, :, :0], out=out[:, :, :0]))]:
        with pytest.raises(zc.ZcError) as e:
            zc.orthogonalize(**{**good, **change})
        assert e.value.code == code, change
    long = torch.zeros(1, 1, 65537, device="cuda")
    with pytest.raises(zc.ZcError) as e:
        zc.orthogonalize(long, long.bfloat16())
    assert e.value.code == ZC_ERR_UNSUPPORTED
