"""One training step of a mixture-of-experts layer around the compressed
all-to-all, on one GPU.

    python examples/moe_layer.py [tokens hidden inner experts topk]

Sending side: tokens are sorted by expert (route, dispatch) and each expert's
rows compressed as a stream of their own.  The exchange is stood in for by
decompressing the streams in place.  Receiving side: the rows go to segments
that begin at multiples of 128 and to 8-bit blocks in one pass, through the
two expert products with a SiLU between them, and back to the order they came
in; the sending side combines them with the router's weights.  The backward
pass takes the same way back: gradients of the combination, of both products
(inputs and weights) and of the dispatch.

The step is compared with the same layer in plain torch, without 8-bit blocks.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import lossless_bf16_exponent_zc_amd as zc  # noqa: E402

BF16 = torch.bfloat16


def exchange(rows, counts, hidden):
    """Compress each expert's rows, decompress them again: what the receiver
    gets.  Returns the received rows and the compressed bytes."""
    plan = zc.Plan([c * hidden for c in counts])
    out, sizes, ws = plan.empty_output(), plan.empty_sizes(), plan.empty_workspace()
    received = torch.empty_like(rows)
    plan.compress(rows.view(torch.int16), out, sizes, ws)
    plan.decompress(out, received.view(torch.int16), ws)
    return received, int(sizes.sum())


def train_step(x, ids, weights, w1, w2, dy):
    """x, dy [tokens, hidden], ids and weights [tokens, topk], w1 [experts,
    inner, hidden], w2 [experts, hidden, inner].  Returns y and the gradients
    of x, weights, w1 and w2, and the bytes exchanged, raw and compressed."""
    (tokens, hidden), topk, (experts, inner, _) = x.shape, ids.shape[1], w1.shape

    # sorted by expert, compressed, sent
    send = zc.ExpertPlan(tokens, topk, experts)
    r = send.empty_routing()
    send.route(ids, r, send.empty_workspace())
    rows = send.empty_rows(hidden)
    send.dispatch(x, r, rows)
    counts = r.counts.tolist()
    live = sum(counts)  # slots without an expert have no row
    got, size = exchange(rows[:live], counts, hidden)

    # received: segments at multiples of 128
    here = zc.ExpertPlan(live, 1, experts, align=128)
    q = here.empty_routing()
    mine = torch.repeat_interleave(torch.arange(experts, dtype=torch.int32, device="cuda"), r.counts)
    here.route(mine[:, None].contiguous(), q, here.empty_workspace())
    used = q.offsets[-1:]

    # forward: two products with a SiLU between
    f1, f1t = zc.empty_fp8_weights(experts, inner, hidden), zc.empty_fp8_weights(experts, hidden, inner)
    f2, f2t = zc.empty_fp8_weights(experts, hidden, inner), zc.empty_fp8_weights(experts, inner, hidden)
    for w, f, ft in ((w1, f1, f1t), (w2, f2, f2t)):
        zc.quantize_weights(w, f)
        zc.quantize_weights(w, ft, transpose=True)
    a = here.empty_fp8(hidden)
    here.dispatch_fp8(got, q, a)
    h, out = here.empty_rows(inner), here.empty_rows(hidden)
    zc.expert_product(a, f1, h, q.offsets, q.counts)
    act = torch.nn.functional.silu(h)
    fact = zc.empty_fp8_rows(here.rows, inner)
    zc.quantize_rows(act, fact, used)
    zc.expert_product(fact, f2, out, q.offsets, q.counts)
    back = send.empty_rows(hidden)
    here.combine(out, None, q, back[:live])
    y = torch.empty_like(x)
    send.combine(back, weights, r, y)

    # backward
    dback, dweights = send.empty_rows(hidden), torch.empty_like(weights)
    send.combine_backward(dy, back, weights, r, dback, dweights)
    dout = here.empty_rows(hidden)
    here.dispatch(dback[:live], q, dout)
    fdout, dact = zc.empty_fp8_rows(here.rows, hidden), here.empty_rows(inner)
    zc.quantize_rows(dout, fdout, used)
    zc.expert_product(fdout, f2t, dact, q.offsets, q.counts)
    s = torch.sigmoid(h.float())
    dh = (dact.float() * s * (1 + h.float() * (1 - s))).to(BF16)
    fdh, drows = zc.empty_fp8_rows(here.rows, inner), here.empty_rows(hidden)
    zc.quantize_rows(dh, fdh, used)
    zc.expert_product(fdh, f1t, drows, q.offsets, q.counts)
    xrows = here.empty_rows(hidden)
    here.dispatch(got, q, xrows)
    dw = []
    for grad, value in ((dh, xrows), (dout, act)):
        cg, cv = zc.empty_fp8_columns(*grad.shape), zc.empty_fp8_columns(*value.shape)
        zc.quantize_columns(grad, cg, used)
        zc.quantize_columns(value, cv, used)
        dw.append(torch.empty(experts, grad.shape[1], value.shape[1], dtype=BF16, device="cuda"))
        zc.expert_weight_grad(cg, cv, dw[-1], q.offsets)
    dgot, dx = send.empty_rows(hidden), torch.empty_like(x)
    here.combine(drows, None, q, dgot[:live])
    send.combine(dgot, None, r, dx)
    return y, dx, dweights, dw[0], dw[1], rows[:live], got, size


def plain_step(x, ids, weights, w1, w2, dy):
    """The same layer and its gradients in 32-bit torch."""
    x, weights, w1, w2 = (t.float().requires_grad_() for t in (x, weights, w1, w2))
    y = torch.zeros_like(x)
    for e in range(w1.shape[0]):
        t, k = torch.nonzero(ids == e, as_tuple=True)
        if t.numel():
            part = torch.nn.functional.silu(x[t] @ w1[e].T) @ w2[e].T
            y = y.index_add(0, t, part * weights[t, k][:, None])
    return (y.detach(),) + torch.autograd.grad(y, (x, weights, w1, w2), dy.float())


def inputs(tokens, hidden, inner, experts, topk, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")
    ids = torch.rand(tokens, experts, generator=g, device="cuda").topk(topk, 1).indices.to(torch.int32)
    weights = torch.softmax(n(tokens, topk), 1)
    return (n(tokens, hidden).to(BF16), ids, weights, (n(experts, inner, hidden) * hidden ** -0.5).to(BF16),
            (n(experts, hidden, inner) * inner ** -0.5).to(BF16), n(tokens, hidden).to(BF16))


def off(a, b):
    """Relative 2-norm of the difference."""
    return float((a.double() - b.double()).norm() / b.double().norm())


def main(tokens=2048, hidden=1024, inner=512, experts=32, topk=4):
    data = inputs(tokens, hidden, inner, experts, topk)
    *got, rows, received, size = train_step(*data)
    assert torch.equal(rows.view(torch.int16), received.view(torch.int16)), "the exchange changed a value"
    print(f"exchanged {rows.numel() * 2} bytes as {size}, values unchanged")
    for name, a, b in zip(("y", "dx", "dweights", "dw1", "dw2"), got, plain_step(*data)):
        print(f"{name:9s} off by {off(a, b):.4f} (8-bit blocks against 32-bit torch)")


if __name__ == "__main__":
    main(*(int(v) for v in sys.argv[1:]))
