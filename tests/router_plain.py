"""The router's choice, its balance loss and their gradient in 64 bits, from
the definitions in include/zc_experts.h, on the CPU."""
import math

import torch

INF = math.inf


def scores(x, score):
    """Scores of float64 logits [tokens, experts]; a token without any open
    expert has none."""
    if score == "sigmoid":
        return torch.sigmoid(x)
    top = x.amax(1, keepdim=True)
    e = torch.exp(x - torch.where(torch.isneginf(top), torch.zeros_like(top), top))
    total = e.sum(1, keepdim=True)
    return torch.where(total == 0, torch.zeros_like(e), e / total)


def shares(s):
    total = s.sum(1, keepdim=True)
    return torch.where(total == 0, torch.zeros_like(s), s / torch.where(total == 0, torch.ones_like(total), total))


def weights_of(x, ids, score, normalize, scale):
    """Weights of given choices, in a form that keeps its digits where every
    score underflows (sigmoid of -800: e^-800)."""
    has = ids >= 0
    at = ids.clamp(min=0).long()
    if not normalize:
        return torch.where(has, scores(x, score).gather(1, at), 0.0) * scale
    log = (torch.nn.functional.logsigmoid(x) if score == "sigmoid" else x).gather(1, at)
    log = torch.where(has, log, -INF)
    return torch.where(has, scores(log, "softmax"), 0.0) * scale


def choose(x, topk, score="softmax", normalize=False, scale=1.0, balance=0.0, bias=None, mask=None):
    """(ids, weights, counts, sums, counted, loss) of float64 logits."""
    T, E = x.shape
    live = torch.ones(T, dtype=torch.bool) if mask is None else mask
    key = x if bias is None else scores(x, score) + bias.double()
    key = torch.where(torch.isneginf(x) | torch.isnan(x) | torch.isnan(key), -INF, key)
    key = torch.where(live[:, None], key, -INF)
    order = [sorted(range(E), key=lambda e: (-row[e], e))[:topk] for row in key.tolist()]
    ids = torch.full((T, topk), -1, dtype=torch.int64)
    for t, o in enumerate(order):
        for k, e in enumerate(o):
            if key[t, e] > -INF:
                ids[t, k] = e
    w = weights_of(x, ids, score, normalize, scale)
    sums = shares(scores(x, score))[live].sum(0)
    counts = torch.bincount(ids[ids >= 0], minlength=E)
    return ids, w, counts, sums, int(live.sum()), loss_of(counts, sums, int(live.sum()), topk, balance)


def loss_of(counts, sums, counted, topk, balance):
    if not counted:
        return sums.sum() * 0
    return balance * len(counts) * (counts.double() / (topk * counted) * sums / counted).sum()


def gradient(x, ids, counts, counted, dweights, dloss, topk, score="softmax", normalize=False, scale=1.0, balance=0.0,
             mask=None):
    """d(sum of dweights * weights + dloss * loss) / dx by torch's derivative
    of the definitions, and a bound on the terms that were added up for it."""
    live = torch.ones(len(x), dtype=torch.bool) if mask is None else mask
    x = torch.where(live[:, None], x, 0.0).requires_grad_()
    v = torch.where(live, 1.0, 0.0)[:, None]
    sums = (shares(scores(x, score)) * v).sum(0)
    total = dloss * loss_of(counts, sums, counted, topk, balance)
    if dweights is not None:
        total = total + (torch.where(ids >= 0, weights_of(x, ids, score, normalize, scale), 0.0) * v * dweights).sum()
    (g,) = torch.autograd.grad(total, x)
    g = torch.where(torch.isnan(g) & torch.isneginf(x.detach()), 0.0, g)  # closed: no gradient
    g = torch.where(live[:, None], g, 0.0)
    with torch.no_grad():
        s = scores(x, score)
        p = shares(s)
        of_loss = abs(dloss * balance) * len(counts) * counts.double() / (topk * max(1, counted) ** 2)
        up = torch.zeros_like(x)
        if dweights is not None:
            t, k = torch.nonzero((ids >= 0) & live[:, None], as_tuple=True)
            w = weights_of(x, ids, score, normalize, scale).abs()
            dw = dweights.abs()
            mean = (dw * w).sum(1) / scale if normalize else dw.sum(1) * 0
            each = (dw[t, k] * abs(scale) + mean[t] * abs(scale)) if normalize else dw[t, k] * abs(scale)
            up[t, ids[t, k]] = each * (w[t, k] / abs(scale))  # times the score
        size = up + p * of_loss + p * (up.sum(1, keepdim=True) + (p * of_loss).sum(1, keepdim=True))
    return g, torch.where(live[:, None], size, 0.0)
