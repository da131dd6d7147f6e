"""Cases, plain forms and exact values of what a mixture-of-experts layer's
training step needs before its routing and after its weights' gradients: the
router's choice of experts with its balance loss, the gradient of both, and the
orthogonalised update of the experts' weights.

`run` takes the plain form in torch arithmetic where `own` is false and the
library's calls where it is true.  Definitions shared by all:

* Scores s[t, e] of one token's logits l: softmax(l), or sigmoid(l).  Chosen
  are the topk experts of largest l, or with a bias of largest s + bias[e], in
  that order, ties to the lower index.  A logit of -inf closes an expert to a
  token: it is never chosen, and where fewer than topk are open the other
  choices are -1 with weight 0.  Weights are scale * s, or with `normalize`
  scale * s / (sum of the chosen s).  A masked token chooses -1 throughout and
  is counted nowhere.
* p[t, e] = s[t, e] / sum over e of s[t, e].  counts[e]: tokens that chose e;
  sums[e] = sum of p[t, e] over the counted tokens, T of them;
  loss = balance * experts / (topk * T^2) * sum over e of counts[e] * sums[e].
  Its gradient takes the counts as constants.
* Orthogonalised update of x [n, k]: X = x / (|x| + eps), |x| the root of the
  sum of squares, then `steps` times
  X <- a X + (b A + c A^2) X,  A = X X^T  (or X <- a X + X (b A + c A^2),
  A = X^T X, the same thing), with a, b, c = 3.4445, -4.7750, 2.0315.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
EPS = 1e-7
STEPS = 5


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one decoding step of a small batch: the choice's latency
        dict(name="choose decode", op="choose", tokens=8, topk=8, experts=256, dtype="fp32", score="sigmoid",
             bias=True, normalize=True, scale=2.5, balance=0.0, masked=0.0, closed=0.0),
        # the MoE batch's 8192 tokens, 32-bit logits, with the balance loss
        dict(name="choose train", op="choose", tokens=8192, topk=8, experts=256, dtype="fp32", score="softmax",
             bias=False, normalize=True, scale=1.0, balance=0.01, masked=0.0, closed=0.0),
        # a long padded batch, sigmoid scores with a bias that balances the choice
        dict(name="choose long", op="choose", tokens=65536, topk=8, experts=256, dtype="bf16", score="sigmoid",
             bias=True, normalize=True, scale=2.5, balance=0.0001, masked=0.125, closed=0.0),
        # sizes that nothing divides, padding, experts closed to some tokens
        dict(name="choose ragged", op="choose", tokens=1021, topk=3, experts=37, dtype="fp16", score="softmax",
             bias=False, normalize=False, scale=1.0, balance=0.01, masked=0.3, closed=0.2),
        # the gradients of the same: the training step's
        dict(name="choose gradient train", op="choose_grad", tokens=8192, topk=8, experts=256, dtype="fp32",
             score="softmax", bias=False, normalize=True, scale=1.0, balance=0.01, masked=0.0, closed=0.0),
        # the long padded batch's
        dict(name="choose gradient long", op="choose_grad", tokens=65536, topk=8, experts=256, dtype="bf16",
             score="sigmoid", bias=True, normalize=True, scale=2.5, balance=0.0001, masked=0.125, closed=0.0),
        # the ragged batch's
        dict(name="choose gradient ragged", op="choose_grad", tokens=1021, topk=3, experts=37, dtype="fp16",
             score="softmax", bias=False, normalize=False, scale=1.0, balance=0.01, masked=0.3, closed=0.2),
        # one small weight: launches alone
        dict(name="update one small", op="update", batch=1, n=64, k=256, dtype="bf16"),
        # the experts of a small layer, first weight
        dict(name="update small experts", op="update", batch=32, n=512, k=1024, dtype="bf16"),
        # widths that no tile divides, 32-bit momentum
        dict(name="update ragged", op="update", batch=37, n=1000, k=1401, dtype="fp32"),
        # a dense layer of the Llama MLP shape: one large weight, more rows than columns
        dict(name="update dense", op="update", batch=1, n=14336, k=4096, dtype="fp32"),
        # one GPU's 32 experts, whose gradients are 2048 x 7168
        dict(name="update experts", op="update", batch=32, n=2048, k=7168, dtype="bf16"),
    ]


def draw(rng):
    def log_int(a, b):
        return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))

    op = rng.choice(["choose", "choose", "choose_grad", "choose_grad", "update", "update", "update"])
    if op == "update":
        while True:
            c = dict(op=op, batch=log_int(1, 128), n=log_int(16, 14336), k=log_int(16, 14336),
                     dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]))
            if rng.random() < 0.5:
                c["n"], c["k"] = (max(16, v // 16 * 16) for v in (c["n"], c["k"]))
            if work(c)["flops"] <= 16 * 2048 * 2048 * 7168 * 16 and c["batch"] * c["n"] * c["k"] <= 32 * 2048 * 7168 // 2:
                return c
    experts = log_int(4, 1024)
    if rng.random() < 0.5:
        experts = max(8, experts // 8 * 8)
    most = min(65536, 65536 * 256 // experts)
    return dict(op=op, tokens=log_int(1, most), topk=rng.randint(1, min(16, experts)), experts=experts,
                dtype=rng.choice(["bf16", "fp16", "fp32"]), score=rng.choice(["softmax", "sigmoid"]),
                bias=rng.random() < 0.5, normalize=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]),
                balance=rng.choice([0.01, 0.001]), masked=rng.choice([0.0, 0.0, 0.25]),
                closed=rng.choice([0.0, 0.0, 0.1]))


def work(case):
    if case["op"] == "update":
        B, s, l = case["batch"], min(case["n"], case["k"]), max(case["n"], case["k"])
        size = 4 if case["dtype"] == "fp32" else 2
        # A and A^2 are symmetric: half of their products
        return {"bytes": B * s * l * (size + 2), "flops": B * STEPS * (3.0 * s * s * l + 1.0 * s * s * s)}
    T, K, E = case["tokens"], case["topk"], case["experts"]
    size = 4 if case["dtype"] == "fp32" else 2
    live = T * (1 - case["masked"])
    mask = T if case["masked"] else 0
    if case["op"] == "choose":
        return {"bytes": live * E * size + T * K * 8 + E * (12 if case["bias"] else 8) + mask, "flops": 8 * live * E}
    return {"bytes": (live + T) * E * size + T * K * 8 + E * 4 + mask, "flops": 12 * live * E}


# --------------------------------------------------------------- the inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) & 0x7FFFFFFFFFFFFFFF)
    return g


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case)
    dev = dict(device="cuda")
    if case["op"] == "update":
        B, n, k = case["batch"], case["n"], case["k"]
        # momentum of gradients: noise with rows and columns of unlike size,
        # and a few directions that most tokens share
        x = torch.randn(B, n, k, generator=g, **dev)
        x *= torch.exp(0.5 * torch.randn(B, n, 1, generator=g, **dev))
        x *= torch.exp(0.5 * torch.randn(B, 1, k, generator=g, **dev))
        strong = torch.randn(B, n, 4, generator=g, **dev) * torch.tensor([2.0, 1.0, 0.5, 0.25], **dev)
        x += torch.bmm(strong, torch.randn(B, 4, k, generator=g, **dev))
        x *= 1e-3
        s["x"] = x.to(DTYPES[case["dtype"]])
        s["out"] = torch.zeros(B, n, k, dtype=torch.bfloat16, **dev)
        return s
    T, K, E = case["tokens"], case["topk"], case["experts"]
    logits = torch.randn(T, E, generator=g, **dev) * 1.5 + 0.5 * torch.randn(E, generator=g, **dev)
    if case["closed"]:
        shut = torch.rand(T, E, generator=g, **dev) < case["closed"]
        logits.masked_fill_(shut, -math.inf)
    s["logits"] = logits.to(DTYPES[case["dtype"]])
    s["bias_of"] = 0.05 * torch.randn(E, generator=g, **dev) if case["bias"] else None
    s["mask"] = torch.rand(T, generator=g, **dev) >= case["masked"] if case["masked"] else None
    i32, f32 = dict(dtype=torch.int32, **dev), dict(dtype=torch.float32, **dev)
    s["choice"] = (torch.zeros(T, K, **i32), torch.zeros(T, K, **f32), torch.zeros(E, **i32), torch.zeros(E, **f32),
                   torch.zeros(1, **i32), torch.zeros(1, **f32))
    if case["op"] == "choose_grad":
        c = _choose(s)
        s["choice"] = tuple(c[name].contiguous() for name in ("ids", "weights", "counts", "sums", "counted", "loss"))
        s["dweights"] = torch.randn(T, K, generator=g, **dev)
        s["dloss"] = torch.ones(1, **dev)
        s["dlogits"] = torch.zeros(T, E, dtype=s["logits"].dtype, **dev)
    return s


# ---------------------------------------------------------- the plain forms

def _scores(s, dtype):
    """(scores, each token's shares p), masked tokens as others."""
    x = s["logits"].to(dtype)
    if s["score"] == "softmax":
        e = torch.exp(x - x.amax(1, keepdim=True))
        e = torch.where(torch.isneginf(x), 0.0, e)  # a row without any open expert
        p = e / e.sum(1, keepdim=True).clamp(min=1e-30)
        return p, p
    v = 1 / (1 + torch.exp(-x))
    return v, v / v.sum(1, keepdim=True).clamp(min=1e-30)


def _choose(s):
    K, E = s["topk"], s["experts"]
    x = s["logits"].float()
    # the border between chosen and not: scores in 64 bits where they are compared with a bias added
    key = x if s["bias_of"] is None else _scores(s, torch.float64)[0] + s["bias_of"].double()
    key = torch.where(torch.isneginf(x), -math.inf, key)
    if s["mask"] is not None:
        key = torch.where(s["mask"][:, None], key, -math.inf)
    top, ids = torch.sort(key, dim=1, descending=True, stable=True)
    open_ = ~torch.isneginf(top[:, :K])
    ids = torch.where(open_, ids[:, :K], -1)
    score, p = _scores(s, torch.float32)
    w = torch.where(open_, score.gather(1, ids.clamp(min=0)), 0.0)
    if s["normalize"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-30)
    w = w * s["scale"]
    live = torch.ones_like(p[:, 0]) if s["mask"] is None else s["mask"].float()
    sums = (p.double() * live[:, None]).sum(0)  # over all tokens
    flat = torch.where(open_, ids, E).reshape(-1)
    counts = torch.zeros(E + 1, dtype=torch.int64, device="cuda").scatter_add_(0, flat, torch.ones_like(flat))[:E]
    counted = live.double().sum()
    loss = s["balance"] * E / K * (counts * sums).sum() / (counted * counted).clamp(min=1)
    return {"ids": ids.to(torch.int32), "weights": w, "counts": counts.to(torch.int32), "sums": sums.float(),
            "counted": counted.to(torch.int32).reshape(1), "loss": loss.float().reshape(1)}


def _choose_grad(s):
    K, E = s["topk"], s["experts"]
    ids, _, counts, _, counted, _ = s["choice"]
    score, p = _scores(s, torch.float32)
    has = ids >= 0
    at = ids.long().clamp(min=0)
    dw = torch.where(has, s["dweights"], 0.0) * s["scale"]
    if s["normalize"]:
        chosen = torch.where(has, score.gather(1, at), 0.0)
        whole = chosen.sum(1, keepdim=True).clamp(min=1e-30)
        share = chosen / whole
        dw = torch.where(has, (dw - (dw * share).sum(1, keepdim=True)) / whole, 0.0)
    dscore = torch.zeros_like(score).scatter_add_(1, at, dw)
    T = counted.float().clamp(min=1)
    dp = (s["balance"] * E / K) * s["dloss"] * counts.float() / (T * T)
    if s["score"] == "softmax":
        d = dscore + dp
        dx = p * (d - (p * d).sum(1, keepdim=True))
    else:
        total = score.sum(1, keepdim=True).clamp(min=1e-30)
        dscore = dscore + (dp - (p * dp).sum(1, keepdim=True)) / total
        dx = dscore * score * (1 - score)
    if s["mask"] is not None:
        dx = torch.where(s["mask"][:, None], dx, 0.0)
    return {"dlogits": dx.to(s["logits"].dtype)}


def _update(s):
    a, b, c = COEFFICIENTS
    x = s["x"].float()
    X = x / (x.square().sum((1, 2), keepdim=True).sqrt() + EPS)
    tall = s["n"] > s["k"]
    for _ in range(STEPS):
        if tall:
            A = torch.bmm(X.transpose(1, 2), X)
            X = a * X + torch.bmm(X, b * A + c * torch.bmm(A, A))
        else:
            A = torch.bmm(X, X.transpose(1, 2))
            X = a * X + torch.bmm(b * A + c * torch.bmm(A, A), X)
    return {"out": X.to(torch.bfloat16)}


# ------------------------------------------------------- the library's calls

def _own(s):
    import lossless_bf16_exponent_zc_amd as zc
    if s["op"] == "update":
        if "ws" not in s:
            s["ws"] = torch.empty(zc.orthogonalize_workspace_bytes(s["batch"], s["n"], s["k"]), dtype=torch.uint8,
                                  device="cuda")
        zc.orthogonalize(s["x"], s["out"], s["ws"], steps=STEPS, coefficients=COEFFICIENTS, eps=EPS)
        return {"out": s["out"]}
    if "router" not in s:
        s["router"] = zc.Router(s["tokens"], s["topk"], s["experts"], score=s["score"], normalize=s["normalize"],
                                scale=s["scale"], balance=s["balance"])
        s["ws"] = s["router"].empty_workspace()
        s["c"] = zc.Choice(*s["choice"])
    router, c = s["router"], s["c"]
    if s["op"] == "choose":
        router.choose(s["logits"], c, s["ws"], bias=s["bias_of"], mask=s["mask"])
        return {"ids": c.ids, "weights": c.weights, "counts": c.counts, "sums": c.sums, "counted": c.counted,
                "loss": c.loss}
    router.choose_backward(s["logits"], c, s["dweights"], s["dloss"], s["dlogits"], mask=s["mask"])
    return {"dlogits": s["dlogits"]}


_PLAIN = {"choose": _choose, "choose_grad": _choose_grad, "update": _update}


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


# ------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "update":
        a, b, c = COEFFICIENTS
        out = torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda")
        for i in range(case["batch"]):
            X = s["x"][i].double()
            X = X / (torch.linalg.vector_norm(X) + EPS)
            wide = X if case["n"] <= case["k"] else X.t().contiguous()
            for _ in range(STEPS):
                A = wide @ wide.t().contiguous()
                P = torch.addmm(A * b, A, A, alpha=c)
                P.diagonal().add_(a)
                wide = P @ wide
            out[i] = wide if case["n"] <= case["k"] else wide.t()
        return {"out": out}
    T, K, E = case["tokens"], case["topk"], case["experts"]
    x = s["logits"].double()
    keep = torch.ones(T, dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"]
    if case["score"] == "softmax":
        log = x - torch.logsumexp(x, 1, keepdim=True)
        score = torch.exp(torch.where(torch.isnan(log), -math.inf, log))
        p = score
    else:
        score = torch.sigmoid(x)
        whole = score.sum(1, keepdim=True)
        p = torch.where(whole > 0, score / whole, 0.0)
    if case["op"] == "choose":  # one choice after the other, the lowest index of the largest
        key = x if s["bias_of"] is None else torch.where(torch.isneginf(x), -math.inf, score + s["bias_of"].double())
        key = torch.where(keep[:, None], key, -math.inf)
        every, ids = torch.arange(E, device="cuda").expand(T, E), []
        for _ in range(K):
            top = key.amax(1, keepdim=True)
            first = torch.where(key == top, every, E).amin(1, keepdim=True)
            ids.append(torch.where(torch.isneginf(top), -1, first))
            key = key.scatter(1, first, -math.inf)
        ids = torch.cat(ids, 1)
    else:
        ids = s["choice"][0].long()
    t, j = torch.nonzero(ids >= 0, as_tuple=True)
    e = ids[t, j]
    picked = torch.zeros(T, K, dtype=torch.float64, device="cuda")
    picked[t, j] = score[t, e]
    of_token = picked.sum(1)
    if case["op"] == "choose":
        w = picked * case["scale"]
        if case["normalize"]:
            w = torch.where(of_token[:, None] > 0, w / of_token[:, None], 0.0)
        sums = p[keep].sum(0)
        counts, n = torch.bincount(e, minlength=E).double(), int(keep.sum())
        loss = case["balance"] * E * torch.dot(counts / max(1, K * n), sums / max(1, n))
        return {"ids": None, "weights": w, "counts": None, "sums": sums, "counted": None, "loss": loss.reshape(1)}
    # the gradient, by one derivative after the other
    counts, n = s["choice"][2].double(), max(1, int(s["choice"][4]))
    up = torch.zeros(T, E, dtype=torch.float64, device="cuda")  # d / d score, by way of the weights
    dw = s["dweights"].double()[t, j] * case["scale"]
    if case["normalize"]:
        mean = torch.zeros(T, dtype=torch.float64, device="cuda").index_add_(0, t, dw * picked[t, j]) / of_token
        dw = (dw - mean[t]) / of_token[t]
    up[t, e] = dw
    share = case["balance"] * E * counts / (K * n * n)  # d / d p, by way of the loss
    if case["score"] == "softmax":
        d = up + share
        dx = p * d - p * (p * d).sum(1, keepdim=True)
    else:
        d = up + torch.where(whole > 0, (share - (p @ share)[:, None]) / whole, 0.0)
        dx = d * score * torch.sigmoid(-x)
    return {"dlogits": torch.where(keep[:, None], dx, 0.0)}
