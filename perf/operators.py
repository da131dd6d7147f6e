"""Cases, plain forms and exact values of the expert operators: tokens sorted
by expert (as they are, or as 8-bit blocks), the weighted way back and its
gradient, and the experts' 8-bit products, forward and for the weights'
gradient.

`run` takes the plain form in 32-bit torch arithmetic where `own` is false and
the library's calls where it is true.  Definitions shared by all:

* A slot is one (token, choice) pair; its expert id is in 0..experts-1, or
  outside (another GPU's expert) and then the slot has no row.  Rows are the
  slots in order of expert, slots of one expert in slot order; every expert's
  segment starts at a multiple of `align`.  Rows of a segment that belong to
  no slot are zeros; rows past the last segment are not written.
* 8-bit blocks: data in E4M3, one power-of-two scale per block (a byte b
  stands for 2^(b-127)), the least with |block| <= 448 * scale, at least
  2^-126, 1 for a block of zeros, over the finite values; a value that is not
  finite is stored as NaN.  A row is stored to a multiple of 128 columns
  (zeros) and its scales to a multiple of 4 (ones).
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BLOCK = 128


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one decoding step of a small batch: latency of sorting 64 slots
        dict(name="dispatch decode", op="dispatch", tokens=8, topk=8, experts=256, hidden=7168,
             dtype="bf16", store="same", align=1, share=1.0),
        # the MoE all-to-all's 65,536 rows of 7168, before they are compressed
        dict(name="dispatch train", op="dispatch", tokens=8192, topk=8, experts=256, hidden=7168,
             dtype="bf16", store="same", align=1, share=1.0),
        # rows cast to 8-bit blocks on the way, segments ready for the products of both directions;
        # half of the experts are elsewhere, sizes that no tile divides
        dict(name="dispatch 8-bit ragged", op="dispatch", tokens=8191, topk=6, experts=67, hidden=5000,
             dtype="fp16", store="fp8", align=128, share=0.5),
        # the way back of a decoding step
        dict(name="combine decode", op="combine", tokens=8, topk=8, experts=256, hidden=7168,
             dtype="bf16", weighted=True, align=1, share=1.0),
        # the way back of the training step's rows
        dict(name="combine train", op="combine", tokens=8192, topk=8, experts=256, hidden=7168,
             dtype="bf16", weighted=True, align=1, share=1.0),
        # its gradient: rows, weights, and the gradient of the dispatch that fed them
        dict(name="combine gradient train", op="combine_grad", tokens=8192, topk=8, experts=256, hidden=7168,
             dtype="bf16", align=1, share=1.0),
        # 32-bit rows of an odd width, experts elsewhere, padded segments
        dict(name="combine gradient ragged", op="combine_grad", tokens=1021, topk=3, experts=37, hidden=1001,
             dtype="fp32", align=16, share=0.5),
        # a decoding step's 64 rows on one GPU's 32 experts: the weights are read once
        dict(name="product decode", op="product", rows=64, experts=32, n=4096, k=7168, source="fp8",
             side="forward", out="bf16"),
        # the training step's rows on all experts, Zipf counts: a few long segments, many short
        dict(name="product train", op="product", rows=65536, experts=256, n=4096, k=7168, source="fp8",
             side="forward", out="bf16"),
        # a dense layer of the Llama MLP shape, both operands cast in the pass, gradient of its input
        dict(name="product dense cast", op="product", rows=4095, experts=1, n=4096, k=14336, source="bf16",
             side="input_grad", out="bf16"),
        # the weights' gradients of one GPU's 32 experts, casts included
        dict(name="weight gradient", op="weight_grad", rows=32768, experts=32, n=2048, k=7168, out="bf16"),
        # few rows an expert, some experts without any, widths that no tile divides
        dict(name="weight gradient ragged", op="weight_grad", rows=1021, experts=37, n=1000, k=1401, out="fp16"),
    ]


def draw(rng):
    def log_int(a, b):
        return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))

    op = rng.choice(["dispatch", "dispatch", "combine", "combine_grad", "product", "product", "weight_grad"])
    if op in ("dispatch", "combine", "combine_grad"):
        topk = rng.randint(1, 8)
        hidden = log_int(64, 8192)
        if rng.random() < 0.5:
            hidden = max(64, hidden // 64 * 64)
        most = 65536 * 7168 // (topk * hidden)
        c = dict(op=op, tokens=log_int(1, min(16384, most)), topk=topk, experts=log_int(max(topk, 2), 512),
                 hidden=hidden, dtype=rng.choice(["bf16", "fp16", "fp32"]),
                 align=rng.choice([1, 8, 16, 128]), share=rng.choice([1.0, 0.5, 0.25]))
        if c["dtype"] == "fp32":
            c["tokens"] = max(1, c["tokens"] // 2)
        c["experts"] = min(c["experts"], 65536 // c["align"])
        if op == "dispatch":
            c["store"] = rng.choice(["same", "fp8"])
        if op == "combine":
            c["weighted"] = rng.random() < 0.7
        return c
    while True:
        c = dict(op=op, rows=log_int(1, 65536), experts=log_int(1, 256), n=log_int(16, 14336), k=log_int(64, 14336),
                 out=rng.choice(["bf16", "bf16", "fp16"]))
        if op == "product":
            c["source"] = rng.choice(["fp8", "fp8", "bf16"])
            c["side"] = rng.choice(["forward", "input_grad"])
            weights = c["experts"] * c["n"] * c["k"] * (1 if c["source"] == "fp8" else 8)
            if weights <= 256 * 4096 * 7168 // 2 and c["rows"] * c["n"] * c["k"] <= 65536 * 4096 * 7168 // 2:
                return c
        elif (c["experts"] * c["n"] * c["k"] <= 32 * 2048 * 7168
              and c["rows"] * c["n"] * c["k"] <= 32768 * 2048 * 7168):
            return c


# ----------------------------------------------------------- shared numbers

def _up(n, m):
    return -(-n // m) * m


def _capacity(slots, experts, align):
    return _up(slots + min(experts, slots) * (align - 1), align)


def _zipf(total, experts, s=1.2):
    """`total` rows over `experts`, proportional to rank^-s: floors, then one
    more each by largest fraction (ties to the lower rank)."""
    w = [r ** -s for r in range(1, experts + 1)]
    whole = sum(w)
    share = [total * v / whole for v in w]
    count = [int(v) for v in share]
    by_fraction = sorted(range(experts), key=lambda i: (count[i] - share[i], i))
    for i in by_fraction[:total - sum(count)]:
        count[i] += 1
    return count


def work(case):
    if case["op"] in ("dispatch", "combine", "combine_grad"):
        T, K, H = case["tokens"], case["topk"], case["hidden"]
        size = 4 if case["dtype"] == "fp32" else 2
        rows = T * K * case["share"]
        # tokens that keep at least one of their slots
        tokens = T * (1 - (1 - case["share"]) ** K)
        table = 4 * T * K
        if case["op"] == "dispatch":
            moved = H * size if case["store"] == "same" else _up(H, BLOCK) + _up(-(-H // BLOCK), 4)
            return {"bytes": tokens * H * size + rows * moved + 3 * table, "flops": 0}
        if case["op"] == "combine":
            return {"bytes": rows * H * size + T * H * size + 2 * table, "flops": 2 * rows * H}
        # dy and the rows in, the rows' and weights' gradients out, then the
        # dispatch's gradient: rows' gradients in, dx out
        return {"bytes": (tokens + 2 * rows) * H * size + (rows + T) * H * size + 3 * table, "flops": 4 * rows * H}
    R, E, N, K = case["rows"], case["experts"], case["n"], case["k"]
    flops = 2.0 * R * N * K
    if case["op"] == "product":
        used = sum(c > 0 for c in _zipf(R, E))
        each = 1 if case["source"] == "fp8" else 2
        return {"bytes": R * K * each + used * N * K * each + R * N * 2, "flops": flops}
    return {"bytes": R * (K + N) * 2 + E * N * K * 2, "flops": flops}


# --------------------------------------------------------------- the inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) & 0x7FFFFFFFFFFFFFFF)
    return g


def _activations(g, rows, cols, dtype):
    """N(0, 1) times a LogNormal(0, 0.5) scale per row."""
    z = torch.randn(rows, cols, generator=g, device="cuda")
    z *= torch.exp(0.5 * torch.randn(rows, 1, generator=g, device="cuda"))
    return z.to(dtype)


def _expert_ids(g, case):
    """topk different experts per token, popularity Zipf(1.2) in an order of
    the seed; only the first `experts` of experts / share are this GPU's."""
    every = max(case["topk"], int(round(case["experts"] / case["share"])))
    p = torch.arange(1, every + 1, device="cuda", dtype=torch.float32) ** -1.2
    p = p[torch.randperm(every, generator=g, device="cuda")]
    ids = torch.multinomial(p.expand(case["tokens"], every), case["topk"], generator=g).to(torch.int32)
    return torch.where(ids < case["experts"], ids, -1).contiguous()


def _segments(g, case, align):
    """Zipf counts over the experts in an order of the seed, and offsets."""
    E = case["experts"]
    count = _zipf(case["rows"], E)
    order = torch.randperm(E, generator=g, device="cuda").tolist()
    count = [count[i] for i in order]
    offset = [0]
    for c in count:
        offset.append(offset[-1] + _up(c, align))
    return count, offset


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    s = dict(case)
    if op in ("dispatch", "combine", "combine_grad"):
        T, K, E, H = case["tokens"], case["topk"], case["experts"], case["hidden"]
        dtype = DTYPES[case["dtype"]]
        cap = _capacity(T * K, E, case["align"])
        s["ids"] = _expert_ids(g, case)
        s["cap"] = cap
        i32 = dict(dtype=torch.int32, device="cuda")
        s["routing"] = (torch.zeros(E + 1, **i32), torch.zeros(E, **i32), torch.zeros(T, K, **i32),
                        torch.zeros(cap, **i32))
        if op == "dispatch":
            s["x"] = _activations(g, T, H, dtype)
            if case["store"] == "same":
                s["rows"] = torch.zeros(cap, H, dtype=dtype, device="cuda")
            else:
                s["data"] = torch.zeros(cap, _up(H, BLOCK), dtype=torch.float8_e4m3fn, device="cuda")
                s["scale"] = torch.zeros(cap, _up(-(-H // BLOCK), 4), dtype=torch.uint8,
                                         device="cuda").view(torch.float8_e8m0fnu)
            return s
        s["routing"] = _route(s["ids"], E, case["align"], cap)
        offsets, _, row, slot = s["routing"]
        rows = _activations(g, cap, H, dtype)
        s["rows"] = torch.where((slot >= 0)[:, None], rows, torch.zeros((), dtype=dtype, device="cuda"))
        w = torch.rand(T, K, generator=g, device="cuda") + 0.05
        s["weights"] = w / w.sum(1, keepdim=True)
        s["y"] = torch.zeros(T, H, dtype=dtype, device="cuda")
        if op == "combine_grad":
            s["dy"] = _activations(g, T, H, dtype)
            s["drows"] = torch.zeros(cap, H, dtype=dtype, device="cuda")
            s["dweights"] = torch.zeros(T, K, device="cuda")
        return s
    R, E, N, K = case["rows"], case["experts"], case["n"], case["k"]
    s["count"], s["offset"] = _segments(g, case, 128 if op == "weight_grad" else 1)
    s["counts"] = torch.tensor(s["count"], dtype=torch.int32, device="cuda")
    s["offsets"] = torch.tensor(s["offset"], dtype=torch.int32, device="cuda")
    cap = s["offset"][-1]
    if op == "weight_grad":
        # rows between a segment's count and its end are zeros, as the dispatch leaves them
        r = torch.arange(cap, device="cuda")
        e = torch.searchsorted(s["offsets"][1:].long(), r, right=True)
        live = (r - s["offsets"].long()[e] < s["counts"].long()[e])[:, None]
        s["x"] = _activations(g, cap, K, torch.bfloat16) * live
        s["dy"] = _activations(g, cap, N, torch.bfloat16) * live
        s["dw"] = torch.zeros(E, N, K, dtype=DTYPES[case["out"]], device="cuda")
        return s
    s["out_rows"] = torch.zeros(R, N, dtype=DTYPES[case["out"]], device="cuda")
    x = _activations(g, R, K, torch.bfloat16)
    if case["source"] == "bf16":
        s["x"] = x
        shape = (E, N, K) if case["side"] == "forward" else (E, K, N)
        s["w"] = (torch.randn(*shape, generator=g, device="cuda") * 0.02).to(torch.bfloat16)
        return s
    s["a"] = _blocks_of_rows(x)
    data = torch.empty(E, N, _up(K, BLOCK), dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty(E, -(-N // BLOCK), _up(-(-K // BLOCK), 4), dtype=torch.uint8,
                        device="cuda").view(torch.float8_e8m0fnu)
    step = max(1, (1 << 28) // (N * K))
    for e in range(0, E, step):
        w = torch.randn(min(step, E - e), N, K, generator=g, device="cuda") * 0.02
        d, c = _blocks_of_weights(w)
        data[e:e + step] = d
        scale.view(torch.uint8)[e:e + step] = c.view(torch.uint8)
    s["wq"] = (data, scale)
    return s


# ---------------------------------------------------------- the plain forms

def _route(ids, experts, align, cap):
    """(offsets, counts, row of each slot or -1, slot of each row or -1)."""
    T, K = ids.shape
    flat = ids.reshape(-1).long()
    has = (flat >= 0) & (flat < experts)
    key = torch.where(has, flat, experts)
    order = torch.argsort(key, stable=True)
    count = torch.zeros(experts + 1, dtype=torch.int64, device=ids.device)
    count.scatter_add_(0, key, torch.ones_like(key))
    padded = (count[:experts] + align - 1) // align * align
    zero = torch.zeros(1, dtype=torch.int64, device=ids.device)
    offsets = torch.cat([zero, torch.cumsum(padded, 0)])
    first = torch.cumsum(count, 0) - count
    key = key[order]
    place = torch.arange(T * K, device=ids.device) - first[key] + offsets[key]
    place = torch.where(key < experts, place, cap)
    slot = torch.full((cap + 1,), -1, dtype=torch.int64, device=ids.device)
    slot[place] = order
    row = torch.empty_like(place)
    row[order] = torch.where(key < experts, place, -1)
    i32 = torch.int32
    return (offsets.to(i32), count[:experts].to(i32), row.reshape(T, K).to(i32), slot[:cap].to(i32))


def _scale_exponent(amax):
    """Least e with amax <= 448 * 2^e (448 = 1.75 * 2^8), at least -126; 0 for 0."""
    m, p = torch.frexp(amax)  # amax = m * 2^p, m in [0.5, 1)
    e = torch.where(m > 0.875, p - 8, p - 9)
    return torch.where(amax == 0, torch.zeros_like(e), e.clamp(min=-126))


def _cast(x, e):
    """E4M3 of x / 2^e, both in 32 bits (exact up to the cast)."""
    y = x * ((127 - e) << 23).view(torch.float32)
    return torch.where(torch.isfinite(x), y, torch.nan).to(torch.float8_e4m3fn)


def _finite(x):
    return torch.where(torch.isfinite(x), x, 0.0).abs()


def _pad(x, rows, cols):
    return torch.nn.functional.pad(x, (0, cols - x.shape[-1], 0, rows - x.shape[-2]))


def _bytes(e, cols4):
    b = torch.nn.functional.pad((e + 127).to(torch.uint8), (0, cols4 - e.shape[-1]), value=127)
    return b.view(torch.float8_e8m0fnu)


def _blocks_of_rows(x):
    """Blocks of 1 x 128."""
    x = _pad(x.float(), x.shape[-2], _up(x.shape[-1], BLOCK))
    b = x.unflatten(-1, (-1, BLOCK))
    e = _scale_exponent(_finite(b).amax(-1))
    return _cast(b, e[..., None]).flatten(-2), _bytes(e, _up(e.shape[-1], 4))


def _blocks_of_weights(w):
    """Blocks of 128 x 128 of [experts, n, k]; the rows past n are not kept."""
    E, N, K = w.shape
    x = _pad(w.float(), _up(N, BLOCK), _up(K, BLOCK))
    b = x.unflatten(-1, (-1, BLOCK)).unflatten(1, (-1, BLOCK))
    e = _scale_exponent(_finite(b).amax(-1).amax(2))
    q = _cast(b, e[:, :, None, :, None]).flatten(-2).flatten(1, 2)
    return q[:, :N].contiguous(), _bytes(e, _up(e.shape[-1], 4))


def _values(data, scale, row_block=1):
    """What 8-bit blocks stand for, in 32 bits."""
    s = scale.float()[..., :data.shape[-1] // BLOCK]
    if row_block > 1:
        s = s.repeat_interleave(row_block, -2)[..., :data.shape[-2], :]
    return (data.float().unflatten(-1, (-1, BLOCK)) * s[..., None]).flatten(-2)


def _plain(s):
    op = s["op"]
    if op == "dispatch":
        offsets, counts, row, slot = _route(s["ids"], s["experts"], s["align"], s["cap"])
        live = slot >= 0
        token = torch.where(live, slot, 0).long() // s["topk"]
        got = {"offsets": offsets, "counts": counts, "row": row, "slot": slot}
        if s["store"] == "same":
            zero = torch.zeros((), dtype=s["x"].dtype, device="cuda")
            return dict(got, rows=torch.where(live[:, None], s["x"][token], zero))
        data, scale = _blocks_of_rows(s["x"])
        data = torch.where(live[:, None], data.view(torch.uint8)[token], 0).view(torch.float8_e4m3fn)
        inside = torch.arange(s["cap"], device="cuda") < offsets[-1]
        rest = torch.where(inside, 127, 0).to(torch.uint8)
        scale = torch.where(live[:, None], scale.view(torch.uint8)[token], rest[:, None])
        return dict(got, data=data, scale=scale.view(torch.float8_e8m0fnu).float())
    if op in ("combine", "combine_grad"):
        row = s["routing"][2].long()
        has = (row >= 0)[..., None]
        at = row.clamp(min=0)
        if op == "combine":
            part = torch.where(has, s["rows"][at].float(), 0.0)
            if s["weighted"]:
                part = torch.where(has, part * s["weights"][..., None], 0.0)
            return {"y": part.sum(1).to(s["rows"].dtype)}
        dy = s["dy"].float()[:, None]
        part = torch.where(has, s["weights"][..., None] * dy, 0.0).to(s["rows"].dtype)
        dw = torch.where(has, s["rows"][at].float() * dy, 0.0).sum(-1)
        drows = torch.zeros(s["cap"] + 1, s["hidden"], dtype=s["rows"].dtype, device="cuda")
        drows[torch.where(row >= 0, row, s["cap"])] = part
        dx = torch.where(has, part.float(), 0.0).sum(1).to(s["rows"].dtype)
        return {"drows": drows[:s["cap"]], "dweights": dw, "dx": dx}
    if op == "weight_grad":
        # blocks of 128 rows x 1 column
        xq, xe = _blocks_of_rows(s["x"].t())
        yq, ye = _blocks_of_rows(s["dy"].t())
        x, y = _values(xq, xe), _values(yq, ye)
        dw = torch.empty_like(s["dw"])
        for e in range(s["experts"]):  # each expert's segment is a product of its own
            a, b = s["offset"][e], s["offset"][e + 1]
            dw[e] = y[:, a:b] @ x[:, a:b].t()
        return {"dw": dw}
    if s["source"] == "bf16":
        a = _blocks_of_rows(s["x"])
        w = _blocks_of_weights(s["w"] if s["side"] == "forward" else s["w"].transpose(1, 2))
    else:
        a, w = s["a"], s["wq"]
    out = torch.empty_like(s["out_rows"])
    for e in range(s["experts"]):  # each expert's segment is a product of its own
        lo, hi = s["offset"][e], s["offset"][e] + s["count"][e]
        if hi > lo:
            out[lo:hi] = _values(a[0][lo:hi], a[1][lo:hi]) @ _values(w[0][e], w[1][e], BLOCK).t()
    return {"out": out}


# ------------------------------------------------------- the library's calls

def _own(s):
    import lossless_bf16_exponent_zc_amd as zc
    op = s["op"]
    if op in ("dispatch", "combine", "combine_grad"):
        if "plan" not in s:
            s["plan"] = zc.ExpertPlan(s["tokens"], s["topk"], s["experts"], s["align"])
            s["ws"] = s["plan"].empty_workspace()
            s["r"] = zc.Routing(*s["routing"])
            if op == "dispatch" and s["store"] == "fp8":
                s["f"] = zc.Fp8Blocks(s["data"], s["scale"], s["hidden"])
        plan, r = s["plan"], s["r"]
        if op == "dispatch":
            plan.route(s["ids"], r, s["ws"])
            got = {"offsets": r.offsets, "counts": r.counts, "row": r.row, "slot": r.slot}
            if s["store"] == "same":
                plan.dispatch(s["x"], r, s["rows"])
                return dict(got, rows=s["rows"])
            plan.dispatch_fp8(s["x"], r, s["f"])
            return dict(got, data=s["data"], scale=s["scale"].float())
        if op == "combine":
            plan.combine(s["rows"], s["weights"] if s["weighted"] else None, r, s["y"])
            return {"y": s["y"]}
        plan.combine_backward(s["dy"], s["rows"], s["weights"], r, s["drows"], s["dweights"])
        plan.combine(s["drows"], None, r, s["y"])
        return {"drows": s["drows"], "dweights": s["dweights"], "dx": s["y"]}
    if op == "weight_grad":
        if "xt" not in s:
            s["xt"] = zc.empty_fp8_columns(s["offset"][-1], s["k"])
            s["yt"] = zc.empty_fp8_columns(s["offset"][-1], s["n"])
        zc.quantize_columns(s["x"], s["xt"])
        zc.quantize_columns(s["dy"], s["yt"])
        zc.expert_weight_grad(s["yt"], s["xt"], s["dw"], s["offsets"])
        return {"dw": s["dw"]}
    if "fa" not in s:
        if s["source"] == "bf16":
            s["fa"] = zc.empty_fp8_rows(s["rows"], s["k"])
            s["fw"] = zc.empty_fp8_weights(s["experts"], s["n"], s["k"])
        else:
            s["fa"] = zc.Fp8Blocks(*s["a"], s["k"])
            s["fw"] = zc.Fp8Blocks(*s["wq"], s["k"])
    if s["source"] == "bf16":
        zc.quantize_rows(s["x"], s["fa"])
        zc.quantize_weights(s["w"], s["fw"], transpose=s["side"] != "forward")
    zc.expert_product(s["fa"], s["fw"], s["out_rows"], s["offsets"], s["counts"])
    return {"out": s["out_rows"]}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------- the definition in 64 bits

def _exact_blocks(x, dim):
    """(values, scales) of blocks of 128 along `dim` of a 2-D tensor, in 64
    bits, from the definition."""
    x = x.double()
    if dim == 0:
        v, s = _exact_blocks(x.t(), 1)
        return v.t(), s.t()
    pad = -x.shape[1] % BLOCK
    b = torch.cat([x, x.new_zeros(x.shape[0], pad)], 1).reshape(x.shape[0], -1, BLOCK)
    finite = torch.isfinite(b)
    top = torch.where(finite, b, 0.0).abs().amax(2, keepdim=True)
    return _exact_round(b, finite, top, x.shape[1] + pad)


def _two_to(e):
    """2^e in 64 bits, whole e (pow may be off by a unit in the last place)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_round(b, finite, top, cols):
    e = torch.ceil(torch.log2(torch.where(top > 0, top, 448.0) / 448.0))
    e = torch.where(top > 448.0 * _two_to(e), e + 1, e)        # log2's rounding, either way
    e = torch.where(top <= 448.0 * _two_to(e - 1), e - 1, e)
    e = torch.where(top > 0, torch.clamp(e, min=-126.0), 0.0)
    scale = _two_to(e)
    v = b / scale
    binade = torch.floor(torch.log2(torch.clamp(v.abs(), min=2.0 ** -6)))
    binade = torch.where(v.abs() >= 2 * _two_to(binade), binade + 1, binade)
    step = _two_to(torch.clamp(binade, min=-6.0) - 3)
    v = torch.where(finite, torch.round(v / step) * step, torch.nan)
    return v.reshape(v.shape[0], cols), scale.reshape(scale.shape[0], -1)


def _exact_weights(w):
    """What the 128 x 128 blocks of one [n, k] matrix stand for."""
    n, k = w.shape
    x = w.new_zeros(_up(n, BLOCK), _up(k, BLOCK), dtype=torch.float64)
    x[:n, :k] = w
    nb, kb = x.shape[0] // BLOCK, x.shape[1] // BLOCK
    b = x.reshape(nb, BLOCK, kb, BLOCK).permute(0, 2, 1, 3).reshape(nb * kb, BLOCK * BLOCK)
    finite = torch.isfinite(b)
    v, s = _exact_round(b, finite, torch.where(finite, b, 0.0).abs().amax(1, keepdim=True), BLOCK * BLOCK)
    return (v * s).reshape(nb, kb, BLOCK, BLOCK).permute(0, 2, 1, 3).reshape(x.shape)[:n]


def _scaled(values, scale):
    return values * scale.repeat_interleave(BLOCK, 1)[:, :values.shape[1]]


def _exact_of_bytes(data, scale):
    s = _two_to(scale.view(torch.uint8).double() - 127)
    return _scaled(data.double(), s)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "dispatch":
        got = {"offsets": None, "counts": None, "row": None, "slot": None}
        routing = _route(s["ids"], s["experts"], s["align"], s["cap"])
        live, end = routing[3] >= 0, int(routing[0][-1])
        token = routing[3][live].long() // s["topk"]
        if case["store"] == "same":
            rows = torch.zeros(s["cap"], s["hidden"], dtype=torch.float64, device="cuda")
            rows[live] = s["x"][token].double()
            return dict(got, rows=rows)
        v, e = _exact_blocks(s["x"], 1)
        data = torch.zeros(s["cap"], v.shape[1], dtype=torch.float64, device="cuda")
        data[live] = v[token]
        scale = torch.full((s["cap"], _up(e.shape[1], 4)), 2.0 ** -127, dtype=torch.float64, device="cuda")
        scale[:end] = 1.0
        scale[live, :e.shape[1]] = e[token]
        scale[live, e.shape[1]:] = 1.0
        return dict(got, data=data, scale=scale)
    if op in ("combine", "combine_grad"):
        row, w = s["routing"][2].long(), s["weights"].double()
        if op == "combine":
            y = torch.zeros(case["tokens"], case["hidden"], dtype=torch.float64, device="cuda")
            for k in range(case["topk"]):
                t = torch.nonzero(row[:, k] >= 0)[:, 0]
                part = s["rows"][row[t, k]].double()
                y[t] += part * w[t, k][:, None] if case["weighted"] else part
            return {"y": y}
        dy = s["dy"].double()
        drows = torch.zeros(s["cap"], case["hidden"], dtype=torch.float64, device="cuda")
        dw, dx = torch.zeros_like(w), torch.zeros_like(dy)
        for k in range(case["topk"]):
            t = torch.nonzero(row[:, k] >= 0)[:, 0]
            part = dy[t] * w[t, k][:, None]
            drows[row[t, k]] = part
            dw[t, k] = (dy[t] * s["rows"][row[t, k]].double()).sum(1)
            dx[t] += part.to(s["rows"].dtype).double()  # the rows' gradient is stored in its type
        return {"drows": drows, "dweights": dw, "dx": dx}
    if op == "weight_grad":
        x, y = _scaled_rows(s["x"]), _scaled_rows(s["dy"])
        dw = torch.zeros(case["experts"], case["n"], case["k"], dtype=torch.float64, device="cuda")
        for e in range(case["experts"]):
            a, b = s["offset"][e], s["offset"][e + 1]
            dw[e] = y[a:b].t() @ x[a:b]
        return {"dw": dw}
    out = torch.zeros(case["rows"], case["n"], dtype=torch.float64, device="cuda")
    for e in range(case["experts"]):
        lo, n = s["offset"][e], s["count"][e]
        if not n:
            continue
        if case["source"] == "bf16":
            a = _scaled(*_exact_blocks(s["x"][lo:lo + n], 1))
            w = _exact_weights(s["w"][e] if case["side"] == "forward" else s["w"][e].t())
        else:
            a = _exact_of_bytes(s["a"][0][lo:lo + n], s["a"][1][lo:lo + n])
            data, scale = s["wq"][0][e], s["wq"][1][e]
            w = _exact_of_bytes(data, scale.view(torch.uint8).repeat_interleave(BLOCK, 0)[:case["n"]])
        out[lo:lo + n] = a @ w.t()
    return {"out": out}


def _scaled_rows(x):
    """What blocks of 128 rows x 1 column of x stand for."""
    v, s = _exact_blocks(x, 0)
    return (v * s.repeat_interleave(BLOCK, 0))[:x.shape[0]]
