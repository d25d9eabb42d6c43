"""What is measured of the linear layers whose rows choose their own weights: the cases, their
inputs, their plain form, their definition in 64 bits and their work.

A token of a mixture of experts meets the weights of a few of many experts, a request with an
adapter those of its own adapter.  The rows of a batch are put in the order of the weights they
meet (a plan), and the products run over the runs of that order, which are ragged.

route    moe_route: the top_k largest of a token's logits, their softmax weights, and the plan of
         the pairs (token, chosen expert): the pairs in order of their experts, where each pair
         lies in that order, and where each expert's run begins.
w4a16    moe_gemm_w4a16: the pairs' products with their experts' INT4 group-128 weights, bf16
         activations (decoding).
w4a4     moe_gemm_w4a4: the same with NVFP4 weights and activations (prompts).
combine  moe_combine: each token's weighted sum over its experts' rows.
lora     lora_add: y + scale * B (A x) with the rows' own low-rank adapters, beside a projection
         that all rows share.

A product's side is "up" (rows taken from the tokens; the weights' first half of rows is a gate:
silu(gate) * up is returned) or "down" (rows in the plan's order, the product itself).  A pair
without an expert (an expert of -1: padding, or a token whose logits are all masked) comes last in
the plan, and its row of a product is zero.
"""

import math
import random

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------

def listed():
    return [
        # one decode step of a batch: the smallest plan, where launches count
        dict(name="route step", op="route", tokens=32, experts=128, top_k=8, x="f32", masked=False,
             renorm=True),
        # a long prompt over many experts
        dict(name="route prompt", op="route", tokens=16384, experts=256, top_k=8, x="f32",
             masked=False, renorm=True),
        # a single sequence's decode step: eight experts' weights read once
        dict(name="experts one", op="w4a16", side="up", tokens=1, experts=64, top_k=8, hidden=4096,
             inter=1024, idle=0.0, out="bf16"),
        # a decode batch: nearly every expert is met, by a few rows each
        dict(name="experts batch", op="w4a16", side="down", tokens=48, experts=128, top_k=8,
             hidden=2048, inter=768, idle=0.0, out="bf16"),
        # a large batch with an odd number of tokens, a tenth of them padding
        dict(name="experts many", op="w4a16", side="up", tokens=509, experts=60, top_k=4,
             hidden=2048, inter=1408, idle=0.1, out="bf16"),
        # a short prompt: uneven runs of some tens of rows
        dict(name="prompt short", op="w4a4", side="up", tokens=1000, experts=60, top_k=4,
             hidden=2048, inter=1408, idle=0.1, out="bf16"),
        # a prompt over few, wide experts
        dict(name="prompt wide", op="w4a4", side="down", tokens=4095, experts=8, top_k=2,
             hidden=4096, inter=2048, idle=0.0, out="bf16"),
        # a long prompt's prefill step, the largest product
        dict(name="prompt long", op="w4a4", side="up", tokens=8192, experts=64, top_k=8, hidden=4096,
             inter=1024, idle=0.0, out="bf16"),
        # the decode batch's way back to its tokens
        dict(name="combine step", op="combine", tokens=48, experts=128, top_k=8, hidden=2048,
             idle=0.0, out="bf16"),
        # the long prompt's
        dict(name="combine prompt", op="combine", tokens=8192, experts=64, top_k=8, hidden=4096,
             idle=0.0, out="bf16"),
        # a decode batch of requests over half as many adapters, beside a qkv projection
        dict(name="lora step", op="lora", tokens=64, adapters=32, rank=16, n=6144, k=4096, runs=False,
             idle=0.2, out="bf16"),
        # prompts of several requests, one adapter each
        dict(name="lora prompt", op="lora", tokens=8190, adapters=8, rank=64, n=7168, k=5120,
             runs=True, idle=0.1, out="bf16"),
    ]


# hidden, inter, experts, top_k
MIXTURES = ((4096, 1024, 64, 8), (2048, 768, 128, 8), (5120, 1280, 32, 4), (2048, 1408, 60, 4),
            (3840, 1920, 16, 2), (4096, 2048, 8, 2))
# n, k of a projection
PROJECTIONS = ((6144, 4096), (4096, 4096), (7168, 5120), (5120, 5120), (3840, 3840), (4096, 12288),
               (256, 512))
MOST_PRODUCT = 8192 * 8 * 2 * 1024 * 4096    # pairs * n * k that a drawn prompt has, at most
MOST_LORA = 8190 * (2 * 7168 + 5120)         # values that a drawn adapter call moves, at most


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("route", "w4a16", "w4a16", "w4a4", "w4a4", "combine", "lora", "lora"))
    if op == "route":
        experts = _spread(rng, 4, 256)
        return dict(op=op, tokens=_spread(rng, 1, 16384), experts=experts,
                    top_k=rng.randint(1, min(8, experts)), x=rng.choice(("f32", "f32", "bf16")),
                    masked=rng.random() < 0.3, renorm=rng.random() < 0.6)
    if op == "lora":
        n, k = rng.choice(PROJECTIONS)
        return dict(op=op, tokens=_spread(rng, 1, min(8190, MOST_LORA // (2 * n + k))),
                    adapters=_spread(rng, 1, 64), rank=rng.choice((8, 16, 32, 64, 128)), n=n, k=k,
                    runs=rng.random() < 0.5, idle=rng.choice((0.0, 0.2)),
                    out=rng.choice(("bf16", "bf16", "f32")))
    hidden, inter, experts, top_k = rng.choice(MIXTURES)
    case = dict(op=op, experts=experts, top_k=top_k, hidden=hidden, idle=rng.choice((0.0, 0.1)),
                out=rng.choice(("bf16", "bf16", "f32")))
    if op == "combine":
        case["tokens"] = _spread(rng, 1, 8192 * 8 * 4096 // (top_k * hidden))
        case["tokens"] = min(case["tokens"], 16384)
        return case
    case["inter"], case["side"] = inter, rng.choice(("up", "down"))
    n, k = _product(case)
    case["tokens"] = (_spread(rng, 1, 512) if op == "w4a16" else
                      _spread(rng, 20, min(8192, MOST_PRODUCT // (top_k * n * k))))
    return case


def _product(case):
    """Rows and columns of an expert's weights."""
    if case["side"] == "up":
        return 2 * case["inter"], case["hidden"]
    return case["hidden"], case["inter"]


# ------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------

_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _choices(case):
    """The experts [tokens, top_k] that the tokens of a case choose, as a trained router chooses
    them: unevenly, no expert twice for one token, and for padded tokens none.  They go by the
    case alone, so that its work is known; a seed shuffles tokens and experts."""
    rng = torch.Generator().manual_seed(case["tokens"] * 1009 + case["experts"])
    score = 0.7 * torch.randn((1, case["experts"]), generator=rng)
    noise = torch.rand((case["tokens"], case["experts"]), generator=rng).clamp(min=1e-9)
    ids = (score - torch.log(-torch.log(noise))).topk(case["top_k"], 1).indices
    ids[torch.rand((case["tokens"],), generator=rng) < case["idle"]] = -1
    return ids


def _adapters(case):
    """The adapters [tokens] of a case's tokens, -1 for none; by the case alone as `_choices`."""
    rng = random.Random(case["tokens"] * 1013 + case["adapters"])
    n, t = case["adapters"], case["tokens"]
    if case["runs"]:      # a few requests' prompts one after another
        cuts = sorted(rng.randrange(t + 1) for _ in range(min(2 * n, t) - 1))
        ids = []
        for a, b in zip([0] + cuts, cuts + [t]):
            ids += [-1 if rng.random() < case["idle"] else rng.randrange(n)] * (b - a)
    else:
        ids = [-1 if rng.random() < case["idle"] else rng.randrange(n) for _ in range(t)]
    return torch.tensor(ids)


def _shuffled(ids, groups, g, tokens=True):
    """The same choices with tokens and groups in another order."""
    names = torch.randperm(groups, generator=g, device=DEV)
    ids = ids.to(DEV)
    if tokens:
        ids = ids[torch.randperm(ids.shape[0], generator=g, device=DEV)]
    return torch.where(ids >= 0, names[ids.clamp(min=0)], ids).int().contiguous()


def _order(ids, groups):
    """(order, where, offsets) of whole numbers ids, those of no group last."""
    flat = ids.flatten().long()
    key = torch.where((flat >= 0) & (flat < groups), flat, torch.full_like(flat, groups))
    order = torch.sort(key, stable=True).indices
    where = torch.empty_like(order)
    where[order] = torch.arange(order.numel(), device=order.device)
    counts = (key[:, None] == torch.arange(groups, device=key.device)).sum(0)
    offsets = torch.cat((torch.zeros_like(counts[:1]), counts.cumsum(0)))
    return order.int(), where.int().view(ids.shape), offsets.int()


def _activations(g, rows, cols):
    """bf16 activations with a few loud channels and rows of uneven size."""
    x = torch.randn((rows, cols), generator=g, device=DEV)
    x *= torch.where(torch.rand((cols,), generator=g, device=DEV) < 0.01, 10.0, 1.0)
    x *= torch.exp(0.3 * torch.randn((rows, 1), generator=g, device=DEV))
    return x.to(torch.bfloat16)


def _int4(w):
    """Symmetric INT4 with groups of 128: codes (q + 8, two to a byte) and bf16 scales."""
    v = w.unflatten(1, (-1, 128))
    s = (v.abs().amax(-1) / 7).to(torch.bfloat16)
    u = ((v / s.float()[..., None]).round().clamp(-7, 7) + 8).flatten(1).to(torch.uint8)
    return u[:, 0::2] | (u[:, 1::2] << 4), s


def _nvfp4(x):
    """NVFP4: codes, E4M3 scales of groups of 16 and the tensor scale."""
    x = x.float()
    ts = x.abs().amax() / 2688
    v = x.unflatten(1, (-1, 16))
    s = (v.abs().amax(-1) / (6 * ts)).clamp(max=448.0).to(torch.float8_e4m3fn)
    p = s.float()[..., None] * ts
    z = torch.where(p > 0, v / p, torch.zeros_like(v)).flatten(1)
    mids = torch.tensor((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0), device=DEV)
    c = torch.bucketize(z.abs(), mids).to(torch.uint8) | (torch.signbit(z).to(torch.uint8) << 3)
    return c[:, 0::2] | (c[:, 1::2] << 4), s.view(torch.uint8), ts.view(1)


def _stack(case, g, fmt):
    """Every expert's weights, quantized: what a program keeps of them."""
    n, k = _product(case)
    parts = []
    for _ in range(case["experts"]):
        w = torch.randn((n, k), generator=g, device=DEV) * k ** -0.5
        parts.append(_int4(w) if fmt == "w4a16" else _nvfp4(w))
    if not own:
        return [torch.stack(p) for p in zip(*parts)]
    from decode_nvfp4_rtn_amd import qlin

    f = qlin.QL_INT4_G128 if fmt == "w4a16" else qlin.QL_NVFP4
    stack = torch.empty((case["experts"], qlin.repack_weights_bytes(f, n, k)), dtype=torch.uint8, device=DEV)
    for blob, p in zip(stack, parts):
        qlin.repack_weights(f, n, k, *(t.contiguous() for t in p), packed=blob)
    return stack


def _plan(state, ids, groups):
    """The plan that a program has of its rows."""
    if own:
        from decode_nvfp4_rtn_amd import qlin
        state["plan"] = qlin.group_rows(ids, groups)
    else:
        state["order"], state["where"], state["offsets"] = _order(ids, groups)


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    op, tokens = case["op"], case["tokens"]
    state = dict(case=case)
    if op == "route":
        x = torch.randn((tokens, case["experts"]), generator=g, device=DEV)
        x += 0.7 * torch.randn((case["experts"],), generator=g, device=DEV)
        if case["masked"]:    # experts that a token may not choose, and tokens that may choose none
            x[torch.rand(x.shape, generator=g, device=DEV) < 0.2] = -math.inf
            x[torch.rand((tokens,), generator=g, device=DEV) < 0.1] = -math.inf
        state["logits"] = x.to(_dtype(case["x"]))
        return state
    if op == "lora":
        n, k, r = case["n"], case["k"], case["rank"]
        ids = _shuffled(_adapters(case), case["adapters"], g, tokens=not case["runs"])
        state["x"] = _activations(g, tokens, k)
        state["y"] = torch.randn((tokens, n), generator=g, device=DEV).to(_dtype(case["out"]))
        state["a"] = (torch.randn((case["adapters"], r, k), generator=g, device=DEV) * k ** -0.5).to(torch.bfloat16)
        state["b"] = (torch.randn((case["adapters"], n, r), generator=g, device=DEV) * r ** -0.5).to(torch.bfloat16)
        state["scale"] = 2 * torch.rand((case["adapters"],), generator=g, device=DEV)
        state["out"] = torch.empty_like(state["y"])
        _plan(state, ids, case["adapters"])
        return state
    ids = _shuffled(_choices(case), case["experts"], g)
    _plan(state, ids, case["experts"])
    pairs = ids.numel()
    if op == "combine":
        state["rows"] = torch.randn((pairs, case["hidden"]), generator=g, device=DEV).to(torch.bfloat16)
        w = torch.rand(ids.shape, generator=g, device=DEV)
        state["weights"] = torch.where(ids >= 0, w / w.sum(1, keepdim=True), torch.zeros_like(w))
        return state
    k = _product(case)[1]
    x = _activations(g, tokens if case["side"] == "up" else pairs, k)
    state["x"] = x if op == "w4a16" else _nvfp4(x)
    state["experts"] = _stack(case, g, op)
    return state


# ------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(state):
    from decode_nvfp4_rtn_amd import qlin

    case = state["case"]
    op = case["op"]
    if op == "route":
        ids, weights, plan = qlin.moe_route(state["logits"], case["top_k"], renormalize=case["renorm"])
        return ids, weights, plan.order, plan.where, plan.offsets
    if op == "lora":
        # binary32 rows are added to in place, as the plain form adds to what no cast copies
        out = state["out"] if case["out"] == "bf16" else state["y"]
        return qlin.lora_add(state["y"], state["x"], state["a"], state["b"], state["plan"],
                             scale=state["scale"], out=out)
    if op == "combine":
        return qlin.moe_combine(state["rows"], state["plan"], state["weights"],
                                out_dtype=_dtype(case["out"]))
    n, k = _product(case)
    up = case["side"] == "up"
    if op == "w4a16":
        return qlin.moe_gemm_w4a16(state["x"], state["experts"], state["plan"], n, k, gather=up,
                                   silu_mul=up, out_dtype=_dtype(case["out"]))
    return qlin.moe_gemm_w4a4(*state["x"], state["experts"], state["plan"], n, k, gather=up,
                              silu_mul=up, out_dtype=_dtype(case["out"]))


def _run_plain(state):
    case = state["case"]
    op, out = case["op"], _dtype(case.get("out"))
    if op == "route":
        x = state["logits"].float()
        ids = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :case["top_k"]]
        chosen = torch.gather(x, 1, ids)
        top = x.amax(1, keepdim=True)
        top = torch.where(top == -math.inf, torch.zeros_like(top), top)
        w = torch.exp(chosen - top)
        total = w.sum(1, keepdim=True) if case["renorm"] else torch.exp(x - top).sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, torch.zeros_like(w))
        ids = torch.where(chosen == -math.inf, torch.full_like(ids, -1), ids)
        return (ids.int(), w, *_order(ids, case["experts"]))
    if op == "combine":
        rows = state["rows"].float()[state["where"].long()]
        return (rows * state["weights"][..., None]).sum(1).to(out)
    offsets = state["offsets"].tolist()
    order = state["order"].long()
    if op == "lora":
        y, x = state["y"].float(), state["x"]
        for i, (a, b) in enumerate(zip(offsets, offsets[1:])):
            if b > a:
                u = torch.matmul(x[order[a:b]].float(), state["a"][i].float().t())
                y[order[a:b]] += torch.matmul(u, state["b"][i].float().t()) * state["scale"][i]
        return y.to(out)
    n, k = _product(case)
    up = case["side"] == "up"
    result = torch.zeros((order.numel(), n // 2 if up else n), dtype=out, device=DEV)
    if op == "w4a4":
        grid = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=DEV)

        def values(codes, scales, ts):
            c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
            s = scales.view(torch.float8_e4m3fn).float()
            return (grid[c.int()].unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2) * ts
    else:
        def values(codes, scales):
            c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float() - 8
            return (c.unflatten(-1, (-1, 128)) * scales.float()[..., None]).flatten(-2)
    x = values(*state["x"]) if op == "w4a4" else state["x"].float()
    for e, (a, b) in enumerate(zip(offsets, offsets[1:])):
        if b > a:
            rows = x[order[a:b] // case["top_k"]] if up else x[a:b]
            y = torch.matmul(rows, values(*(t[e] for t in state["experts"])).t())
            if up:
                gate, y = y[:, :n // 2], y[:, n // 2:]
                y = gate / (1 + torch.exp(-gate)) * y
            result[a:b] = y.to(out)
    return result


# ------------------------------------------------------------------------------------------
# the definition in 64 bits
# ------------------------------------------------------------------------------------------

def _e4m3_64(b):
    """The value of E4M3 bytes, from the format's definition."""
    b = b.int()
    sign, e, m = 1.0 - 2.0 * (b >> 7).double(), (b >> 3) & 15, (b & 7).double()
    return sign * torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2((e - 10).double()))


def _e2m1_64(codes):
    c = torch.stack((codes % 16, codes // 16), -1).flatten(-2).int()
    e, m = (c >> 1) & 3, (c & 1).double()
    v = torch.where(e == 0, m * 0.5, (1 + m * 0.5) * torch.exp2((e - 1).double()))
    return torch.where(c >= 8, -v, v)


def _weights_64(op, parts):
    if op == "w4a4":
        codes, scales, ts = parts
        return (_e2m1_64(codes) * _e4m3_64(scales).repeat_interleave(16, -1)) * ts.double()
    codes, scales = parts
    q = torch.stack((codes % 16, codes // 16), -1).flatten(-2).double() - 8
    return q * scales.double().repeat_interleave(128, -1)


def exact(case, seed):
    global own
    op = case["op"]
    if op in ("w4a4", "w4a16"):
        n, k = _product(case)
        if case["tokens"] * case["top_k"] * n * k > 2 ** 38:
            return None
    was, own = own, False
    try:
        state = prepare(case, seed)
    finally:
        own = was
    if op == "route":
        x = state["logits"].double()
        e = torch.exp(x - x.amax(1, keepdim=True).clamp(min=-1e300))
        ids = torch.argsort(x, dim=1, descending=True, stable=True)[:, :case["top_k"]]
        w = e.gather(1, ids)
        w = w / (w if case["renorm"] else e).sum(1, keepdim=True)
        w[x.gather(1, ids) == -math.inf] = 0
        ids[x.gather(1, ids) == -math.inf] = -1
        flat = ids.flatten().tolist()
        runs = [[] for _ in range(case["experts"] + 1)]
        for p, i in enumerate(flat):
            runs[i].append(p)              # those of -1 into the last run
        order = torch.tensor(sum(runs, []), device=DEV)
        offsets, at = [0], 0
        for r in runs[:-1]:
            at += len(r)
            offsets.append(at)
        return ids, w, order, order.argsort().view(ids.shape), torch.tensor(offsets, device=DEV)
    if op == "combine":
        out = torch.zeros((case["tokens"], case["hidden"]), dtype=torch.float64, device=DEV)
        for j in range(case["top_k"]):
            out += state["rows"].double()[state["where"][:, j].long()] * state["weights"][:, j:j + 1].double()
        return out
    order, offsets = state["order"].long(), state["offsets"].tolist()
    if op == "lora":
        y = state["y"].double()
        for i in range(case["adapters"]):
            at = order[offsets[i]:offsets[i + 1]]
            if at.numel():
                u = state["x"][at].double() @ state["a"][i].double().t()
                y[at] = y[at] + state["scale"][i].double() * (u @ state["b"][i].double().t())
        return y
    up = case["side"] == "up"
    x = _weights_64(op, state["x"]) if op == "w4a4" else state["x"].double()
    out = torch.zeros((order.numel(), n // 2 if up else n), dtype=torch.float64, device=DEV)
    for e in range(case["experts"]):
        a, b = offsets[e], offsets[e + 1]
        if a == b:
            continue
        rows = x[torch.div(order[a:b], case["top_k"], rounding_mode="floor")] if up else x[a:b]
        y = rows @ _weights_64(op, [t[e] for t in state["experts"]]).t()
        if up:
            y = y[:, :n // 2] * torch.sigmoid(y[:, :n // 2]) * y[:, n // 2:]
        out[a:b] = y
    return out


# ------------------------------------------------------------------------------------------
# work
# ------------------------------------------------------------------------------------------

def work(case):
    """Each input read once, each output written once, and the products' operations."""
    op, t = case["op"], case["tokens"]
    o = 2 if case.get("out") == "bf16" else 4
    if op == "route":
        pairs = t * case["top_k"]
        size = 2 if case["x"] == "bf16" else 4
        return dict(bytes=t * case["experts"] * size + pairs * 16 + (case["experts"] + 1) * 4,
                    flops=4 * t * case["experts"])
    if op == "lora":
        ids = _adapters(case)
        met, used = len(set(ids[ids >= 0].tolist())), int((ids >= 0).sum())
        n, k, r = case["n"], case["k"], case["rank"]
        return dict(bytes=used * k * 2 + 2 * t * n * o + met * r * (n + k) * 2 + 8 * t,
                    flops=2 * used * r * (n + k))
    ids = _choices(case)
    met, used = len(set(ids[ids >= 0].tolist())), int((ids >= 0).sum())
    pairs = ids.numel()
    if op == "combine":
        return dict(bytes=used * case["hidden"] * 2 + pairs * 8 + t * case["hidden"] * o,
                    flops=2 * used * case["hidden"])
    n, k = _product(case)
    up = case["side"] == "up"
    weight = n * k // 2 + (n * k // 64 if op == "w4a16" else n * k // 16)
    rows = int((ids[:, 0] >= 0).sum()) if up else used
    x = rows * (k * 2 if op == "w4a16" else k // 2 + k // 16)
    return dict(bytes=met * weight + x + pairs * (n // 2 if up else n) * o + pairs * 4,
                flops=2 * used * n * k)
