"""What is measured of the key/value-cache operators: the cases, their inputs, their plain
form, their definition in 64 bits and their work.

Four operators of a decoder layer stand between its qkv and its output projection.

norm    qkv_norm_rope_append: every query and key head of a token is RMS-normalised and
        rotated by its position, the queries are returned and keys and values are written
        into the paged cache; kv_gather reads the same tokens back.
append  kv_append: rows of keys and values are quantised into the paged cache; kv_gather
        reads them back.
attend  kv_attention: the queries of one or more drafted tokens of each sequence (a token's
        children form a tree; one token is ordinary decoding) over the cached context and
        the drafted tokens' own keys.
commit  kv_commit: once a path of each tree is accepted, its tokens' rows move to the
        places right behind the context; kv_gather reads the drafted places back.

The cache is one buffer of bytes.  A page holds `page` tokens of every kv head in blocks of
16 tokens; all blocks' codes [pages, n_kv, page/16, 2 * 16 * row bytes] come first (a
block's keys, then its values), then all blocks' scales [pages, n_kv, page/16, S].
Formats of a row of d values:

bf16   the values; S = 0.
e4m3   E4M3 codes of x / 2^e with the smallest e for which max|x| <= 448 * 2^e; S = 32.
nvfp4  E2M1 codes in groups of 16 with an E4M3 scale for each group, x / 2^e as above with
       2688 = 6 * 448 in the place of 448; S = 2 * d + 32.

Where byte b of token t's row lies in its block is what `_offsets` says.
"""

import math

import torch

own = False

DEV = "cuda"
E_MIN = -100  # the smallest row exponent that is stored (as e + 127; 127 for a row of zeros)
ROW_BYTES = {"bf16": lambda d: 2 * d, "e4m3": lambda d: d, "nvfp4": lambda d: d // 2}
SCALE_BYTES = {"bf16": lambda d: 0, "e4m3": lambda d: 32, "nvfp4": lambda d: 2 * d + 32}


# ------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------

def listed():
    return [
        # one decode step of eight sequences: the smallest write, where launches count
        dict(name="norm step", op="norm", fmt="e4m3", tokens=8, n_q=32, n_kv=8, d=128,
             page=16, x="bf16", rot=128, style="half"),
        # a prompt's prefill chunk, the widest qkv projection's output read once
        dict(name="norm prompt", op="norm", fmt="e4m3", tokens=8192, n_q=32, n_kv=8, d=128,
             page=64, x="bf16", rot=128, style="half"),
        # odd token count, fp32 projections, interleaved pairs over half of the head
        dict(name="norm odd", op="norm", fmt="bf16", tokens=1537, n_q=40, n_kv=8, d=128,
             page=32, x="f32", rot=64, style="pairs"),
        # a decode batch's write at four bits
        dict(name="append step", op="append", fmt="nvfp4", tokens=32, n_q=32, n_kv=8, d=128,
             page=16, x="bf16"),
        # a long prompt's write at four bits
        dict(name="append prompt", op="append", fmt="nvfp4", tokens=16384, n_q=32, n_kv=8,
             d=128, page=128, x="bf16"),
        # one short chat, one token, narrow unquantised heads: latency alone
        dict(name="attend one", op="attend", fmt="bf16", seqs=1, ctx=500, nodes=1, ragged=False,
             draft="chain", n_q=60, n_kv=12, d=64, page=16),
        # a decode batch of uneven lengths over a four-bit cache
        dict(name="attend batch", op="attend", fmt="nvfp4", seqs=32, ctx=8192, nodes=1,
             ragged=True, draft="chain", n_q=32, n_kv=8, d=128, page=64),
        # one long document, one token: the context is the only axis to split
        dict(name="attend long", op="attend", fmt="e4m3", seqs=1, ctx=131071, nodes=1,
             ragged=False, draft="chain", n_q=40, n_kv=8, d=128, page=128),
        # drafted trees of 16 tokens to be verified at once
        dict(name="attend tree", op="attend", fmt="e4m3", seqs=8, ctx=4096, nodes=16,
             ragged=True, draft="tree", n_q=32, n_kv=8, d=128, page=16),
        # the widest heads and nearly the largest trees
        dict(name="attend wide tree", op="attend", fmt="nvfp4", seqs=4, ctx=16000, nodes=63,
             ragged=True, draft="tree", n_q=15, n_kv=5, d=256, page=64),
        # the accepted paths of a small batch
        dict(name="commit step", op="commit", fmt="nvfp4", seqs=4, ctx=1000, nodes=8,
             ragged=True, draft="tree", n_q=32, n_kv=8, d=128, page=16),
        # the accepted paths of many large trees
        dict(name="commit batch", op="commit", fmt="e4m3", seqs=64, ctx=2000, nodes=63,
             ragged=True, draft="tree", n_q=20, n_kv=4, d=256, page=64),
    ]


HEADS = ((32, 8, 128), (40, 8, 128), (15, 5, 256), (60, 12, 64), (16, 16, 64), (8, 1, 128),
         (30, 30, 128), (20, 4, 256))
MOST_ROWS = 16384 * 8 * 128      # values of K that a drawn write has, at most
MOST_QKV = 8192 * 48 * 128       # values of qkv that a drawn norm has, at most
MOST_CACHE = 32 * 8192 * 8 * 128  # values of K that a drawn attention reads, at most
MOST_SCORES = 4 * 16000 * 63 * 15


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "append", "attend", "attend", "attend", "commit"))
    n_q, n_kv, d = rng.choice(HEADS)
    case = dict(op=op, n_q=n_q, n_kv=n_kv, d=d, page=rng.choice((16, 32, 64, 128)))
    if op == "attend":
        seqs = _spread(rng, 1, 64)
        ctx = _spread(rng, 16, min(131072, MOST_CACHE // (seqs * n_kv * d)))
        nodes = _spread(rng, 1, min(64, max(1, MOST_SCORES // (seqs * ctx * n_q))))
        case.update(fmt=rng.choice(("bf16", "e4m3", "nvfp4")), seqs=seqs, ctx=ctx, nodes=nodes,
                    ragged=rng.random() < 0.7, draft=rng.choice(("tree", "chain")))
        return case
    if op == "commit":
        case.update(fmt=rng.choice(("bf16", "e4m3", "nvfp4")), seqs=_spread(rng, 1, 64),
                    ctx=_spread(rng, 16, 2048), nodes=_spread(rng, 2, 64), ragged=rng.random() < 0.7,
                    draft="tree")
        return case
    case["x"] = rng.choice(("bf16", "bf16", "f32"))
    if op == "append":
        case["tokens"] = _spread(rng, 1, min(16384, MOST_ROWS // (n_kv * d)))
        case["fmt"] = rng.choice(("bf16", "e4m3", "nvfp4"))
    else:
        case["tokens"] = _spread(rng, 1, min(8192, MOST_QKV // ((n_q + 2 * n_kv) * d)))
        # not at four bits: one step of such a code is half of its value, and two sums of
        # squares that are both right to 32 bits can come down on either side of it
        case["fmt"] = rng.choice(("bf16", "e4m3"))
        case["rot"] = rng.choice((d, d, d // 2, 16))
        case["style"] = rng.choice(("half", "pairs"))
    return case


def _contexts(case):
    """Cached tokens of each sequence before its drafted ones."""
    c = case["ctx"]
    if not case["ragged"]:
        return [c] * case["seqs"]
    return [c if b == 0 else max(1, int(c * (0.25 + 0.75 * (b * 0.6180339887 % 1.0))))
            for b in range(case["seqs"])]


def _nodes(case):
    """Drafted tokens of each sequence."""
    n = case["nodes"]
    return [max(1, n - b % 3) if case["ragged"] else n for b in range(case["seqs"])]


# ------------------------------------------------------------------------------------------
# the cache's bytes
# ------------------------------------------------------------------------------------------

def _geometry(case, tokens):
    pages = -(-tokens // case["page"])
    rb, sb = ROW_BYTES[case["fmt"]](case["d"]), SCALE_BYTES[case["fmt"]](case["d"])
    blocks = pages * case["n_kv"] * (case["page"] // 16)
    return pages, blocks, 32 * rb, sb


def _offsets(fmt, d):
    """Byte offsets in a block: of K's and V's row bytes [16, row bytes] in its codes, of K's
    and V's group scales [16, d/16] and row exponents [16] in its scales."""
    t = torch.arange(16, device=DEV)[:, None]
    rb = ROW_BYTES[fmt](d)
    b = torch.arange(rb, device=DEV)[None, :]
    chunk = min(16, rb // 4)
    k = b // chunk * (16 * chunk) + t * chunk + b % chunk
    size = 2 if fmt == "bf16" else 1                    # bytes that stay together in V
    seg = {"bf16": 32, "e4m3": 64, "nvfp4": min(d, 128) // 2}[fmt]
    u = b // size
    v = size * (u // seg * (16 * seg) + t // 4 * (4 * seg) + u % seg * 4 + t % 4) + b % size
    v = v + 16 * rb
    g = torch.arange(d // 16, device=DEV)[None, :]
    per = chunk // 8 if fmt == "nvfp4" else 1
    ks = g // per * (16 * per) + t * per + g % per
    vs = d + g * 16 + t
    t = t[:, 0]
    e = (2 * d if fmt == "nvfp4" else 0) + t // 4 * 8 + t % 4
    return dict(k=k, v=v, ks=ks, vs=vs, ke=e, ve=e + 4)


E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _power(e):
    """2^e in 32 bits, for whole e of the normal range."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _row_exponent(amax, top):
    m, e = torch.frexp(amax)
    tm, te = math.frexp(top)
    e = (e - te + (m > tm)).clamp(min=E_MIN)
    return torch.where(amax > 0, e, torch.zeros_like(e))


def _e4m3(x):
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _encode(fmt, x):
    """Rows x [..., d] in 32 bits: (row bytes, group scales, stored exponents), None where
    the format has none."""
    if fmt == "bf16":
        return x.to(torch.bfloat16).contiguous().view(torch.uint8), None, None
    amax = x.abs().amax(-1)
    e = _row_exponent(amax, 448.0 if fmt == "e4m3" else 2688.0)
    y = x * _power(-e)[..., None]
    stored = (e + 127).to(torch.uint8)
    if fmt == "e4m3":
        return _e4m3(y), None, stored
    g = y.unflatten(-1, (-1, 16))
    s = _e4m3(g.abs().amax(-1) / 6.0)
    sv = s.view(torch.float8_e4m3fn).float()
    inv = torch.where(sv > 0, 1.0 / sv, torch.zeros_like(sv))
    z = (g * inv[..., None]).flatten(-2)
    a = z.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75).to(torch.uint8) + (a > 1.25).to(torch.uint8)
            + (a >= 1.75).to(torch.uint8) + (a > 2.5).to(torch.uint8)
            + (a >= 3.5).to(torch.uint8) + (a > 5.0).to(torch.uint8))
    code = code | (torch.signbit(z).to(torch.uint8) << 3)
    return code[..., 0::2] | (code[..., 1::2] << 4), s, stored


def _decode(fmt, row, scales, stored):
    """The values of rows in 32 bits."""
    if fmt == "bf16":
        return row.contiguous().view(torch.bfloat16).float()
    p = _power(stored.int() - 127)[..., None]
    if fmt == "e4m3":
        return row.contiguous().view(torch.float8_e4m3fn).float() * p
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=row.device)
    c = torch.stack((row & 15, row >> 4), -1).flatten(-2)
    s = scales.contiguous().view(torch.float8_e4m3fn).float()
    return (table[c.int()].unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2) * p


def _write(case, state, which, x, slots):
    """Rows x [tokens, n_kv, d] into the cache's bytes at their slots."""
    block, t, off = _blocks(case, slots), slots % 16, state["off"]
    row, scales, stored = _encode(case["fmt"], x)
    cb, sb, codes_end = state["code_bytes"], state["scale_bytes"], state["codes_end"]
    cache = state["cache"]
    cache[block[..., None] * cb + off[which][t][:, None, :]] = row
    if scales is not None:
        at = codes_end + block[..., None] * sb + off[which + "s"][t][:, None, :]
        cache[at] = scales
    if stored is not None:
        cache[codes_end + block * sb + off[which + "e"][t][:, None]] = stored


def _read(case, state, which, slots):
    """The values [..., n_kv, d] of the cache at slots [...]."""
    block, t, off = _blocks(case, slots), slots % 16, state["off"]
    cb, sb, codes_end = state["code_bytes"], state["scale_bytes"], state["codes_end"]
    cache, fmt = state["cache"], case["fmt"]
    row = cache[block[..., None] * cb + off[which][t][..., None, :]]
    scales = stored = None
    if fmt == "nvfp4":
        scales = cache[codes_end + block[..., None] * sb + off[which + "s"][t][..., None, :]]
    if fmt != "bf16":
        stored = cache[codes_end + block * sb + off[which + "e"][t][..., None]]
    return _decode(fmt, row, scales, stored)


def _blocks(case, slots):
    """Block indices [..., n_kv] of slots [...]."""
    page, per = case["page"], case["page"] // 16
    h = torch.arange(case["n_kv"], device=slots.device)
    return ((slots // page)[..., None] * case["n_kv"] + h) * per + (slots % page // 16)[..., None]


# ------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------

def _rows(g, tokens, heads, d):
    """Keys or values as projections give them: unit spread, a few loud channels, rows of
    uneven size."""
    x = torch.randn((tokens, heads, d), generator=g, device=DEV)
    loud = torch.rand((heads, d), generator=g, device=DEV) < 0.02
    x *= torch.where(loud, 8.0, 1.0)
    x *= torch.exp(0.3 * torch.randn((tokens, heads, 1), generator=g, device=DEV))
    return x


def _empty_cache(case, tokens):
    pages, blocks, cb, sb = _geometry(case, tokens)
    return dict(cache=torch.zeros(blocks * (cb + sb), dtype=torch.uint8, device=DEV),
                pages=pages, code_bytes=cb, scale_bytes=sb, codes_end=blocks * cb,
                off=_offsets(case["fmt"], case["d"]))


def _table(g, case, counts):
    """A block table [seqs, most pages] over shuffled pages, -1 past a sequence's last, and
    the number of pages."""
    need = [-(-n // case["page"]) for n in counts]
    perm = torch.randperm(sum(need), generator=g, device=DEV).int()
    n = torch.tensor(need, device=DEV)[:, None]
    j = torch.arange(max(need), device=DEV)
    table = torch.where(j < n, perm[(n.cumsum(0) - n + j).clamp(max=sum(need) - 1)], -1)
    return table.int().contiguous(), sum(need)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    d, n_q, n_kv = case["d"], case["n_q"], case["n_kv"]
    if case["op"] in ("norm", "append"):
        tokens = case["tokens"]
        dtype = torch.bfloat16 if case["x"] == "bf16" else torch.float32
        table, pages = _table(g, case, [tokens])
        state = _empty_cache(case, pages * case["page"])
        i = torch.arange(tokens, device=DEV)
        state["slots"] = table[0, i // case["page"]].long() * case["page"] + i % case["page"]
        if case["op"] == "append":
            state["k"] = _rows(g, tokens, n_kv, d).to(dtype)
            state["v"] = _rows(g, tokens, n_kv, d).to(dtype)
        else:
            state["qkv"] = _rows(g, tokens, n_q + 2 * n_kv, d).to(dtype).flatten(1)
            state["q_weight"] = 1 + 0.1 * torch.randn(d, generator=g, device=DEV)
            state["k_weight"] = 1 + 0.1 * torch.randn(d, generator=g, device=DEV)
            # the prompt starts somewhere in the model's range of positions
            start = int(torch.randint(0, 1024, (1,), generator=g, device=DEV))
            state["positions"] = (start + i).int()
            half = case["rot"] // 2
            f = 1e6 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half)
            a = torch.arange(start + tokens, device=DEV, dtype=torch.float64)[:, None] * f
            state["rope"] = torch.cat((a.cos(), a.sin()), 1).float()
        state["case"] = case
        return state
    ctx, nodes = _contexts(case), _nodes(case)
    lens = [c + n for c, n in zip(ctx, nodes)]
    table, pages = _table(g, case, lens)
    state = _empty_cache(case, pages * case["page"])
    every = torch.arange(pages * case["page"], device=DEV)
    for part in every.split(1 << 16):
        for which in ("k", "v"):
            _write(case, state, which, _rows(g, part.numel(), n_kv, d), part)
    total = sum(nodes)
    if case["op"] == "attend":
        state["q"] = _rows(g, total, n_q, d).to(torch.bfloat16)
    state["cu_q"] = torch.tensor([0] + nodes, device=DEV).cumsum(0).int()
    state["kv_lens"] = torch.tensor(lens, device=DEV).int()
    state["table"] = table
    state["tree"] = None
    if case["draft"] == "tree":
        # each drafted token hangs under an earlier one of its sequence, or is a root
        r = torch.rand((total,), generator=g, device=DEV).tolist()
        masks, at = [], 0
        for n in nodes:
            m = []
            for j in range(n):
                parent = int(r[at + j] * (j + 1)) - 1
                m.append((m[parent] if parent >= 0 else 0) | 1 << j)
            masks += m
            at += n
        state["tree"] = torch.tensor([m - (1 << 64) if m >> 63 else m for m in masks], device=DEV)
    if case["op"] == "commit":
        # the path from a root to one drafted token of each tree, chosen at random
        ends = [at + int(x * n) for at, n, x in
                zip(state["cu_q"].tolist(), nodes, torch.rand(len(nodes), generator=g, device=DEV).tolist())]
        paths = [[j for j in range(64) if masks[e] >> j & 1] for e in ends]
        state["path"] = torch.tensor([p + [-1] * (max(nodes) - len(p)) for p in paths], device=DEV).int()
        i = torch.arange(max(nodes), device=DEV)
        at = torch.tensor(ctx, device=DEV)[:, None] + i
        slots = torch.gather(table, 1, (at // case["page"]).clamp(max=table.shape[1] - 1)).long()
        state["slots"] = (slots * case["page"] + at % case["page"])[i < torch.tensor(nodes, device=DEV)[:, None]]
    state["max_q"], state["max_kv"] = max(nodes), max(lens)
    state["case"] = case
    return state


# ------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(state):
    from decode_nvfp4_rtn_amd import qlin

    case = state["case"]
    fmt = {"bf16": qlin.QL_KV_BF16, "e4m3": qlin.QL_KV_E4M3, "nvfp4": qlin.QL_KV_NVFP4}[case["fmt"]]
    cache = qlin.KVCache(fmt, state["pages"], case["page"], case["n_kv"], case["d"],
                         data=state["cache"])
    if case["op"] == "attend":
        return qlin.kv_attention(cache, state["q"], state["cu_q"], state["kv_lens"],
                                 state["table"], state["max_q"], state["max_kv"],
                                 tree=state["tree"])
    if case["op"] == "commit":
        qlin.kv_commit(cache, state["cu_q"], state["kv_lens"], state["table"], state["path"])
        return qlin.kv_gather(cache, state["slots"])
    if case["op"] == "append":
        qlin.kv_append(cache, state["k"], state["v"], state["slots"])
        return qlin.kv_gather(cache, state["slots"])
    q = qlin.qkv_norm_rope_append(cache, state["qkv"], case["n_q"], state["slots"],
                                  state["positions"], state["rope"], state["q_weight"],
                                  state["k_weight"], eps=1e-6,
                                  interleaved=case["style"] == "pairs")
    return (q, *qlin.kv_gather(cache, state["slots"]))


def _norm_rope(case, x, weight, c, s):
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight
    half = case["rot"] // 2
    if case["style"] == "half":
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat((a * c - b * s, b * c + a * s), -1)
    else:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    return torch.cat((turned, x[..., 2 * half:]), -1)


def _run_plain(state):
    case = state["case"]
    if case["op"] == "attend":
        return _attend_plain(state, case)
    if case["op"] == "commit":
        return _commit_plain(state, case)
    slots, n_q, n_kv = state["slots"], case["n_q"], case["n_kv"]
    if case["op"] == "append":
        out, k, v = (), state["k"].float(), state["v"].float()
    else:
        x = state["qkv"].float().unflatten(1, (-1, case["d"]))
        c, s = state["rope"][state["positions"].long()][:, None, :].chunk(2, -1)
        q = _norm_rope(case, x[:, :n_q], state["q_weight"], c, s)
        k = _norm_rope(case, x[:, n_q:n_q + n_kv], state["k_weight"], c, s)
        out, v = (q.to(torch.bfloat16),), x[:, n_q + n_kv:]
    _write(case, state, "k", k, slots)
    _write(case, state, "v", v, slots)
    k, v = _read(case, state, "k", slots), _read(case, state, "v", slots)
    return (*out, k.to(torch.bfloat16), v.to(torch.bfloat16))


def _commit_plain(state, case):
    path, table = state["path"].long(), state["table"]
    cu = state["cu_q"].long()
    ctx = (state["kv_lens"].long() - (cu[1:] - cu[:-1]))[:, None]
    there = path >= 0
    cb, sb, end, off, cache = (state[x] for x in ("code_bytes", "scale_bytes", "codes_end", "off", "cache"))

    def places(at):
        """Byte places [moves, n_kv, bytes] of the whole rows at positions [seqs, moves]."""
        slots = torch.gather(table, 1, (at // case["page"]).clamp(max=table.shape[1] - 1)).long()
        slots = (slots * case["page"] + at % case["page"])[there]
        block, t = _blocks(case, slots)[..., None], slots % 16
        rows = [block * cb + off[x][t][:, None, :] for x in ("k", "v")]
        if case["fmt"] == "nvfp4":
            rows += [end + block * sb + off[x][t][:, None, :] for x in ("ks", "vs")]
        if case["fmt"] != "bf16":
            rows += [end + block * sb + off[x][t][:, None, None] for x in ("ke", "ve")]
        return torch.cat(rows, -1)

    to = places(ctx + torch.arange(path.shape[1], device=DEV))
    cache[to] = cache[places(ctx + path.clamp(min=0))]
    k, v = (_read(case, state, x, state["slots"]) for x in ("k", "v"))
    return k.to(torch.bfloat16), v.to(torch.bfloat16)


def _attend_plain(state, case):
    n_kv, d, group = case["n_kv"], case["d"], case["n_q"] // case["n_kv"]
    cu, lens, table = state["cu_q"].long(), state["kv_lens"].long(), state["table"]
    seqs, most, length = lens.numel(), state["max_q"], state["max_kv"]
    # the queries of each sequence, padded: [seqs, n_kv, most * group, d]
    i = torch.arange(most, device=DEV)
    count = cu[1:] - cu[:-1]
    real = i < count[:, None]
    at = torch.where(real, cu[:-1, None] + i, torch.zeros_like(cu[:1]))
    q = state["q"][at].float().unflatten(2, (n_kv, group)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    # the keys and values of each sequence, padded: [seqs, length, n_kv, d]
    p = torch.arange(length, device=DEV)
    slots = table[:, p // case["page"]].long().clamp(min=0) * case["page"] + p % case["page"]
    k, v = _read(case, state, "k", slots), _read(case, state, "v", slots)
    scores = torch.matmul(q, k.permute(0, 2, 3, 1).contiguous()) * d ** -0.5
    # what a drafted token sees: the context, and of the drafted tokens those of its path
    node = p - (lens - count)[:, None]                              # [seqs, length]
    if state["tree"] is None:
        path = node[:, None, :] <= i[None, :, None]
    else:
        bits = state["tree"][at][:, :, None] >> node[:, None, :].clamp(0, 63)
        path = (bits & 1).bool()
    sees = (node < 0)[:, None, :] | path
    sees = sees & (p < lens[:, None])[:, None, :]
    sees = sees.repeat_interleave(group, 1)[:, None]                # [seqs, 1, most * group, length]
    scores = scores.masked_fill(~sees, -math.inf)
    top = scores.amax(-1, keepdim=True)
    w = torch.exp(scores - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = w.sum(-1, keepdim=True)
    y = torch.matmul(w, v.permute(0, 2, 1, 3).contiguous())
    y = torch.where(total > 0, y / total, torch.zeros_like(y))
    y = y.unflatten(2, (most, group)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    return y[real].to(torch.bfloat16)


# ------------------------------------------------------------------------------------------
# the definition in 64 bits
# ------------------------------------------------------------------------------------------

def _table_e4m3():
    """The 256 values of E4M3, from its definition."""
    low = [m * 2.0 ** -9 for m in range(8)]
    high = [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)]
    half = low + high[:-1] + [math.nan]
    return torch.tensor(half + [-x for x in half], dtype=torch.float64, device=DEV)


def _nearest_even(x, values):
    """The values of a sorted table (non-negative, even places first) nearest to x >= 0, ties to even."""
    x = x.clamp(max=float(values[-1]))
    hi = torch.searchsorted(values, x).clamp(max=values.numel() - 1)
    lo = (hi - 1).clamp(min=0)
    a, b = x - values[lo], values[hi] - x
    take = torch.where((b < a) | ((a == b) & (hi % 2 == 0)), hi, lo)
    return values[torch.where(x == values[hi], hi, take)]


def _quantised_64(fmt, x):
    """What rows x [..., d] (64 bits) stand for once quantised."""
    if fmt == "bf16":
        return x.float().to(torch.bfloat16).double()
    e4 = _table_e4m3()[:127]
    top = 448.0 if fmt == "e4m3" else 2688.0
    amax = x.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(torch.where(amax > 0, amax / top, torch.ones_like(amax))))
    e = torch.where(amax > top * torch.exp2(e), e + 1, e)     # where log2 was rounded
    e = torch.where((amax > 0) & (amax <= top * torch.exp2(e - 1)), e - 1, e).clamp(min=E_MIN)
    y = x * torch.exp2(-e)
    if fmt == "e4m3":
        return torch.sign(y) * _nearest_even(y.abs(), e4) * torch.exp2(e)
    g = y.unflatten(-1, (-1, 16))
    # the scale and its inverse are defined in binary32
    s = _nearest_even((g.abs().amax(-1, keepdim=True) / 6).float().double(), e4)
    inv = torch.where(s > 0, (1 / s).float().double(), torch.zeros_like(s))
    grid = torch.tensor(E2M1, dtype=torch.float64, device=DEV)
    z = (g * inv).float().double()
    return (torch.sign(z) * _nearest_even(z.abs(), grid) * s).flatten(-2) * torch.exp2(e)


def _pages_64(case, state):
    """Keys and values [pages, n_kv, page, d] that the cache's bytes stand for, in 64 bits."""
    fmt, d, n_kv, page, pages = case["fmt"], case["d"], case["n_kv"], case["page"], state["pages"]
    lead = (pages, n_kv, page // 16)
    raw = state["cache"]
    codes = raw[:state["codes_end"]].view(*lead, 2, -1)
    scales = raw[state["codes_end"]:].view(*lead, -1)
    if fmt == "bf16":
        k = codes[..., 0, :].view(torch.bfloat16).view(*lead, d // 8, 16, 8).permute(0, 1, 2, 4, 3, 5)
        v = codes[..., 1, :].view(torch.bfloat16).view(*lead, d // 32, 4, 32, 4).permute(0, 1, 2, 4, 6, 3, 5)
        return (k.reshape(pages, n_kv, page, d).double(), v.reshape(pages, n_kv, page, d).double())
    power = torch.exp2(scales[..., -32:].reshape(*lead, 4, 2, 4).double() - 127)
    e4 = _table_e4m3()
    if fmt == "e4m3":
        k = codes[..., 0, :].reshape(*lead, d // 16, 16, 16).permute(0, 1, 2, 4, 3, 5)
        v = codes[..., 1, :].reshape(*lead, d // 64, 4, 64, 4).permute(0, 1, 2, 4, 6, 3, 5)
        k, v = (e4[x.reshape(*lead, 16, d).int()] for x in (k, v))
    else:
        c = min(16, d // 8)
        w = min(d, 128) // 2
        k = codes[..., 0, :].reshape(*lead, d // 2 // c, 16, c).permute(0, 1, 2, 4, 3, 5)
        v = codes[..., 1, :].reshape(*lead, d // 2 // w, 4, w, 4).permute(0, 1, 2, 4, 6, 3, 5)
        grid = torch.tensor(E2M1 + tuple(-x for x in E2M1), dtype=torch.float64, device=DEV)
        k, v = (x.reshape(*lead, 16, d // 2).int() for x in (k, v))
        k, v = (grid[torch.stack((x % 16, x // 16), -1)].reshape(*lead, 16, d // 16, 16) for x in (k, v))
        ks = scales[..., :d].reshape(*lead, -1, 16, c // 8).permute(0, 1, 2, 4, 3, 5).reshape(*lead, 16, d // 16)
        vs = scales[..., d:2 * d].reshape(*lead, d // 16, 16).transpose(-1, -2)
        k, v = ((x * e4[s.int()][..., None]).reshape(*lead, 16, d) for x, s in ((k, ks), (v, vs)))
    k, v = (x * power[..., j, :].reshape(*lead, 16, 1) for j, x in enumerate((k, v)))
    return k.reshape(pages, n_kv, page, d), v.reshape(pages, n_kv, page, d)


def exact(case, seed):
    state = prepare(case, seed)
    n_q, n_kv, d = case["n_q"], case["n_kv"], case["d"]
    if case["op"] == "append":
        return tuple(_quantised_64(case["fmt"], state[w].double()) for w in ("k", "v"))
    if case["op"] == "norm":
        x = state["qkv"].double().view(-1, n_q + 2 * n_kv, d)
        w = torch.cat((state["q_weight"].double().expand(n_q, d), state["k_weight"].double().expand(n_kv, d)))
        r = x[:, :n_q + n_kv]
        r = r / torch.sqrt(torch.mean(r ** 2, -1, keepdim=True) + 1e-6) * w
        half = case["rot"] // 2
        at = torch.arange(half, device=DEV)
        first, second = (at, at + half) if case["style"] == "half" else (2 * at, 2 * at + 1)
        turn = state["rope"].double()[state["positions"].long()]
        z = torch.complex(r[..., first], r[..., second]) * torch.complex(turn[:, :half], turn[:, half:])[:, None]
        r = r.clone()
        r[..., first], r[..., second] = z.real, z.imag
        return r[:, :n_q], _quantised_64(case["fmt"], r[:, n_q:]), _quantised_64(case["fmt"], x[:, n_q + n_kv:])
    k, v = _pages_64(case, state)
    if case["op"] == "commit":
        out, cu = [], state["cu_q"].tolist()
        for b, length in enumerate(state["kv_lens"].tolist()):
            n = cu[b + 1] - cu[b]
            ids = state["table"][b, :-(-length // case["page"])].long()
            both = [x[ids].transpose(0, 1).reshape(n_kv, -1, d)[:, length - n:length] for x in (k, v)]
            taken = [j for j in state["path"][b].tolist() if j >= 0]
            order = torch.tensor(taken + list(range(len(taken), n)), device=DEV)
            out.append([x[:, order].transpose(0, 1) for x in both])
        return tuple(torch.cat(x) for x in zip(*out))
    out, cu = [], state["cu_q"].tolist()
    for b, length in enumerate(state["kv_lens"].tolist()):
        n = cu[b + 1] - cu[b]
        pages = state["table"][b, :-(-length // case["page"])].long()
        kb, vb = (x[pages].transpose(0, 1).reshape(n_kv, -1, d)[:, :length] for x in (k, v))
        q = state["q"][cu[b]:cu[b + 1]].double().view(n, n_kv, -1, d)
        sees = torch.ones(n, length, dtype=torch.bool, device=DEV)
        if state["tree"] is None:
            sees[:, length - n:] = torch.ones(n, n, device=DEV).tril().bool()
        else:
            m = state["tree"][cu[b]:cu[b + 1]].tolist()
            sees[:, length - n:] = torch.tensor([[bool(x >> j & 1) for j in range(n)] for x in m], device=DEV)
        s = torch.einsum("nhgd,hld->hngl", q, kb) / math.sqrt(d)
        s = s.masked_fill(~sees[None, :, None, :], -math.inf)
        out.append(torch.einsum("hngl,hld->nhgd", torch.softmax(s, -1), vb).reshape(n, n_q, d))
    return torch.cat(out)


# ------------------------------------------------------------------------------------------
# work
# ------------------------------------------------------------------------------------------

def work(case):
    n_q, n_kv, d, fmt = case["n_q"], case["n_kv"], case["d"], case["fmt"]
    row = 2 * n_kv * (ROW_BYTES[fmt](d) + SCALE_BYTES[fmt](d) / 32)  # K and V of a token, cached
    if case["op"] == "commit":
        # a path of a random tree is about ln(n) + 1 tokens long; every drafted row is read back
        nodes = _nodes(case)
        moved = sum(math.log(n) + 1 for n in nodes)
        return {"bytes": moved * 2 * row + sum(nodes) * (row + 2 * n_kv * d * 2 + 8), "flops": sum(nodes) * 2 * n_kv * d}
    if case["op"] == "attend":
        ctx, nodes = _contexts(case), _nodes(case)
        tokens, queries = sum(ctx) + sum(nodes), sum(nodes)
        pages = sum(-(-(c + n) // case["page"]) for c, n in zip(ctx, nodes))
        scores = sum((c + n) * n for c, n in zip(ctx, nodes)) * n_q
        return {"bytes": tokens * row + queries * n_q * d * 4 + pages * 4 + queries * 8,
                "flops": 4 * scores * d}
    tokens, size = case["tokens"], 2 if case["x"] == "bf16" else 4
    plain = 2 * n_kv * d                                             # values of K and V of a token
    back = row + plain * 2                                           # kv_gather: cache read, bf16 out
    if case["op"] == "append":
        return {"bytes": tokens * (plain * size + row + 8 + back + 8), "flops": tokens * plain * 4}
    qkv = (n_q + 2 * n_kv) * d
    return {"bytes": tokens * (qkv * size + n_q * d * 2 + row + 12 + back + 8 + case["rot"] * 4),
            "flops": tokens * ((n_q + n_kv) * d * 8 + plain * 4)}
