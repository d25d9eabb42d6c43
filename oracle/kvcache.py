"""Paged key/value cache (oracle; test infrastructure).

Definition of the cache's row formats, of its byte layout and of the operators
on it: head norm and rotation, attention of new tokens (a chain or a tree of
drafts) over a cached context.  The reference pages hand a KV cache from the
prefill half to the decode half (Disaggregated Quantization; Mix-Quant, section
2, system-level deployment) and compare 8-bit with 16-bit caches (the qiita
article on f16 and q8_0); they define no format, so the 4-bit rows follow the
NVFP4 reading of ``nvfp4.py`` with a power of two for each row in the place of
the tensor scale, and the 8-bit ones are E4M3 codes under the same kind of
scale.

Steps for a row x of d values, binary32 (keys that were just normed: binary64),
each rounded once to binary32:
  e = the smallest integer >= -100 with max|x| <= Q 2^e, -100 for a row of zeros;
      Q = 448 (E4M3) or 2688 = 6 * 448 (NVFP4); stored as the byte e + 127
  E4M3:  code = E4M3(x 2^-e)
  NVFP4: s_g = E4M3(rn32(max|x_g| 2^-e / 6)); code = E2M1(rn32(x 2^-e rn32(1 / s_g))),
         the sign alone where s_g == 0
"""

import numpy as np

from .formats import (rn32, enc_e2m1, dec_e2m1, enc_e4m3, dec_e4m3, rn_bf16_bits,
                      bf16_bits_to_f32)

BF16, E4M3, NVFP4 = 0, 1, 2
E_MIN = -100
TOP = {E4M3: 448.0, NVFP4: 2688.0}


def row_bytes(fmt, d):
    return {BF16: 2 * d, E4M3: d, NVFP4: d // 2}[fmt]


def scale_bytes(fmt, d):
    return {BF16: 0, E4M3: 32, NVFP4: 2 * d + 32}[fmt]


def row_exponent(amax, top):
    """The exponent e of rows of the given maxima (float64 array); 0 where there
    is nothing to scale."""
    amax = np.asarray(amax, dtype=np.float64)
    e = np.zeros(amax.shape, dtype=np.int64)
    for i, a in np.ndenumerate(amax):
        if a > 0:
            k = E_MIN
            while a > top * 2.0 ** k:
                k += 1
            e[i] = k
    return e


def sticky32(v):
    """Binary32 values that round on to fewer bits as the float64 v do: the last
    bit says that something was dropped."""
    f = np.asarray(v, dtype=np.float64).astype(np.float32)
    f = np.where(np.abs(f.astype(np.float64)) > np.abs(v), np.nextafter(f, np.float32(0)), f)
    return (f.view(np.uint32) | (f.astype(np.float64) != v)).view(np.float32)


def enc_e4m3_signed(v):
    """E4M3 codes of binary32 values, sign included, saturating at 448."""
    v = np.asarray(v, dtype=np.float32)
    return enc_e4m3(np.abs(v)) | (np.signbit(v).astype(np.uint8) << 7)


def dec_e4m3_signed(c):
    c = np.asarray(c, dtype=np.uint8)
    return np.where(c >> 7, -1.0, 1.0) * dec_e4m3(c & 0x7F)


def quantize(fmt, x):
    """Rows x [n, d] (binary32 or, as float64, binary64 values) -> dict with "row" (bytes [n, row_bytes]),
    "scales" ([n, d/16] or None), "exp" ([n] stored bytes or None) and "value"
    (float64 [n, d], what the bytes stand for)."""
    x = np.asarray(x)
    x = x if x.dtype == np.float64 else x.astype(np.float32)
    n, d = x.shape
    if fmt == BF16:
        bits = rn_bf16_bits(sticky32(x))
        return dict(row=bits.view(np.uint8).reshape(n, 2 * d), scales=None, exp=None,
                    value=bf16_bits_to_f32(bits).astype(np.float64))
    amax = np.max(np.abs(x), axis=1)
    e = np.where(amax > 0, row_exponent(amax, TOP[fmt]), E_MIN)
    y = x.astype(np.float64) * 2.0 ** -e[:, None]
    stored = (e + 127).astype(np.uint8)
    p = 2.0 ** e[:, None].astype(np.float64)
    if fmt == E4M3:
        c = enc_e4m3_signed(sticky32(y))
        return dict(row=c, scales=None, exp=stored, value=dec_e4m3_signed(c) * p)
    g = y.reshape(n, d // 16, 16)
    s = enc_e4m3(rn32(np.max(np.abs(g), axis=2).astype(np.float64) / 6.0))
    sv = dec_e4m3(s)
    inv = np.where(sv > 0, rn32(1.0 / np.where(sv > 0, sv, 1.0)), 0.0).astype(np.float64)
    z = rn32(g.astype(np.float64) * inv[:, :, None])
    c = np.where((sv > 0)[:, :, None], enc_e2m1(z), np.signbit(g).astype(np.uint8) << 3)
    value = (dec_e2m1(c) * sv[:, :, None]).reshape(n, d) * p
    c = c.reshape(n, d)
    return dict(row=(c[:, 0::2] | (c[:, 1::2] << 4)).astype(np.uint8), scales=s.astype(np.uint8),
                exp=stored, value=value)


# ---------------------------------------------------------------------------
# Layout
# ---------------------------------------------------------------------------

def offsets(fmt, d):
    """Where token t's bytes lie in a block: dict of index arrays into the
    block's codes ("k", "v": [16, row_bytes]) and scales ("ks", "vs": [16,
    d/16]; "ke", "ve": [16])."""
    rb = row_bytes(fmt, d)
    c = min(16, rb // 4)
    size = 2 if fmt == BF16 else 1
    seg = {BF16: 32, E4M3: 64, NVFP4: min(d, 128) // 2}[fmt]
    per = max(1, c // 8)
    out = dict(k=np.zeros((16, rb), int), v=np.zeros((16, rb), int), ks=np.zeros((16, d // 16), int),
               vs=np.zeros((16, d // 16), int), ke=np.zeros(16, int), ve=np.zeros(16, int))
    for t in range(16):
        for b in range(rb):
            out["k"][t, b] = (b // c) * 16 * c + t * c + b % c
            u, r = divmod(b, size)
            out["v"][t, b] = 16 * rb + size * ((u // seg) * 16 * seg + (t // 4) * 4 * seg
                                               + (u % seg) * 4 + t % 4) + r
        for g in range(d // 16):
            out["ks"][t, g] = (g // per) * 16 * per + t * per + g % per
            out["vs"][t, g] = d + 16 * g + t
        at = (2 * d if fmt == NVFP4 else 0) + (t // 4) * 8 + t % 4
        out["ke"][t], out["ve"][t] = at, at + 4
    return out


class Cache:
    """The bytes of a cache and the values they stand for, row by row."""

    def __init__(self, fmt, n_pages, page_size, n_kv, d, fill=0):
        self.fmt, self.page, self.n_kv, self.d, self.n_pages = fmt, page_size, n_kv, d, n_pages
        self.blocks = n_pages * n_kv * (page_size // 16)
        self.cb, self.sb = 32 * row_bytes(fmt, d), scale_bytes(fmt, d)
        self.bytes = np.full(self.blocks * (self.cb + self.sb), fill, dtype=np.uint8)
        self.off = offsets(fmt, d)
        self.value = {w: np.full((n_pages * page_size, n_kv, d), np.nan) for w in "kv"}
        self.exp = {w: np.zeros((n_pages * page_size, n_kv), dtype=np.int64) for w in "kv"}

    def _places(self, which, slot, head):
        """Indices of a row's codes, group scales and exponent."""
        page, at = divmod(int(slot), self.page)
        block = (page * self.n_kv + head) * (self.page // 16) + at // 16
        t = at % 16
        code = block * self.cb + self.off[which][t]
        scale = self.blocks * self.cb + block * self.sb
        return code, scale + self.off[which + "s"][t], scale + self.off[which + "e"][t]

    def places(self, which, slot, head):
        """Those that the format has."""
        codes, scales, exp = self._places(which, slot, head)
        return {BF16: [codes], E4M3: [codes, exp], NVFP4: [codes, scales, exp]}[self.fmt]

    def write(self, which, x, slots):
        """Rows x [tokens, n_kv, d] (binary32) to slots; slots < 0 are skipped."""
        x = np.asarray(x)
        for h in range(self.n_kv):
            q = quantize(self.fmt, x[:, h])
            for i, s in enumerate(slots):
                if s < 0:
                    continue
                code, scale, exp = self._places(which, s, h)
                self.bytes[code] = q["row"][i]
                if q["scales"] is not None:
                    self.bytes[scale] = q["scales"][i]
                if q["exp"] is not None:
                    self.bytes[exp] = q["exp"][i]
                    self.exp[which][s, h] = int(q["exp"][i]) - 127
                self.value[which][s, h] = q["value"][i]

    def move(self, pairs):
        """Rows from slot a to slot b for every (a, b) at once."""
        for which in "kv":
            for h in range(self.n_kv):
                places = {s: self.places(which, s, h) for pair in pairs for s in pair}
                held = [([self.bytes[p].copy() for p in places[a]], self.value[which][a, h].copy(),
                         self.exp[which][a, h]) for a, _ in pairs]
                for (_, b), (rows, value, exp) in zip(pairs, held):
                    for p, row in zip(places[b], rows):
                        self.bytes[p] = row
                    self.value[which][b, h], self.exp[which][b, h] = value, exp


# ---------------------------------------------------------------------------
# Operators in float64
# ---------------------------------------------------------------------------

def norm_rope(x, weight, eps, table, positions, interleaved):
    """x [tokens, heads, d] float64 -> normed by weight (None: not) and rotated
    by table [max_pos, rot] (None: not) at positions."""
    x = np.asarray(x, dtype=np.float64)
    if weight is not None:
        x = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    if table is None or table.shape[1] == 0:
        return x
    half = table.shape[1] // 2
    row = np.asarray(table, np.float64)[np.clip(positions, 0, table.shape[0] - 1)]
    c, s = row[:, None, :half], row[:, None, half:]
    first = 2 * np.arange(half) if interleaved else np.arange(half)
    second = first + 1 if interleaved else first + half
    y = x.copy()
    y[..., first] = x[..., first] * c - x[..., second] * s
    y[..., second] = x[..., second] * c + x[..., first] * s
    return y


def visible(nodes, length, tree=None):
    """bool [nodes, length]: what each of a sequence's `nodes` newest tokens sees
    of its `length` keys."""
    ctx = max(length - nodes, 0)
    v = np.zeros((nodes, length), dtype=bool)
    v[:, :ctx] = True
    for i in range(nodes):
        for p in range(ctx, length):
            j = p - ctx
            v[i, p] = j <= i if tree is None else j < 64 and bool(int(tree[i]) >> j & 1)
    return v


def attention(q, k, v, sees, scale, v_exp=None):
    """q [nodes, n_q, d], k, v [length, n_kv, d], sees [nodes, length], v_exp
    [length, n_kv] the exponents of V's rows (None: zeros): (y, mean |v| under
    the weights, largest sum of |q k| scale, sum of |v 2^-e| times the largest
    weight 2^e) -- the last three bound the error that rounded weights and
    scores may cause."""
    nodes, n_q, d = q.shape
    group = n_q // k.shape[1]
    y, mag, top, unit = (np.zeros((nodes, n_q) + s) for s in ((d,), (d,), (), (d,)))
    v_exp = np.zeros(k.shape[:2]) if v_exp is None else v_exp
    for i in range(nodes):
        at = np.flatnonzero(sees[i])
        if at.size == 0:
            continue
        for h in range(n_q):
            kk, vv = k[at, h // group], v[at, h // group]
            s = kk @ q[i, h] * scale
            w = np.exp(s - s.max())
            w /= w.sum()
            y[i, h], mag[i, h] = w @ vv, w @ np.abs(vv)
            top[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() * abs(scale)
            p = 2.0 ** v_exp[at, h // group]
            unit[i, h] = (w * p).max() * (np.abs(vv) / p[:, None]).sum(0)
    return y, mag, top, unit
