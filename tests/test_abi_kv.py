"""C-ABI checks of the key/value cache that need no GPU: every call below is
refused, or has nothing to do, before any device work."""

import ctypes
import os

import pytest

from tests.test_abi import LIB, _declared, A, B, C, D, E
from tests.test_abi import (QL_OK, QL_EINVAL, QL_ESHAPE, QL_EALIGN, QL_EDTYPE, QL_EWORKSPACE,
                            QL_EFORMAT)

vp, i64, sz, i32, u = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int, ctypes.c_uint
f32 = ctypes.c_float
BF16, E4M3, NVFP4 = 0, 1, 2
QF32, QBF16 = 0, 1


class KV(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int32), ("n_kv", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("n_pages", i64), ("data", vp), ("bytes", sz)]


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB):
        pytest.fail(f"{LIB} not built (python -m decode_nvfp4_rtn_amd.build)")
    L = ctypes.CDLL(LIB)
    for name, res, args in (
            ("kv_cache_bytes", sz, [i32, i64, i64, i64, i64]),
            ("kv_append", i32, [vp, vp, vp, i32, i64, i64, i64, vp, vp]),
            ("kv_gather", i32, [vp, vp, i64, vp, vp, i32, vp]),
            ("qkv_norm_rope_append", i32, [vp, vp, i32, i64, i64, i64, vp, vp, f32, vp, vp, i64, i64,
                                           u, vp, vp, vp]),
            ("kv_attention_workspace", sz, [vp, i64, i64, i64, i64, i64]),
            ("kv_attention", i32, [vp, vp, i64, i64, i64, i64, vp, vp, vp, i64, i64, i64, i64, vp,
                                   f32, vp, vp, sz, vp]),
            ("kv_commit", i32, [vp, i64, vp, vp, vp, i64, i64, vp, i64, vp])):
        f = getattr(L, name)
        f.restype, f.argtypes = res, args
    return L


def cache(lib, **kw):
    a = dict(format=E4M3, n_kv=2, head_dim=128, page_size=16, n_pages=4, data=A, bytes=1 << 40)
    a.update(kw)
    return KV(**a)


def test_header_declares_the_calls():
    assert {"kv_cache_bytes", "kv_append", "kv_gather", "qkv_norm_rope_append", "kv_attention",
            "kv_attention_workspace", "kv_commit"} <= set(_declared())


@pytest.mark.parametrize("d", [64, 128, 256])
def test_cache_bytes(lib, d):
    for fmt, row, scales in ((BF16, 2 * d, 0), (E4M3, d, 32), (NVFP4, d // 2, 2 * d + 32)):
        assert lib.kv_cache_bytes(fmt, 5, 64, 3, d) == 5 * 3 * 4 * (32 * row + scales)
    for bad in ((3, 5, 64, 3, d), (0, 0, 64, 3, d), (0, -1, 64, 3, d), (0, 5, 8, 3, d),
                (0, 5, 48, 3, d), (0, 5, 8192, 3, d), (0, 5, 64, 0, d), (0, 5, 64, 1025, d),
                (0, 5, 64, 3, 96), (0, 1 << 31, 64, 3, d), (0, (1 << 31) - 1, 4096, 1024, d)):
        assert lib.kv_cache_bytes(*bad) == 0


BAD_CACHES = [(dict(format=3), QL_EFORMAT), (dict(format=-1), QL_EFORMAT), (dict(n_kv=0), QL_ESHAPE),
              (dict(head_dim=96), QL_ESHAPE), (dict(page_size=24), QL_ESHAPE),
              (dict(page_size=-16), QL_ESHAPE), (dict(n_pages=0), QL_ESHAPE), (dict(data=0), QL_EINVAL),
              (dict(data=A + 8), QL_EALIGN), (dict(bytes=4 * 2 * (32 * 128 + 32) - 1), QL_EWORKSPACE)]


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_every_call_checks_its_cache(lib, kw, status):
    c = ctypes.byref(cache(lib, **kw))
    assert lib.kv_append(c, B, C, QBF16, 3, 256, 256, D, 0) == status
    assert lib.kv_gather(c, D, 3, B, C, QBF16, 0) == status
    assert lib.qkv_norm_rope_append(c, B, QBF16, 3, 1024, 4, 0, 0, 1e-6, C, D, 8, 128, 0, E, B, 0) == status
    assert lib.kv_attention(c, B, 512, 3, 4, 1, C, C, D, 4, 4, 1, 64, 0, 1.0, E, 0, 0, 0) == status
    assert lib.kv_commit(c, 1, C, C, D, 4, 4, E, 4, 0) == status


def test_null_cache(lib):
    assert lib.kv_append(None, B, C, QBF16, 3, 256, 256, D, 0) == QL_EINVAL
    assert lib.kv_attention_workspace(None, 3, 4, 1, 1, 64) == 0


def test_append_and_gather(lib):
    c = ctypes.byref(cache(lib))

    def append(k=B, v=C, dt=QBF16, tokens=3, ks=256, vs=256, slots=D):
        return lib.kv_append(c, k, v, dt, tokens, ks, vs, slots, 0)
    for kw, status in ((dict(k=0), QL_EINVAL), (dict(slots=0), QL_EINVAL), (dict(tokens=-1), QL_EINVAL),
                       (dict(dt=2), QL_EDTYPE), (dict(ks=255), QL_ESHAPE), (dict(vs=260), QL_EALIGN),
                       (dict(dt=QF32, ks=258), QL_EALIGN), (dict(v=C + 4), QL_EALIGN),
                       (dict(slots=D + 4), QL_EALIGN), (dict(tokens=1 << 31), QL_ESHAPE),
                       (dict(tokens=0), QL_OK), (dict(tokens=0, k=0, slots=0), QL_OK)):
        assert append(**kw) == status, kw

    def gather(slots=D, tokens=3, k=B, v=C, dt=QBF16):
        return lib.kv_gather(c, slots, tokens, k, v, dt, 0)
    for kw, status in ((dict(k=0), QL_EINVAL), (dict(tokens=-2), QL_EINVAL), (dict(dt=7), QL_EDTYPE),
                       (dict(k=B + 2), QL_EALIGN), (dict(tokens=0), QL_OK)):
        assert gather(**kw) == status, kw


def test_norm_rope(lib):
    c = ctypes.byref(cache(lib))

    def run(x=B, dt=QBF16, tokens=3, stride=1024, n_q=4, qw=0, kw=0, pos=C, rope=D, max_pos=8, rot=128,
            flags=0, out=E, slots=B):
        return lib.qkv_norm_rope_append(c, x, dt, tokens, stride, n_q, qw, kw, 1e-6, pos, rope, max_pos,
                                        rot, flags, out, slots, 0)
    for kw, status in ((dict(x=0), QL_EINVAL), (dict(out=0), QL_EINVAL), (dict(slots=0), QL_EINVAL),
                       (dict(pos=0), QL_EINVAL), (dict(rope=0), QL_EINVAL), (dict(flags=2), QL_EINVAL),
                       (dict(tokens=-1), QL_EINVAL), (dict(dt=3), QL_EDTYPE), (dict(n_q=0), QL_ESHAPE),
                       (dict(n_q=65537), QL_ESHAPE), (dict(rot=3), QL_ESHAPE), (dict(rot=130), QL_ESHAPE),
                       (dict(rot=-2), QL_ESHAPE), (dict(max_pos=0), QL_ESHAPE),
                       (dict(stride=1016), QL_ESHAPE), (dict(stride=1028), QL_EALIGN),
                       (dict(x=B + 8), QL_EALIGN), (dict(out=E + 8), QL_EALIGN), (dict(qw=2), QL_EALIGN),
                       (dict(pos=C + 2), QL_EALIGN), (dict(tokens=0), QL_OK)):
        assert run(**kw) == status, kw


def test_attention(lib):
    c = ctypes.byref(cache(lib))

    def run(q=B, stride=512, tokens=3, n_q=4, seqs=1, cu=C, lens=C, table=D, ts=4, cols=4, max_q=1,
            max_kv=64, tree=0, y=E, ws=0, wsb=0):
        return lib.kv_attention(c, q, stride, tokens, n_q, seqs, cu, lens, table, ts, cols, max_q, max_kv,
                                tree, 1.0, y, ws, wsb, 0)
    for kw, status in ((dict(q=0), QL_EINVAL), (dict(y=0), QL_EINVAL), (dict(cu=0), QL_EINVAL),
                       (dict(table=0), QL_EINVAL), (dict(tokens=-1), QL_EINVAL), (dict(seqs=-1), QL_EINVAL),
                       (dict(max_q=-1), QL_EINVAL), (dict(max_kv=-1), QL_EINVAL), (dict(n_q=3), QL_ESHAPE),
                       (dict(n_q=0), QL_ESHAPE), (dict(seqs=65536), QL_ESHAPE), (dict(ts=3), QL_ESHAPE),
                       (dict(cols=-1), QL_ESHAPE), (dict(max_q=65, tree=A), QL_ESHAPE),
                       (dict(stride=511), QL_ESHAPE), (dict(stride=516), QL_EALIGN),
                       (dict(q=B + 8), QL_EALIGN), (dict(cu=C + 1), QL_EALIGN), (dict(tree=A + 4), QL_EALIGN),
                       (dict(max_kv=1 << 31), QL_ESHAPE), (dict(tokens=0), QL_OK), (dict(seqs=0), QL_OK),
                       (dict(max_q=0), QL_OK)):
        assert run(**kw) == status, kw
    # a workspace is asked for where keys are split, and only there
    assert lib.kv_attention_workspace(c, 3, 4, 1, 1, 512) == 0
    need = lib.kv_attention_workspace(c, 3, 4, 1, 1, 100000)
    assert need > 8 and (need - 8) % (4 * (128 + 2) * 4) == 0
    assert run(max_kv=100000) == QL_EINVAL
    assert run(max_kv=100000, ws=A + 8, wsb=need) == QL_EALIGN
    assert run(max_kv=100000, ws=A, wsb=need - 1) == QL_EWORKSPACE
    assert lib.kv_attention_workspace(c, 3, 3, 1, 1, 100000) == 0      # a refused shape


def test_commit(lib):
    c = ctypes.byref(cache(lib))

    def run(seqs=1, cu=C, lens=C, table=D, ts=4, cols=4, path=E, most=4):
        return lib.kv_commit(c, seqs, cu, lens, table, ts, cols, path, most, 0)
    for kw, status in ((dict(seqs=-1), QL_EINVAL), (dict(most=-1), QL_EINVAL), (dict(most=65), QL_ESHAPE),
                       (dict(seqs=65536), QL_ESHAPE), (dict(ts=3), QL_ESHAPE), (dict(path=0), QL_EINVAL),
                       (dict(cu=0), QL_EINVAL), (dict(path=E + 2), QL_EALIGN), (dict(seqs=0), QL_OK),
                       (dict(most=0), QL_OK)):
        assert run(**kw) == status, kw
