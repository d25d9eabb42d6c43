"""C-ABI checks of plans, experts and adapters that need no GPU: every call
below is refused, or has nothing to do, before any device work."""

import ctypes
import os

import pytest

from tests.test_abi import LIB, _declared, A, B, C, D, E
from tests.test_abi import QL_OK, QL_EINVAL, QL_ESHAPE, QL_EALIGN, QL_EDTYPE, QL_EWORKSPACE

vp, i64, sz, i32, u = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int, ctypes.c_uint
QF32, QBF16 = 0, 1
MOST = (1 << 24) - 1


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB):
        pytest.fail(f"{LIB} not built (python -m decode_nvfp4_rtn_amd.build)")
    L = ctypes.CDLL(LIB)
    for name, res, args in (
            ("repack_weights_bytes", sz, [i32, i64, i64]),
            ("group_rows_workspace", sz, [i64, i64]),
            ("group_rows", i32, [vp, i64, i64, vp, vp, vp, vp, sz, vp]),
            ("moe_route_workspace", sz, [i64, i64, i64]),
            ("moe_route", i32, [vp, i32, i64, i64, i64, i64, u, vp, vp, vp, vp, vp, vp, sz, vp]),
            ("moe_gemm_w4a16", i32, [vp, vp, i64, i64, vp, vp, i64, i64, i64, i64, u, vp, i32, vp]),
            ("moe_gemm_w4a4", i32, [vp, vp, vp, vp, i64, i64, vp, vp, i64, i64, i64, i64, u, vp, i32, vp]),
            ("moe_combine", i32, [vp, i32, vp, vp, i64, vp, i64, i64, i64, vp, i32, vp]),
            ("lora_add_workspace", sz, [i64, i64, i64, i64]),
            ("lora_add", i32, [vp, i64, vp, i64, vp, vp, vp, i64, i64, vp, vp, i64, i64, i64, vp, i64, i32,
                               vp, sz, vp])):
        f = getattr(L, name)
        f.restype, f.argtypes = res, args
    return L


def test_header_declares_the_calls():
    assert {"group_rows", "group_rows_workspace", "moe_route", "moe_route_workspace", "moe_gemm_w4a16",
            "moe_gemm_w4a4", "moe_combine", "lora_add", "lora_add_workspace"} <= set(_declared())


def test_group_rows(lib):
    def run(ids=A, rows=100, groups=7, order=B, where=C, offsets=D, ws=0, wsb=0):
        return lib.group_rows(ids, rows, groups, order, where, offsets, ws, wsb, 0)
    for kw, status in ((dict(ids=0), QL_EINVAL), (dict(order=0), QL_EINVAL), (dict(where=0), QL_EINVAL),
                       (dict(offsets=0), QL_EINVAL), (dict(rows=-1), QL_EINVAL), (dict(groups=0), QL_ESHAPE),
                       (dict(groups=1025), QL_ESHAPE), (dict(rows=MOST + 1), QL_ESHAPE),
                       (dict(ids=A + 2), QL_EALIGN), (dict(offsets=D + 1), QL_EALIGN),
                       (dict(rows=0, offsets=0), QL_EINVAL)):
        assert run(**kw) == status, kw
    # one block's rows need no workspace; more need their blocks' counts
    assert lib.group_rows_workspace(1024, 1024) == 0
    need = lib.group_rows_workspace(1025, 7)
    assert need == 3 * 8 * 4
    assert run(rows=1025) == QL_EINVAL
    assert run(rows=1025, ws=E + 8, wsb=need) == QL_EALIGN
    assert run(rows=1025, ws=E, wsb=need - 1) == QL_EWORKSPACE
    # the counts stay small however many rows
    assert 0 < lib.group_rows_workspace(MOST, 1024) <= 256 * 1028 * 4
    for bad in ((-1, 7), (MOST + 1, 7), (2000, 0), (2000, 1025)):
        assert lib.group_rows_workspace(*bad) == 0


def test_route(lib):
    def run(x=A, dt=QF32, tokens=3, experts=8, stride=8, top_k=2, flags=1, ids=B, weights=C, order=D, where=E,
            offsets=A, ws=0, wsb=0):
        return lib.moe_route(x, dt, tokens, experts, stride, top_k, flags, ids, weights, order, where, offsets,
                             ws, wsb, 0)
    for kw, status in ((dict(x=0), QL_EINVAL), (dict(ids=0), QL_EINVAL), (dict(weights=0), QL_EINVAL),
                       (dict(order=0), QL_EINVAL), (dict(where=0), QL_EINVAL), (dict(offsets=0), QL_EINVAL),
                       (dict(flags=2), QL_EINVAL), (dict(tokens=-1), QL_EINVAL), (dict(dt=2), QL_EDTYPE),
                       (dict(top_k=0), QL_ESHAPE), (dict(top_k=9), QL_ESHAPE), (dict(stride=7), QL_ESHAPE),
                       (dict(experts=1025, stride=1025), QL_ESHAPE),
                       (dict(experts=100, stride=100, top_k=65), QL_ESHAPE),
                       (dict(tokens=MOST // 2 + 1), QL_ESHAPE), (dict(x=A + 2), QL_EALIGN),
                       (dict(dt=QBF16, x=A + 1), QL_EALIGN), (dict(weights=C + 2), QL_EALIGN),
                       (dict(tokens=600), QL_EINVAL)):
        assert run(**kw) == status, kw
    assert lib.moe_route_workspace(512, 8, 2) == 0 < lib.moe_route_workspace(513, 8, 2)
    assert lib.moe_route_workspace(MOST // 2 + 1, 8, 2) == 0 == lib.moe_route_workspace(5, 8, 65)


PRODUCTS = [(dict(x=0), QL_EINVAL), (dict(experts=0), QL_EINVAL), (dict(offsets=0), QL_EINVAL),
            (dict(y=0), QL_EINVAL), (dict(order=0), QL_EINVAL), (dict(flags=4), QL_EINVAL),
            (dict(pairs=-2), QL_EINVAL), (dict(n=-16), QL_EINVAL), (dict(dt=3), QL_EDTYPE),
            (dict(count=0), QL_ESHAPE), (dict(count=1025), QL_ESHAPE), (dict(top_k=0), QL_ESHAPE),
            (dict(top_k=65, pairs=65), QL_ESHAPE), (dict(pairs=5), QL_ESHAPE), (dict(n=40), QL_ESHAPE),
            (dict(n=48, flags=3), QL_ESHAPE), (dict(n=0), QL_ESHAPE), (dict(k=0), QL_ESHAPE),
            (dict(k=100), QL_ESHAPE), (dict(n=1 << 22, k=1024), QL_ESHAPE),
            (dict(pairs=(MOST // 2 + 1) * 2), QL_ESHAPE), (dict(step=-1), QL_EWORKSPACE),
            (dict(step=8), QL_EALIGN), (dict(x=A + 8), QL_EALIGN), (dict(experts=B + 8), QL_EALIGN),
            (dict(y=E + 4), QL_EALIGN), (dict(offsets=D + 2), QL_EALIGN), (dict(order=C + 2), QL_EALIGN),
            (dict(pairs=0, x=0, y=0, order=0, offsets=0, experts=0), QL_OK)]


@pytest.mark.parametrize("kw,status", PRODUCTS)
@pytest.mark.parametrize("name", ["moe_gemm_w4a16", "moe_gemm_w4a4"])
def test_products(lib, name, kw, status):
    a = dict(x=A, experts=B, count=6, order=C, offsets=D, pairs=8, top_k=2, n=64, k=256, flags=1, y=E, dt=QBF16)
    step = kw.get("step", 0)
    a.update({k: v for k, v in kw.items() if k != "step"})
    each = lib.repack_weights_bytes(1 if name == "moe_gemm_w4a16" else 0, 64, 256) + (-16 if step == -1 else step)
    first = [a["x"]] if name == "moe_gemm_w4a16" else [a["x"], B, C]
    assert getattr(lib, name)(*first, a["experts"], a["count"], each, a["order"], a["offsets"], a["pairs"],
                              a["top_k"], a["n"], a["k"], a["flags"], a["y"], a["dt"], 0) == status


def test_w4a4_operands(lib):
    each = lib.repack_weights_bytes(0, 64, 1 << 20)
    run = lib.moe_gemm_w4a4
    assert run(A, 0, C, B, 6, each, C, D, 8, 2, 64, 256, 1, E, 1, 0) == QL_EINVAL
    assert run(A, B, 0, B, 6, each, C, D, 8, 2, 64, 256, 1, E, 1, 0) == QL_EINVAL
    assert run(A, B + 8, C, B, 6, each, C, D, 8, 2, 64, 256, 1, E, 1, 0) == QL_EALIGN
    # codes past 31 bits of offset
    assert run(A, B, C, B, 6, each, C, D, 4096, 1, 64, 1 << 20, 1, E, 1, 0) == QL_ESHAPE


def test_combine(lib):
    def run(rows=A, xt=QBF16, where=B, offsets=C, experts=6, weights=D, tokens=3, top_k=2, n=64, out=E, ot=QBF16):
        return lib.moe_combine(rows, xt, where, offsets, experts, weights, tokens, top_k, n, out, ot, 0)
    for kw, status in ((dict(rows=0), QL_EINVAL), (dict(where=0), QL_EINVAL), (dict(offsets=0), QL_EINVAL),
                       (dict(weights=0), QL_EINVAL), (dict(out=0), QL_EINVAL), (dict(tokens=-1), QL_EINVAL),
                       (dict(n=-8), QL_EINVAL), (dict(xt=2), QL_EDTYPE), (dict(ot=-1), QL_EDTYPE),
                       (dict(n=60), QL_ESHAPE), (dict(experts=0), QL_ESHAPE), (dict(top_k=65), QL_ESHAPE),
                       (dict(tokens=MOST), QL_ESHAPE), (dict(rows=A + 8), QL_EALIGN),
                       (dict(out=E + 8), QL_EALIGN), (dict(where=B + 1), QL_EALIGN),
                       (dict(tokens=0, rows=0), QL_OK), (dict(n=0, out=0), QL_OK)):
        assert run(**kw) == status, kw


def test_lora(lib):
    need = lib.lora_add_workspace(200, 3, 16, 256)
    assert need and need % (200 * 16 * 4) == 0
    assert lib.lora_add_workspace(10, 3, 16, 256) == 0      # few rows: one launch

    def run(y=A, ys=64, x=B, xs=256, a=C, b=D, scale=0, adapters=3, rank=16, order=E, offsets=A, rows=200, n=64,
            k=256, out=B, os_=64, dt=QBF16, ws=C, wsb=need):
        return lib.lora_add(y, ys, x, xs, a, b, scale, adapters, rank, order, offsets, rows, n, k, out, os_, dt,
                            ws, wsb, 0)
    for kw, status in ((dict(y=0), QL_EINVAL), (dict(x=0), QL_EINVAL), (dict(a=0), QL_EINVAL),
                       (dict(b=0), QL_EINVAL), (dict(order=0), QL_EINVAL), (dict(offsets=0), QL_EINVAL),
                       (dict(out=0), QL_EINVAL), (dict(ws=0), QL_EINVAL), (dict(rows=-1), QL_EINVAL),
                       (dict(out=A, os_=72), QL_EINVAL), (dict(dt=2), QL_EDTYPE), (dict(adapters=0), QL_ESHAPE),
                       (dict(adapters=1025), QL_ESHAPE), (dict(rank=4), QL_ESHAPE), (dict(rank=20), QL_ESHAPE),
                       (dict(rank=136), QL_ESHAPE), (dict(rows=MOST + 1), QL_ESHAPE), (dict(n=40), QL_ESHAPE),
                       (dict(k=100), QL_ESHAPE), (dict(n=0), QL_ESHAPE), (dict(k=0), QL_ESHAPE),
                       (dict(ys=63), QL_ESHAPE), (dict(xs=255), QL_ESHAPE), (dict(os_=48), QL_ESHAPE),
                       (dict(ys=68), QL_EALIGN), (dict(xs=260), QL_EALIGN), (dict(dt=QF32, os_=66), QL_EALIGN),
                       (dict(y=A + 8), QL_EALIGN), (dict(x=B + 2), QL_EALIGN), (dict(scale=C + 2), QL_EALIGN),
                       (dict(ws=C + 8), QL_EALIGN), (dict(wsb=need - 1), QL_EWORKSPACE),
                       (dict(rows=MOST, n=1 << 24, ys=1 << 24, os_=1 << 24), QL_ESHAPE),
                       (dict(rows=0, y=0, x=0), QL_OK)):
        assert run(**kw) == status, kw
    for bad in ((0, 3, 16, 256), (10, 0, 16, 256), (10, 3, 12, 256), (10, 3, 136, 256), (10, 3, 16, 100)):
        assert lib.lora_add_workspace(*bad) == 0


MB = 1 << 20      # addresses that no call below reads


def test_outputs_that_share_bytes_with_inputs_are_refused(lib):
    """Refused whatever part is shared; each call has all else in order."""
    each = lib.repack_weights_bytes(1, 256, 256)
    for y, dt in ((64 * MB, QBF16), (64 * MB + 512, QBF16), (64 * MB - 512, QBF16), (64 * MB - 7 * 1024, QF32)):
        assert lib.moe_gemm_w4a16(64 * MB, A, 6, each, B, C, 8, 1, 256, 256, 1, y, dt, 0) == QL_EINVAL, (y, dt)
    each = lib.repack_weights_bytes(0, 256, 256)
    for y in (64 * MB, 64 * MB + 128 * 7, 80 * MB + 16 * 7):
        assert lib.moe_gemm_w4a4(64 * MB, 80 * MB, A, B, 6, each, B, C, 8, 1, 256, 256, 1, y, QBF16, 0) == QL_EINVAL
    for out in (64 * MB, 64 * MB + 5 * 128, 64 * MB - 2 * 128):
        assert lib.moe_combine(64 * MB, QBF16, B, C, 6, D, 3, 2, 64, out, QBF16, 0) == QL_EINVAL

    def lora(y=64 * MB, ys=256, x=80 * MB, xs=256, out=64 * MB, os_=256, dt=QBF16, n=256, rows=10):
        return lib.lora_add(y, ys, x, xs, A, B, 0, 3, 16, C, D, rows, n, 256, out, os_, dt, 0, 0, 0)
    for kw in (dict(x=64 * MB), dict(out=80 * MB), dict(out=80 * MB + 512 * 9), dict(out=80 * MB - 512 * 9 - 16),
               dict(out=64 * MB + 16), dict(out=64 * MB + 512), dict(out=64 * MB - 512),
               dict(out=64 * MB, y=64 * MB + 256, n=144, ys=256),              # half a column of the same rows
               dict(x=64 * MB + 256, xs=512, ys=512, os_=512),                 # columns 128 .. 255 are both's
               dict(x=64 * MB + 512 + 496, xs=512, ys=512, os_=512, n=512),    # wraps into the next row
               dict(x=64 * MB + 512, xs=264)):                                 # of two strides
        assert lora(**kw) == QL_EINVAL, kw


def test_more_blocks_than_a_launch_has_are_refused(lib):
    def run(pairs, n, k=4096, count=6):
        each = lib.repack_weights_bytes(1, n, k)
        return lib.moe_gemm_w4a16(64 * MB, A, count, each, B, C, pairs, 1, n, k, 1, 0, QBF16, 0)
    # y is missing, which is seen only where the sizes are in order
    for pairs, n, status in ((32 * 131072, 16384, QL_ESHAPE), (32 * 131064, 16384, QL_EINVAL),
                             (MOST, 8 * 512, QL_ESHAPE), (MOST, 7 * 512, QL_EINVAL)):
        assert run(pairs, n) == status, (pairs, n)


def test_w4a4_blocks_are_those_of_the_launch(lib):
    """Tiles of 64 places up to 256 rows of an expert on average, of 256 above."""
    def run(pairs, n, k=128, count=6, y=0):
        each = lib.repack_weights_bytes(0, n, k)
        return lib.moe_gemm_w4a4(64 * MB, A, B, A, count, each, C, D, pairs, 1, n, k, 1, y, QBF16, 0)
    # y is missing, which is seen only where the sizes are in order
    for pairs, n, count, status in ((MOST, 127 * 256, 6, QL_EINVAL), (MOST, 128 * 256, 6, QL_ESHAPE),
                                    (1 << 22, 32768, 6, QL_EINVAL), (1 << 22, 511 * 256, 6, QL_EINVAL),
                                    (1 << 22, 512 * 256, 6, QL_ESHAPE),
                                    (256 * 1024, 1637 * 256, 1024, QL_EINVAL),
                                    (256 * 1024, 1638 * 256, 1024, QL_ESHAPE),
                                    (256 * 1024 + 1, 4000 * 256, 1024, QL_EINVAL)):
        assert run(pairs, n, count=count) == status, (pairs, n, count)


def test_lora_sizes_are_those_of_memory(lib):
    """What a call's rows span is limited (2^47 bytes), not the blocks of a launch."""
    def run(rows, n=64, xs=128, ys=None, os_=None, dt=QBF16):
        ys = n if ys is None else ys
        return lib.lora_add(A, ys, B, xs, C, D, 0, 3, 16, E, A, rows, n, 128, 1 << 50, os_ or ys, dt, 1 << 49, 0, 0)
    # the workspace is too small, which is seen only where the sizes are in order
    for rows, kw, status in ((1 << 22, dict(n=32768), QL_EWORKSPACE), (MOST, dict(n=16384), QL_EWORKSPACE),
                             (MOST, dict(n=1 << 24), QL_ESHAPE),
                             (1 << 20, dict(xs=1 << 26), QL_EWORKSPACE), (1 << 20, dict(xs=(1 << 26) + 8), QL_ESHAPE),
                             (1 << 20, dict(ys=1 << 26), QL_EWORKSPACE), (1 << 20, dict(ys=(1 << 26) + 8), QL_ESHAPE),
                             (1 << 20, dict(ys=1 << 25, dt=QF32), QL_EWORKSPACE),
                             (1 << 20, dict(ys=(1 << 25) + 4, dt=QF32), QL_ESHAPE),
                             (1 << 20, dict(os_=(1 << 26) + 8), QL_ESHAPE),
                             (MOST, dict(xs=1 << 40), QL_ESHAPE), (MOST, dict(ys=1 << 40), QL_ESHAPE),
                             (1 << 20, dict(xs=1 << 62), QL_ESHAPE)):
        assert run(rows, **kw) == status, (rows, kw)


def test_plans_written_over_their_input_are_refused(lib):
    """Blocks read choices, and logits, that other blocks would have written over."""
    def group(order=2 * MB, where=3 * MB, offsets=4 * MB, rows=1000):
        return lib.group_rows(MB, rows, 7, order, where, offsets, 0, 0, 0)
    for kw in (dict(order=MB), dict(order=MB + 3996), dict(order=MB - 3996), dict(where=MB), dict(where=MB + 4),
               dict(offsets=MB + 400), dict(offsets=MB - 28)):
        assert group(**kw) == QL_EINVAL, kw

    def route(ids=2 * MB, weights=3 * MB, order=4 * MB, where=5 * MB, offsets=6 * MB, dt=QF32, stride=100):
        return lib.moe_route(MB, dt, 50, 100, stride, 4, 1, ids, weights, order, where, offsets, 0, 0, 0)
    end = MB + 4 * (49 * 100 + 100)
    for kw in (dict(ids=MB), dict(weights=MB), dict(weights=end - 4), dict(order=MB + 8), dict(where=MB - 796),
               dict(offsets=MB + 4000), dict(offsets=MB - 400), dict(ids=end, stride=101),
               dict(dt=QBF16, weights=MB + 2 * (49 * 100 + 98))):
        assert route(**kw) == QL_EINVAL, kw
