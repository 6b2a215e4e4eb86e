"""Argument refusals of the 8-bit cache's calls and of the norm and rotation of heads, on the host before any
launch (no GPU needed): the pointers below are never dereferenced."""
import ctypes

import pytest

from tests.test_serving_overlaps import _check
from tests.test_serving_refusals import INVALID, ODD, UNSUPPORTED, lib, pytestmark  # noqa: F401

at = ctypes.c_void_p


def _apart(names, start):
    return {n: at(start + (i << 32)) for i, n in enumerate(names)}


def _append(lib, **kw):  # noqa: F811
    a = dict(L=1, B=2, N=8, A=8, Hkv=2, d=64, page=16, num=10, mp=4, S=8, it=1, adv=1,
             **_apart(("k", "v", "node", "cnt", "tab", "plen", "kp", "vp", "ks", "vs", "st"), 1 << 40))
    a.update(kw)
    return lib.ddt_append_paged_quant(*(a[x] for x in ("L", "B", "N", "A", "Hkv", "d", "page", "num", "mp", "S", "it", "k", "v", "node",
                                                       "cnt", "tab", "plen", "adv", "kp", "vp", "ks", "vs", "st")), None)


def _read(lib, **kw):  # noqa: F811
    a = dict(L=1, B=2, Hkv=2, d=64, Pcap=64, page=16, num=10, mp=4, S=8, ot=1,
             **_apart(("kp", "vp", "ks", "vs", "tab", "plen", "ko", "vo", "st"), 1 << 40))
    a.update(kw)
    return lib.ddt_read_paged_quant(*(a[x] for x in ("L", "B", "Hkv", "d", "Pcap", "page", "num", "mp", "S", "ot", "kp", "vp", "ks",
                                                     "vs", "tab", "plen", "ko", "vo", "st")), None)


def _decode(lib, **kw):  # noqa: F811
    a = dict(L=1, B=2, Hq=8, Hkv=2, d=64, page=16, num=10, mp=4, S=8, it=1, ot=1, scale=1.0, n=1 << 30,
             **_apart(("q", "kn", "vn", "kp", "vp", "ks", "vs", "tab", "plen", "o", "st", "ws"), 1 << 40))
    a.update(kw)
    return lib.ddt_decode_attn_paged_quant(*(a[x] for x in ("L", "B", "Hq", "Hkv", "d", "page", "num", "mp", "S", "it", "ot", "q", "kn",
                                                            "vn", "kp", "vp", "ks", "vs", "tab", "plen", "scale", "o", "st", "ws",
                                                            "n")), None)


def _strides(*x):
    return (ctypes.c_int64 * 4)(*x)


def _norm(lib, **kw):  # noqa: F811
    a = dict(L=1, B=2, N=5, Hq=8, Hkv=2, d=64, rot=32, theta=1e4, eps=1e-6, off=0.0, dt=1, qs=_strides(5120, 2560, 512, 64),
             ks=_strides(1280, 640, 128, 64), **_apart(("q", "k", "qw", "kw", "pos", "nn", "qo", "ko"), 1 << 40))
    a.update(kw)
    return lib.ddt_qk_norm_rope(*(a[x] for x in ("L", "B", "N", "Hq", "Hkv", "d", "rot", "theta", "eps", "off", "dt", "q", "qs", "k", "ks",
                                                 "qw", "kw", "pos", "nn", "qo", "ko")), None)


def test_append(lib):  # noqa: F811
    before = lib.ddt_launch_count()
    for kw in (dict(L=0), dict(B=0), dict(N=0), dict(A=0), dict(Hkv=0), dict(num=0), dict(mp=0), dict(it=2), dict(node=None, A=9),
               *(dict([(x, None)]) for x in ("k", "v", "cnt", "tab", "plen", "kp", "vp", "ks", "vs", "st")),
               *(dict([(x, ODD)]) for x in ("k", "v", "kp", "vp"))):
        assert _append(lib, **kw) == INVALID, kw
    for kw in (dict(d=96), dict(page=12), dict(page=100), dict(S=4), dict(S=12), dict(S=32), dict(S=256, page=256), dict(mp=1 << 27),
               dict(num=1 << 30), dict(A=1025), dict(L=300, B=300), dict(page=192, S=128)):
        assert _append(lib, **kw) == UNSUPPORTED, kw
    assert lib.ddt_launch_count() == before


def test_read(lib):  # noqa: F811
    before = lib.ddt_launch_count()
    for kw in (dict(L=0), dict(B=0), dict(Hkv=0), dict(Pcap=0), dict(num=0), dict(mp=0), dict(ot=5),
               *(dict([(x, None)]) for x in ("kp", "vp", "ks", "vs", "tab", "plen", "ko", "vo", "st")),
               *(dict([(x, ODD)]) for x in ("kp", "vp", "ko", "vo"))):
        assert _read(lib, **kw) == INVALID, kw
    for kw in (dict(d=80), dict(page=24), dict(S=2), dict(S=24, page=192), dict(L=300, B=300), dict(mp=1 << 27), dict(num=1 << 30)):
        assert _read(lib, **kw) == UNSUPPORTED, kw
    assert lib.ddt_launch_count() == before


def test_decode(lib):  # noqa: F811
    before = lib.ddt_launch_count()
    small = lib.ddt_decode_attn_paged_quant_workspace(1, 2, 8, 2, 64, 1)
    assert small > 0
    for kw in (dict(L=0), dict(B=0), dict(Hq=7), dict(Hq=0), dict(Hkv=0), dict(num=0), dict(mp=0), dict(it=2), dict(ot=-1),
               *(dict([(x, None)]) for x in ("q", "kn", "vn", "kp", "vp", "ks", "vs", "tab", "plen", "o", "st", "ws")),
               *(dict([(x, ODD)]) for x in ("q", "kn", "vn", "kp", "vp", "o", "ws")), dict(n=small - 1)):
        assert _decode(lib, **kw) == INVALID, kw
    for kw in (dict(d=96), dict(page=12), dict(page=8192), dict(S=1), dict(S=48, page=192), dict(mp=1 << 27), dict(num=1 << 30),
               dict(Hq=1 << 12, Hkv=1), dict(L=1 << 20, B=1 << 20)):
        assert _decode(lib, **kw) == UNSUPPORTED, kw
    assert lib.ddt_launch_count() == before
    assert lib.ddt_decode_attn_paged_quant_workspace(1, 2, 7, 2, 64, 1) == 0
    assert lib.ddt_decode_attn_paged_quant_workspace(1, 2, 8, 2, 64, 7) == 0


def test_norm(lib):  # noqa: F811
    before = lib.ddt_launch_count()
    inf, nan = float("inf"), float("nan")
    for kw in (dict(L=0), dict(B=0), dict(N=0), dict(Hq=0), dict(Hkv=0), dict(dt=3), dict(rot=-16), dict(rot=80), dict(theta=1.0),
               dict(theta=nan), dict(theta=inf), dict(eps=-1e-6), dict(eps=nan), dict(eps=inf), dict(off=nan), dict(off=inf),
               *(dict([(x, None)]) for x in ("q", "k", "qs", "ks", "qw", "kw", "pos", "qo", "ko")),
               *(dict([(x, at(257))]) for x in ("q", "k", "qw", "kw", "qo", "ko")), dict(qs=_strides(5120, 2560, -512, 64))):
        assert _norm(lib, **kw) == INVALID, kw
    for kw in (dict(d=80), dict(rot=8), dict(rot=24), dict(L=70000), dict(B=1 << 16, N=1 << 16), dict(qs=_strides(5120, 1 << 60, 512, 64)),
               dict(ks=_strides(1280, 640, 128, 1 << 30)), dict(qs=_strides(5120, 2560, 512, 107374177))):
        assert _norm(lib, **kw) == UNSUPPORTED, kw
    # in place over rows that lie otherwise than the output's
    q = at(1 << 36)
    assert _norm(lib, q=q, qo=q, qs=_strides(5120, 2560, 640, 64)) == INVALID
    assert _norm(lib, q=q, qo=at((1 << 36) + 16)) == INVALID
    assert lib.ddt_launch_count() == before


@pytest.mark.parametrize("node", [True, False])
def test_append_buffers_that_overlap(lib, node):  # noqa: F811
    L, B, N, A, Hkv, d, page, num, mp, S = 2, 4, 5, 5, 2, 64, 16, 10, 4, 8
    rows, pool = L * B * N * Hkv * d * 2, L * num * Hkv * page
    sizes = dict(kp=pool * d, vp=pool * d, ks=pool // S, vs=pool // S, st=4 * B, plen=4 * B, k=rows, v=rows, cnt=4 * B, tab=4 * B * mp)
    more = dict(L=L, B=B, N=N, A=A, Hkv=Hkv, d=d, page=page, num=num, mp=mp, S=S)
    if node:
        sizes["node"] = 4 * B * A
    else:
        more["node"] = None
    before = lib.ddt_launch_count()
    _check(lambda **kw: _append(lib, **kw), sizes, ("kp", "vp", "ks", "vs", "st", "plen"), more)
    assert lib.ddt_launch_count() == before


def test_read_and_decode_buffers_that_overlap(lib):  # noqa: F811
    L, B, Hq, Hkv, d, page, num, mp, S, Pcap = 2, 4, 4, 2, 64, 16, 10, 4, 8, 48
    pool = L * num * Hkv * page
    cache = dict(kp=pool * d, vp=pool * d, ks=pool // S, vs=pool // S, tab=4 * B * mp, plen=4 * B)
    before = lib.ddt_launch_count()
    out = L * B * Hkv * Pcap * d * 2
    _check(lambda **kw: _read(lib, **kw), dict(ko=out, vo=out, st=4 * B, **cache), ("ko", "vo", "st"),
           dict(L=L, B=B, Hkv=Hkv, d=d, Pcap=Pcap, page=page, num=num, mp=mp, S=S))
    ws = lib.ddt_decode_attn_paged_quant_workspace(L, B, Hq, Hkv, d, 1)
    _check(lambda **kw: _decode(lib, **kw),
           dict(o=L * B * Hq * d * 2, st=4 * B, ws=ws, q=L * B * Hq * d * 2, kn=L * B * Hkv * d * 2, vn=L * B * Hkv * d * 2, **cache),
           ("o", "st", "ws"), dict(L=L, B=B, Hq=Hq, Hkv=Hkv, d=d, page=page, num=num, mp=mp, S=S))
    assert lib.ddt_launch_count() == before


def test_norm_buffers_that_overlap(lib):  # noqa: F811
    L, B, N, Hq, Hkv, d = 2, 3, 4, 4, 2, 64
    nq, nk = L * B * N * Hq * d * 2, L * B * N * Hkv * d * 2
    sizes = dict(qo=nq, ko=nk, qw=L * d * 2, kw=L * d * 2, pos=4 * B * N, nn=4 * B)
    more = dict(L=L, B=B, N=N, Hq=Hq, Hkv=Hkv, d=d, qs=_strides(B * N * Hq * d, N * Hq * d, Hq * d, d),
                ks=_strides(B * N * Hkv * d, N * Hkv * d, Hkv * d, d), q=at(1 << 44), k=at(1 << 45))
    before = lib.ddt_launch_count()
    _check(lambda **kw: _norm(lib, **{**more, **kw}), sizes, ("qo", "ko"), {})
    # outputs over inputs that are not theirs, or lie across them
    for kw in (dict(qo=at(1 << 45)), dict(ko=at(1 << 44)), dict(qo=at((1 << 44) + 16)), dict(ko=at((1 << 45) - 16))):
        assert _norm(lib, **{**more, **kw}) == INVALID, kw
    assert lib.ddt_launch_count() == before
