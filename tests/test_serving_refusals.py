"""Argument refusals of the single-token attention, eviction and log-probability calls, on the
host before any launch (no GPU needed): the pointers below are never dereferenced."""
import ctypes
import os
import shutil

import pytest

from tree_speculative_decoding_02_gb300 import ddt

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="nvcc not available")

OK, INVALID, UNSUPPORTED = 0, 1, 2
P, ODD = ctypes.c_void_p(256), ctypes.c_void_p(264)   # 16-byte aligned, and not
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    return ddt.load()


def _decode(lib, **kw):
    a = dict(L=1, B=2, Hq=8, Hkv=2, d=64, page=16, num=10, mp=4, it=1, ot=1, q=P, kn=P, vn=P, kp=P, vp=P, tab=P, plen=P,
             scale=1.0, o=P, w=None, st=P, ws=P, n=BIG)
    a.update(kw)
    return lib.ddt_decode_attn_paged(*(a[k] for k in ("L", "B", "Hq", "Hkv", "d", "page", "num", "mp", "it", "ot", "q", "kn",
                                                      "vn", "kp", "vp", "tab", "plen", "scale", "o", "w", "st", "ws", "n")),
                                     None)


def _evict(lib, **kw):
    a = dict(L=1, B=2, Hkv=2, d=64, page=16, num=10, mp=4, tab=P, dt=1, keep=8, sink=1, recent=2, kp=P, vp=P, seq=P, w=P,
             pos=P, plen=P, np=P, st=P, ws=P, n=BIG)
    a.update(kw)
    return lib.ddt_evict_paged(*(a[k] for k in ("L", "B", "Hkv", "d", "page", "num", "mp", "tab", "dt", "keep", "sink", "recent",
                                                "kp", "vp", "seq", "w", "pos", "plen", "np", "st", "ws", "n")), None)


def _logprobs(lib, **kw):
    a = dict(B=2, N=5, V=100, A=3, top=4, T=1.0, dt=1, x=P, node=P, tok=P, lp=P, en=P, tt=P, tl=P, st=P, ws=P, n=BIG)
    a.update(kw)
    return lib.ddt_token_logprobs(*(a[k] for k in ("B", "N", "V", "A", "top", "T", "dt", "x", "node", "tok", "lp", "en", "tt",
                                                   "tl", "st", "ws", "n")), None)


def test_decode(lib):
    before = lib.ddt_launch_count()
    for kw in (dict(L=0), dict(B=0), dict(Hq=7), dict(Hq=0), dict(Hkv=0), dict(num=0), dict(mp=0), dict(it=2), dict(ot=-1),
               dict(q=None), dict(kp=None), dict(vp=None), dict(tab=None), dict(plen=None), dict(o=None), dict(st=None),
               dict(ws=None), dict(kn=None), dict(vn=None), dict(n=64), dict(q=ODD), dict(kp=ODD), dict(vn=ODD), dict(o=ODD),
               dict(ws=ODD), dict(w=ODD)):
        assert _decode(lib, **kw) == INVALID, kw
    for kw in (dict(d=96), dict(page=12), dict(page=100), dict(page=8192), dict(mp=1 << 27), dict(num=1 << 30),
               dict(Hq=1 << 12, Hkv=1), dict(L=1 << 20, B=1 << 20)):
        assert _decode(lib, **kw) == UNSUPPORTED, kw
    # a workspace without room for the scores of the weights
    small = lib.ddt_decode_attn_paged_workspace(1, 2, 8, 2, 64, 16, 4, 1, 0)
    assert 0 < small < lib.ddt_decode_attn_paged_workspace(1, 2, 8, 2, 64, 16, 4, 1, 1)
    assert _decode(lib, w=P, n=small) == INVALID
    assert lib.ddt_launch_count() == before
    assert lib.ddt_decode_attn_paged_workspace(1, 2, 7, 2, 64, 16, 4, 1, 0) == 0
    assert lib.ddt_decode_attn_paged_workspace(1, 2, 8, 2, 64, 12, 4, 1, 0) == 0


def test_evict(lib):
    before = lib.ddt_launch_count()
    for kw in (dict(L=0), dict(B=0), dict(Hkv=0), dict(d=0), dict(num=0), dict(mp=0), dict(dt=7), dict(keep=0), dict(sink=-1),
               dict(recent=-1), dict(sink=6, recent=3), dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1), dict(tab=None), dict(kp=None),
               dict(vp=None), dict(seq=None), dict(w=None), dict(pos=None), dict(plen=None), dict(np=None), dict(st=None),
               dict(ws=None), dict(n=100), dict(kp=ODD), dict(vp=ODD), dict(w=ODD), dict(pos=ODD), dict(ws=ODD)):
        assert _evict(lib, **kw) == INVALID, kw
    for kw in (dict(page=24), dict(d=7), dict(d=12), dict(d=1 << 20), dict(num=1 << 28), dict(mp=1 << 27)):
        assert _evict(lib, **kw) == UNSUPPORTED, kw
    assert lib.ddt_launch_count() == before
    assert lib.ddt_evict_paged_workspace(1, 2, 2, 24, 10, 4) == 0
    assert lib.ddt_evict_paged_workspace(1, 2, 2, 16, 10, 4) > 0


def test_logprobs(lib):
    before = lib.ddt_launch_count()
    for kw in (dict(B=0), dict(N=0), dict(V=0), dict(A=0), dict(top=-1), dict(dt=5), dict(T=0.0), dict(T=-1.0),
               dict(T=float("nan")), dict(T=float("inf")), dict(T=1e-40), dict(node=None), dict(x=None), dict(tok=None),
               dict(lp=None), dict(st=None), dict(ws=None), dict(tt=None), dict(tl=None), dict(n=64), dict(ws=ODD),
               dict(x=ctypes.c_void_p(257))):
        assert _logprobs(lib, **kw) == INVALID, kw
    for kw in (dict(top=33), dict(top=4, V=3), dict(V=(1 << 30) + 1), dict(B=1 << 15, A=1 << 15, V=1 << 20)):
        assert _logprobs(lib, **kw) == UNSUPPORTED, kw
    assert lib.ddt_launch_count() == before
    assert lib.ddt_token_logprobs_workspace(0, 3, 100, 4) == 0
    assert lib.ddt_token_logprobs_workspace(2, 3, 100, 4) > lib.ddt_token_logprobs_workspace(2, 3, 100, 0) > 0


def test_buffers_that_overlap(lib):
    """o over q, and the three lengths of an eviction in one array (seq_len would be cut with prefix_len)."""
    before = lib.ddt_launch_count()
    at = lambda x: ctypes.c_void_p(x)  # noqa: E731
    q = 4096                                               # 2 * 8 * 64 bf16: 2048 bytes
    for o in (q, q + 2032, q - 2032):
        assert _decode(lib, q=at(q), o=at(o)) == INVALID
    assert _decode(lib, q=at(q), o=at(q - 2048), ot=0) == INVALID
    for kw in (dict(seq=P, plen=P, np=at(512)), dict(seq=at(512), plen=P, np=P), dict(seq=P, plen=at(512), np=P),
               dict(seq=P, plen=at(260), np=at(512))):
        assert _evict(lib, **kw) == INVALID, kw
    assert lib.ddt_launch_count() == before
