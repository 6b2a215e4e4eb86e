"""Buffers that a single-token call would read, or write again, after it has begun to write them
are refused on the host (no GPU needed: the pointers are never dereferenced)."""
import ctypes
import itertools

import pytest

from tests.test_serving_refusals import INVALID, _decode, _evict, _logprobs, lib, pytestmark  # noqa: F401

at = ctypes.c_void_p


def _apart(sizes):
    """Places for buffers of these bytes, each directly behind the one before (to 16 bytes)."""
    places, x = {}, 1 << 30
    for name, n in sizes.items():
        places[name] = x
        x += (n + 15) // 16 * 16
    return places


def _check(call, sizes, outputs, more):
    """Every output over every other buffer: its last 16 bytes over the other's first, the same place,
    and its first bytes over the other's last."""
    places = _apart(sizes)
    for out, other in itertools.product(outputs, sizes):
        if out == other:
            continue
        y, n, m = places[other], sizes[out], sizes[other]
        for x in {y, y - (n - 1) // 16 * 16, y + (m - 1) // 16 * 16}:
            kw = {k: at(v) for k, v in places.items()}
            kw[out] = at(x)
            assert call(**kw, **more) == INVALID, (out, other, x - y)


@pytest.mark.parametrize("G", [1, 4])
def test_decode(lib, G):  # noqa: F811
    L, B, Hkv, d, page, mp = 2, 4, 2, 64, 16, 4
    Hq = G * Hkv
    ws = lib.ddt_decode_attn_paged_workspace(L, B, Hq, Hkv, d, page, mp, 1, 1)
    sizes = dict(o=L * B * Hq * d * 2, w=L * B * Hkv * page * mp * 4, st=4 * B, ws=ws, q=L * B * Hq * d * 2,
                 kn=L * B * Hkv * d * 2, vn=L * B * Hkv * d * 2, tab=4 * B * mp, plen=4 * B)
    before = lib.ddt_launch_count()
    _check(lambda **kw: _decode(lib, **kw), sizes, ("o", "w", "st", "ws"), dict(L=L, B=B, Hq=Hq, Hkv=Hkv, d=d, page=page, mp=mp))
    assert lib.ddt_launch_count() == before


def test_evict(lib):  # noqa: F811
    L, B, Hkv, page, mp = 2, 4, 2, 16, 4
    rows = L * B * Hkv * page * mp * 4
    sizes = dict(w=rows, pos=rows, plen=4 * B, np=4 * B, st=4 * B, ws=lib.ddt_evict_paged_workspace(L, B, Hkv, page, 10, mp),
                 tab=4 * B * mp, seq=4 * B)
    before = lib.ddt_launch_count()
    _check(lambda **kw: _evict(lib, **kw), sizes, ("w", "pos", "plen", "np", "st", "ws"),
           dict(L=L, B=B, Hkv=Hkv, page=page, mp=mp))
    pool = L * 10 * Hkv * page * 64 * 2
    places = {k: at(v) for k, v in _apart({**sizes, "kp": pool, "vp": pool}).items()}
    for x in (16, pool - 16, 16 - pool):
        places["vp"] = at(places["kp"].value + x)
        assert _evict(lib, **places, L=L, B=B, Hkv=Hkv, page=page, mp=mp) == INVALID, x
    assert lib.ddt_launch_count() == before


def test_logprobs(lib):  # noqa: F811
    B, N, V, A, top = 3, 5, 200, 4, 6
    n = 4 * B * A
    sizes = dict(lp=n, en=n, tt=n * top, tl=n * top, st=n, ws=lib.ddt_token_logprobs_workspace(B, A, V, top), x=B * N * V * 2,
                 node=n, tok=n)
    before = lib.ddt_launch_count()
    _check(lambda **kw: _logprobs(lib, **kw), sizes, ("lp", "en", "tt", "tl", "st", "ws"), dict(B=B, N=N, V=V, A=A, top=top))
    assert lib.ddt_launch_count() == before
