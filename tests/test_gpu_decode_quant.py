"""ddt_decode_attn_paged_quant against a plain 64-bit softmax over the cache's values.  Every row that is not a
prefix row holds NaN, so a read past a prefix, or of a page of another request, shows."""
import math

import numpy as np
import pytest
import torch

from tests import _quant as Q
from tree_speculative_decoding_02_gb300 import ddt, synth

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _case(workload, L, B, Hq, Hkv, d, lens, page, block, dtype, *, new=True, cap_rows=None, q_std=1.5, spread=0.0):
    g = synth.gen(workload, 82)
    c = Q.cache(workload, L, B, Hkv, d, lens, page, block, cap_rows=cap_rows, spread=spread)
    c.update(q=synth.normal((L, B, Hq, d), q_std, g=g, dtype=dtype), scale=1 / math.sqrt(d), k_new=None, v_new=None)
    if new:
        c["k_new"] = synth.normal((L, B, Hkv, d), g=g, dtype=dtype)
        c["v_new"] = synth.normal((L, B, Hkv, d), g=g, dtype=dtype)
    return c


def _args(c):
    k, v, ks, vs, table, lens = Q.to_gpu(c)
    new = [None if c[x] is None else c[x].cuda() for x in ("k_new", "v_new")]
    return (c["q"].cuda(), *new, k, v, ks, vs, table, lens)


def _run(c, **kw):
    r = ddt.ddt_decode_attn_paged_quant(*_args(c), scale=c["scale"], **kw)
    torch.cuda.synchronize()
    return r


def _check(c, r):
    f = lambda t: None if t is None else Q.f64(t)  # noqa: E731
    want, bound = Q.decode_ref(f(c["q"]), f(c["k_new"]), f(c["v_new"]), c, c["scale"], c["q"].dtype)
    got = Q.f64(r["o"])
    tol = bound + Q.HALF[r["o"].dtype] * (np.abs(want) + bound) + 1e-30
    err = np.abs(got - want)
    assert bool((err <= tol).all()), f"{np.nanmax(err / tol):.3g} of the tolerance, error {np.nanmax(err):.3g}"
    assert (r["status"].cpu() == 0).all()


# head groups 1 to 40 (in and across head blocks), page and block sizes of every kind, lengths 0, 1, tile and
# page edges
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hq,Hkv,d,page,block", [(24, 4, 256, 64, 16), (4, 4, 64, 16, 8), (16, 2, 128, 8, 8), (10, 2, 64, 32, 32),
                                                 (12, 1, 128, 192, 64), (6, 3, 256, 128, 128), (40, 1, 64, 64, 16),
                                                 (17, 1, 128, 256, 128), (34, 2, 256, 16, 16), (20, 1, 256, 64, 64)])
def test_matches_softmax(dtype, Hq, Hkv, d, page, block):
    lens = [0, 1, page, 127, 128, 129, 3 * page + 5, 700]
    c = _case(31, 2, len(lens), Hq, Hkv, d, lens, page, block, dtype, cap_rows=701)
    r = _run(c, out_dtype=F32)
    _check(c, r)
    # the rounded output is the fp32 one rounded
    assert torch.equal(_run(c, out_dtype=BF)["o"], r["o"].to(BF))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_blocks_of_different_scales(dtype, d):
    """Blocks whose values differ by powers of two up to some 2^16 (K's by less: scores stay finite)."""
    c = _case(32, 1, 3, 8, 2, d, [900, 300, 61], 32, 16, dtype, spread=4.0)
    c["ks"] = np.clip(c["ks"], 115, 123).astype(np.uint8)
    _check(c, _run(c, out_dtype=F32))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_blocks_of_zeros(dtype):
    """Byte 0: rows of zero, weights as any other row's; at a prefix's start, inside it and everywhere."""
    c = _case(33, 1, 3, 8, 2, 128, [300, 300, 40], 16, 16, dtype)
    for b, blocks in enumerate(([0, 1, 7], [3, 18], [0, 1, 2])):
        for i in blocks:
            pg = c["table"][b, i]
            n = min(16, c["lens"][b] - 16 * i)
            c["k"][:, pg, :, :n] = c["v"][:, pg, :, :n] = 0
            c["ks"][:, pg] = c["vs"][:, pg] = 0
    r = _run(c, out_dtype=F32)
    _check(c, r)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_without_a_new_row(dtype):
    """The prefix alone; a request with no rows gets zeros."""
    c = _case(34, 1, 3, 8, 2, 128, [0, 5, 300], 16, 16, dtype, new=False)
    r = _run(c, out_dtype=F32)
    assert (r["o"][:, 0] == 0).all()
    _check(c, r)


@pytest.mark.parametrize("dtype,n,d", [(BF, 40001, 128), (BF, 30011, 256), (BF, 50003, 64), (F32, 20011, 128)])
def test_long_prefix_is_split_and_joined(dtype, n, d):
    c = _case(35, 1, 2, 16, 2, d, [n, 77], 64, 16, dtype)
    _check(c, _run(c, out_dtype=F32))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 256])
def test_many_short_units(dtype, d):
    """More (layer, request, head) units than CTAs: several whole units a CTA, ragged, some empty."""
    lens = [(37 * i) % 400 if i % 5 else 0 for i in range(60)]
    c = _case(36, 3, 60, 10, 5, d, lens, 32, 32, dtype)
    _check(c, _run(c, out_dtype=F32))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_growing_maximum(dtype):
    """Keys whose scores climb far along the prefix (the scale byte of every page is larger) and fall: the
    references move, and earlier tiles are rescaled."""
    lens = [1500, 640]
    c = _case(37, 1, 2, 4, 2, 64, lens, 64, 64, dtype, q_std=1.0)
    for b, n in enumerate(lens):
        for i in range(-(-n // 64)):
            pg = c["table"][b, i]
            c["ks"][:, pg] = np.clip(c["ks"][:, pg].astype(int) + (i // 4 if b == 0 else 3 - i // 2), 1, 200)
    _check(c, _run(c, out_dtype=F32))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_value_scales_that_climb(dtype):
    """Values that grow by 2^5 a page: the weights' reference goes by score and scale together."""
    c = _case(38, 1, 1, 8, 1, 128, [640], 64, 64, dtype)
    for i in range(10):
        c["vs"][:, c["table"][0, i]] = 90 + 5 * i
    _check(c, _run(c, out_dtype=F32))
    for i in range(10):
        c["vs"][:, c["table"][0, i]] = 160 - 5 * i
    _check(c, _run(c, out_dtype=F32))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("first,rest", [(60, 140), (180, 100), (0, 47), (0, 207)])
def test_value_scales_far_apart(dtype, first, rest):
    """2^80 between blocks in one tile: sums keep every weight that counts (2^17 rows below 2^-38 are 2^-21 at most)."""
    c = _case(39, 1, 2, 8, 2, 64, [300, 40], 16, 16, dtype, new=False)
    c["vs"][:] = rest
    c["vs"][:, c["table"][:, 0]] = first
    if not first:
        c["v"][:, c["table"][:, 0]] = 0
    _check(c, _run(c, out_dtype=F32))


@pytest.mark.parametrize("first,rest", [(27, 247), (247, 27), (60, 141), (180, 99), (0, 208)])
def test_value_scales_too_far_apart(first, rest):
    """Farther apart than the sums reach: NaN, not a wrong value; a head without such blocks is as it was."""
    c = _case(40, 1, 2, 8, 2, 64, [300, 40], 16, 16, BF, new=False)
    want = _run(c, out_dtype=F32)["o"]
    c["vs"][:, :, 0] = rest
    head = slice(0, 1 if first else 8)  # a tile of zeros counts as 1
    c["vs"][:, c["table"][0, head], 0] = first
    if not first:
        c["v"][:, c["table"][0, head], 0] = 0
    r = _run(c, out_dtype=F32)
    assert r["status"].tolist() == [0, 0]
    assert torch.equal(r["o"][:, :, 4:], want[:, :, 4:])
    far = r["o"][:, 0, :4]
    if first:  # both in one tile
        assert torch.isnan(far).all()
    else:      # in two, which may be two CTAs': right there
        exact, bound = Q.decode_ref(Q.f64(c["q"]), None, None, c, c["scale"], BF)
        assert (torch.isnan(far).cpu().numpy() | (np.abs(Q.f64(far) - exact[:, 0, :4]) <= bound[:, 0, :4] + 1e-30)).all()
    # the other request has no such blocks; (with byte 247 it has values up to 448 * 2^120 = 2^128.8, past fp32: infinities)
    assert not torch.isnan(r["o"][:, 1]).any()
    assert rest == 247 or torch.isfinite(r["o"][:, 1]).all()


def test_non_finite():
    """A NaN code of a cached row, and a NaN or infinity of q, show in the heads that they enter and nowhere else."""
    c = _case(39, 1, 3, 8, 2, 64, [200, 200, 200], 16, 16, BF)
    want = _run(c)["o"].clone()
    c["k"][0, c["table"][0, 3], 1, 4, 9] = 0xFF
    c["v"][0, c["table"][1, 2], 0, 4, 9] = Q.NAN_CODE
    c["q"][0, 2, 5, 7] = float("inf")
    r = _run(c)
    nan = torch.isnan(r["o"][0])
    expect = torch.zeros_like(nan)
    expect[0, 4:] = True
    expect[1, :4, 9] = True
    expect[2, 5] = True
    assert torch.equal(nan, expect)
    assert torch.equal(r["o"][0][~expect], want[0][~expect]) and r["status"].tolist() == [0, 0, 0]


def test_statuses():
    """Lengths outside the cache and pages that do not exist: zeros and a status, beside requests that are right."""
    c = _case(40, 2, 6, 8, 2, 128, [100, 64, 64, 64, 64, 30], 16, 16, BF, cap_rows=112)
    good = _run(c)["o"].clone()
    a = list(_args(c))
    a[8] = torch.tensor([100, -1, 113, 64, 64, 30], dtype=torch.int32).cuda()
    a[7][3, 2], a[7][4, 0], a[7][5, 2] = -5, 1 << 20, 1 << 30   # the last is behind its request's prefix
    r = ddt.ddt_decode_attn_paged_quant(*a, scale=c["scale"])
    assert r["status"].tolist() == [0, 3, 3, 1, 1, 0]
    assert (r["o"][:, 1:5] == 0).all()
    assert torch.equal(r["o"][:, [0, 5]], good[:, [0, 5]])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_same_bits_and_shared_pages(dtype):
    """The same call gives the same bits, alone or with another beside it on a second stream; requests may share pages."""
    c = _case(41, 1, 4, 16, 2, 256, [5000, 1200, 5000, 3], 64, 16, dtype)
    a = _args(c)
    first = ddt.ddt_decode_attn_paged_quant(*a, scale=c["scale"])["o"].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = []
    for i in range(4):
        with torch.cuda.stream(side):
            outs.append(ddt.ddt_decode_attn_paged_quant(*a, scale=c["scale"])["o"])
        outs.append(ddt.ddt_decode_attn_paged_quant(*a, scale=c["scale"])["o"])
    torch.cuda.synchronize()
    assert all(torch.equal(o, first) for o in outs)
    # (request 2's rows may be cut elsewhere than request 0's: within the bound, not to the bit)
    c["table"][2] = c["table"][0]
    r = _run(c)
    assert torch.equal(r["o"][:, 0], first[:, 0])
    _check(c, r)


def test_captured_call_follows_the_lengths():
    """A captured call replayed with other lengths, and beside a second graph with a workspace of its own."""
    c = _case(42, 1, 3, 24, 4, 128, [2000, 900, 10], 64, 16, BF)
    a = list(_args(c))
    graphs = []
    for _ in range(2):
        ws = ddt.decode_attn_paged_quant_workspace(a[0], a[3], a[7])
        out = torch.empty_like(a[0])
        st = torch.empty(3, dtype=torch.int32, device="cuda")
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            ddt.ddt_decode_attn_paged_quant(*a, scale=c["scale"], out=out, status=st, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ddt.ddt_decode_attn_paged_quant(*a, scale=c["scale"], out=out, status=st, workspace=ws)
        graphs.append((g, out, st, ws))
    for lens in ([2000, 900, 10], [77, 0, 1999], [1, 2000, 500]):
        a[8].copy_(torch.tensor(lens, dtype=torch.int32))
        want = ddt.ddt_decode_attn_paged_quant(*a, scale=c["scale"])["o"]
        for g, out, st, _ in graphs:
            out.fill_(9.0)
            g.replay()
        torch.cuda.synchronize()
        # rows past a request's own prefix hold NaN codes: only lengths up to it are compared
        for b in range(3):
            if lens[b] <= c["lens"][b]:
                assert torch.equal(graphs[0][1][:, b], want[:, b]) and torch.equal(graphs[1][1][:, b], want[:, b])
