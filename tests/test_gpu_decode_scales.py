"""ddt_decode_attn_paged_quant where V's blocks have scales far from one another: neither a block's scale nor a block
of zeros costs the rows of other blocks their weights, in the sums or in any channel."""
import math

import numpy as np
import pytest
import torch

from tests import _quant as Q
from tests.test_gpu_decode_quant import _args, _case, _run
from tree_speculative_decoding_02_gb300 import ddt

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
NEAR = 2.0 ** 8     # blocks whose rows go through the products together are at most this far apart


def _want(c):
    """o in 64 bits and the bound on its error: decode_ref's, whose floor of 2^-26 (fp32: 2^-34) of the largest weight is
    one of the largest product of weight and scale, so up to NEAR times that of a row of a smaller scale.  A channel's
    error counts the rows by their values in that channel alone."""
    f = lambda t: None if t is None else Q.f64(t)  # noqa: E731
    o, bound = Q.decode_ref(f(c["q"]), f(c["k_new"]), f(c["v_new"]), c, c["scale"], c["q"].dtype)
    floor = NEAR * (2.0 ** -26 if c["q"].dtype == BF else 2.0 ** -34)
    L, B, Hq, _ = c["q"].shape
    Hkv = c["k"].shape[2]
    G = Hq // Hkv
    for b, n in enumerate(c["lens"]):
        K, V = (Q.rows_of(c[x], c[x + "s"], c["table"], b, n) for x in "kv")
        for l in range(L):
            for g in range(Hkv if n else 0):
                at = slice(g * G, (g + 1) * G)
                s = Q.f64(c["q"])[l, b, at] @ K[l, g].T * c["scale"]
                if c["k_new"] is not None:
                    mine = Q.f64(c["q"])[l, b, at] @ Q.f64(c["k_new"])[l, b, g] * c["scale"]
                    s = np.concatenate([s, mine[:, None]], axis=1)
                p = np.exp(s - s.max(axis=1, keepdims=True))
                p /= p.sum(axis=1, keepdims=True)
                bound[l, b, at] += 2.2 * floor * p[:, :n].max(axis=1, keepdims=True) * np.abs(V[l, g]).sum(axis=0)
    return o, bound


def _check(c, r, heads=slice(None)):
    want, bound = _want(c)
    got = Q.f64(r["o"])
    tol = bound + Q.HALF[r["o"].dtype] * (np.abs(want) + bound) + 1e-30
    ok = np.abs(got - want) <= tol
    assert ok[:, :, heads].all(), f"{np.nanmax((np.abs(got - want) / tol)[:, :, heads]):.3g} of the tolerance, {np.isnan(got).sum()} NaN"
    assert (r["status"].cpu() == 0).all()


def _blocks(c, b):
    """(page, block in it) of request b's blocks, in order."""
    per = c["page"] // c["block"]
    return [(c["table"][b, i // per], i % per) for i in range(-(-c["lens"][b] // c["block"]))]


def _set(c, at, byte, channel=None, zero=False):
    """A block's scale in all layers and heads; its values in one channel only, or nowhere."""
    pg, i = at
    c["vs"][:, pg, :, i] = byte
    v = c["v"][:, pg, :, i * c["block"]:(i + 1) * c["block"]]      # [L][Hkv][block][d]
    live = (v & 0x7F) != Q.NAN_CODE
    if zero:
        v[live] = 0
    elif channel is not None:
        live[..., channel] = False
        v[live] = 0


SHAPES = [(4, 2, 64, 16, 8), (8, 2, 128, 16, 16), (16, 2, 256, 64, 64), (24, 2, 64, 32, 32), (24, 1, 128, 128, 128), (24, 1, 256, 16, 16),
          (40, 1, 128, 64, 16), (3, 3, 128, 8, 8)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("up", [5, 9, 20, 36])
@pytest.mark.parametrize("Hq,Hkv,d,page,block", SHAPES)
def test_a_large_block_in_one_channel(Hq, Hkv, d, page, block, up, dtype):
    """One block has a single large channel and zeros elsewhere: the other channels are the other rows' mean."""
    lens = [700, 129, 61, 300]
    c = _case(51, 1, 4, Hq, Hkv, d, lens, page, block, dtype)
    c["vs"][:] = 120
    for b, i in enumerate((1, 0, 0, -1)):
        at = _blocks(c, b)
        _set(c, at[i % len(at)], 120 + up, channel=5 * b)
    _check(c, _run(c, out_dtype=F32))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hq,Hkv,d,page,block", SHAPES)
def test_scales_of_every_size(Hq, Hkv, d, page, block, dtype):
    """Blocks up to 2^78 from one another at random places, whole or in one channel, among blocks of zeros, while the keys'
    scales climb, so that references move with sums of far blocks behind them."""
    lens = [1500, 640, 77, 1, 0, 256]
    c = _case(52, 2, 6, Hq, Hkv, d, lens, page, block, dtype, q_std=1.0)
    c["vs"][:] = 120
    r = np.random.default_rng(7)
    for b in range(6):
        for i, at in enumerate(_blocks(c, b)):
            c["ks"][:, at[0], :, at[1]] = 116 + min(6, i * block // 128) if b % 2 == 0 else 122 - min(6, i * block // 128)
            if (x := r.random()) < 0.3:
                _set(c, at, 120 + int(r.integers(-39, 40)), channel=int(r.integers(d)) if x < 0.2 else None)
            elif x < 0.4:
                _set(c, at, 0, zero=True)
    _check(c, _run(c, out_dtype=F32))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("byte", [40, 47, 60, 124, 130, 194, 201, 202, 207, 230])
def test_a_tile_of_zeros_counts_in_the_sums(byte, dtype):
    """The first 128 rows are zeros, the others of one scale, several tiles of a request in one CTA: the zeros' weights
    stay in the sums."""
    B, Hkv = 200, 4
    lens = [300 + b % 3 for b in range(B)]
    c = _case(53, 1, B, 2 * Hkv, Hkv, 64, lens, 16, 16, dtype, new=False, q_std=0.1)
    c["vs"][:] = byte
    for b in range(B):
        for at in _blocks(c, b)[:8]:
            _set(c, at, 0, zero=True)
    _check(c, _run(c, out_dtype=F32))


@pytest.mark.parametrize("bytes_", [(127, 57, 197), (127, 197, 57), (127, 82, 172), (87, 127, 168)])
def test_far_apart_on_both_sides_of_the_first(bytes_):
    """Two blocks more than 2^80 apart give NaN, also where neither is that far from the first one."""
    c = _case(54, 1, 2, 8, 2, 64, [100, 100], 16, 16, BF, new=False)
    c["vs"][:] = 120
    for at, byte in zip(_blocks(c, 0), bytes_):
        c["vs"][:, at[0], 0, at[1]] = byte
    r = _run(c, out_dtype=F32)
    assert torch.isnan(r["o"][:, 0, :4]).all()
    c["lens"] = [0, 100]                                            # the bound of what is left
    o, bound = _want(c)
    assert (np.abs(Q.f64(r["o"]) - o)[:, 1] <= bound[:, 1] + 1e-30).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("bytes_", [(127, 87, 167), (167, 127, 87), (127, 167, 87, 0, 127)])
def test_as_far_apart_as_is_allowed(bytes_, dtype):
    c = _case(55, 1, 2, 8, 2, 64, [100, 400], 16, 16, dtype)
    for b in range(2):
        for i, at in enumerate(_blocks(c, b)):
            byte = bytes_[i % len(bytes_)]
            _set(c, at, byte, channel=i % 64 if byte > 127 else None, zero=not byte)
    _check(c, _run(c, out_dtype=F32))


def test_non_finite_in_a_far_block():
    """A NaN code of a far block shows in its channel, a NaN of K in its kv head, and nowhere else."""
    c = _case(56, 1, 3, 8, 2, 64, [200, 200, 200], 16, 16, BF)
    for b in range(3):
        c["vs"][:, c["table"][b, 2]] = 150
    want = _run(c)["o"].clone()
    c["v"][0, c["table"][0, 2], 1, 4, 9] = Q.NAN_CODE
    c["k"][0, c["table"][1, 2], 0, 4, 9] = Q.NAN_CODE
    r = _run(c)
    nan = torch.isnan(r["o"][0])
    expect = torch.zeros_like(nan)
    expect[0, 4:, 9] = True
    expect[1, :4] = True
    assert torch.equal(nan, expect)
    assert torch.equal(r["o"][0][~expect], want[0][~expect]) and r["status"].tolist() == [0, 0, 0]


def test_pages_that_do_not_exist():
    """A request with a bad page among far blocks gets zeros and a status; the others are as they were."""
    c = _case(57, 1, 3, 12, 1, 128, [300, 300, 300], 16, 16, BF)
    for b in range(3):
        c["vs"][:, c["table"][b, 5]] = 150
    want = _run(c)["o"].clone()
    a = list(_args(c))
    a[7][1, 4] = -1
    r = ddt.ddt_decode_attn_paged_quant(*a, scale=c["scale"])
    assert r["status"].tolist() == [0, 1, 0] and (r["o"][:, 1] == 0).all()
    assert torch.equal(r["o"][:, [0, 2]], want[:, [0, 2]])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_same_bits_with_far_blocks(dtype):
    """Any workspace, and a replayed call: the same bits."""
    c = _case(58, 1, 40, 16, 4, 128, [(53 * i) % 700 for i in range(40)], 32, 16, dtype)
    c["vs"][:, ::5] = 150
    c["vs"][:, 2::7] = 90
    a = _args(c)
    ws = ddt.decode_attn_paged_quant_workspace(a[0], a[3], a[7])
    ws.zero_()
    first = ddt.ddt_decode_attn_paged_quant(*a, scale=c["scale"], workspace=ws)["o"].clone()
    ws.fill_(255)
    assert torch.equal(ddt.ddt_decode_attn_paged_quant(*a, scale=c["scale"], workspace=ws)["o"], first)
    out, st = torch.empty_like(first), torch.empty(40, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ddt.ddt_decode_attn_paged_quant(*a, scale=c["scale"], out=out, status=st, workspace=ws)
    for _ in range(3):
        out.fill_(math.nan)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hq,block,every", [(4, 128, 2), (8, 16, 1), (20, 64, 3)])
def test_many_far_blocks_a_cta(Hq, block, every, dtype):
    """400 requests over the same pages, so that a CTA meets dozens of tiles with far blocks: each as it is alone."""
    c = _case(59, 1, 1, Hq, 4, 64, [4000], 128, block, dtype)
    c["vs"][:] = 120
    for i, at in enumerate(_blocks(c, 0)):
        if i * block // 128 % every == 0 and i % 2 == 0:
            _set(c, at, 120 + (9 if i % 3 else -20), channel=None if i % 3 else 7)
    a = _args(c)
    wide = [x.expand(-1, 400, *x.shape[2:]).contiguous() for x in a[:3]]
    r = ddt.ddt_decode_attn_paged_quant(*wide, *a[3:7], a[7].expand(400, -1).contiguous(), a[8].expand(400).contiguous(), scale=c["scale"],
                                        out_dtype=F32)
    want, bound = _want(c)
    assert (r["status"] == 0).all()
    tol = torch.from_numpy(bound + Q.U * np.abs(want)).cuda()
    err = (r["o"].double() - torch.from_numpy(want).cuda()).abs()
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("zeros", [31, 32, 33, 49])
def test_far_blocks_behind_many_blocks_of_zeros(zeros, dtype):
    """Zeros over the 32 blocks that the scale the others are near is looked for in, then ordinary and far blocks: several
    requests a CTA, cut anywhere."""
    B = 100
    lens = [520 + b % 9 for b in range(B)]
    c = _case(60, 1, B, 8, 4, 64, lens, 16, 8, dtype, new=False, q_std=0.1)
    c["vs"][:] = 120
    for b in range(B):
        for i, at in enumerate(_blocks(c, b)):
            if i < zeros:
                _set(c, at, 0, zero=True)
            elif i % 7 == b % 7:
                _set(c, at, 131 if i % 2 else 95, channel=b % 64 if i % 2 else None)
    _check(c, _run(c, out_dtype=F32))
