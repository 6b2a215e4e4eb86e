"""ddt_decode_attn_paged against a plain 64-bit softmax over the gathered rows.  Every row that
is not a prefix row holds NaN, so a read past a prefix, or of a page of another request, shows."""
import math

import numpy as np
import pytest
import torch

from tests import _serving as S
from tree_speculative_decoding_02_gb300 import ddt, synth

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _case(workload, L, B, Hq, Hkv, d, lens, page, dtype, *, new=True, cap_rows=None, q_std=1.5):
    g = synth.gen(workload, 71)
    c = dict(q=synth.normal((L, B, Hq, d), q_std, g=g, dtype=dtype), lens=lens, scale=1 / math.sqrt(d))
    c["k_new"] = synth.normal((L, B, Hkv, d), g=g, dtype=dtype) if new else None
    c["v_new"] = synth.normal((L, B, Hkv, d), g=g, dtype=dtype) if new else None
    c["k"], c["v"], c["table"] = S.paged_cache(workload, L, B, Hkv, d, lens, page, dtype=dtype, cap_rows=cap_rows)
    return c


def _dev(t):
    return None if t is None else t.cuda()


def _run(c, *, weight=None, out_dtype=None, **kw):
    r = ddt.ddt_decode_attn_paged(_dev(c["q"]), _dev(c["k_new"]), _dev(c["v_new"]), _dev(c["k"]), _dev(c["v"]),
                                  _dev(c["table"]), torch.tensor(c["lens"], dtype=torch.int32).cuda(), scale=c["scale"],
                                  attn_weight=weight, out_dtype=out_dtype, **kw)
    torch.cuda.synchronize()
    return r


def _ref(c):
    f = lambda t: None if t is None else S.f64(t)  # noqa: E731
    return S.decode_ref(f(c["q"]), f(c["k_new"]), f(c["v_new"]), f(c["k"]), f(c["v"]), c["table"].numpy(), c["lens"],
                        c["scale"])


def _check(c, r, weight=None, before=0.0):
    want, weights, size = _ref(c)
    got = S.f64(r["o"])
    L, B, Hq, d = got.shape
    Hkv = c["k"].shape[2]
    half = S.HALF[r["o"].dtype]
    for b, n in enumerate(c["lens"]):
        delta = S.decode_delta(d, n, size[:, b].repeat(Hq // Hkv, axis=1))[..., None]
        big = 5.0   # |v| of N(0, 1) entries; a weighted mean of values moves by at most 2 delta max |v|
        tol = 2.2 * delta * big + half * np.abs(want[:, b]) + 1e-30
        err = np.abs(got[:, b] - want[:, b])
        assert bool((err <= tol).all()), f"request {b}: {(err / tol).max():.3g} of the tolerance"
        if weight is not None:
            w = S.f64(weight)[:, b]
            m = min(weights[b].shape[2], w.shape[2])
            exact = weights[b][:, :, :m]
            dw = S.decode_delta(d, n, size[:, b])[..., None]
            assert (np.abs(w[:, :, :m] - before - exact) <= 2.5 * dw * exact + 4 * S.U * (exact + before) + 1e-30).all(), b
            assert (w[:, :, m:] == before).all()
    assert (r["status"].cpu() == 0).all()


# head groups 1 to 40 (in and across head blocks), page sizes of every kind, lengths 0, 1, tile
# and page edges
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hq,Hkv,d,page", [(24, 4, 256, 64), (4, 4, 64, 16), (16, 2, 128, 8), (10, 2, 64, 32),
                                           (12, 1, 128, 192), (6, 3, 256, 128), (40, 1, 64, 64), (17, 1, 128, 256),
                                           (34, 2, 256, 16)])
def test_matches_softmax(dtype, Hq, Hkv, d, page):
    lens = [0, 1, page, 127, 128, 129, 3 * page + 5, 700]
    c = _case(11, 2, len(lens), Hq, Hkv, d, lens, page, dtype, cap_rows=701)
    w = torch.zeros((2, len(lens), Hkv, c["table"].shape[1] * page), device="cuda")
    r = _run(c, weight=w, out_dtype=F32)
    _check(c, r, w)
    # without the sums: the same output
    assert torch.equal(_run(c, out_dtype=F32)["o"], r["o"])
    # the rounded output is the fp32 one rounded
    assert torch.equal(_run(c, out_dtype=BF)["o"], r["o"].to(BF))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_without_a_new_row(dtype):
    """The prefix alone; a request with no rows gets zeros (and nothing in its sums)."""
    lens = [0, 5, 300]
    c = _case(12, 1, 3, 8, 2, 128, lens, 16, dtype, new=False)
    w = torch.full((1, 3, 2, c["table"].shape[1] * 16), 0.5, device="cuda")
    r = _run(c, weight=w, out_dtype=F32)
    assert (r["o"][:, 0] == 0).all()
    _check(c, r, w, before=0.5)


@pytest.mark.parametrize("dtype,n", [(BF, 70001), (F32, 30011)])
def test_long_prefix_is_split_and_joined(dtype, n):
    c = _case(13, 1, 2, 16, 2, 128, [n, 77], 64, dtype)
    w = torch.zeros((1, 2, 2, c["table"].shape[1] * 64), device="cuda")
    _check(c, _run(c, weight=w, out_dtype=F32), w)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_short_units(dtype):
    """More (layer, request, head) units than CTAs: several whole units a CTA, ragged, some empty."""
    lens = [(37 * i) % 400 if i % 5 else 0 for i in range(60)]
    c = _case(14, 3, 60, 10, 5, 64, lens, 32, dtype)
    _check(c, _run(c, out_dtype=F32))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_growing_maximum(dtype):
    """Keys whose scores climb far along the prefix (every tile raises the running maximum by
    more than any lazy bound) and far below zero: the rescaling of earlier tiles is exact."""
    lens = [1500, 640]
    c = _case(15, 1, 2, 4, 2, 64, lens, 64, dtype, q_std=1.0)
    k = c["k"]
    for b, n in enumerate(lens):
        for i in range(-(-n // 64)):
            k[:, int(c["table"][b, i])] *= (0.2 + i) if b == 0 else (3.0 - 0.2 * i)
    c["k"] = k
    w = torch.zeros((1, 2, 2, c["table"].shape[1] * 64), device="cuda")
    _check(c, _run(c, weight=w, out_dtype=F32), w)


def test_scale_is_taken_as_given():
    for scale in (0.0, -0.3):
        c = _case(16, 1, 2, 6, 2, 64, [200, 65], 16, BF)
        c["scale"] = scale
        _check(c, _run(c, out_dtype=F32))


def test_sums_accumulate_over_calls_and_the_last_place():
    """Two calls add up; a request whose cache is full has no place for its new row's weight."""
    lens = [64, 63, 10]
    c = _case(17, 1, 3, 4, 2, 64, lens, 32, BF, cap_rows=64)
    assert c["table"].shape[1] * 32 == 64
    w = torch.zeros((1, 3, 2, 64), device="cuda")
    _run(c, weight=w)
    once = w.clone()
    _run(c, weight=w)
    assert torch.equal(w, once + once)
    sums = once.sum(-1)[0]
    assert (sums[0] < 2).all() and torch.allclose(sums[1:], torch.full_like(sums[1:], 2.0), rtol=1e-4)


def test_bad_requests_are_flagged_and_left_alone():
    lens = [100, 100, 100, 100]
    c = _case(18, 2, 4, 4, 1, 64, lens, 32, BF)
    good = _run(c)["o"]
    c["table"] = c["table"].clone()
    c["table"][1, 2] = 10 ** 6
    c["table"][2, 3] = -1
    c["lens"] = [100, 100, 100, 129]
    w = torch.full((2, 4, 1, 128), 3.0, device="cuda")
    r = _run(c, weight=w)
    assert r["status"].cpu().tolist() == [0, 1, 1, 3]
    assert (r["o"][:, 1:] == 0).all() and torch.equal(r["o"][:, 0], good[:, 0])
    assert (w[:, 1:] == 3).all() and (w[:, 0] != 3).any()


def test_table_entries_past_the_prefix_are_not_read():
    c = _case(19, 1, 2, 4, 2, 64, [33, 40], 32, BF, cap_rows=200)
    c["table"] = c["table"].clone()
    c["table"][:, 2:] = -7
    _check(c, _run(c, out_dtype=F32))


def test_shared_pages():
    """Two requests on the same pages with the same query agree bit for bit."""
    c = _case(20, 1, 2, 8, 2, 128, [300, 300], 16, BF)
    c["table"][1] = c["table"][0]
    for k in ("q", "k_new", "v_new"):
        c[k][:, 1] = c[k][:, 0]
    c["k"], c["v"] = c["k"].nan_to_num(0.5), c["v"].nan_to_num(0.5)
    r = _run(c, out_dtype=F32)
    _check(c, r)
    assert (r["o"][:, 0] - r["o"][:, 1]).abs().max() <= 1e-5   # the cuts into segments may differ
    assert torch.equal(r["o"], _run(c, out_dtype=F32)["o"])    # and a second call is the same


def test_equals_the_tree_call_on_a_root():
    """ddt_tree_attn_paged on trees of the root alone computes the same attention (to the
    tolerance both are held to)."""
    lens = [0, 200, 999]
    c = _case(21, 2, 3, 24, 4, 256, lens, 64, BF)
    anc = torch.ones((3, 1, 1), dtype=torch.int32, device="cuda")
    one = torch.ones(3, dtype=torch.int32, device="cuda")
    t = ddt.ddt_tree_attn_paged(c["q"][:, :, None].contiguous().cuda(), c["k_new"][:, :, None].contiguous().cuda(),
                                c["v_new"][:, :, None].contiguous().cuda(), c["k"].cuda(), c["v"].cuda(), c["table"].cuda(),
                                torch.tensor(lens, dtype=torch.int32).cuda(), one, anc, scale=c["scale"], out_dtype=F32)
    r = _run(c, out_dtype=F32)
    assert (t["o"][:, :, 0] - r["o"]).abs().max() <= 2e-3 * r["o"].abs().max()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_two_launches_captured_follow_the_lengths(dtype):
    lens = [4900, 40, 0]
    c = _case(25, 1, 3, 8, 2, 64, lens, 16, dtype, cap_rows=9000)
    c["k"], c["v"] = c["k"].nan_to_num(0.25), c["v"].nan_to_num(0.25)
    d = {k: _dev(c[k]) for k in ("q", "k_new", "v_new", "k", "v", "table")}
    P = torch.tensor(lens, dtype=torch.int32).cuda()
    w = torch.zeros((1, 3, 2, c["table"].shape[1] * 16), device="cuda")
    ws = ddt.decode_attn_paged_workspace(d["q"], d["k"], d["table"], weights=True)
    out = torch.empty((1, 3, 8, 64), dtype=F32, device="cuda")
    st = torch.empty(3, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ddt.ddt_decode_attn_paged(d["q"], d["k_new"], d["v_new"], d["k"], d["v"], d["table"], P, scale=c["scale"],
                                  attn_weight=w, out=out, status=st, workspace=ws)
    for lens in ([4900, 40, 0], [1, 5000, 2600], [0, 0, 0]):
        P.copy_(torch.tensor(lens, dtype=torch.int32))
        w.zero_()
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        c["lens"] = lens
        _check(c, {"o": out, "status": st}, w)


# One launch (a cluster of 1, 2, 4 or 8 blocks a unit joins its own partials) or two (the table's
# rows are too many for that): either is chosen by the table's capacity, not by the lengths.
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hq,Hkv,d,B", [(8, 1, 64, 1), (6, 2, 128, 30), (24, 4, 256, 20), (16, 16, 64, 13)])
@pytest.mark.parametrize("cap_rows", [120, 300, 900, 5000])
def test_any_table_capacity(dtype, Hq, Hkv, d, B, cap_rows):
    lens = [(37 * i + 1) * 53 % (min(cap_rows, 900) + 1) for i in range(B)]
    lens[-1] = min(cap_rows, 900) - 1
    c = _case(24, 1, B, Hq, Hkv, d, lens, 16, dtype, cap_rows=cap_rows)
    w = torch.zeros((1, B, Hkv, c["table"].shape[1] * 16), device="cuda")
    r = _run(c, weight=w, out_dtype=F32)
    _check(c, r, w)
    if B > 2:  # flagged requests beside others
        c["table"] = c["table"].clone()
        c["table"][1, 0] = -7
        lens[1], lens[2] = 16, c["table"].shape[1] * 16 + 1
        w2 = torch.zeros_like(w)
        bad = _run(c, weight=w2, out_dtype=F32)
        assert bad["status"].cpu().tolist() == [0, 1, 3] + [0] * (B - 3)
        assert (bad["o"][:, 1:3] == 0).all() and (w2[:, 1:3] == 0).all()
        # (not bit for bit: where two launches split the rows, the split follows all lengths)
        rest = [0] + list(range(3, B))
        c2 = dict(c, lens=[lens[b] for b in rest], table=c["table"][rest], **{k: c[k][:, rest] for k in ("q", "k_new", "v_new")})
        _check(c2, {"o": bad["o"][:, rest], "status": bad["status"][rest]}, w2[:, rest])


def test_side_stream_and_graph_replay_follow_the_lengths():
    """A captured call runs on its stream, and a replay takes the lengths it finds."""
    lens = [500, 40, 0]
    c = _case(22, 1, 3, 8, 2, 128, lens, 16, BF, cap_rows=600)
    c["k"], c["v"] = c["k"].nan_to_num(0.25), c["v"].nan_to_num(0.25)
    d = {k: _dev(c[k]) for k in ("q", "k_new", "v_new", "k", "v", "table")}
    P = torch.tensor(lens, dtype=torch.int32).cuda()
    w = torch.zeros((1, 3, 2, c["table"].shape[1] * 16), device="cuda")
    ws = ddt.decode_attn_paged_workspace(d["q"], d["k"], d["table"], weights=True)
    out = torch.empty((1, 3, 8, 128), dtype=F32, device="cuda")
    st = torch.empty(3, dtype=torch.int32, device="cuda")

    def call():
        ddt.ddt_decode_attn_paged(d["q"], d["k_new"], d["v_new"], d["k"], d["v"], d["table"], P, scale=c["scale"],
                                  attn_weight=w, out=out, status=st, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    _check(c, {"o": out, "status": st}, w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lens in ([500, 40, 0], [1, 300, 600], [0, 0, 0]):
        P.copy_(torch.tensor(lens, dtype=torch.int32))
        w.zero_()
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        c["lens"] = lens
        _check(c, {"o": out, "status": st}, w)


def test_refusals():
    c = _case(23, 1, 2, 4, 2, 64, [10, 20], 16, BF)
    d = {k: _dev(c[k]) for k in ("q", "k_new", "v_new", "k", "v", "table")}
    P = torch.tensor([10, 20], dtype=torch.int32).cuda()

    def call(**kw):
        a = {**d, "P": P, **{k: v for k, v in kw.items() if k in d or k == "P"}}
        o = {k: v for k, v in kw.items() if k not in a}
        return ddt.ddt_decode_attn_paged(a["q"], a["k_new"], a["v_new"], a["k"], a["v"], a["table"], a["P"], scale=1.0, **o)
    launched = ddt.ddt_launch_count()
    for kw in (dict(v_new=None), dict(q=d["q"].half()), dict(q=d["q"][..., :32].contiguous()), dict(k=d["k"].float()),
               dict(q=d["q"].transpose(0, 1)), dict(P=P.long()), dict(P=P.cpu()), dict(table=d["table"][:1]),
               dict(attn_weight=torch.zeros((1, 2, 2, 5), device="cuda")), dict(out=torch.empty((1, 2, 4, 64))),
               dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda")),
               dict(out=torch.empty((1, 2, 4, 64), dtype=torch.float16, device="cuda"))):
        with pytest.raises(ddt.DDTError):
            call(**kw)
    assert ddt.ddt_launch_count() == launched
