"""ddt_decode_attn_paged on scores at the edges of fp32 (-inf, NaN), and on scores that move the
exponents' reference many times a segment, for every head block and head size, in one launch and
in two; against a plain 64-bit softmax."""
import math

import numpy as np
import pytest
import torch

from tests import _serving as S
from tests.test_gpu_decode import BF, F32, _case, _run
from tree_speculative_decoding_02_gb300 import synth

pytestmark = pytest.mark.gpu


def _near(c, r, want, weights, size, spread, w=None, skip=()):
    """Of request b's o: each weight is off by a relative 2.2 decode_delta after normalisation, so a
    channel by that times sum_p w_p |v_p| (`spread`), and by its rounding to the output type."""
    got, half = S.f64(r["o"]), S.HALF[r["o"].dtype]
    Hq, Hkv, d = c["q"].shape[2], c["k"].shape[2], c["q"].shape[3]
    for b, n in enumerate(c["lens"]):
        if b in skip:
            continue
        delta = S.decode_delta(d, n, size[:, b].repeat(Hq // Hkv, axis=1))[..., None]
        tol = 2.2 * delta * spread[:, b] + half * np.abs(want[:, b]) + 1e-30
        err = np.abs(got[:, b] - want[:, b])
        assert (err <= tol).all(), f"request {b}: {np.nanmax(err / tol):.3g} of the tolerance"
        if w is not None:
            m = min(weights[b].shape[2], w.shape[-1])
            x, exact = S.f64(w)[:, b], weights[b][:, :, :m]
            dw = S.decode_delta(d, n, size[:, b])[..., None]
            assert (np.abs(x[:, :, :m] - exact) <= 2.5 * dw * exact + 4 * S.U * exact + 1e-30).all(), b
            assert (x[:, :, m:] == 0).all()


def _plain(c):
    """o, weights, |q||k| of the finite scores, and sum w |v|; scores of -inf have weight 0, and a
    head with no others has no rows (o and weights 0)."""
    f = lambda t: None if t is None else S.f64(t)  # noqa: E731
    q, kp, vp, kn, vn = f(c["q"]), f(c["k"]), f(c["v"]), f(c["k_new"]), f(c["v_new"])
    L, B, Hq, d = q.shape
    Hkv = kp.shape[2]
    G = Hq // Hkv
    o, spread, size, weights = np.zeros(q.shape), np.zeros(q.shape), np.zeros((L, B, Hkv)), []
    for b, n in enumerate(c["lens"]):
        K, V = S.rows_of(kp, c["table"].numpy(), b, n), S.rows_of(vp, c["table"].numpy(), b, n)
        if kn is not None:
            K, V = (np.concatenate([x, y[:, b][:, :, None]], axis=2) for x, y in ((K, kn), (V, vn)))
        w = np.zeros((L, Hkv, K.shape[2]))
        for l in range(L):
            for g in range(Hkv):
                h = slice(g * G, (g + 1) * G)
                with np.errstate(invalid="ignore"):
                    s = q[l, b, h] @ K[l, g].T * c["scale"]
                s[s < -3e38] = -np.inf                       # past fp32
                m = s.max(axis=1, keepdims=True, initial=-np.inf)
                e = np.exp(s - np.where(np.isinf(m), 0.0, m))
                p = e / np.maximum(e.sum(axis=1, keepdims=True), 1e-300)
                o[l, b, h], spread[l, b, h] = p @ V[l, g], p @ np.abs(V[l, g])
                w[l, g] = p.sum(axis=0)
                a = np.abs(q[l, b, h]) @ np.abs(np.where(np.abs(K[l, g]) > 1e37, 0, K[l, g])).T
                size[l, b, g] = (a.max(initial=0.0) + 4.0) * abs(c["scale"])   # (4: the products left out here)
        weights.append(w)
    return o, weights, size, spread


def _set_rows(c, b, rows, channel, value):
    page = c["k"].shape[3]
    for i in rows:
        c["k"][:, int(c["table"][b, i // page]), :, i % page, channel] = value


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 64), (12, 1, 128), (24, 4, 256), (40, 2, 64)])
@pytest.mark.parametrize("cap_rows", [1024, 9000])
@pytest.mark.parametrize("kind", ["inf", "overflow"])
def test_scores_of_minus_infinity(dtype, Hq, Hkv, d, cap_rows, kind):
    """Cached rows whose score is -inf (a key of -inf, or a product past fp32, the latter for every
    second head only) have weight 0, however the rows are cut: the row alone in the last tile, whole
    first tiles, all but the new row, and all."""
    lens = [129, 700, 300, 200, 640]
    c = _case(26, 1, len(lens), Hq, Hkv, d, lens, 64, dtype, cap_rows=cap_rows)
    c["q"][..., 0] = 4.0
    c["k_new"][..., 0] = 0.5
    low = -math.inf
    if kind == "overflow":
        low = -3e38
        c["scale"] = 1.0
        c["q"][..., 1:] *= 0.1
        c["q"][..., ::2, 0] = 2.0 ** -126                     # 3e38 of it: 3.5
    _set_rows(c, 0, [128], 0, low)
    _set_rows(c, 1, range(0, 512), 0, low)
    _set_rows(c, 2, range(300), 0, low)
    _set_rows(c, 3, range(200), 0, low)
    _set_rows(c, 4, range(0, 640, 2), 0, low)
    if kind == "inf":
        c["k_new"][:, 3, :, 0] = low
    w = torch.zeros((1, len(lens), Hkv, c["table"].shape[1] * 64), device="cuda")
    r = _run(c, weight=w, out_dtype=F32)
    assert (r["status"] == 0).all()
    _near(c, r, *_plain(c), w)
    if kind == "inf":
        assert (r["o"][:, 3] == 0).all() and (w[:, 3] == 0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cap_rows", [512, 9000])
def test_a_nan_key_makes_its_heads_and_their_sums_nan(dtype, cap_rows):
    """By the definition every weight of a head with a NaN score is NaN; other requests are not touched."""
    lens = [400, 400, 10]
    c = _case(27, 1, 3, 8, 2, 64, lens, 64, dtype, cap_rows=cap_rows)
    c["k"][:, int(c["table"][1, 3]), 0, 5, 7] = math.nan      # kv head 0 of request 1
    w = torch.zeros((1, 3, 2, c["table"].shape[1] * 64), device="cuda")
    r = _run(c, weight=w, out_dtype=F32)
    o = r["o"].cpu()
    assert o[0, 1, :4].isnan().all() and o[0, [0, 2]].isfinite().all() and o[0, 1, 4:].isfinite().all()
    assert w[0, 1, 0, :401].isnan().all() and (w[0, 1, 0, 401:] == 0).all()
    assert w[0, [0, 2]].isfinite().all() and w[0, 1, 1].isfinite().all()


def _steps(workload, G, d, n, dtype):
    """40 requests on the same pages.  Channel 0 of the keys climbs by 9.5 (log2 of the weight, for a
    head whose q has 1 there) from tile to tile, seven tiles and then from the start again, and the
    values shrink by as much, so that every tile counts; heads take it whole, not at all, by half
    (a new reference every second tile) and reversed."""
    B = 40
    c = _case(workload, 1, 1, G, 1, d, [n], 64, dtype, q_std=0.5)
    g = synth.gen(workload, 72)
    c["q"] = synth.normal((1, B, G, d), 0.5, g=g, dtype=dtype)
    c["q"][..., 0] = torch.tensor([1.0, 0.0, 0.5, -1.0])[torch.arange(G) % 4].to(dtype)
    c["k_new"], c["v_new"] = (synth.normal((1, B, 1, d), g=g, dtype=dtype) for _ in range(2))
    for i in range(n):
        page, row, level = int(c["table"][0, i // 64]), i % 64, i // 128 % 7
        c["k"][:, page, :, row, 0] = 9.5 * level / (c["scale"] * math.log2(math.e))
        c["v"][:, page, :, row] *= 2.0 ** (9.5 * (6 - level))
    c["table"] = c["table"].repeat(B, 1)
    c["lens"] = [max(0, n - 61 * b) for b in range(B)]
    return c


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("G", [2, 12, 24])
@pytest.mark.parametrize("n", [1530, 6000])
def test_the_reference_moves_many_times_a_segment(dtype, d, G, n):
    c = _steps(28, G, d, n, dtype)
    w = torch.zeros((1, len(c["lens"]), 1, c["table"].shape[1] * 64), device="cuda")
    r = _run(c, weight=w, out_dtype=F32)
    assert (r["status"] == 0).all()
    _near(c, r, *_plain(c), w)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,G", [(64, 12), (64, 2), (128, 24)])
def test_bad_pages_deep_in_long_segments(dtype, d, G):
    """Segments of many more tiles than are in flight, a page that does not exist in a tile of its own
    for every third request."""
    c = _case(29, 1, 1, G, 1, d, [6000], 64, dtype)
    B = 40
    g = synth.gen(29, 72)
    c["q"] = synth.normal((1, B, G, d), 1.5, g=g, dtype=dtype)
    c["k_new"], c["v_new"] = (synth.normal((1, B, 1, d), g=g, dtype=dtype) for _ in range(2))
    c["table"], c["lens"] = c["table"].repeat(B, 1), [6000 - 37 * b for b in range(B)]
    bad = list(range(0, B, 3))
    for b in bad:
        c["table"][b, (7 * b) % 70] = 10 ** 6 if b % 2 else -1
    w = torch.zeros((1, B, 1, c["table"].shape[1] * 64), device="cuda")
    r = _run(c, weight=w, out_dtype=F32)
    assert r["status"].cpu().tolist() == [int(b in bad) for b in range(B)]
    assert (r["o"][:, bad] == 0).all() and (w[:, bad] == 0).all()
    for b in bad:
        c["table"][b] = c["table"][1]
    _near(c, r, *_plain(c), w, skip=bad)
