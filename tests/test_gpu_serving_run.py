"""The single-token calls together, as a server uses them next to the verification round: plain
steps whose weights are summed while the cache grows through ddt_commit_paged, an eviction by
those sums, more steps, and a verification round over what is left; every step against plain
64-bit arithmetic or the oracle.  And the emitted tokens' log probabilities of a round."""
import math

import numpy as np
import pytest
import torch

import oracle
from tests import _cases as C
from tests import _serving as S
from tests._parity import TOL, normwise
from tree_speculative_decoding_02_gb300 import ddt, synth
from tree_speculative_decoding_02_gb300.round import Round

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def test_steps_eviction_and_a_round():
    L, B, Hq, Hkv, d, page, keep = 2, 3, 12, 2, 128, 16, 150
    lens = np.array([160, 40, 0], np.int64)
    g = synth.gen(60, 1)
    k, v, table = S.paged_cache(60, L, B, Hkv, d, lens.tolist(), page, dtype=BF, cap_rows=320, poison=False)
    cap = table.shape[1] * page
    dev = dict(k=k.cuda(), v=v.cuda(), table=table.cuda(), P=torch.tensor(lens, dtype=torch.int32).cuda(),
               seq=torch.tensor(lens, dtype=torch.int32).cuda(), placed=torch.zeros(B, dtype=torch.int32, device="cuda"),
               w=torch.zeros((L, B, Hkv, cap), device="cuda"),
               pos=torch.zeros((L, B, Hkv, cap), dtype=torch.int32, device="cuda"))
    zero = torch.zeros((B, 1), dtype=torch.int32, device="cuda")
    none = torch.zeros(B, dtype=torch.int32, device="cuda")
    ws = ddt.decode_attn_paged_workspace(torch.empty((L, B, Hq, d), dtype=BF, device="cuda"), dev["k"], dev["table"],
                                         weights=True)
    sums = np.zeros((L, B, Hkv, cap))
    scale, evictions = 1 / math.sqrt(d), 0
    for step in range(40):
        q, kn, vn = (synth.normal((L, B, h, d), g=g, dtype=BF) for h in (Hq, Hkv, Hkv))
        now = dev["P"].cpu().numpy()
        r = ddt.ddt_decode_attn_paged(q.cuda(), kn.cuda(), vn.cuda(), dev["k"], dev["v"], dev["table"], dev["P"], scale=scale,
                                      attn_weight=dev["w"], out_dtype=F32, workspace=ws)
        o, weights, _ = S.decode_ref(S.f64(q), S.f64(kn), S.f64(vn), S.f64(dev["k"]), S.f64(dev["v"]), table.numpy(),
                                     now.tolist(), scale)
        assert normwise(S.f64(r["o"]), o, axes=-1).max() <= TOL
        for b in range(B):
            sums[:, b, :, :now[b] + 1] += weights[b]
        assert np.abs(S.f64(dev["w"]) - sums).max() <= 1e-3
        c = ddt.ddt_commit_paged(zero, none, dev["P"], dev["table"], k_tree=kn[:, :, None].contiguous().cuda(),
                                 v_tree=vn[:, :, None].contiguous().cuda(), k_pages=dev["k"], v_pages=dev["v"])
        dev["seq"] += 1
        assert (c["status"] == 0).all() and (dev["P"].cpu().numpy() == now + 1).all()
        if (now + 1).max() < keep + 24:
            continue
        # eviction: exact, from the sums the steps left on the GPU
        hk, hv = (dev[x].cpu().view(torch.int16).numpy().copy() for x in ("k", "v"))
        hw, hp = dev["w"].cpu().numpy().copy(), dev["pos"].cpu().numpy().copy()
        P1, placed = S.evict_ref(hk, hv, table.numpy(), now + 1, dev["placed"].cpu().numpy(), dev["seq"].cpu().numpy(), hw, hp,
                                 keep, 4, 16)
        e = ddt.ddt_evict_paged(dev["k"], dev["v"], dev["table"], dev["P"], dev["placed"], dev["seq"], dev["w"], dev["pos"],
                                keep=keep, n_sink=4, n_recent=16)
        assert (e["status"] == 0).all()
        np.testing.assert_array_equal(dev["P"].cpu().numpy(), P1)
        np.testing.assert_array_equal(dev["placed"].cpu().numpy(), placed)
        np.testing.assert_array_equal(dev["pos"].cpu().numpy(), hp)
        np.testing.assert_array_equal(dev["k"].cpu().view(torch.int16).numpy(), hk)
        np.testing.assert_array_equal(dev["v"].cpu().view(torch.int16).numpy(), hv)
        np.testing.assert_array_equal(dev["w"].cpu().numpy(), hw)
        # the recent positions are among the rows that stay
        for b in np.flatnonzero(now + 1 > keep):
            have = set(hp[0, b, 0, :keep].tolist())
            s = int(dev["seq"][b])
            assert have >= set(range(s - 16, s)) | set(range(4)) and len(have) == keep
        sums = hw.astype(np.float64)
        evictions += 1
    assert evictions >= 2

    # a verification round's attention over the cut cache: positions go on from seq_len
    prefix = dev["P"].cpu().numpy()
    tree, _ = C.tree_from_logits(61, B, 6, 300, 4, 20, std=2.0, boost=0.0, prefix=dev["seq"].cpu().numpy())
    t = C.tree_to_dev(tree)
    N = 21
    q, kt, vt = (synth.normal((L, B, N, h, d), g=g, dtype=BF) for h in (Hq, Hkv, Hkv))
    r = ddt.ddt_tree_attn_paged(q.cuda(), kt.cuda(), vt.cuda(), dev["k"], dev["v"], dev["table"], dev["P"], t["n_nodes"],
                                t["anc"], scale=scale, out_dtype=F32)
    kc = oracle.gather_pages(C.f64(dev["k"]), table.numpy(), prefix, cap)
    vc = oracle.gather_pages(C.f64(dev["v"]), table.numpy(), prefix, cap)
    want = oracle.tree_attn(C.f64(q), C.f64(kt), C.f64(vt), kc, vc, prefix, tree["n_nodes"], tree["anc"], scale)["o"]
    for b in range(B):
        n = int(tree["n_nodes"][b])
        assert normwise(C.f64(r["o"])[:, b, :n], want[:, b, :n], axes=-1).max() <= TOL


@pytest.mark.parametrize("temperature", [0.0, 0.8])
def test_log_probabilities_of_a_round(temperature):
    cfg = dict(synth.WORKLOADS[1], V=3000, budget=24, B=3, temperature=temperature, dtype=BF, Lf=0, Lg=0)
    r = Round(cfg, device="cuda", workload=1)
    ddt.ddt_build_tree(r.draft_logits, r.root_token, r.prefix_len, cfg["top_k"], cfg["budget"], out=r.tree,
                       workspace=r.build_ws)
    tl = r.target_logits.float().cpu()
    synth.plant_path(tl, r.tree["token"].cpu().numpy(), r.tree["parent"].cpu().numpy(), r.tree["n_nodes"].cpu().numpy(),
                     [2, 0, 3], boost=14.0)
    r.target_logits.copy_(tl.to(BF))
    r.step()
    got = r.emitted_logprobs(top_n=4)
    torch.cuda.synchronize()
    node, token = r.walk["acc_nodes"].cpu().numpy(), r.walk["emitted"].cpu().numpy()
    n = r.walk["n_emitted"].cpu().numpy()
    assert n.max() >= 2
    lp, en, ids, tlp = S.logprobs_ref(S.f64(r.target_logits), node, token, 4, temperature or 1.0)
    assert np.abs(S.f64(got["logprob"]) - lp).max() <= 1e-5 and np.abs(S.f64(got["entropy"]) - en).max() <= 1e-4
    np.testing.assert_array_equal(got["top_token"].cpu().numpy(), ids)
    for b in range(3):   # greedy: every emitted token is its row's first alternative
        if not temperature:
            np.testing.assert_array_equal(ids[b, :n[b], 0], token[b, :n[b]])
        assert (got["logprob"][b, n[b]:] == 0).all() and (got["top_token"][b, n[b]:] == -1).all()


def test_offsets_past_32_bits():
    """Pages that lie more than 2^32 elements into the pools."""
    num, Hkv, page, d = 66000, 4, 64, 256
    k = torch.empty((1, num, Hkv, page, d), dtype=BF, device="cuda")
    v = torch.empty_like(k)
    assert k.numel() > 1 << 32
    table = torch.tensor([[num - 1, 3, num - 2, 7]], dtype=torch.int32)
    n = 200
    small_k = synth.normal((1, 4, Hkv, page, d), g=synth.gen(62, 1), dtype=BF)
    small_v = synth.normal((1, 4, Hkv, page, d), g=synth.gen(62, 2), dtype=BF)
    k[:, table[0].long().cuda()] = small_k.cuda()
    v[:, table[0].long().cuda()] = small_v.cuda()
    q = synth.normal((1, 1, 8, d), g=synth.gen(62, 3), dtype=BF)
    P = torch.tensor([n], dtype=torch.int32, device="cuda")
    w = torch.zeros((1, 1, Hkv, 256), device="cuda")
    r = ddt.ddt_decode_attn_paged(q.cuda(), None, None, k, v, table.cuda(), P, scale=1 / 16, attn_weight=w, out_dtype=F32)
    local = np.arange(4)[None]
    o, _, _ = S.decode_ref(S.f64(q), None, None, S.f64(small_k), S.f64(small_v), local, [n], 1 / 16)
    assert normwise(S.f64(r["o"]), o, axes=-1).max() <= TOL
    hk, hv = (x.view(torch.int16).numpy().copy() for x in (small_k, small_v))
    hw, pos = w.cpu().numpy().copy(), np.zeros((1, 1, Hkv, 256), np.int32)
    S.evict_ref(hk, hv, local, np.array([n]), np.array([0]), np.array([n]), hw, pos, 100, 0, 0)
    placed, seq = torch.zeros_like(P), P.clone()
    gp = torch.zeros((1, 1, Hkv, 256), dtype=torch.int32, device="cuda")
    assert int(ddt.ddt_evict_paged(k, v, table.cuda(), P, placed, seq, w, gp, keep=100)["status"][0]) == 0
    at = table[0].long().cuda()
    np.testing.assert_array_equal(k[:, at].cpu().view(torch.int16).numpy(), hk)
    np.testing.assert_array_equal(v[:, at].cpu().view(torch.int16).numpy(), hv)
    np.testing.assert_array_equal(gp.cpu().numpy()[..., :n], pos[..., :n])


def test_two_streams_at_once():
    """Calls of each kind on two streams, each with a workspace of its own, agree with calls alone."""
    cases = []
    for wl in (63, 64):
        k, v, table = S.paged_cache(wl, 1, 4, 2, 64, [700, 90, 0, 300], 16, dtype=BF, poison=False)
        q = synth.normal((1, 4, 8, 64), g=synth.gen(wl, 3), dtype=BF).cuda()
        x = synth.normal((2, 40, 5000), 2.0, g=synth.gen(wl, 4), dtype=BF).cuda()
        tok = torch.randint(0, 5000, (2, 40), generator=synth.gen(wl, 5)).to(torch.int32).cuda()
        P = torch.tensor([700, 90, 0, 300], dtype=torch.int32, device="cuda")
        cases.append((q, k.cuda(), v.cuda(), table.cuda(), P, x, tok))

    def calls(c):
        q, k, v, table, P, x, tok = c
        w = torch.zeros((1, 4, 2, table.shape[1] * 16), device=q.device)
        o = ddt.ddt_decode_attn_paged(q, None, None, k, v, table, P, scale=0.125, attn_weight=w)["o"]
        lp = ddt.ddt_token_logprobs(x, tok, top_n=3)
        k2, v2, P2 = k.clone(), v.clone(), P.clone()
        pos = torch.zeros_like(w, dtype=torch.int32)
        ddt.ddt_evict_paged(k2, v2, table, P2, torch.zeros_like(P), P, w, pos, keep=200, n_recent=10)
        return [o, w, k2, v2, pos, P2, *lp.values()]
    want = [calls(c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = []
        for s, c in zip(streams, cases):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(calls(c))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            for x, y in zip(a, b):
                assert torch.equal(x, y)
