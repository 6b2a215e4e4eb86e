"""The 8-bit cache's calls together, as a server uses them: plain steps (heads normalised and rotated, attention over
the cache, the row appended) from a prompt on, and whole verification rounds over 8-bit prefixes; every step against
plain 64-bit arithmetic or the oracle."""
import math

import numpy as np
import pytest
import torch

import oracle
from tests import _cases as C
from tests import _quant as Q
from tests._parity import TOL, normwise
from tree_speculative_decoding_02_gb300 import ddt, synth
from tree_speculative_decoding_02_gb300.round import Round

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_prompt_and_steps(dtype):
    L, B, Hq, Hkv, d, page, S, rot = 2, 3, 12, 2, 128, 32, 16, 64
    g = synth.gen(90, 1)
    prompt = [75, 1, 0]
    weights = [(1 + synth.normal((L, d), 0.2, g=g, dtype=dtype)).cuda() for _ in range(2)]
    pools = ddt.quant_cache(L, B * 4 + 2, Hkv, page, d, block=S)
    table = torch.randperm(B * 4 + 2, generator=g)[:B * 4].reshape(B, 4).to(torch.int32).cuda()
    P = torch.zeros(B, dtype=torch.int32, device="cuda")
    host = dict(k=pools[0].view(torch.uint8).cpu().numpy(), v=pools[1].view(torch.uint8).cpu().numpy(), ks=pools[2].cpu().numpy(),
                vs=pools[3].cpu().numpy(), table=table.cpu().numpy(), lens=[0] * B)

    def heads(N):
        """A projection's rows, and q and k of them normalised and rotated at the positions behind the prefix."""
        x = synth.normal((L, B, N, Hq + 2 * Hkv, d), 1.5, g=g, dtype=dtype).cuda()
        at = (P[:, None] + torch.arange(N, device="cuda", dtype=torch.int32)).contiguous()
        q, k = ddt.ddt_qk_norm_rope(x[..., :Hq, :], x[..., Hq:Hq + Hkv, :], *weights, at, rot_dim=rot)
        for got, of, w in ((q, x[..., :Hq, :], weights[0]), (k, x[..., Hq:Hq + Hkv, :], weights[1])):
            want, bound = Q.norm_ref(Q.f64(of), Q.f64(w), at.cpu().numpy(), rot, 10000.0, 1e-6, 0.0)
            assert (np.abs(Q.f64(got) - want) <= bound + Q.HALF[dtype] * (np.abs(want) + bound)).all()
        return q, k, x[..., Hq + Hkv:, :].contiguous()

    def append(k, v, count):
        r = ddt.ddt_append_paged_quant(k, v, *pools, table, P, torch.tensor(count, dtype=torch.int32).cuda())
        assert r["status"].tolist() == [0] * B
        for x, codes, scale in ((k, "k", "ks"), (v, "v", "vs")):
            Q.append_ref(Q.f64(x), host[codes], host[scale], host["table"], host["lens"], count, None)
        host["lens"] = [p + n for p, n in zip(host["lens"], count)]
        assert P.tolist() == host["lens"]
        for have, want in zip(pools, (host["k"], host["v"], host["ks"], host["vs"])):
            assert Q.same_codes(have.view(torch.uint8).cpu().numpy(), want).all()

    _, k, v = heads(max(prompt))
    append(k, v, prompt)
    for step in range(20):
        q, k, v = heads(1)
        k1, v1 = k[:, :, 0].contiguous(), v[:, :, 0].contiguous()
        r = ddt.ddt_decode_attn_paged_quant(q[:, :, 0].contiguous(), k1, v1, *pools, table, P, scale=d ** -0.5, out_dtype=F32)
        want, bound = Q.decode_ref(Q.f64(q[:, :, 0]), Q.f64(k1), Q.f64(v1), host, d ** -0.5, dtype)
        assert r["status"].tolist() == [0] * B
        assert (np.abs(Q.f64(r["o"]) - want) <= bound + Q.U * np.abs(want)).all()
        append(k, v, [1, 1, step % 2])


@pytest.mark.parametrize("Lg,rope,qk_norm,dtype", [(0, 0, False, BF), (1, 64, False, BF), (0, 64, True, BF), (1, 0, True, F32)])
def test_rounds_over_8_bit_prefixes(Lg, rope, qk_norm, dtype):
    """Two rounds in a row: attention over the values that the cache holds, accepted rows appended in 8 bits; then a third
    one replayed from a graph."""
    cfg = dict(synth.WORKLOADS[1], B=3, V=2000, budget=24, Lf=2, Hq=8, Hkv=2, d=128, dtype=dtype, page=32, kv_quant=16, rope=rope,
               qk_norm=qk_norm, P_lo=40, P_hi=300, Lg=Lg, Pcap=400)
    cfg.pop("P", None)
    if not Lg:
        cfg.pop("Lg")
    r = Round(cfg, device="cuda", workload=1, poison=True, attn_out_dtype=F32, gdn_out_dtype=F32)
    scale = 1 / math.sqrt(cfg["d"])
    for turn in range(2):
        now = r.prefix_len.cpu().numpy()
        host = [x.view(torch.uint8).cpu().numpy() for x in (r.k_pages, r.v_pages, r.k_scale, r.v_scale)]
        table = r.block_table.cpu().numpy()
        kt0 = Q.f64(r.attn.k_tree)
        r.step()
        torch.cuda.synchronize()
        for st in (r.tree["status"], r.attn_status, r.walk["status"], r.append_status):
            assert (st == 0).all()
        tree = {k: v.cpu().numpy() for k, v in r.tree.items()}
        nn, pos = tree["n_nodes"], tree["position"]
        q, kt, vt = Q.f64(r.attn.q), kt0, Q.f64(r.attn.v_tree)
        if qk_norm:
            half = Q.HALF[dtype]
            for x, w, got in ((q, r.q_weight, r.q_heads), (kt0, r.k_weight, r.k_heads)):
                want, bound = Q.norm_ref(x, Q.f64(w), pos, rope, 10000.0, 1e-6, 0.0)
                for b in range(3):
                    g, t = Q.f64(got)[:, b, :nn[b]], want[:, b, :nn[b]]
                    assert (np.abs(g - t) <= bound[:, b, :nn[b]] + half * (np.abs(t) + bound[:, b, :nn[b]])).all()
            q, kt = Q.f64(r.q_heads), Q.f64(r.k_heads)
        elif rope:
            kt = Q.f64(r.attn.k_tree)          # rotated in place; q inside the attention call, rounded once
            q = Q.f64(torch.from_numpy(oracle.rope_tree(q, pos, nn, rope, 10000.0)).to(dtype))
        cap = table.shape[1] * 32
        kc, vc = np.zeros((2, 3, 2, cap, 128)), np.zeros((2, 3, 2, cap, 128))
        for b in range(3):
            kc[:, b, :, :now[b]] = Q.rows_of(host[0], host[2], table, b, now[b])
            vc[:, b, :, :now[b]] = Q.rows_of(host[1], host[3], table, b, now[b])
        want = oracle.tree_attn(q, kt, vt, kc, vc, now, nn, tree["anc"].view(np.uint32), scale)["o"]
        for b in range(3):
            assert normwise(C.f64(r.attn_o)[:, b, :nn[b]], want[:, b, :nn[b]], axes=-1).max() <= TOL
        # the accepted rows in the cache
        acc, n = r.walk["acc_nodes"].cpu().numpy(), r.walk["n_emitted"].cpu().numpy()
        for x, codes, sc in ((kt, host[0], host[2]), (vt, host[1], host[3])):
            Q.append_ref(x, codes, sc, table, now.tolist(), n.tolist(), acc)
        for have, w in zip((r.k_pages, r.v_pages, r.k_scale, r.v_scale), host):
            assert Q.same_codes(have.view(torch.uint8).cpu().numpy(), w).all()
        assert (r.prefix_len.cpu().numpy() == now + n).all()
        if rope and not qk_norm:
            r.attn.k_tree.copy_(torch.from_numpy(kt0).to(dtype))
    # captured: the same round from the same state gives the same bits
    state = [r.prefix_len, r.k_pages, r.v_pages, r.k_scale, r.v_scale, r.attn.k_tree] + ([r.gdn.S, r.gdn.conv_state] if Lg else [])
    saved = [x.clone() for x in state]
    r.step()
    torch.cuda.synchronize()
    want = [x.clone() for x in state + [r.attn_o]]
    for x, y in zip(state, saved):
        x.copy_(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r.step()
    for x, y in zip(state, saved):
        x.copy_(y)
    r.attn_o.fill_(0)
    graph.replay()
    torch.cuda.synchronize()
    bits = lambda x: x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x  # noqa: E731
    nn = r.tree["n_nodes"].tolist()
    for x, y in zip(state, want[:-1]):
        assert torch.equal(bits(x), bits(y))
    for b in range(3):
        assert torch.equal(r.attn_o[:, b, :nn[b]], want[-1][:, b, :nn[b]])


@pytest.mark.parametrize("Lg", [0, 1])
def test_a_full_request_is_left_as_it_is(Lg):
    """A request whose rows do not fit is committed nowhere: neither its length nor its recurrent state moves."""
    cfg = dict(synth.WORKLOADS[1], B=3, V=2000, budget=24, Lf=2, Hq=8, Hkv=2, d=128, dtype=BF, page=32, kv_quant=16,
               P_lo=40, P_hi=300, Lg=Lg, Pcap=416)
    cfg.pop("P", None)
    if not Lg:
        cfg.pop("Lg")
    r = Round(cfg, device="cuda", workload=1, poison=True, attn_out_dtype=F32, gdn_out_dtype=F32)
    full = r.block_table.shape[1] * 32
    r.prefix_len[1] = full
    before = r.prefix_len.tolist()
    state = [x.clone() for x in ((r.gdn.S, r.gdn.conv_state) if Lg else ())]
    r.step()
    torch.cuda.synchronize()
    n, acc = r.walk["n_emitted"].tolist(), r.walk["acc_nodes"].tolist()
    assert r.append_status.tolist() == r.commit["status"].tolist() == [0, 3, 0]
    assert r.prefix_len.tolist() == [before[0] + n[0], full, before[2] + n[2]]
    for b in (0, 2):
        assert r.commit["src_row"][b, :n[b]].tolist() == acc[b][:n[b]]
        assert r.commit["dst_pos"][b, :n[b]].tolist() == list(range(before[b], before[b] + n[b]))
    for x, y in zip((r.gdn.S, r.gdn.conv_state) if Lg else (), state):
        assert torch.equal(x[:, 1], y[:, 1]) and not torch.equal(x[:, 0], y[:, 0])


def test_kv_quant_needs_pages():
    with pytest.raises(ValueError):
        Round(dict(synth.WORKLOADS[1], kv_quant=16), device="cuda", workload=1)


def test_on_a_stream_of_their_own():
    """Every call on a stream other than the default one, whose inputs are made there too."""
    s = torch.cuda.Stream()
    c = Q.cache(91, 1, 2, 2, 64, [50, 7], 16, 8, cap_rows=64)
    with torch.cuda.stream(s):
        gpu = Q.to_gpu(c)
        x = synth.normal((1, 2, 1, 8, 64), g=synth.gen(91, 5), dtype=BF).cuda()
        one = torch.ones((1, 64), dtype=BF, device="cuda")
        q, k = ddt.ddt_qk_norm_rope(x[..., :4, :], x[..., 4:6, :], one, one, gpu[5][:, None].contiguous())
        v = x[..., 6:, :].contiguous()
        o = ddt.ddt_decode_attn_paged_quant(q[:, :, 0].contiguous(), k[:, :, 0].contiguous(), v[:, :, 0].contiguous(), *gpu, scale=0.125,
                                            out_dtype=F32)["o"]
        want, bound = Q.decode_ref(Q.f64(q[:, :, 0]), Q.f64(k[:, :, 0]), Q.f64(v[:, :, 0]), c, 0.125, BF)
        ddt.ddt_append_paged_quant(k, v, *gpu, torch.ones(2, dtype=torch.int32, device="cuda"))
        back = [torch.zeros((1, 2, 2, 64, 64), device="cuda") for _ in range(2)]
        ddt.ddt_read_paged_quant(*gpu, *back)
    s.synchronize()
    assert (np.abs(Q.f64(o) - want) <= bound + Q.U * np.abs(want)).all()
    assert gpu[5].tolist() == [51, 8]
    for x, codes, scale, t in ((k, "k", "ks", back[0]), (v, "v", "vs", back[1])):
        Q.append_ref(Q.f64(x), c[codes], c[scale], c["table"], [50, 7], [1, 1], None)
        for b, n in enumerate((51, 8)):
            assert np.array_equal(Q.f64(t)[:, b, :, :n], Q.rows_of(c[codes], c[scale], c["table"], b, n))
