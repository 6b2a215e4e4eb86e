"""Operators of the serving path beside the verification round, and the cases they are measured on.

  decode_attn     attention of one new token a request over the paged key-value cache, with the sums of the
                  attention weights that every cached row has received
  evict           eviction from that cache by those sums, in place
  token_logprobs  log probabilities of given tokens under the target's logits, with entropy and top alternatives

`run` computes an operator from elementary torch operations in 32 bits where `own` is false, and calls the
library's entry point of that operator where it is true.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one user's plain step at the head shape of the batched round's attention layers: latency
        dict(name="decode one short", op="decode", L=1, B=1, Hq=24, Hkv=4, d=256, page=64, lo=1000, hi=1000, weights=False,
             dtype="bf16", lens=1),
        # the batched round's 32 requests in a step without drafts, the weights kept for a later eviction
        dict(name="decode batch ragged", op="decode", L=1, B=32, Hq=24, Hkv=4, d=256, page=64, lo=1024, hi=32768,
             weights=True, dtype="bf16", lens=2),
        # one very long document, small pages, grouped heads of 128
        dict(name="decode one long", op="decode", L=1, B=1, Hq=32, Hkv=8, d=128, page=16, lo=131071, hi=131071, weights=True,
             dtype="bf16", lens=3),
        # many short chats, every head with keys of its own (no sharing), heads of 64, both layers of a draft model at once
        dict(name="decode many short", op="decode", L=2, B=96, Hq=16, Hkv=16, d=64, page=32, lo=0, hi=2500, weights=False,
             dtype="bf16", lens=4),
        # the fp32 configuration, as used to check a model: a few short requests
        dict(name="decode fp32", op="decode", L=1, B=8, Hq=8, Hkv=2, d=64, page=16, lo=255, hi=4097, weights=True,
             dtype="fp32", lens=5),
        # one request's cache of one layer cut to half
        dict(name="evict one", op="evict", L=1, B=1, Hkv=4, d=256, page=64, lo=2001, hi=2001, keep=1000, sink=4, recent=128,
             placed=0.0, dtype="bf16", lens=6),
        # the steady state of a batch under a budget: every request is a little over it
        dict(name="evict steady", op="evict", L=4, B=32, Hkv=8, d=128, page=16, lo=4100, hi=4224, keep=4096, sink=4,
             recent=256, placed=0.96, dtype="bf16", lens=7),
        # long ragged prompts cut to the budget after their prefill; some are already under it
        dict(name="evict prompts", op="evict", L=2, B=16, Hkv=4, d=256, page=64, lo=3000, hi=32768, keep=8192, sink=16,
             recent=1024, placed=0.0, dtype="bf16", lens=8),
        # the log probabilities of one round's emitted tokens, one request
        dict(name="logprobs one", op="logprobs", B=1, N=65, V=151936, A=16, valid=3, top=5, T=1.0, std=3.0, dtype="bf16"),
        # the same for the batched round, at a temperature
        dict(name="logprobs batch", op="logprobs", B=32, N=65, V=151936, A=16, valid=5, top=5, T=0.7, std=3.0, dtype="bf16"),
        # every token of a prompt scored
        dict(name="logprobs prompt", op="logprobs", B=1, N=2047, V=151936, A=0, valid=0, top=20, T=1.0, std=3.0, dtype="bf16"),
        # fp32 logits over a vocabulary of odd size, entropy and log probabilities alone
        dict(name="logprobs fp32", op="logprobs", B=4, N=300, V=32003, A=0, valid=0, top=0, T=1.3, std=2.0, dtype="fp32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("decode", "decode", "evict", "evict", "logprobs", "logprobs"))
    if op == "logprobs":
        dtype = rng.choice(("bf16", "bf16", "fp32"))
        V = _log_int(rng, 40, 200000)
        rows = max(1, min(_log_int(rng, 1, 4096), 150_000_000 // V))
        B = _log_int(rng, 1, max(1, min(32, rows)))
        N = max(1, rows // B)
        walk = rng.random() < 0.5
        A = rng.randint(1, 17) if walk else 0
        return dict(op=op, B=B, N=N, V=V, A=A, valid=rng.randint(1, A) if walk else 0, top=rng.choice((0, 1, 5, 20, 32)),
                    T=round(rng.uniform(0.3, 2.0), 2), std=round(rng.uniform(0.5, 5.0), 2), dtype=dtype)
    dtype = rng.choice(("bf16", "bf16", "bf16", "fp32"))
    d = rng.choice((64, 128, 256))
    Hkv = rng.choice((1, 2, 4, 8, 16))
    L = rng.choice((1, 1, 1, 2, 3))
    page = rng.choice((8, 16, 32, 64, 128, 192, 256))
    row = 2 * d * Hkv * L * (2 if dtype == "bf16" else 4)
    if op == "decode":
        G = rng.choice((1, 2, 3, 4, 5, 6, 8, 12, 16))
        rows = min(_log_int(rng, 500, 400_000), 1_500_000_000 // row)
        B = min(_log_int(rng, 1, 128), max(1, rows // 100))
        hi = max(1, 2 * rows // B - 1) if B > 1 else rows
        return dict(op=op, L=L, B=B, Hq=G * Hkv, Hkv=Hkv, d=d, page=page, lo=rng.choice((0, 1, hi // 8)) if B > 1 else rows,
                    hi=hi, weights=rng.random() < 0.5, dtype=dtype, lens=rng.randint(100, 1 << 30))
    rows = min(_log_int(rng, 500, 200_000), 1_000_000_000 // row)
    B = min(_log_int(rng, 1, 64), max(1, rows // 200))
    hi = max(64, rows // B)
    keep = max(32, int(hi * rng.uniform(0.1, 0.95)))
    return dict(op=op, L=L, B=B, Hkv=Hkv, d=d, page=page, lo=min(hi, keep + 1) if rng.random() < 0.5 else hi // 4, hi=hi,
                keep=keep, sink=rng.randint(0, 8), recent=rng.randint(0, keep // 4), placed=rng.choice((0.0, 0.5, 0.9)),
                dtype=dtype, lens=rng.randint(100, 1 << 30))


def _lengths(case):
    """The requests' cached rows: part of the case, so that every seed does the same work."""
    r = random.Random(case["lens"])
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["B"])]


def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed((int(seed) * 1000003 + salt) & ((1 << 62) - 1))
    return g


# ------------------------------------------------------------------------------------------------ inputs
def _paged_cache(case, g, rows):
    """Pages of normal values behind a shuffled block table with two spare pages."""
    dt, page = DTYPES[case["dtype"]], case["page"]
    max_pages = max(1, -(-rows // page))
    num_pages = case["B"] * max_pages + 2
    shape = (case["L"], num_pages, case["Hkv"], page, case["d"])
    k = torch.randn(shape, generator=g, device="cuda", dtype=dt)
    v = torch.randn(shape, generator=g, device="cuda", dtype=dt)
    table = torch.randperm(num_pages, generator=g, device="cuda")[:case["B"] * max_pages].reshape(case["B"], max_pages)
    return k, v, table.to(torch.int32).contiguous()


def _prepare_decode(case, seed):
    g = _gen(seed, 1)
    L, B, Hq, Hkv, d = (case[k] for k in ("L", "B", "Hq", "Hkv", "d"))
    dt, lens = DTYPES[case["dtype"]], _lengths(case)
    k_pages, v_pages, table = _paged_cache(case, g, max(lens) + 1)
    cap = table.shape[1] * case["page"]
    s = dict(case=case, k_pages=k_pages, v_pages=v_pages, table=table,
             q=(1.5 * torch.randn((L, B, Hq, d), generator=g, device="cuda")).to(dt),
             k_new=torch.randn((L, B, Hkv, d), generator=g, device="cuda", dtype=dt),
             v_new=torch.randn((L, B, Hkv, d), generator=g, device="cuda", dtype=dt),
             prefix_len=torch.tensor(lens, dtype=torch.int32, device="cuda"), scale=1.0 / math.sqrt(d),
             weight=torch.zeros((L, B, Hkv, cap), device="cuda") if case["weights"] else None)
    if own:
        from tree_speculative_decoding_02_gb300 import ddt
        s["out"] = torch.empty((L, B, Hq, d), dtype=dt, device="cuda")
        s["status"] = torch.empty((B,), dtype=torch.int32, device="cuda")
        s["workspace"] = ddt.decode_attn_paged_workspace(s["q"], k_pages, table, weights=case["weights"])
    return s


def _prepare_evict(case, seed):
    g = _gen(seed, 2)
    L, B, Hkv = (case[k] for k in ("L", "B", "Hkv"))
    lens = _lengths(case)
    k_pages, v_pages, table = _paged_cache(case, g, max(lens))
    cap = table.shape[1] * case["page"]
    P = torch.tensor(lens, dtype=torch.int32, device="cuda")
    # sums of attention weights are heavy-tailed; a fifth of the rows has never been looked at
    w = torch.exp(2.0 * torch.randn((L, B, Hkv, cap), generator=g, device="cuda"))
    w *= torch.rand((L, B, Hkv, cap), generator=g, device="cuda") >= 0.2
    w *= torch.arange(cap, device="cuda") < P[:, None, None]
    # rows left by an earlier eviction hold tokens of any position, in no order
    placed = torch.clamp((P * case["placed"]).to(torch.int32), max=case["keep"])
    gone = torch.where(placed > 0, P // 2, torch.zeros_like(P))   # tokens that earlier evictions dropped
    seq = (P + gone).to(torch.int32)
    most = int(max(lens)) + int(max(lens)) // 2 + 1
    order = torch.rand((L, B, Hkv, most), generator=g, device="cuda")
    order.masked_fill_(torch.arange(most, device="cuda") >= (placed + gone)[:, None, None], 2.0)
    pos = torch.argsort(order, dim=-1)[..., :cap].to(torch.int32)
    pos = torch.nn.functional.pad(pos, (0, cap - pos.shape[-1]), value=-1)
    pos = torch.where(torch.arange(cap, device="cuda") < placed[:, None, None], pos, torch.full_like(pos, -1)).contiguous()
    s = dict(case=case, k_pages=k_pages, v_pages=v_pages, table=table, weight=w, row_pos=pos, prefix_len=P,
             n_placed=placed.contiguous(), seq_len=seq)
    if own:
        from tree_speculative_decoding_02_gb300 import ddt
        s["status"] = torch.empty((B,), dtype=torch.int32, device="cuda")
        s["workspace"] = ddt.evict_paged_workspace(k_pages, table)
    return s


def _prepare_logprobs(case, seed):
    g = _gen(seed, 3)
    B, N, V, A = (case[k] for k in ("B", "N", "V", "A"))
    logits = torch.empty((B, N, V), dtype=DTYPES[case["dtype"]], device="cuda")
    for b in range(B):   # a few tokens of every row stand out, as in a trained model's output
        x = case["std"] * torch.randn((N, V), generator=g, device="cuda")
        top = torch.randint(0, V, (N, 3), generator=g, device="cuda")
        x.scatter_add_(1, top, 4.0 * case["std"] * torch.rand((N, 3), generator=g, device="cuda"))
        logits[b] = x
    if A:   # a walk's accepted rows (ascending, -1 behind the last) and its emitted tokens
        r = random.Random(int(seed))
        node = torch.full((B, A), -1, dtype=torch.int32)
        for b in range(B):
            n = min(r.randint(max(1, case["valid"] - 2), case["valid"]), N)
            node[b, :n] = torch.tensor([0] + sorted(r.sample(range(1, N), n - 1)), dtype=torch.int32)
        node = node.cuda()
    else:
        node = None
    token = torch.randint(0, V, (B, A or N), generator=g, device="cuda", dtype=torch.int32)
    best = logits.float().argmax(-1).to(torch.int32)
    if A:
        best = torch.gather(best, 1, node.clamp(min=0).long())
    token = torch.where(torch.rand((B, A or N), generator=g, device="cuda") < 0.6, best, token)
    if A:
        token = torch.where(node < 0, torch.full_like(token, -1), token)
    s = dict(case=case, logits=logits, node=node, token=token.contiguous())
    if own:
        from tree_speculative_decoding_02_gb300 import ddt
        s["workspace"] = ddt.token_logprobs_workspace(logits, s["token"])
        one, top = tuple(token.shape), tuple(token.shape) + (case["top"],)
        s["out"] = {"logprob": torch.empty(one, device="cuda"), "entropy": torch.empty(one, device="cuda"),
                    "status": torch.empty(one, dtype=torch.int32, device="cuda")}
        if case["top"]:
            s["out"].update(top_token=torch.empty(top, dtype=torch.int32, device="cuda"),
                            top_logprob=torch.empty(top, device="cuda"))
    return s


def prepare(case, seed):
    return {"decode": _prepare_decode, "evict": _prepare_evict, "logprobs": _prepare_logprobs}[case["op"]](case, seed)


# ------------------------------------------------------------------------------------------------ plain forms
def _rows(pages, table):
    """[L][num_pages][Hkv][page][d] through a table [B][n] -> [L][B][Hkv][n * page][d] in 32 bits."""
    x = pages[:, table.long()]
    L, B, n, Hkv, page, d = x.shape
    return x.permute(0, 1, 3, 2, 4, 5).reshape(L, B, Hkv, n * page, d).float()


def _plain_decode(s):
    case = s["case"]
    L, B, Hq, Hkv, d = (case[k] for k in ("L", "B", "Hq", "Hkv", "d"))
    P = s["prefix_len"]
    K, V = _rows(s["k_pages"], s["table"]), _rows(s["v_pages"], s["table"])
    cap = K.shape[3]
    q = s["q"].float().reshape(L, B, Hkv, Hq // Hkv, d)
    score = torch.matmul(q, K.transpose(-1, -2)) * s["scale"]
    score.masked_fill_(torch.arange(cap, device="cuda") >= P[:, None, None, None], -math.inf)
    mine = (q * s["k_new"].float()[:, :, :, None]).sum(-1, keepdim=True) * s["scale"]
    m = torch.maximum(score.amax(-1, keepdim=True), mine)
    e, em = torch.exp(score - m), torch.exp(mine - m)
    z = e.sum(-1, keepdim=True) + em
    o = (torch.matmul(e, V) + em * s["v_new"].float()[:, :, :, None]) / z
    out = [o.reshape(L, B, Hq, d).to(s["q"].dtype)]
    if s["weight"] is not None:
        at = P.long()[None, :, None, None].expand(L, B, Hkv, 1)
        s["weight"] += (e / z).sum(-2)
        s["weight"].scatter_add_(-1, at, (em / z).sum(-2))
        out.append(s["weight"])
    return out


def _plain_evict(s, w, pos, P, placed):
    case = s["case"]
    keep, page, cap = case["keep"], case["page"], w.shape[-1]
    i = torch.arange(cap, device="cuda")
    n, seq = P[:, None, None], s["seq_len"][:, None, None]
    cut = n > keep
    where = torch.where(i < placed[:, None, None], pos, seq - n + i)
    live = i < n
    guard = live & ((where < case["sink"]) | (where >= seq - case["recent"]))
    key = torch.where(guard, math.inf, torch.where(live, w, -math.inf))
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    kept = torch.zeros_like(live.expand_as(w)).scatter_(-1, order, (i < keep).expand_as(w)) & live
    hole, mover = cut & (i < keep) & ~kept, cut & (i >= keep) & kept
    l, b, g, dst = hole.nonzero(as_tuple=True)
    src = mover.nonzero(as_tuple=True)[3]
    to, of = s["table"][b, dst // page].long(), s["table"][b, src // page].long()
    s["k_pages"][l, to, g, dst % page] = s["k_pages"][l, of, g, src % page]
    s["v_pages"][l, to, g, dst % page] = s["v_pages"][l, of, g, src % page]
    new = torch.where(cut & (i < keep), where, pos).to(torch.int32)
    new[l, b, g, dst] = where[l, b, g, src].to(torch.int32)
    w[l, b, g, dst] = w[l, b, g, src]
    w.masked_fill_(cut & (i >= keep) & live, 0.0)
    pos.copy_(torch.where(cut & (i >= keep) & live, torch.full_like(new, -1), new))
    placed.copy_(torch.where(P > keep, torch.full_like(P, keep), placed))
    P.clamp_(max=keep)


def _plain_logprobs(s):
    case = s["case"]
    x, token = s["logits"], s["token"]
    if s["node"] is not None:
        x = torch.gather(x, 1, s["node"].clamp(min=0).long()[..., None].expand(-1, -1, x.shape[-1]))
    x = x.float()
    u = (x - x.amax(-1, keepdim=True)) / case["T"]
    e = torch.exp(u)
    z = e.sum(-1, keepdim=True)
    lse = torch.log(z)
    fine = (token >= 0)
    logprob = torch.gather(u - lse, -1, token.clamp(min=0).long()[..., None])[..., 0]
    out = [torch.where(fine, logprob, torch.zeros_like(logprob)),
           torch.where(fine, lse[..., 0] - ((e * u).sum(-1, keepdim=True) / z)[..., 0], torch.zeros_like(logprob))]
    if case["top"]:
        ids = torch.sort(x, dim=-1, descending=True, stable=True).indices[..., :case["top"]]
        out.append(torch.where(fine[..., None], ids, torch.full_like(ids, -1)).to(torch.int32))
        out.append(torch.where(fine[..., None], torch.gather(u, -1, ids) - lse, torch.zeros_like(lse)))
    return out


def run(s):
    case = s["case"]
    if own:
        from tree_speculative_decoding_02_gb300 import ddt
    if case["op"] == "decode":
        if not own:
            return _plain_decode(s)
        ddt.ddt_decode_attn_paged(s["q"], s["k_new"], s["v_new"], s["k_pages"], s["v_pages"], s["table"], s["prefix_len"],
                                  scale=s["scale"], attn_weight=s["weight"], out=s["out"], status=s["status"],
                                  workspace=s["workspace"])
        return [s["out"]] + ([s["weight"]] if s["weight"] is not None else [])
    if case["op"] == "evict":
        # the eviction updates its sums, positions and lengths in place: a pass takes a copy of them (a few
        # bytes a row) so that the next pass on this state has as much to evict
        w, pos, P, placed = s["weight"].clone(), s["row_pos"].clone(), s["prefix_len"].clone(), s["n_placed"].clone()
        if own:
            ddt.ddt_evict_paged(s["k_pages"], s["v_pages"], s["table"], P, placed, s["seq_len"], w, pos, keep=case["keep"],
                                n_sink=case["sink"], n_recent=case["recent"], status=s["status"], workspace=s["workspace"])
        else:
            _plain_evict(s, w, pos, P, placed)
        return [s["k_pages"], s["v_pages"], w, pos, P, placed]
    if not own:
        return _plain_logprobs(s)
    r = ddt.ddt_token_logprobs(s["logits"], s["token"], node=s["node"], top_n=case["top"], temperature=case["T"],
                               out=s["out"], workspace=s["workspace"])
    return [r["logprob"], r["entropy"]] + ([r["top_token"], r["top_logprob"]] if case["top"] else [])


# ------------------------------------------------------------------------------------------------ work
def work(case):
    esz = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "decode":
        L, B, Hq, Hkv, d = (case[k] for k in ("L", "B", "Hq", "Hkv", "d"))
        rows = sum(_lengths(case)) + B
        return {"bytes": L * (2 * rows * Hkv * d * esz + 2 * B * Hq * d * esz + (8 * rows * Hkv if case["weights"] else 0)),
                "flops": 4 * L * Hq * d * rows}
    if case["op"] == "evict":
        L, Hkv, d, keep = (case[k] for k in ("L", "Hkv", "d", "keep"))
        total = 0.0
        for n in _lengths(case):
            total += 8 * n   # the weights read, the positions or weights written
            if n > keep:
                # of the rows behind the budget's last the recent ones stay, and of the others as large a part as of all
                recent = min(case["recent"], n - keep)
                part = max(0.0, (keep - case["sink"] - case["recent"]) / max(1, n - case["sink"] - case["recent"]))
                total += (recent + (n - keep - recent) * part) * 2 * 2 * d * esz
        return {"bytes": L * Hkv * total, "flops": 0}
    rows = case["B"] * ((case["valid"] if case["valid"] < 3 else case["valid"] - 1) if case["A"] else case["N"])
    return {"bytes": rows * (case["V"] * esz + 12 + 8 * case["top"]), "flops": 5 * rows * case["V"]}


# ------------------------------------------------------------------------------------------------ in 64 bits
def _exact_decode(case, seed):
    s = _prepare_decode(case, seed)
    page, G = case["page"], case["Hq"] // case["Hkv"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    w = torch.zeros(s["weight"].shape, dtype=torch.float64, device="cuda") if case["weights"] else None
    for b, n in enumerate(_lengths(case)):
        pages = s["table"][b, :-(-n // page)].long()
        for l in range(case["L"]):
            for g in range(case["Hkv"]):
                k = s["k_pages"][l, pages, g].reshape(-1, case["d"])[:n]
                v = s["v_pages"][l, pages, g].reshape(-1, case["d"])[:n]
                k = torch.cat([k, s["k_new"][l, b, g][None]]).double()
                v = torch.cat([v, s["v_new"][l, b, g][None]]).double()
                p = torch.softmax(s["q"][l, b, g * G:(g + 1) * G].double() @ k.T * s["scale"], dim=-1)
                o[l, b, g * G:(g + 1) * G] = p @ v
                if w is not None:
                    w[l, b, g, :n + 1] = p.sum(0)
    return [o] + ([w] if w is not None else [])


def _exact_evict(case, seed):
    s = _prepare_evict(case, seed)
    page, keep = case["page"], case["keep"]
    w, pos, table = s["weight"].cpu().numpy(), s["row_pos"].cpu().numpy(), s["table"].cpu().numpy()
    P, placed, seq = (s[k].cpu().numpy().copy() for k in ("prefix_len", "n_placed", "seq_len"))
    at = []
    for b in range(case["B"]):
        n = int(P[b])
        if n <= keep:
            continue
        idx = np.arange(n)
        for l in range(case["L"]):
            for g in range(case["Hkv"]):
                p = np.where(idx < placed[b], pos[l, b, g, :n], seq[b] - n + idx)
                safe = (p < case["sink"]) | (p >= seq[b] - case["recent"])
                best = np.lexsort((idx, -w[l, b, g, :n].astype(np.float64), ~safe))[:keep]
                holes, moved = np.setdiff1d(idx[:keep], best), np.sort(best[best >= keep])
                at.append((np.full(len(holes), l), np.full(len(holes), b), np.full(len(holes), g), holes, moved))
                w[l, b, g, holes], p[holes] = w[l, b, g, moved], p[moved]
                pos[l, b, g, :keep] = p[:keep]
                w[l, b, g, keep:n], pos[l, b, g, keep:n] = 0, -1
        P[b] = placed[b] = keep
    if at:
        l, b, g, dst, src = (np.concatenate(x) for x in zip(*at))
        to, of = torch.from_numpy(table[b, dst // page]).long(), torch.from_numpy(table[b, src // page]).long()
        l, g, dst, src = (torch.from_numpy(x) for x in (l, g, dst % page, src % page))
        for t in (s["k_pages"], s["v_pages"]):
            t[l.cuda(), to.cuda(), g.cuda(), dst.cuda()] = t[l.cuda(), of.cuda(), g.cuda(), src.cuda()]
    return [s["k_pages"], s["v_pages"], w.astype(np.float64), pos, P, placed]


def _exact_logprobs(case, seed):
    s = _prepare_logprobs(case, seed)
    B, A = s["token"].shape
    logprob, entropy = torch.zeros((B, A), dtype=torch.float64), torch.zeros((B, A), dtype=torch.float64)
    ids = torch.full((B, A, case["top"]), -1, dtype=torch.int32)
    best = torch.zeros((B, A, case["top"]), dtype=torch.float64)
    token = s["token"].cpu()
    for b in range(B):
        of = s["node"][b] if s["node"] is not None else torch.arange(A, device="cuda")
        for lo in range(0, A, 256):
            row = of[lo:lo + 256]
            row = row[row >= 0].long()
            n = len(row)
            if not n:
                continue
            x = s["logits"][b, row].double()
            lp = torch.log_softmax(x / case["T"], dim=-1)
            logprob[b, lo:lo + n] = torch.gather(lp, 1, token[b, lo:lo + n].long().cuda()[:, None])[:, 0].cpu()
            entropy[b, lo:lo + n] = -(torch.exp(lp) * lp).sum(-1).cpu()
            if case["top"]:
                pick = torch.argsort(-x, dim=-1, stable=True)[:, :case["top"]]
                ids[b, lo:lo + n] = pick.to(torch.int32).cpu()
                best[b, lo:lo + n] = torch.gather(lp, 1, pick).cpu()
    return [logprob, entropy] + ([ids, best] if case["top"] else [])


def exact(case, seed):
    global own
    mine, own = own, False   # inputs alone, without the library
    try:
        return {"decode": _exact_decode, "evict": _exact_evict, "logprobs": _exact_logprobs}[case["op"]](case, seed)
    finally:
        own = mine
