"""Operators of a paged key-value cache held in 8 bits, and the cases they are measured on.

  norm_rope  root-mean-square norms of every query and key head, with the rotation by position in the same pass
  append     rows quantised as they are written to the cache: e4m3 codes, a power-of-two scale for each block of
             tokens and head
  read       the cache's rows read back into a contiguous cache of 16 or 32 bits
  decode     attention of one new token a request over that cache

`run` computes an operator from elementary torch operations in 32 bits where `own` is false, and calls the
library's entry point of that operator where it is true.
"""
import math
import random

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one token of one user, at the head shape of the batched round's attention layers: latency
        dict(name="norm one token", op="norm", L=1, B=1, N=1, Hq=24, Hkv=4, d=256, rot=64, fused=True, pad=False, pos=1000,
             dtype="bf16"),
        # the tree rows of the batched round: 32 requests, 16 layers, rows past a request's nodes left alone
        dict(name="norm round", op="norm", L=16, B=32, N=65, Hq=24, Hkv=4, d=256, rot=64, fused=False, pad=True, pos=32768,
             dtype="bf16"),
        # prompts of an odd length, q and k as they lie in one projection, fp32 as used to check a model
        dict(name="norm prompt fp32", op="norm", L=1, B=3, N=1471, Hq=16, Hkv=2, d=128, rot=128, fused=True, pad=False,
             pos=131072, dtype="fp32"),
        # the row of one token of one request, one layer: latency
        dict(name="append one", op="append", L=1, B=1, N=1, A=0, Hkv=4, d=256, page=64, block=16, lo=1000, hi=1000, clo=1,
             chi=1, dtype="bf16", lens=1),
        # the accepted rows of the batched round's trees
        dict(name="append commit", op="append", L=16, B=32, N=65, A=16, Hkv=4, d=256, page=64, block=16, lo=256, hi=2048, clo=1,
             chi=5, dtype="bf16", lens=2),
        # ragged prompts into an empty cache, small pages
        dict(name="append prompts", op="append", L=1, B=6, N=16384, A=0, Hkv=8, d=128, page=16, block=16, lo=0, hi=0, clo=2001,
             chi=16384, dtype="bf16", lens=3),
        # one layer of the batched round's prefixes, read back for the tree attention
        dict(name="read layer", op="read", L=1, B=32, Hkv=4, d=256, page=64, block=16, lo=1024, hi=32768, dtype="bf16", lens=4),
        # a few short requests, fp32
        dict(name="read fp32", op="read", L=2, B=5, Hkv=2, d=64, page=32, block=32, lo=1, hi=4097, dtype="fp32", lens=5),
        # one user's plain step: latency
        dict(name="decode one short", op="decode", L=1, B=1, Hq=24, Hkv=4, d=256, page=64, block=16, lo=1000, hi=1000,
             dtype="bf16", lens=6),
        # the batched round's 32 requests in a step without drafts
        dict(name="decode batch ragged", op="decode", L=1, B=32, Hq=24, Hkv=4, d=256, page=64, block=64, lo=1024, hi=32768,
             dtype="bf16", lens=7),
        # one very long document, small pages
        dict(name="decode one long", op="decode", L=1, B=1, Hq=32, Hkv=8, d=128, page=16, block=16, lo=131071, hi=131071,
             dtype="bf16", lens=8),
        # many short chats, every head with keys of its own, both layers of a draft model at once
        dict(name="decode many short", op="decode", L=2, B=96, Hq=16, Hkv=16, d=64, page=32, block=32, lo=0, hi=2500,
             dtype="bf16", lens=9),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "append", "read", "decode", "decode"))
    dtype = rng.choice(("bf16", "bf16", "bf16", "fp32"))
    d, Hkv = rng.choice((64, 128, 256)), rng.choice((1, 2, 4, 8))
    if op == "norm":
        Hq, L = Hkv * rng.choice((1, 2, 4, 6, 8)), rng.choice((1, 1, 2, 4))
        rows = min(_log_int(rng, 1, 60_000), 400_000_000 // (L * (Hq + Hkv) * d * (4 if dtype == "fp32" else 2)))
        B = _log_int(rng, 1, max(1, min(32, rows)))
        return dict(op=op, L=L, B=B, N=max(1, rows // B), Hq=Hq, Hkv=Hkv, d=d, rot=16 * rng.randint(1, d // 16),
                    fused=rng.random() < 0.5, pad=rng.random() < 0.5, pos=_log_int(rng, 10, 1_000_000), dtype=dtype)
    page = rng.choice((8, 16, 32, 64, 128, 192, 256))
    block = rng.choice([s for s in (8, 16, 32, 64, 128) if page % s == 0])
    L = rng.choice((1, 1, 1, 2, 3))
    same = dict(op=op, L=L, Hkv=Hkv, d=d, page=page, block=block, dtype=dtype, lens=rng.randint(100, 1 << 30))
    if op == "append":
        rows = min(_log_int(rng, 1, 60_000), 300_000_000 // (L * Hkv * d * (4 if dtype == "fp32" else 2)))
        B = _log_int(rng, 1, max(1, min(48, rows)))
        N = max(1, rows // B)
        A = rng.randint(1, min(N, 17)) if rng.random() < 0.5 else 0
        hi = _log_int(rng, 1, 3000)
        return dict(same, B=B, N=N, A=A, lo=rng.choice((0, hi)), hi=hi, clo=rng.choice((0, 1)), chi=A or N)
    row = L * Hkv * d
    if op == "read":
        rows = min(_log_int(rng, 100, 300_000), 500_000_000 // row)
        B = _log_int(rng, 1, max(1, min(32, rows // 50)))
        hi = max(1, rows // B)
        return dict(same, B=B, lo=rng.choice((0, hi // 8, hi)), hi=hi)
    G = rng.choice((1, 2, 3, 4, 6, 8, 12, 16))
    rows = min(_log_int(rng, 500, 400_000), 700_000_000 // row)
    B = min(_log_int(rng, 1, 128), max(1, rows // 100))
    hi = max(1, 2 * rows // B - 1) if B > 1 else rows
    return dict(same, B=B, Hq=G * Hkv, lo=rng.choice((0, 1, hi // 8)) if B > 1 else rows, hi=hi)


def _lengths(case, lo="lo", hi="hi", salt=0):
    """The requests' cached (or new) rows: part of the case, so that every seed does the same work."""
    r = random.Random(case["lens"] + salt)
    return [r.randint(case[lo], case[hi]) for _ in range(case["B"])]


def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed((int(seed) * 1000003 + salt) & ((1 << 62) - 1))
    return g


# ------------------------------------------------------------------------------------------------ the 8-bit format
def _scale(byte):
    """2^(byte - 127); 0 for byte 0, the mark of a block of zeros."""
    return (byte.to(torch.int32) << 23).view(torch.float32)


def _byte(amax):
    """The byte of the smallest e in [-100, 120] with amax <= 448 * 2^e; 0 for amax 0."""
    bits = amax.contiguous().view(torch.int32)
    e = torch.clamp((bits >> 23) - 135 + ((bits & 0x7FFFFF) > 0x600000), -100, 120)
    return torch.where(amax > 0, e + 127, torch.zeros_like(e)).to(torch.uint8)


def _codes(x, byte):
    """The e4m3 codes of x under the scales: to nearest, ties to even; what is not finite becomes NaN."""
    inv = torch.where(byte > 0, _scale(254 - byte.to(torch.int32)), torch.zeros((), device=x.device))
    return torch.where(torch.isfinite(x), x * inv, math.nan).to(torch.float8_e4m3fn).view(torch.uint8)


def _cache(case, g, rows):
    """Quantised pages of normal values (layers and heads of different sizes) behind a shuffled block table with two
    spare pages."""
    L, B, Hkv, page, d, S = (case[k] for k in ("L", "B", "Hkv", "page", "d", "block"))
    max_pages = max(1, -(-rows // page))
    num = B * max_pages + 2
    out = []
    for _ in range(2):
        codes = torch.empty((L, num, Hkv, page, d), dtype=torch.uint8, device="cuda")
        byte = torch.empty((L, num, Hkv, page // S), dtype=torch.uint8, device="cuda")
        size = torch.exp(0.5 * torch.randn((L, 1, Hkv, 1, 1), generator=g, device="cuda"))
        step = max(1, (1 << 26) // (Hkv * page * d))
        for l in range(L):
            for i in range(0, num, step):
                x = torch.randn((min(step, num - i), Hkv, page // S, S * d), generator=g, device="cuda") * size[l]
                b = _byte(x.abs().amax(-1))
                byte[l, i:i + step] = b
                codes[l, i:i + step] = _codes(x, b[..., None]).view(-1, Hkv, page, d)
        out += [codes.view(torch.float8_e4m3fn), byte]
    table = torch.randperm(num, generator=g, device="cuda")[:B * max_pages].reshape(B, max_pages)
    return dict(k_pages=out[0], v_pages=out[2], k_scale=out[1], v_scale=out[3], table=table.to(torch.int32).contiguous())


# ------------------------------------------------------------------------------------------------ inputs
def _prepare_norm(case, seed):
    g = _gen(seed, 1)
    L, B, N, Hq, Hkv, d = (case[k] for k in ("L", "B", "N", "Hq", "Hkv", "d"))
    dt = DTYPES[case["dtype"]]
    if case["fused"]:   # as one projection leaves them, values behind the keys
        x = (1.5 * torch.randn((L, B, N, Hq + 2 * Hkv, d), generator=g, device="cuda")).to(dt)
        q, k = x[..., :Hq, :], x[..., Hq:Hq + Hkv, :]
    else:
        q = (1.5 * torch.randn((L, B, N, Hq, d), generator=g, device="cuda")).to(dt)
        k = (1.5 * torch.randn((L, B, N, Hkv, d), generator=g, device="cuda")).to(dt)
    r = random.Random(int(seed))
    start = torch.tensor([r.randint(0, case["pos"]) for _ in range(B)], device="cuda")
    if case["pad"]:     # a tree's rows share a depth with their siblings; the rows past the nodes are padding
        depth = torch.sort(torch.randint(0, 16, (B, N), generator=g, device="cuda"), dim=-1).values
        nodes = torch.tensor([r.randint(max(1, N // 2), N) for _ in range(B)], dtype=torch.int32, device="cuda")
    else:
        depth, nodes = torch.arange(N, device="cuda")[None], None
    return dict(case=case, q=q, k=k, qw=(1 + 0.2 * torch.randn((L, d), generator=g, device="cuda")).to(dt),
                kw=(1 + 0.2 * torch.randn((L, d), generator=g, device="cuda")).to(dt),
                position=(start[:, None] + depth).to(torch.int32).contiguous(), nodes=nodes,
                q_out=torch.zeros((L, B, N, Hq, d), dtype=dt, device="cuda"),
                k_out=torch.zeros((L, B, N, Hkv, d), dtype=dt, device="cuda"))


def _prepare_append(case, seed):
    g = _gen(seed, 2)
    L, B, N, Hkv, d = (case[k] for k in ("L", "B", "N", "Hkv", "d"))
    dt, lens, count = DTYPES[case["dtype"]], _lengths(case), _lengths(case, "clo", "chi", 1)
    s = dict(case=case, **_cache(case, g, max(p + c for p, c in zip(lens, count))))
    size = torch.exp(torch.randn((L, B, 1, Hkv, 1), generator=g, device="cuda"))   # some raise the scale of their first block
    s.update(k=(size * torch.randn((L, B, N, Hkv, d), generator=g, device="cuda")).to(dt),
             v=(size * torch.randn((L, B, N, Hkv, d), generator=g, device="cuda")).to(dt),
             prefix_len=torch.tensor(lens, dtype=torch.int32, device="cuda"),
             count=torch.tensor(count, dtype=torch.int32, device="cuda"), node=None,
             status=torch.empty((B,), dtype=torch.int32, device="cuda"))
    if case["A"]:       # a walk's accepted rows: ascending, -1 behind the last
        r = random.Random(int(seed))
        node = torch.full((B, case["A"]), -1, dtype=torch.int32)
        for b, c in enumerate(count):
            node[b, :c] = torch.tensor(([0] + sorted(r.sample(range(1, N), c - 1))) if c else [], dtype=torch.int32)
        s["node"] = node.cuda()
    return s


def _prepare_read(case, seed):
    g = _gen(seed, 3)
    lens = _lengths(case)
    s = dict(case=case, **_cache(case, g, max(lens)))
    shape = (case["L"], case["B"], case["Hkv"], max(1, max(lens)) + 3, case["d"])
    s.update(prefix_len=torch.tensor(lens, dtype=torch.int32, device="cuda"),
             k_out=torch.zeros(shape, dtype=DTYPES[case["dtype"]], device="cuda"),
             v_out=torch.zeros(shape, dtype=DTYPES[case["dtype"]], device="cuda"),
             status=torch.empty((case["B"],), dtype=torch.int32, device="cuda"))
    return s


def _prepare_decode(case, seed):
    g = _gen(seed, 4)
    L, B, Hq, Hkv, d = (case[k] for k in ("L", "B", "Hq", "Hkv", "d"))
    dt, lens = DTYPES[case["dtype"]], _lengths(case)
    s = dict(case=case, **_cache(case, g, max(lens) + 1))
    s.update(q=(1.5 * torch.randn((L, B, Hq, d), generator=g, device="cuda")).to(dt),
             k_new=torch.randn((L, B, Hkv, d), generator=g, device="cuda", dtype=dt),
             v_new=torch.randn((L, B, Hkv, d), generator=g, device="cuda", dtype=dt),
             prefix_len=torch.tensor(lens, dtype=torch.int32, device="cuda"), scale=1.0 / math.sqrt(d))
    if own:
        from tree_speculative_decoding_02_gb300 import ddt
        s["out"] = torch.empty((L, B, Hq, d), dtype=dt, device="cuda")
        s["status"] = torch.empty((B,), dtype=torch.int32, device="cuda")
        s["workspace"] = ddt.decode_attn_paged_quant_workspace(s["q"], s["k_pages"], s["table"])
    return s


def prepare(case, seed):
    op = {"norm": _prepare_norm, "append": _prepare_append, "read": _prepare_read, "decode": _prepare_decode}[case["op"]]
    return op(case, seed)


# ------------------------------------------------------------------------------------------------ plain forms
def _norm_one(x, w, cos, sin, eps, rot):
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w.float()[:, None, None, None]
    a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., rot:]], dim=-1)


def _plain_norm(s):
    rot, N = s["case"]["rot"], s["case"]["N"]
    freq = 10000.0 ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64, device="cuda") / rot)
    a = (s["position"].double()[..., None] * freq)[None, :, :, None]
    cos, sin = torch.cos(a).float(), torch.sin(a).float()
    out = []
    for name, w in (("q", "qw"), ("k", "kw")):
        y = _norm_one(s[name], s[w], cos, sin, 1e-6, rot).to(s[name].dtype)
        old = s[name + "_out"]
        if s["nodes"] is not None:
            y = torch.where((torch.arange(N, device="cuda") < s["nodes"][:, None])[None, :, :, None, None], y, old)
        old.copy_(y)
        out.append(old)
    return out


def _plain_append(s, P):
    case = s["case"]
    page, S, N = case["page"], case["block"], case["N"]
    A = case["A"] or N
    j = torch.arange(A, device="cuda")
    live = j < s["count"][:, None]
    at = P.long()[:, None] + j                                   # [B][A] positions
    first = (P // S).long()
    nb = A // S + 2
    blocks = first[:, None] + torch.arange(nb, device="cuda")     # the blocks that the new rows can fall into
    last = s["table"].shape[1] * page // S - 1
    bpage = torch.gather(s["table"].long(), 1, blocks.clamp(max=last) * S // page)
    inside = blocks.clamp(max=last) % (page // S)
    used = torch.zeros_like(blocks).scatter_add_(1, at // S - first[:, None], live.long()) > 0
    row = torch.arange(S, device="cuda")
    head = torch.arange(case["Hkv"], device="cuda")[:, None]
    for name in ("k", "v"):
        x = s[name].float()
        if s["node"] is not None:
            of = s["node"].clamp(min=0).long()[None, :, :, None, None]
            x = torch.gather(x, 2, of.expand(x.shape[0], -1, -1, *x.shape[3:]))
        size = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x)).amax(-1) * live[None, :, :, None]
        to = (at // S - first[:, None])[None, :, :, None].expand_as(size)
        amax = torch.zeros((x.shape[0], *blocks.shape, x.shape[3]), device="cuda").scatter_reduce(2, to, size, "amax")
        byte = _byte(amax)                                       # [L][B][nb][Hkv]
        scale, codes = s[name + "_scale"], s[name + "_pages"].view(torch.uint8)
        old = scale[:, bpage, :, inside].permute(2, 0, 1, 3)
        filled = (P % S > 0)[:, None] & (torch.arange(nb, device="cuda") == 0)
        old = torch.where(filled[None, :, :, None], old, torch.zeros_like(old))
        byte = torch.maximum(byte, old)
        raised = (byte > old) & (filled & used)[None, :, :, None]
        # rows that the first block has already, under its new scale
        l, b, _, h = raised[:, :, :1].nonzero(as_tuple=True)
        where = (l[:, None], bpage[b, 0][:, None], h[:, None], inside[b, 0][:, None] * S + row)
        have = codes[where]
        ratio = _scale(torch.clamp(127 + old[l, b, 0, h].to(torch.int32) - byte[l, b, 0, h].to(torch.int32), min=0))
        new = (have.view(torch.float8_e4m3fn).float() * ratio[:, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        codes[where] = torch.where((row < (P % S)[b][:, None])[..., None], new, have)
        b, n = used.nonzero(as_tuple=True)
        scale[:, bpage[b, n], :, inside[b, n]] = byte[:, b, n].permute(1, 0, 2)
        b, i = live.nonzero(as_tuple=True)
        pos = at[b, i]
        mine = byte[:, b, pos // S - first[b]]                   # [L][rows][Hkv]
        codes[:, s["table"][b, pos // page].long(), head, pos % page] = _codes(x[:, b, i], mine[..., None]).transpose(1, 2)
    P += s["count"]


def _values(codes, byte, table):
    """[L][num_pages][Hkv][page][d] codes through a table [B][n] -> [L][B][Hkv][n * page][d] in 32 bits."""
    x, e = codes.view(torch.uint8)[:, table.long()], byte[:, table.long()]
    L, B, n, Hkv, page, d = x.shape
    x = x.view(torch.float8_e4m3fn).float().view(L, B, n, Hkv, e.shape[-1], -1) * _scale(e)[..., None]
    return x.view(L, B, n, Hkv, page, d).permute(0, 1, 3, 2, 4, 5).reshape(L, B, Hkv, n * page, d)


def _plain_read(s):
    P, out = s["prefix_len"], []
    for name in ("k", "v"):
        x, to = _values(s[name + "_pages"], s[name + "_scale"], s["table"]), s[name + "_out"]
        n = min(x.shape[3], to.shape[3])
        live = (torch.arange(n, device="cuda") < P[:, None])[None, :, None, :, None]
        to[:, :, :, :n] = torch.where(live, x[:, :, :, :n].to(to.dtype), to[:, :, :, :n])
        out.append(to)
    return out


def _plain_decode(s):
    case = s["case"]
    L, B, Hq, Hkv, d = (case[k] for k in ("L", "B", "Hq", "Hkv", "d"))
    P = s["prefix_len"]
    K = _values(s["k_pages"], s["k_scale"], s["table"])
    q = s["q"].float().reshape(L, B, Hkv, Hq // Hkv, d)
    score = torch.matmul(q, K.transpose(-1, -2)) * s["scale"]
    del K
    score.masked_fill_(torch.arange(score.shape[-1], device="cuda") >= P[:, None, None, None], -math.inf)
    mine = (q * s["k_new"].float()[:, :, :, None]).sum(-1, keepdim=True) * s["scale"]
    m = torch.maximum(score.amax(-1, keepdim=True), mine)
    e, em = torch.exp(score - m), torch.exp(mine - m)
    V = _values(s["v_pages"], s["v_scale"], s["table"])
    o = (torch.matmul(e, V) + em * s["v_new"].float()[:, :, :, None]) / (e.sum(-1, keepdim=True) + em)
    return [o.reshape(L, B, Hq, d).to(s["q"].dtype)]


def run(s):
    op = s["case"]["op"]
    if own:
        from tree_speculative_decoding_02_gb300 import ddt
    if op == "norm":
        if not own:
            return _plain_norm(s)
        ddt.ddt_qk_norm_rope(s["q"], s["k"], s["qw"], s["kw"], s["position"], n_nodes=s["nodes"], rot_dim=s["case"]["rot"],
                             theta=10000.0, eps=1e-6, q_out=s["q_out"], k_out=s["k_out"])
        return [s["q_out"], s["k_out"]]
    if op == "append":
        P = s["prefix_len"].clone()   # advanced by the call: the next pass on this state starts where this one did
        if own:
            ddt.ddt_append_paged_quant(s["k"], s["v"], s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"], s["table"], P,
                                       s["count"], node=s["node"], status=s["status"])
        else:
            _plain_append(s, P)
        return [s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"], P]
    if op == "read":
        if not own:
            return _plain_read(s)
        ddt.ddt_read_paged_quant(s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"], s["table"], s["prefix_len"],
                                 s["k_out"], s["v_out"], status=s["status"])
        return [s["k_out"], s["v_out"]]
    if not own:
        return _plain_decode(s)
    ddt.ddt_decode_attn_paged_quant(s["q"], s["k_new"], s["v_new"], s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"],
                                    s["table"], s["prefix_len"], scale=s["scale"], out=s["out"], status=s["status"],
                                    workspace=s["workspace"])
    return [s["out"]]


# ------------------------------------------------------------------------------------------------ work
def work(case):
    esz = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm":
        rows = case["L"] * case["B"] * case["N"] * (0.75 if case["pad"] else 1.0)   # half to all of the rows are nodes
        n = rows * (case["Hq"] + case["Hkv"]) * case["d"]
        return {"bytes": 2 * esz * n, "flops": 8 * n}
    n = case["L"] * case["Hkv"] * case["d"]   # elements of K, and of V, in a row of all layers and heads
    if case["op"] == "append":
        count = sum(_lengths(case, "clo", "chi", 1))
        return {"bytes": 2 * n * count * (esz + 1), "flops": 4 * n * count}
    rows = sum(_lengths(case))
    if case["op"] == "read":
        return {"bytes": max(1, 2 * n * rows * (esz + 1)), "flops": 2 * n * rows}
    q = case["L"] * case["B"] * case["Hq"] * case["d"]
    return {"bytes": 2 * n * rows + 2 * n * rows // (case["block"] * case["d"]) + 2 * q * esz + 2 * n * case["B"] * esz,
            "flops": 4 * case["L"] * case["Hq"] * case["d"] * (rows + case["B"])}


# ------------------------------------------------------------------------------------------------ in 64 bits
def _exact_norm(case, seed):
    s, rot = _prepare_norm(case, seed), case["rot"]
    out = []
    for name, w in (("q", "qw"), ("k", "kw")):
        if s[name].numel() > 300_000_000:
            return None
        x = s[name].double()
        x /= torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6)
        x *= s[w].double()[:, None, None, None]
        z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous())
        turn = s["position"].double()[..., None] / 10000.0 ** (torch.arange(0, rot, 2, device="cuda").double() / rot)
        z *= torch.polar(torch.ones_like(turn), turn)[None, :, :, None]
        x[..., :rot // 2], x[..., rot // 2:rot] = z.real, z.imag
        if s["nodes"] is not None:
            for b, n in enumerate(s["nodes"].tolist()):
                x[:, b, n:] = 0
        out.append(x)
    return out


def _real(codes, byte, l, table, g, n, page, S):
    """Rows 0..n-1 of one layer, request and head in 64 bits."""
    pages = table[:-(-n // page)].long()
    x = codes[l, pages, g].double().reshape(-1, codes.shape[-1])[:n]
    e = byte[l, pages, g].double().reshape(-1).repeat_interleave(S)[:n]
    return x * torch.where(e > 0, torch.exp2(e - 127), torch.zeros_like(e))[:, None]


def _exact_append(case, seed):
    s, S, page = _prepare_append(case, seed), case["block"], case["page"]
    table, lens, count = s["table"].tolist(), _lengths(case), _lengths(case, "clo", "chi", 1)
    if s["k_pages"].numel() > 1_250_000_000 or case["L"] * case["B"] * case["Hkv"] * (max(count) // S + 2) > 60_000:
        return None
    out = []
    for name in ("k", "v"):
        byte, real = s[name + "_scale"].cpu(), s[name + "_pages"].double()
        x = s[name].double()
        for b, (p, c) in enumerate(zip(lens, count)):
            rows = x[:, b, :c] if s["node"] is None else x[:, b, s["node"][b, :c].long()]
            size, at = rows.abs().amax(-1).cpu(), 0
            while at < c:      # block after block
                n = min(c - at, S - (p + at) % S)
                pg, blk = table[b][(p + at) // page], (p + at) % page // S
                for l in range(case["L"]):
                    for g in range(case["Hkv"]):
                        top, was = float(size[l, at:at + n, g].max()), int(byte[l, pg, g, blk]) if (p + at) % S else 0
                        e = max(-100, min(120, math.ceil(math.log2(top / 448)))) if top > 0 else -127
                        now = max(was, e + 127)
                        if was and now > was:
                            real[l, pg, g, blk * S:blk * S + (p + at) % S] *= 2.0 ** (was - now)
                        byte[l, pg, g, blk] = now
                        real[l, pg, g, (p + at) % page:(p + at) % page + n] = rows[l, at:at + n, g] * 2.0 ** (127 - now)
                at += n
        out.append((real, byte))
    return [out[0][0], out[1][0], out[0][1], out[1][1], s["prefix_len"] + s["count"]]


def _exact_read(case, seed):
    s, S, page = _prepare_read(case, seed), case["block"], case["page"]
    if s["k_out"].numel() > 1_200_000_000:
        return None
    out = []
    for name in ("k", "v"):
        x = torch.zeros(s[name + "_out"].shape, dtype=torch.float64, device="cuda")
        for b, n in enumerate(_lengths(case)):
            for l in range(case["L"]):
                for g in range(case["Hkv"]):
                    x[l, b, g, :n] = _real(s[name + "_pages"], s[name + "_scale"], l, s["table"][b], g, n, page, S)
        out.append(x)
    return out


def _exact_decode(case, seed):
    s, S, page, G = _prepare_decode(case, seed), case["block"], case["page"], case["Hq"] // case["Hkv"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lengths(case)):
        for l in range(case["L"]):
            for g in range(case["Hkv"]):
                k = _real(s["k_pages"], s["k_scale"], l, s["table"][b], g, n, page, S)
                v = _real(s["v_pages"], s["v_scale"], l, s["table"][b], g, n, page, S)
                k = torch.cat([k, s["k_new"][l, b, g][None].double()])
                v = torch.cat([v, s["v_new"][l, b, g][None].double()])
                heads = slice(g * G, (g + 1) * G)
                o[l, b, heads] = torch.softmax(s["q"][l, b, heads].double() @ k.T * s["scale"], dim=-1) @ v
    return [o]


def exact(case, seed):
    global own
    mine, own = own, False   # inputs alone, without the library
    try:
        op = {"norm": _exact_norm, "append": _exact_append, "read": _exact_read, "decode": _exact_decode}[case["op"]]
        return op(case, seed)
    finally:
        own = mine
