"""ddt_token_logprobs against a plain 64-bit log-softmax."""
import numpy as np
import pytest
import torch

from tests import _serving as S
from tree_speculative_decoding_02_gb300 import ddt, synth

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _logits(workload, B, N, V, dtype, std=3.0):
    return synth.normal((B, N, V), std, g=synth.gen(workload, 90), dtype=dtype)


def _run(logits, token, **kw):
    node = kw.pop("node", None)
    r = ddt.ddt_token_logprobs(logits.cuda(), token.cuda(), node=None if node is None else node.cuda(), **kw)
    torch.cuda.synchronize()
    return {k: v.cpu() for k, v in r.items()}


def _check(r, logits, token, node=None, top_n=0, T=1.0):
    """Z has a relative error of at most 2^-22 (exponential) + (64 + 16) U (fp32 sums of 64 terms a
    lane and five levels across) + U (its reference), a term's exponent one of 3 U |u|; log p is off
    by that plus its rounding.  A term of the entropy is p u: the same errors times |u|, which the
    weights p keep at the size of the entropy itself plus log Z."""
    lp, en, ids, tl = S.logprobs_ref(S.f64(logits), None if node is None else node.numpy(), token.numpy(), top_n, T)
    ez = 2.0 ** -22 + 84 * S.U

    def near(got, want, extra):
        got = got.double().numpy()
        same = got == want               # -inf where the reference has it, 0 for padding
        with np.errstate(invalid="ignore"):
            err = np.abs(got - want)
            tol = ez + 4 * S.U * (np.abs(want) + extra) + S.U * np.abs(want)
        assert (same | (err <= tol)).all(), np.where(same, 0, err).max()
    span = float(np.log(logits.shape[2])) + 20.0
    near(r["logprob"], lp, span)
    got, want = r["entropy"].double().numpy(), en
    assert (np.abs(got - want) <= (ez + 6 * S.U * span) * (2 * span) + S.U * want).all(), np.abs(got - want).max()
    if top_n:
        np.testing.assert_array_equal(r["top_token"].numpy(), ids)
        near(r["top_logprob"], tl, span)
    assert (r["status"] == 0).all()


@pytest.mark.parametrize("dtype,V,top_n", [(BF, 20001, 7), (BF, 20001, 0), (F32, 20000, 32), (F32, 45001, 3), (BF, 9000, 32)])
def test_more_rows_than_fit_at_once(dtype, V, top_n):
    """One block a row, its units' largest entries in shared memory or (45001 fp32 entries) not."""
    logits = _logits(49, 1, 470, V, dtype)
    logits[0, 3, 100:] = float("-inf")                                   # a masked row
    logits[0, 4, ::2] = logits[0, 4].max()                               # many ties
    token = torch.randint(0, V, (1, 470), generator=synth.gen(49, 91)).to(torch.int32)
    _check(_run(logits, token, top_n=top_n), logits, token, top_n=top_n)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [1, 7, 8, 33, 1000, 2047, 2048, 2049, 20001, 151936])
def test_every_row_scored(dtype, V):
    B, N = (2, 3) if V > 5000 else (2, 19)
    logits = _logits(41, B, N, V, dtype)
    token = torch.randint(0, V, (B, N), generator=synth.gen(41, 91)).to(torch.int32)
    token[0, 0], token[1, -1] = 0, V - 1
    for top_n, T in ((min(5, V), 1.0), (min(32, V), 0.6), (0, 1.7)):
        _check(_run(logits, token, top_n=top_n, temperature=T), logits, token, top_n=top_n, T=T)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_of_a_walk(dtype):
    """node / token as a walk leaves them (-1 behind the last), a row without a token, one row twice."""
    B, N, V, A = 3, 9, 5003, 6
    logits = _logits(42, B, N, V, dtype)
    node = torch.tensor([[0, 2, 5, -1, -1, -1], [0, 8, 8, 1, -1, -1], [0, -1, -1, -1, -1, -1]], dtype=torch.int32)
    token = torch.tensor([[7, 5002, 0, -1, -1, -1], [3, 1, 2, -1, -1, -1], [4000, -1, -1, -1, -1, -1]], dtype=torch.int32)
    r = _run(logits, token, node=node, top_n=20, temperature=0.8)
    _check(r, logits, token, node, 20, 0.8)
    assert (r["top_token"][0, 3:] == -1).all() and (r["top_logprob"][0, 3:] == 0).all() and r["logprob"][1, 3] == 0


def test_rows_that_are_not_asked_for_may_hold_anything():
    logits = _logits(43, 1, 4, 3000, BF)
    logits[0, 1] = float("nan")
    node = torch.tensor([[3, 0]], dtype=torch.int32)
    token = torch.tensor([[5, 6]], dtype=torch.int32)
    _check(_run(logits, token, node=node, top_n=3), logits, token, node, 3)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_ties_and_masks(dtype):
    """Constant rows, rows of few distinct values, rows masked with -inf or with the type's lowest
    value but for a few tokens, one finite entry, one token with nearly all the mass."""
    V = 70001
    g = synth.gen(44, 90)
    low = float(torch.finfo(dtype).min)
    rows = [torch.full((V,), 1.25), torch.randint(0, 3, (V,), generator=g).float(), torch.full((V,), float("-inf")),
            torch.full((V,), low), torch.full((V,), float("-inf")), torch.randn(V, generator=g) * 0.01,
            torch.full((V,), float("-inf")), torch.full((V,), low)]
    rows[2][[69000, 3, 40000]] = torch.tensor([1.0, 2.0, 1.0])
    rows[3][[69999, 70000]] = torch.tensor([-3.0, -3.0])
    rows[4][70000] = 5.0
    rows[5][12345] = 40.0
    rows[6][::2] = torch.randn((V + 1) // 2, generator=g)
    logits = torch.stack(rows)[None].to(dtype)
    token = torch.tensor([[0, 5, 3, 70000, 70000, 12345, 1, 4]], dtype=torch.int32)
    for top_n in (1, 32):
        _check(_run(logits, token, top_n=top_n), logits, token, top_n=top_n)
    assert _run(logits, token)["logprob"][0, 6] == float("-inf")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,N,V", [(1, 1031, 2500), (3, 500, 4099), (2, 2300, 129)])
def test_many_rows(dtype, B, N, V):
    """Calls of many rows (shared out over persistent warps): more rows than are listed, rows of a
    few units cut anywhere."""
    logits = _logits(49, B, N, V, dtype)
    token = torch.randint(0, V, (B, N), generator=synth.gen(49, 91)).to(torch.int32)
    _check(_run(logits, token, top_n=7, temperature=0.9), logits, token, top_n=7, T=0.9)


@pytest.mark.parametrize("B", [20, 90])
def test_many_padded_rows(B):
    """Walks of many requests, most of whose entries are padding, some without a token, one that
    names no row and one that names no token; rows of no request hold NaN."""
    N, V, A = 60, 3001, 60
    g = synth.gen(50, 90)
    logits = _logits(50, B, N, V, BF)
    node = torch.full((B, A), -1, dtype=torch.int32)
    token = torch.full((B, A), -1, dtype=torch.int32)
    for b in range(B):
        n = b % 9
        node[b, :n] = torch.randperm(N, generator=g)[:n].to(torch.int32)
        token[b, :n] = torch.randint(-1, V, (n,), generator=g).to(torch.int32)
        unused = torch.ones(N, dtype=torch.bool)
        unused[node[b, :n].long()] = False
        logits[b, unused] = float("nan")
    r = _run(logits, token, node=node, top_n=3)
    _check(r, logits, token, node, 3)
    node[3, 0], token[4, 1] = N, V
    r = _run(logits, token, node=node, top_n=3)
    assert r["status"][3, 0] == 1 and r["status"][4, 1] == 1 and int(r["status"].sum()) == 2
    assert r["logprob"][3, 0] == 0 and (r["top_token"][4, 1] == -1).all()


def test_many_masked_rows():
    """The ties of test_ties_and_masks in a call of many rows."""
    V, N = 6001, 1100
    logits = torch.full((1, N, V), float("-inf"), dtype=BF)
    g = synth.gen(51, 90)
    for i in range(N):
        k = i % 40
        at = torch.randperm(V, generator=g)[:k + 1]
        logits[0, i, at] = torch.randint(0, 3, (k + 1,), generator=g).to(BF)
    logits[0, 5] = 2.0
    logits[0, 7] = float("-inf")
    token = logits[0].float().argmax(-1).to(torch.int32)[None]
    r = _run(logits, token, top_n=20)
    assert r["status"][0, 7] == 6 and int((r["status"] != 0).sum()) == 1
    keep = torch.arange(N) != 7
    _check({k: v[:, keep] for k, v in r.items()}, logits[:, keep], token[:, keep], top_n=20)


def test_statuses():
    V = 500
    logits = _logits(45, 1, 7, V, F32)
    logits[0, 1, 17] = float("nan")
    logits[0, 2, 499] = float("inf")
    logits[0, 3] = float("-inf")
    node = torch.tensor([[0, 1, 2, 3, 7, 4, -2, 5]], dtype=torch.int32)
    token = torch.tensor([[1, 1, 1, 1, 1, 500, 1, -1]], dtype=torch.int32)
    r = _run(logits, token, node=node, top_n=2)
    assert r["status"].tolist() == [[0, 6, 6, 6, 1, 1, 0, 0]]
    for a in (1, 2, 3):
        assert r["logprob"][0, a].isnan() and r["entropy"][0, a].isnan()
        assert (r["top_token"][0, a] == -1).all() and r["top_logprob"][0, a].isnan().all()
    for a in (4, 5, 6):
        assert r["logprob"][0, a] == 0 and r["entropy"][0, a] == 0 and (r["top_token"][0, a] == -1).all()
    assert r["logprob"][0, 7] == 0 and r["entropy"][0, 7] > 0 and (r["top_token"][0, 7] >= 0).all()


def test_rows_at_any_alignment():
    """A logits buffer that starts one element behind a 16-byte boundary."""
    B, N, V = 1, 5, 4001
    for dtype in (BF, F32):
        base = _logits(46, 1, 1, N * V + 1, dtype).flatten().cuda()
        logits = base[1:].view(B, N, V)
        token = torch.arange(N, dtype=torch.int32)[None]
        r = ddt.ddt_token_logprobs(logits, token.cuda(), top_n=4)
        torch.cuda.synchronize()
        _check({k: v.cpu() for k, v in r.items()}, logits.cpu(), token, top_n=4)


def test_graph_replay_is_the_same():
    logits = _logits(47, 2, 30, 9001, BF).cuda()
    token = torch.randint(0, 9001, (2, 30), generator=synth.gen(47, 91)).to(torch.int32).cuda()
    ws = ddt.token_logprobs_workspace(logits, token, top_n=8)
    out = ddt.ddt_token_logprobs(logits, token, top_n=8, workspace=ws)
    want = {k: v.clone() for k, v in out.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ddt.ddt_token_logprobs(logits, token, top_n=8, out=out, workspace=ws)
    for v in out.values():
        v.fill_(-9)
    graph.replay()
    torch.cuda.synchronize()
    for k, v in want.items():
        assert torch.equal(out[k], v), k


def test_refusals():
    logits = _logits(48, 1, 4, 100, BF).cuda()
    token = torch.zeros((1, 4), dtype=torch.int32, device="cuda")
    launched = ddt.ddt_launch_count()
    for kw in (dict(temperature=0.0), dict(temperature=-1.0), dict(temperature=float("inf")), dict(temperature=1e-40),
               dict(top_n=33), dict(top_n=-1), dict(node=token.long()), dict(out={"logprob": torch.zeros((1, 3), device="cuda")}),
               dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ddt.DDTError):
            ddt.ddt_token_logprobs(logits, token, **kw)
    for args in ((logits, token[:, :3]), (logits.half(), token), (logits, token.long()), (logits.cpu(), token),
                 (logits[:, :, :50], token)):
        with pytest.raises((ddt.DDTError, RuntimeError)):
            ddt.ddt_token_logprobs(*args)
    with pytest.raises(ddt.DDTError):
        ddt.ddt_token_logprobs(logits[:, :, :3].contiguous(), token, top_n=4)
    assert ddt.ddt_launch_count() == launched
