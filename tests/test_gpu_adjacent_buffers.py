"""Buffers of the single-token calls that lie directly behind one another in one allocation are
accepted, and the results are those of buffers of their own."""
import pytest
import torch

from tests import _serving as S
from tree_speculative_decoding_02_gb300 import ddt, synth

pytestmark = pytest.mark.gpu

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def _carve(tensors):
    """Copies of the tensors side by side (to 16 bytes) in one allocation."""
    n = [(t.nbytes + 15) // 16 * 16 for t in tensors]
    base, at, out = torch.zeros(sum(n), dtype=torch.uint8, device="cuda"), 0, []
    for t, size in zip(tensors, n):
        v = base[at:at + t.nbytes].view(t.dtype).view(t.shape)
        v.copy_(t)
        out.append(v)
        at += size
    return out


@pytest.mark.parametrize("cap", [256, 9008])
def test_decode(cap):
    k, v, table = S.paged_cache(70, 2, 3, 4, 64, [100, 0, 77], 16, dtype=BF, cap_rows=cap)
    g = synth.gen(70, 71)
    q, kn, vn = (synth.normal((2, 3, 4, 64), g=g, dtype=BF) for _ in range(3))
    w, st = torch.zeros((2, 3, 4, table.shape[1] * 16)), torch.zeros(3, dtype=I32)
    P = torch.tensor([100, 0, 77], dtype=I32)
    own = [t.cuda() for t in (q, kn, vn, torch.zeros_like(q), w, st, table, P)]
    ws = ddt.decode_attn_paged_workspace(own[0], k.cuda(), table, weights=True)
    side = _carve([*own, torch.zeros_like(ws)])
    k, v = k.cuda(), v.cuda()
    for x in ([*own, ws], side):
        ddt.ddt_decode_attn_paged(x[0], x[1], x[2], k, v, x[6], x[7], scale=0.125, attn_weight=x[4], out=x[3], status=x[5],
                                  workspace=x[8])
    for a, b in zip(own, side):
        assert torch.equal(a, b)


def test_evict():
    k, v, table = S.paged_cache(71, 1, 3, 2, 64, [100, 9, 90], 16, dtype=BF, cap_rows=128, poison=False)
    w = torch.rand((1, 3, 2, table.shape[1] * 16), generator=synth.gen(71, 71))
    P = torch.tensor([100, 9, 90], dtype=I32)
    own = [t.cuda() for t in (w, torch.zeros_like(w, dtype=I32), P, torch.zeros_like(P), torch.full_like(P, 7), table, P)]
    ws = ddt.evict_paged_workspace(k.cuda(), table)
    side = _carve([*own, torch.zeros_like(ws)])
    pools = []
    for x in ([*own, ws], side):
        pools.append((k.cuda(), v.cuda()))
        ddt.ddt_evict_paged(*pools[-1], x[5], x[2], x[3], x[6], x[0], x[1], keep=50, n_recent=3, status=x[4], workspace=x[7])
    assert own[4].tolist() == [0, 0, 0]
    for a, b in zip([*own, *pools[0]], [*side[:7], *pools[1]]):
        assert torch.equal(a, b)
    x = [t.cuda() for t in (w, torch.zeros_like(w, dtype=I32), P, torch.zeros_like(P), torch.full_like(P, 7), table, P)]
    one = k.cuda()                                              # keys that are the values too
    ddt.ddt_evict_paged(one, one, x[5], x[2], x[3], x[6], x[0], x[1], keep=50, n_recent=3, status=x[4], workspace=ws)
    assert torch.equal(one, pools[0][0]) and torch.equal(x[1], own[1])


@pytest.mark.parametrize("top", [0, 5])
def test_logprobs(top):
    x = synth.normal((2, 5, 200), g=synth.gen(72, 71), dtype=BF)
    node = torch.tensor([[0, 3, -1], [4, 1, 1]], dtype=I32)
    token = torch.tensor([[9, 199, -1], [0, 5, -1]], dtype=I32)
    names = ["logprob", "entropy", "status"] + (["top_token", "top_logprob"] if top else [])
    like = dict(logprob=torch.zeros((2, 3)), entropy=torch.zeros((2, 3)), status=torch.zeros((2, 3), dtype=I32),
                top_token=torch.zeros((2, 3, top), dtype=I32), top_logprob=torch.zeros((2, 3, top)))
    own = [t.cuda() for t in (x, node, token, *(like[n] for n in names))]
    ws = ddt.token_logprobs_workspace(own[0], own[2], top_n=top)
    side = _carve([*own, torch.zeros_like(ws)])
    for t in ([*own, ws], side):
        ddt.ddt_token_logprobs(t[0], t[2], node=t[1], top_n=top, out=dict(zip(names, t[3:])), workspace=t[-1])
    assert (own[5] == 0).all()
    if not top:   # where no alternatives are asked for, their pointers are not looked at
        p = [t.data_ptr() for t in side]
        rc = ddt.load().ddt_token_logprobs(2, 5, 200, 3, 0, 1.0, 1, p[0], p[1], p[2], p[3], p[4], p[0] + 16, p[0] + 32, p[5], p[6],
                                           ws.nbytes, torch.cuda.current_stream().cuda_stream)
        assert rc == 0
    for a, b in zip(own, side):
        assert torch.equal(a, b)
