"""Rounds over 8-bit prefixes with a request whose prefix cannot be read: its output rows are zeros and its status says
why, and the other requests' rounds are as they are without it."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from tree_speculative_decoding_02_gb300 import ddt, synth
from tree_speculative_decoding_02_gb300.round import Round

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _round(rope=0):
    cfg = dict(synth.WORKLOADS[1], B=3, V=2000, budget=24, Lf=3, Hq=8, Hkv=2, d=128, dtype=BF, page=32, kv_quant=16, rope=rope,
               P_lo=40, P_hi=300, Lg=1, Pcap=416)
    cfg.pop("P", None)
    return Round(cfg, device="cuda", workload=1, poison=True, attn_out_dtype=F32, gdn_out_dtype=F32)


@pytest.mark.parametrize("rope", [0, 64])
@pytest.mark.parametrize("what,status", [("page", 1), ("last page", 1), ("length", 3), ("negative length", 3)])
def test_a_prefix_that_cannot_be_read(what, status, rope):
    good = _round(rope)
    good.step()
    r = _round(rope)
    used = -(-int(r.prefix_len[1]) // 32)
    if what == "page":
        r.block_table[1, 0] = -1
    elif what == "last page":       # the page that the new rows go to as well, unless it is full
        r.block_table[1, used - 1] = 1 << 20
    else:
        r.prefix_len[1] = 417 if what == "length" else -1
    before = r.prefix_len.tolist()
    r.step()
    torch.cuda.synchronize()
    assert r.attn_status.tolist() == [0, status, 0]
    assert (r.attn_o[:, 1] == 0).all()
    for b in (0, 2):
        n = int(r.tree["n_nodes"][b])
        assert torch.equal(r.attn_o[:, b, :n], good.attn_o[:, b, :n])
        assert r.prefix_len[b] == good.prefix_len[b] and r.commit["status"][b] == 0
    if what != "page":              # its rows cannot be written either
        assert r.append_status[1] == status and r.commit["status"][1] == status and r.prefix_len[1] == before[1]


def test_replayed_with_and_without_a_bad_page():
    """One captured round, replayed while a page is bad and when it is right again."""
    r = _round()
    state = [r.prefix_len, r.k_pages.view(torch.uint8), r.v_pages.view(torch.uint8), r.k_scale, r.v_scale, r.gdn.S, r.gdn.conv_state]
    saved = [x.clone() for x in state]

    def restore():
        for x, y in zip(state, saved):
            x.copy_(y)

    r.step()
    torch.cuda.synchronize()
    want, nn = r.attn_o.clone(), r.tree["n_nodes"].tolist()
    restore()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r.step()
    page = int(r.block_table[2, 0])
    for bad in (True, False, True):
        restore()
        r.block_table[2, 0] = -7 if bad else page
        r.attn_o.fill_(5)
        g.replay()
        torch.cuda.synchronize()
        assert r.attn_status.tolist() == [0, 0, 1 if bad else 0]
        for b in range(3):
            zero = bad and b == 2
            assert torch.equal(r.attn_o[:, b, :nn[b]], torch.zeros_like(want[:, b, :nn[b]]) if zero else want[:, b, :nn[b]])


@pytest.mark.parametrize("n,B", [(1, 1), (3, 5), (17, 300), (2, 129)])
def test_chain_status(n, B):
    g = torch.Generator().manual_seed(n * 1000 + B)
    st = torch.randint(0, 8, (n, B), generator=g, dtype=torch.int32) * (torch.rand((n, B), generator=g) < 0.3)
    length = torch.randint(0, 1 << 30, (B,), generator=g, dtype=torch.int32)
    first = [next((int(x) for x in st[:, b] if x), 0) for b in range(B)]
    out, so = (torch.full((B + 1,), 77, dtype=torch.int32, device="cuda") for _ in range(2))
    ddt.ddt_chain_status(st.to(torch.int32).cuda(), length=length.cuda(), length_out=out[:B], status_out=so[:B])
    assert so.tolist() == first + [77]
    assert out.tolist() == [-1 if s else int(x) for s, x in zip(first, length)] + [77]
    alone = torch.empty(B, dtype=torch.int32, device="cuda")
    ddt.ddt_chain_status(st.to(torch.int32).cuda(), status_out=alone)
    assert alone.tolist() == first


class _Ops(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.names = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        if not func.is_view and "empty" not in str(func):
            self.names.append(str(func))
        return func(*args, **(kwargs or {}))


@pytest.mark.parametrize("rope", [0, 64])
def test_a_round_is_the_librarys_calls_alone(rope):
    """No arithmetic of torch's between the calls, which the launch counter would not see."""
    r = _round(rope)
    r.step()
    with _Ops() as ops:
        r.step()
    assert ops.names == []
    torch.cuda.synchronize()
    assert (r.commit["status"] == 0).all()
