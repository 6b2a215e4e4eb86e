"""ddt_evict_paged against a plain selection and the same moves on the host: every output is
exact (whole numbers and copies)."""
import numpy as np
import pytest
import torch

from tests import _serving as S
from tree_speculative_decoding_02_gb300 import ddt, synth

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _case(workload, L, B, Hkv, d, lens, page, dtype, *, placed=None, cap_rows=None):
    g = synth.gen(workload, 80)
    c = dict(lens=np.asarray(lens, np.int32))
    c["k"], c["v"], c["table"] = S.paged_cache(workload, L, B, Hkv, d, lens, page, dtype=dtype, cap_rows=cap_rows, poison=False)
    cap = c["table"].shape[1] * page
    w = torch.exp(2 * torch.randn((L, B, Hkv, cap), generator=g))
    w[torch.rand(w.shape, generator=g) < 0.3] = 0.0            # ties
    c["w"] = w
    c["placed"] = np.asarray(placed if placed is not None else [0] * B, np.int32)
    gone = np.where(c["placed"] > 0, 50, 0).astype(np.int32)   # tokens evicted before
    c["seq"] = c["lens"] + gone
    pos = torch.full((L, B, Hkv, cap), -5, dtype=torch.int32)
    for b in range(B):
        n = int(c["placed"][b])
        for l in range(L):
            for h in range(Hkv):
                pos[l, b, h, :n] = torch.randperm(n + int(gone[b]), generator=g)[:n].to(torch.int32)
    c["pos"] = pos
    return c


def _run(c, keep, n_sink=0, n_recent=0, **kw):
    d = dict(k=c["k"].cuda(), v=c["v"].cuda(), table=c["table"].cuda(), P=torch.as_tensor(c["lens"]).cuda(),
             placed=torch.as_tensor(c["placed"]).cuda(), seq=torch.as_tensor(c["seq"]).cuda(), w=c["w"].cuda(),
             pos=c["pos"].cuda())
    r = ddt.ddt_evict_paged(d["k"], d["v"], d["table"], d["P"], d["placed"], d["seq"], d["w"], d["pos"], keep=keep,
                            n_sink=n_sink, n_recent=n_recent, **kw)
    torch.cuda.synchronize()
    d["status"] = r["status"]
    return d


def _bits(t):
    return t.cpu().view(torch.int16 if t.dtype == BF else torch.int32).numpy()


def _check(c, d, keep, n_sink=0, n_recent=0, skip=()):
    k, v = _bits(c["k"]).copy(), _bits(c["v"]).copy()
    w, pos = c["w"].numpy().copy(), c["pos"].numpy().copy()
    lens = c["lens"].copy()
    for b in skip:                      # refused requests: as within the budget
        lens[b] = 0
    P, placed = S.evict_ref(k, v, c["table"].numpy(), lens, c["placed"], c["seq"], w, pos, keep, n_sink, n_recent)
    for b in skip:
        P[b] = c["lens"][b]
    np.testing.assert_array_equal(d["P"].cpu().numpy(), P)
    np.testing.assert_array_equal(d["placed"].cpu().numpy(), placed)
    np.testing.assert_array_equal(d["pos"].cpu().numpy(), pos)
    np.testing.assert_array_equal(_bits(d["w"]), w.view(np.int32))
    np.testing.assert_array_equal(_bits(d["k"]), k)
    np.testing.assert_array_equal(_bits(d["v"]), v)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,page,keep,n_sink,n_recent", [(64, 16, 100, 4, 20), (128, 8, 1, 0, 0), (256, 64, 500, 0, 500),
                                                         (8, 32, 129, 129, 0), (40, 192, 300, 1, 17), (128, 256, 999, 0, 1)])
def test_matches_plain_eviction(dtype, d, page, keep, n_sink, n_recent):
    lens = [0, 1, keep, keep + 1, 700, 1000]
    c = _case(31, 2, len(lens), 3, d, lens, page, dtype, placed=[0, 1, min(keep, 50), keep, 350, 0])
    r = _run(c, keep, n_sink, n_recent)
    assert (r["status"].cpu() == 0).all()
    _check(c, r, keep, n_sink, n_recent)


@pytest.mark.parametrize("kind", ["equal", "zero", "nan", "signs", "inf", "close"])
def test_sums_of_every_kind(kind):
    """All equal, all zero (-0 among them), NaN, negative, infinite, and neighbouring floats:
    the order is by value, NaN last, ties by the lower row."""
    c = _case(32, 1, 2, 2, 64, [2500, 1300], 64, BF)
    w, g = c["w"], synth.gen(32, 81)
    if kind == "equal":
        w.fill_(0.37)
    elif kind == "zero":
        w.zero_()
        w[torch.rand(w.shape, generator=g) < 0.5] = -0.0
    elif kind == "nan":
        w[torch.rand(w.shape, generator=g) < 0.7] = float("nan")
    elif kind == "signs":
        w *= torch.randn(w.shape, generator=g)
    elif kind == "inf":
        w[torch.rand(w.shape, generator=g) < 0.3] = float("inf")
        w[torch.rand(w.shape, generator=g) < 0.3] = float("-inf")
    else:
        w.view(torch.int32).copy_(torch.randint(0, 40, w.shape, generator=g).to(torch.int32) + 0x3f800000)
    _check(c, _run(c, 1000, 2, 100), 1000, 2, 100)


def test_long_cache():
    c = _case(33, 1, 1, 2, 64, [70001], 64, BF, placed=[30000])
    _check(c, _run(c, 40000, 8, 1024), 40000, 8, 1024)


# one block a unit, or a cluster of 2, 4 or 8 with a slice of the rows each: chosen by the table's
# rows and the number of units
@pytest.mark.parametrize("kind", ["random", "equal", "zero", "nan", "close"])
@pytest.mark.parametrize("B,Hkv,lens,cap_rows,keep,n_recent",
                         [(1, 1, [33000], 33024, 20000, 0), (20, 2, [17000 - 800 * i for i in range(20)], 17024, 4000, 9), (1, 4, [16500], 16640, 16499, 100), (2, 3, [9000, 17000], 17024, 33, 32),
                          (12, 2, [8200 - 300 * i for i in range(12)], 8256, 5003, 7), (1, 2, [4100], 20032, 4090, 64)])
def test_a_unit_in_slices(kind, B, Hkv, lens, cap_rows, keep, n_recent):
    c = _case(35, 1, B, Hkv, 8, lens, 64, BF, cap_rows=cap_rows, placed=[n // 3 for n in lens])
    w, g = c["w"], synth.gen(35, 81)
    if kind == "equal":
        w.fill_(0.37)
    elif kind == "zero":
        w.zero_()
    elif kind == "nan":
        w[torch.rand(w.shape, generator=g) < 0.7] = float("nan")
    elif kind == "close":
        w.view(torch.int32).copy_(torch.randint(0, 40, w.shape, generator=g).to(torch.int32) + 0x3f800000)
    _check(c, _run(c, keep, 1, n_recent), keep, 1, n_recent)


def test_slices_captured_and_refused():
    """Clusters of eight: refused requests between others, and a replay on the same state."""
    c = _case(38, 1, 4, 2, 8, [33000, 20000, 16000, 17000], 64, BF, cap_rows=33024)
    c["table"][1, 5] = c["table"][1, 6]
    c["lens"][2] = 33025
    keep = 9001
    eager = _run(c, keep, 3, 500)
    assert eager["status"].cpu().tolist() == [0, 1, 3, 0]
    _check(c, eager, keep, 3, 500, skip=[1, 2])
    d = dict(k=c["k"].cuda(), v=c["v"].cuda(), table=c["table"].cuda(), P=torch.as_tensor(c["lens"]).cuda(),
             placed=torch.as_tensor(c["placed"]).cuda(), seq=torch.as_tensor(c["seq"]).cuda(), w=c["w"].cuda(),
             pos=c["pos"].cuda())
    start = {k: x.clone() for k, x in d.items()}
    st = torch.empty(4, dtype=torch.int32, device="cuda")
    ws = ddt.evict_paged_workspace(d["k"], d["table"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ddt.ddt_evict_paged(d["k"], d["v"], d["table"], d["P"], d["placed"], d["seq"], d["w"], d["pos"], keep=keep,
                            n_sink=3, n_recent=500, status=st, workspace=ws)
    for _ in range(2):
        for k, x in start.items():
            d[k].copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        for k in ("k", "v", "P", "placed", "pos", "w"):
            assert (_bits(d[k]) == _bits(eager[k])).all() if d[k].is_floating_point() else torch.equal(d[k], eager[k]), k
        assert torch.equal(st, eager["status"])


def test_slices_beyond_shared_memory():
    c = _case(36, 1, 1, 1, 8, [400003], 256, BF, placed=[100000])
    _check(c, _run(c, 150001, 4, 1000), 150001, 4, 1000)


def test_second_eviction_and_the_steady_state():
    """Evict, append rows, evict again (the appended ones' positions follow from seq_len)."""
    c = _case(34, 1, 2, 2, 64, [600, 300], 16, BF, cap_rows=640)
    for step in range(3):
        r = _run(c, 400, 2, 64)
        _check(c, r, 400, 2, 64)
        c.update(k=r["k"].cpu(), v=r["v"].cpu(), w=r["w"].cpu(), pos=r["pos"].cpu(), placed=r["placed"].cpu().numpy())
        more = 33 + 7 * step
        c["lens"] = r["P"].cpu().numpy() + more
        c["seq"] = c["seq"] + more
        for b in range(2):
            assert (c["w"][:, b, :, int(c["placed"][b]):600] == 0).all() or c["placed"][b] == 0


def test_bad_requests_are_left_alone():
    """Lengths, positions and block tables that make no sense, and shared pages."""
    c = _case(35, 1, 9, 2, 64, [200] * 9, 16, BF, cap_rows=256)
    c["table"][1, 3] = -1
    c["table"][2, 12] = 10 ** 6
    c["table"][3, 5] = c["table"][4, 7]        # shared by two requests that would both evict
    c["table"][5, 1] = c["table"][5, 2]        # twice in one request
    c["placed"][6] = 201
    c["seq"][7] = 199
    c["lens"][8] = 300                         # past the capacity
    r = _run(c, 150)
    assert r["status"].cpu().tolist() == [0, 1, 1, 1, 1, 1, 1, 1, 3]
    _check(c, r, 150, skip=range(1, 9))


def test_a_page_shared_with_a_request_within_its_budget():
    """The small request reads the page: the large one may not rewrite it; unused entries of a
    block table (here the same page again) do not count."""
    c = _case(36, 1, 3, 2, 64, [200, 40, 200], 16, BF, cap_rows=256)
    c["table"][1, 0] = c["table"][0, 0]
    c["table"][2, 13:] = int(c["table"][2, 0])
    r = _run(c, 150)
    assert r["status"].cpu().tolist() == [1, 0, 0]
    _check(c, r, 150, skip=[0])


def test_graph_replay_and_side_stream():
    c = _case(37, 2, 2, 2, 128, [900, 500], 32, BF)
    d = dict(k=c["k"].cuda(), v=c["v"].cuda(), table=c["table"].cuda(), P=torch.as_tensor(c["lens"]).cuda(),
             placed=torch.as_tensor(c["placed"]).cuda(), seq=torch.as_tensor(c["seq"]).cuda(), w=c["w"].cuda(),
             pos=c["pos"].cuda())
    start = {k: v.clone() for k, v in d.items()}
    ws = ddt.evict_paged_workspace(d["k"], d["table"])
    st = torch.empty(2, dtype=torch.int32, device="cuda")

    def call():
        ddt.ddt_evict_paged(d["k"], d["v"], d["table"], d["P"], d["placed"], d["seq"], d["w"], d["pos"], keep=300,
                            n_sink=1, n_recent=30, status=st, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    _check(c, d, 300, 1, 30)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(2):
        for k, v in start.items():
            d[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        _check(c, d, 300, 1, 30)


def test_refusals():
    c = _case(38, 1, 2, 2, 64, [100, 200], 16, BF)
    launched = ddt.ddt_launch_count()
    for kw in (dict(keep=0), dict(keep=10, n_sink=6, n_recent=5), dict(keep=10, n_sink=-1), dict(keep=10, n_recent=-1),
               dict(keep=10, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ddt.DDTError):
            _run(c, **kw)
    for bad in (dict(w=c["w"].double()), dict(pos=c["pos"].long()), dict(v=c["v"].float()), dict(w=c["w"][..., :5])):
        with pytest.raises(ddt.DDTError):
            _run({**c, **bad}, 10)
    assert ddt.ddt_launch_count() == launched
