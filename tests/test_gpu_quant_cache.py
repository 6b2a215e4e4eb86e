"""ddt_append_paged_quant and ddt_read_paged_quant against a plain quantiser: codes, scale bytes and values
are exact, and nothing that is not written changes."""
import numpy as np
import pytest
import torch

from tests import _quant as Q
from tree_speculative_decoding_02_gb300 import ddt, synth

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _rows(workload, L, B, N, Hkv, d, dtype, std=1.0):
    g = synth.gen(workload, 81)
    return [synth.normal((L, B, N, Hkv, d), std, g=g, dtype=dtype) for _ in range(2)]


def _append(c, k, v, count, *, node=None, advance=True, **kw):
    """Runs the call on a cache() and the plain form beside it; compares everything."""
    gpu = Q.to_gpu(c)
    cnt = torch.tensor(count, dtype=torch.int32).cuda()
    nd = None if node is None else torch.from_numpy(node.astype(np.int32)).cuda()
    r = ddt.ddt_append_paged_quant(k.cuda(), v.cuda(), *gpu, cnt, node=nd, advance=advance, **kw)
    torch.cuda.synchronize()
    for x, codes, scale in ((k, "k", "ks"), (v, "v", "vs")):
        Q.append_ref(Q.f64(x), c[codes], c[scale], c["table"], c["lens"], count, node)
    got = [t.view(torch.uint8).cpu().numpy() for t in gpu[:4]]
    for have, want in zip(got[2:], (c["ks"], c["vs"])):
        assert np.array_equal(have, want)
    for have, want in zip(got[:2], (c["k"], c["v"])):
        assert Q.same_codes(have, want).all(), f"{(~Q.same_codes(have, want)).sum()} codes differ"
    assert gpu[5].tolist() == [p + (n if advance else 0) for p, n in zip(c["lens"], count)]
    assert r["status"].tolist() == [0] * len(count)
    return gpu


# lengths at, before and behind the edges of blocks and pages; counts of 0, 1 and over several pages
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,page,block,Hkv", [(64, 8, 8, 3), (128, 16, 16, 2), (256, 64, 16, 4), (64, 192, 64, 1), (128, 128, 128, 1),
                                              (256, 128, 128, 2), (64, 32, 8, 5), (256, 256, 32, 1)])
def test_append(dtype, d, page, block, Hkv):
    lens = [0, 1, block - 1, block, block + 1, page, 2 * page - 1, 5]
    count = [3, 1, 1, block, 2 * block + 3, 0, page + 1, 2 * page + block + 1]
    N = max(count)
    c = Q.cache(21, 2, len(lens), Hkv, d, lens, page, block, cap_rows=max(p + n for p, n in zip(lens, count)), spread=2.0)
    k, v = _rows(21, 2, len(lens), N, Hkv, d, dtype)
    k[:, :, 1:] *= 3.0          # the first row of each fits its block, later ones may raise it
    v[:, ::2] *= 0.01
    _append(c, k, v, count)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_append_of_a_walk(dtype):
    """Accepted rows by index, -1 behind the last; the same row may be named twice."""
    lens, count = [100, 31, 64, 0], [1, 5, 3, 0]
    node = np.full((4, 6), -1)
    node[0, :1], node[1, :5], node[2, :3] = [0], [0, 2, 3, 7, 12], [4, 4, 12]
    c = Q.cache(22, 3, 4, 2, 128, lens, 32, 16, cap_rows=110)
    k, v = _rows(22, 3, 4, 13, 2, 128, dtype, 4.0)
    _append(c, k, v, count, node=node)


def test_one_row_at_a_time():
    """A block filled row by row, every row larger than those before: its rows are rescaled each time.  One CTA has all
    of a request here (and prefix_len with it)."""
    c = Q.cache(23, 1, 2, 2, 64, [0, 7], 16, 8, cap_rows=40)
    for i in range(12):
        k, v = _rows(230 + i, 1, 2, 1, 2, 64, BF, 1.7 ** i)
        gpu = _append(c, k, v, [1, 1])
        c["lens"] = gpu[5].tolist()
    assert c["lens"] == [12, 19]


def test_without_advance():
    c = Q.cache(24, 2, 2, 2, 64, [5, 6], 16, 16, cap_rows=20)
    k, v = _rows(24, 2, 2, 3, 2, 64, BF)
    _append(c, k, v, [3, 2], advance=False)


def test_zeros_infinities_and_extremes():
    """Blocks of zeros (and what joins them), NaN and infinite channels, the smallest and largest magnitudes."""
    lens, count = [0, 0, 8, 0, 0, 3], [5, 8, 4, 8, 8, 4]
    c = Q.cache(25, 1, 6, 1, 64, lens, 16, 8, cap_rows=16)
    k, v = _rows(25, 1, 6, 8, 1, 64, F32)
    k[0, 0] = 0.0
    v[0, 0, 1:] = -0.0
    k[0, 1, 2, 0, 5], k[0, 1, 3, 0, 6], k[0, 1, 3, 0, 7] = float("nan"), float("inf"), -float("inf")
    v[0, 1, 4] = float("nan")
    v[0, 2] = float("inf")
    k[0, 3] *= 1e-36
    v[0, 3] *= 1e36
    k[0, 4] = 1e-42
    k[0, 4, 3] = 3.4e38
    v[0, 4] = torch.linspace(-448, 448, 8 * 64).reshape(8, 1, 64)    # ties and every binade
    k[0, 5] = 0.0
    _append(c, k, v, count)
    # zeros first, then rows that are not: the block's scale is theirs
    c["lens"] = [p + n for p, n in zip(lens, count)]
    k, v = _rows(26, 1, 6, 3, 1, 64, F32, 1e-3)
    _append(c, k, v, [3, 0, 0, 0, 0, 1])


def test_bad_requests_are_left_alone():
    """Every status, beside requests that are written; the bad ones' pages, scales and lengths stay."""
    page, S, mp = 16, 8, 4
    lens = [10, -1, 65, 60, 10, 10, 10, 62, 0]
    c = Q.cache(27, 1, 9, 2, 64, [max(0, min(p, 64)) for p in lens], page, S, cap_rows=64)
    c["lens"] = lens
    count = [4, 1, 0, 5, -1, 9, 4, 2, 4]
    node = np.tile(np.arange(8), (9, 1))
    node[6, 3], node[8, 0] = 8, -1
    table = c["table"].copy()
    k, v = _rows(27, 1, 9, 8, 2, 64, BF)
    gpu = Q.to_gpu(c)
    gpu[4][0, 1] = 1000              # not among the pages that request 0 writes now (row 10 to 13 are in page 0)
    st = torch.full((9,), -1, dtype=torch.int32).cuda()
    ddt.ddt_append_paged_quant(k.cuda(), v.cuda(), *gpu, torch.tensor(count, dtype=torch.int32).cuda(),
                               node=torch.from_numpy(node.astype(np.int32)).cuda(), status=st)
    torch.cuda.synchronize()
    assert st.tolist() == [0, 3, 3, 3, 1, 1, 1, 0, 1]
    good = [n if s == 0 else 0 for n, s in zip(count, st.tolist())]
    c["lens"] = [max(0, p) for p in lens]
    for x, codes, scale in ((k, "k", "ks"), (v, "v", "vs")):
        Q.append_ref(Q.f64(x), c[codes], c[scale], table, c["lens"], good, node)
    assert gpu[5].tolist() == [p + n for p, n in zip(lens, good)]
    for have, want in zip(gpu[:4], (c["k"], c["v"], c["ks"], c["vs"])):
        assert Q.same_codes(have.view(torch.uint8).cpu().numpy(), want).all()
    # a page that does not exist
    before = [t.view(torch.uint8).clone() for t in gpu[:4]]
    gpu[4][7, 3] = -1
    gpu[5][:] = torch.tensor([5, 0, 0, 0, 0, 0, 0, 62, 0], dtype=torch.int32)
    one = torch.tensor([0] * 7 + [1, 0], dtype=torch.int32).cuda()
    r = ddt.ddt_append_paged_quant(k.cuda(), v.cuda(), *gpu, one)
    assert r["status"].tolist() == [0] * 7 + [1, 0] and gpu[5].tolist()[7] == 62
    assert all(torch.equal(a, b.view(torch.uint8)) for a, b in zip(before, gpu[:4]))


@pytest.mark.parametrize("L,A", [(1, 1), (2, 1), (1, 20), (1, 3000)])
def test_no_rows_no_page(L, A):
    """Requests that append nothing: no page of theirs is looked at, whatever the table says behind the prefix (or in it),
    in one CTA a request, in several, and where a kernel of its own checks the pages."""
    c = Q.cache(31, L, 3, 2, 64, [5, 13, 8], 8, 8, cap_rows=A + 24)
    gpu = Q.to_gpu(c)
    gpu[4][:2] = torch.tensor([1 << 30, -7], dtype=torch.int32, device="cuda")[:, None]
    k, v = _rows(31, L, 3, A, 2, 64, BF)
    count = [0, 0, min(A, 2)]
    r = ddt.ddt_append_paged_quant(k.cuda(), v.cuda(), *gpu, torch.tensor(count, dtype=torch.int32).cuda())
    assert r["status"].tolist() == [0, 0, 0] and gpu[5].tolist() == [5, 13, 8 + count[2]]
    for x, codes, scale in ((k, "k", "ks"), (v, "v", "vs")):
        Q.append_ref(Q.f64(x), c[codes], c[scale], c["table"], c["lens"], count, None)
    for have, want in zip(gpu[:4], (c["k"], c["v"], c["ks"], c["vs"])):
        assert Q.same_codes(have.view(torch.uint8).cpu().numpy(), want).all()
    # and nothing at all
    before = [t.view(torch.uint8).clone() for t in gpu[:4]]
    r = ddt.ddt_append_paged_quant(k.cuda(), v.cuda(), *gpu, torch.zeros(3, dtype=torch.int32).cuda())
    assert r["status"].tolist() == [0, 0, 0] and all(torch.equal(x.view(torch.uint8), y) for x, y in zip(gpu[:4], before))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_long_prompts(dtype):
    """Rows over hundreds of pages, where the pages are checked by a kernel of its own: beside requests that are refused (a
    page that does not exist at the far end, lengths and counts that are wrong) and ones that append nothing."""
    lens, count = [3, 40, 0, -1, 0, 9, 2200], [2300, 2100, 0, 100, 2301, 2300, 300]
    c = Q.cache(32, 1, 7, 2, 64, [max(0, p) for p in lens], 8, 8, cap_rows=2400)
    c["lens"] = lens
    k, v = _rows(32, 1, 7, 2300, 2, 64, dtype)
    k[:, 0, 1000, 0, 3] = float("inf")
    gpu = Q.to_gpu(c)
    gpu[4][5, 2300 // 8] = 1 << 29
    r = ddt.ddt_append_paged_quant(k.cuda(), v.cuda(), *gpu, torch.tensor(count, dtype=torch.int32).cuda())
    assert r["status"].tolist() == [0, 0, 0, 3, 1, 1, 3]
    good = [n if s == 0 else 0 for n, s in zip(count, r["status"].tolist())]
    assert gpu[5].tolist() == [p + n for p, n in zip(lens, good)]
    c["lens"] = [max(0, p) for p in lens]
    for x, codes, scale in ((k, "k", "ks"), (v, "v", "vs")):
        Q.append_ref(Q.f64(x), c[codes], c[scale], c["table"], c["lens"], good, None)
    for have, want in zip(gpu[:4], (c["k"], c["v"], c["ks"], c["vs"])):
        assert Q.same_codes(have.view(torch.uint8).cpu().numpy(), want).all()


def test_long_prompts_a_call_a_layer():
    """The same a layer at a time (prefix_len moves with the last one), and replayed from a graph behind what it wrote."""
    L, count = 2, [2300, 2101]
    c = Q.cache(33, L, 2, 2, 64, [3, 16], 8, 8, cap_rows=4700)
    k, v = (x.cuda() for x in _rows(33, L, 2, 2300, 2, 64, BF))
    gpu = Q.to_gpu(c)
    n = torch.tensor(count, dtype=torch.int32).cuda()
    st = torch.zeros((L, 2), dtype=torch.int32).cuda()

    def run():
        for l in range(L):
            at = slice(l, l + 1)
            ddt.ddt_append_paged_quant(k[at], v[at], *(x[at] for x in gpu[:4]), *gpu[4:], n, advance=l == L - 1, status=st[l])

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    graph.replay()
    torch.cuda.synchronize()
    for _ in range(2):
        for x, codes, scale in ((k, "k", "ks"), (v, "v", "vs")):
            Q.append_ref(Q.f64(x), c[codes], c[scale], c["table"], c["lens"], count, None)
        c["lens"] = [p + m for p, m in zip(c["lens"], count)]
    assert st.tolist() == [[0, 0]] * L and gpu[5].tolist() == c["lens"]
    for have, want in zip(gpu[:4], (c["k"], c["v"], c["ks"], c["vs"])):
        assert Q.same_codes(have.view(torch.uint8).cpu().numpy(), want).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,page,block,Hkv", [(64, 8, 8, 3), (128, 16, 16, 2), (256, 64, 16, 4), (64, 192, 64, 1), (128, 128, 128, 1)])
def test_read_back(dtype, d, page, block, Hkv):
    lens = [0, 1, page, page - 1, 3 * page + 5, 333]
    c = Q.cache(28, 2, len(lens), Hkv, d, lens, page, block, spread=3.0)
    c["ks"][:, ::5] = np.maximum(c["ks"][:, ::5], 100)
    gpu = Q.to_gpu(c)
    out = [torch.full((2, len(lens), Hkv, max(lens) + 17, d), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
    r = ddt.ddt_read_paged_quant(*gpu, *out)
    assert r["status"].tolist() == [0] * len(lens)
    for t, codes, scale in ((out[0], "k", "ks"), (out[1], "v", "vs")):
        got = Q.f64(t)
        for b, n in enumerate(lens):
            assert np.array_equal(got[:, b, :, :n], Q.rows_of(c[codes], c[scale], c["table"], b, n))
            assert (got[:, b, :, n:] == 7.0).all()


def test_read_back_statuses():
    lens = [20, -3, 200, 50, 33]
    c = Q.cache(29, 1, 5, 2, 64, [20, 0, 64, 50, 33], 16, 8, cap_rows=64)
    c["lens"] = lens
    gpu = Q.to_gpu(c)
    gpu[4][3, 1] = 99999
    gpu[4][4, 3] = -1        # behind the prefix: never looked at
    out = [torch.full((1, 5, 2, 52, 64), 7.0, device="cuda") for _ in range(2)]
    r = ddt.ddt_read_paged_quant(*gpu, *out)
    assert r["status"].tolist() == [0, 3, 3, 1, 0]
    k = Q.f64(out[0])
    assert (k[:, 1:3] == 7.0).all() and (k[:, 3, :, 16:32] == 7.0).all()
    assert np.array_equal(k[:, 3, :, 32:50], Q.rows_of(c["k"], c["ks"], c["table"], 3, 50)[:, :, 32:])
    # an output of fewer rows than the prefix
    short = [torch.full((1, 5, 2, 32, 64), 7.0, device="cuda") for _ in range(2)]
    r = ddt.ddt_read_paged_quant(*gpu, *short)
    assert r["status"].tolist() == [0, 3, 3, 3, 3] and (short[0][:, 3:] == 7.0).all()


def test_large_offsets():
    """Codes past 2^32 bytes of a pool: 70000 pages of 64 rows, 4 heads, 256 channels are 4.6 GB each for K and V."""
    L, num, Hkv, page, d, S = 1, 70000, 4, 64, 256, 16
    pools = ddt.quant_cache(L, num, Hkv, page, d, block=S)
    table = torch.tensor([[num - 1, 3], [num - 2, 69000]], dtype=torch.int32).cuda()
    plen = torch.tensor([60, 0], dtype=torch.int32).cuda()
    k, v = _rows(30, 1, 2, 70, Hkv, d, BF)
    count = torch.tensor([8, 70], dtype=torch.int32).cuda()
    r = ddt.ddt_append_paged_quant(k.cuda(), v.cuda(), *pools, table, plen, count)
    assert r["status"].tolist() == [0, 0] and plen.tolist() == [68, 70]
    out = [torch.zeros((1, 2, Hkv, 72, d), device="cuda") for _ in range(2)]
    ddt.ddt_read_paged_quant(*pools, table, plen, *out)
    for x, t in ((k, out[0]), (v, out[1])):
        x = Q.f64(x)[0].transpose(0, 2, 1, 3)       # [B][Hkv][N][d]
        got = Q.f64(t)[0]
        # half a step of a value, or of the smallest normal code of a block of values up to 6
        assert (np.abs(got[1, :, :70] - x[1]) <= np.abs(x[1]) * 2.0 ** -4 + 6 * 2.0 ** -17).all()
        assert (np.abs(got[0, :, 60:68] - x[0, :, :8]) <= np.abs(x[0, :, :8]) * 2.0 ** -4 + 6 * 2.0 ** -17).all()
        assert (got[0, :, :60] == 0).all()
    # and attention over them
    q = synth.normal((1, 2, 8, d), g=synth.gen(30, 84), dtype=BF).cuda()
    o = ddt.ddt_decode_attn_paged_quant(q, None, None, *pools, table, plen, scale=d ** -0.5, out_dtype=F32)["o"]
    for b, n in enumerate((68, 70)):
        s = torch.einsum("ghd,gnd->ghn", q[0, b].double().reshape(Hkv, 2, d), out[0][0, b, :, :n].double()) * d ** -0.5
        want = (torch.softmax(s, -1) @ out[1][0, b, :, :n].double()).reshape(8, d)
        assert (o[0, b].double() - want).abs().max() <= 1e-3     # (weights to 2^-16, values up to 6, outputs in fp32)
