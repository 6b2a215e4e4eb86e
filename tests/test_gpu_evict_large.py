"""ddt_evict_paged on a pool of more pages than one window of its page check covers, and on rows
wider than a block's copy."""
import numpy as np
import pytest
import torch

from tests import _serving as S
from tests.test_gpu_evict import BF, F32, _bits, _case, _check, _run
from tree_speculative_decoding_02_gb300 import ddt

pytestmark = pytest.mark.gpu


def test_a_pool_of_over_a_million_pages():
    """Pages of both windows (the border is page 2^20): one request that is cut, two that share a page
    behind the border, one that has a page there twice, one with a page past the pool."""
    num, page, d, keep = (1 << 20) + 5000, 8, 8, 60
    c = _case(39, 1, 6, 1, d, [100, 100, 100, 100, 100, 40], page, BF)
    at = c["table"].long()                                        # the small pool's pages
    n = int(at.max()) + 1
    rng = np.random.default_rng(39)
    where = torch.as_tensor(np.concatenate([rng.choice(1 << 20, 40, replace=False),
                                            (1 << 20) + rng.choice(5000, n - 40, replace=False)]))
    where = where[torch.as_tensor(rng.permutation(len(where)))]
    where[at[0, 0]], where[at[0, 1]] = (1 << 20) - 1, 1 << 20     # both sides of the border
    assert len(set(where.tolist())) == len(where)
    k = torch.zeros((1, num, 1, page, d), dtype=BF, device="cuda")
    v = torch.zeros_like(k)
    used = where[:n].cuda()
    k[:, used], v[:, used] = c["k"][:, :n].cuda(), c["v"][:, :n].cuda()
    table = where[at].to(torch.int32)
    high = next(int(x) for x in table[1] if x > 1 << 20)
    free = next(x for x in range((1 << 20) + 4999, 0, -1) if x not in where.tolist())
    table[2, 7] = high
    table[3, 2] = table[3, 9] = free
    table[4, 4] = num
    P, placed, seq = (torch.as_tensor(c[x]).cuda() for x in ("lens", "placed", "seq"))
    w, pos = c["w"].cuda(), c["pos"].cuda()
    r = ddt.ddt_evict_paged(k, v, table.cuda(), P, placed, seq, w, pos, keep=keep, n_sink=2, n_recent=9)
    assert r["status"].cpu().tolist() == [0, 1, 1, 1, 1, 0]
    got = dict(k=k[:, used], v=v[:, used], P=P, placed=placed, pos=pos, w=w)
    c["k"], c["v"] = c["k"][:, :n], c["v"][:, :n]
    _check(c, got, keep, 2, 9, skip=range(1, 5))
    rest = torch.ones(num, dtype=torch.bool, device="cuda")
    rest[used] = False
    assert not k[0, rest].any() and not v[0, rest].any()


@pytest.mark.parametrize("dtype,d", [(F32, 4096), (BF, 4104), (BF, 2056)])
def test_rows_of_several_copies(dtype, d):
    """Up to 16384 bytes a row: more than the 4096 that the threads of a block copy at once."""
    c = _case(40, 1, 2, 2, d, [90, 33], 16, dtype, placed=[20, 0])
    r = _run(c, 30, 1, 5)
    assert (r["status"].cpu() == 0).all()
    _check(c, r, 30, 1, 5)
