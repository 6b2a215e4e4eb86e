"""ddt_qk_norm_rope against the formula in 64 bits."""
import numpy as np
import pytest
import torch

from tests import _quant as Q
from tree_speculative_decoding_02_gb300 import ddt, synth

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _case(workload, L, B, N, Hq, Hkv, d, dtype, pos=5000, std=1.5):
    g = synth.gen(workload, 83)
    c = dict(q=synth.normal((L, B, N, Hq, d), std, g=g, dtype=dtype), k=synth.normal((L, B, N, Hkv, d), std, g=g, dtype=dtype),
             qw=synth.normal((L, d), g=g, dtype=dtype), kw=synth.normal((L, d), g=g, dtype=dtype),
             position=torch.randint(0, pos, (B, N), generator=g).to(torch.int32))
    return {k: v.cuda() for k, v in c.items()}


def _check(c, got, rot, theta=10000.0, eps=1e-6, offset=0.0, rows=None):
    for x, w, y in ((c["q"], c["qw"], got[0]), (c["k"], c["kw"], got[1])):
        want, bound = Q.norm_ref(Q.f64(x), Q.f64(w), c["position"].cpu().numpy(), rot, theta, eps, offset)
        tol = bound + Q.HALF[y.dtype] * (np.abs(want) + bound) + 1e-37
        err = np.abs(Q.f64(y) - want)
        if rows is not None:
            err = np.where(rows[None, :, :, None, None], err, 0.0)
        assert (err <= tol).all(), f"{(err / tol).max():.3g} of the tolerance"


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("L,B,N,Hq,Hkv,d,rot", [(1, 1, 1, 1, 1, 64, 64), (1, 1, 1, 24, 4, 256, 64), (2, 3, 7, 8, 2, 128, 128),
                                                (1, 2, 33, 5, 3, 64, 16), (3, 1, 5, 7, 7, 256, 256), (1, 1, 700, 2, 1, 128, 112),
                                                (1, 4, 600, 6, 1, 64, 48), (2, 2, 3, 40, 8, 128, 0)])
def test_matches_the_formula(dtype, L, B, N, Hq, Hkv, d, rot):
    c = _case(51, L, B, N, Hq, Hkv, d, dtype)
    got = ddt.ddt_qk_norm_rope(c["q"], c["k"], c["qw"], c["kw"], c["position"], rot_dim=rot)
    _check(c, got, rot)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_offset_eps_theta(dtype):
    c = _case(52, 2, 2, 5, 4, 2, 128, dtype, std=1e-3)
    got = ddt.ddt_qk_norm_rope(c["q"], c["k"], c["qw"], c["kw"], c["position"], theta=1e6, eps=1e-5, weight_offset=1.0)
    _check(c, got, 128, theta=1e6, eps=1e-5, offset=1.0)


def test_far_and_negative_positions():
    """Angles are reduced exactly: positions up to the ends of 32 bits.  (The reference multiplies in 64 bits, off by 2^-22
    of a turn at 2^31: allowed for on top.)"""
    c = _case(53, 1, 1, 6, 2, 2, 128, F32)
    c["position"] = torch.tensor([[0, -1, 131071, 1 << 20, (1 << 31) - 1, -(1 << 31)]], dtype=torch.int32).cuda()
    got = ddt.ddt_qk_norm_rope(c["q"], c["k"], c["qw"], c["kw"], c["position"])
    for x, w, y in ((c["q"], c["qw"], got[0]), (c["k"], c["kw"], got[1])):
        want, bound = Q.norm_ref(Q.f64(x), Q.f64(w), c["position"].cpu().numpy(), 128, 10000.0, 1e-6, 0.0)
        far = np.abs(c["position"].cpu().numpy().astype(np.float64))[None, :, :, None, None] * 2.0 ** -52
        assert (np.abs(Q.f64(y) - want) <= bound * (1 + far / 2.0 ** -23) + Q.U * (np.abs(want) + bound)).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_padding_rows_stay(dtype):
    c = _case(54, 2, 4, 9, 4, 2, 64, dtype)
    nodes = [9, 1, 0, 10]     # the last is malformed: the whole request stays
    q_out, k_out = torch.full_like(c["q"], 7.0), torch.full_like(c["k"], 7.0)
    got = ddt.ddt_qk_norm_rope(c["q"], c["k"], c["qw"], c["kw"], c["position"], n_nodes=torch.tensor(nodes, dtype=torch.int32).cuda(),
                               q_out=q_out, k_out=k_out)
    assert got[0] is q_out and got[1] is k_out
    rows = np.zeros((4, 9), bool)
    for b, n in enumerate(nodes):
        rows[b, :n if n <= 9 else 0] = True
    _check(c, got, 64, rows=rows)
    for y in got:
        assert (Q.f64(y)[:, ~rows] == 7.0).all()
    # outputs that the call makes: zeros there
    q2, _ = ddt.ddt_qk_norm_rope(c["q"], c["k"], c["qw"], c["kw"], c["position"], n_nodes=torch.tensor(nodes, dtype=torch.int32).cuda())
    assert (Q.f64(q2)[:, ~rows] == 0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_strides_and_alignment(dtype):
    """Slices of one projection, rows of an odd pitch, an odd offset, broadcast rows: the same as contiguous copies."""
    L, B, N, Hq, Hkv, d = 2, 3, 5, 4, 2, 64
    c = _case(55, L, B, N, Hq, Hkv, d, dtype)
    want = ddt.ddt_qk_norm_rope(c["q"], c["k"], c["qw"], c["kw"], c["position"])
    fused = torch.cat([c["q"], c["k"], c["k"]], dim=3)
    views = [(fused[:, :, :, :Hq], fused[:, :, :, Hq:Hq + Hkv])]
    odd = torch.zeros((L, B, N, (Hq + Hkv) * d + 3), dtype=dtype, device="cuda")
    odd[..., 1:1 + Hq * d], odd[..., 1 + Hq * d:1 + (Hq + Hkv) * d] = c["q"].flatten(3), c["k"].flatten(3)
    views.append((odd[..., 1:1 + Hq * d].unflatten(-1, (Hq, d)), odd[..., 1 + Hq * d:1 + (Hq + Hkv) * d].unflatten(-1, (Hkv, d))))
    views.append((c["q"].permute(3, 2, 0, 1, 4).contiguous().permute(2, 3, 1, 0, 4), c["k"].transpose(0, 2).contiguous().transpose(0, 2)))
    for q, k in views:
        assert not q.is_contiguous()
        got = ddt.ddt_qk_norm_rope(q, k, c["qw"], c["kw"], c["position"])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    wide = c["q"][:, :1].expand(-1, B, -1, -1, -1)
    got = ddt.ddt_qk_norm_rope(wide, c["k"], c["qw"], c["kw"], c["position"][:1].expand(B, -1).contiguous())
    assert torch.equal(got[0][:, 2], got[0][:, 0]) and torch.equal(got[0][:, 0], want[0][:, 0])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_in_place(dtype):
    c = _case(56, 1, 2, 300, 6, 2, 256, dtype)
    want = ddt.ddt_qk_norm_rope(c["q"], c["k"], c["qw"], c["kw"], c["position"], rot_dim=64)
    q, k = c["q"].clone(), c["k"].clone()
    ddt.ddt_qk_norm_rope(q, k, c["qw"], c["kw"], c["position"], rot_dim=64, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


def test_zero_and_non_finite_rows():
    """A row of zeros with eps stays zero; a NaN or infinity makes its own row NaN (an infinite mean) and no other."""
    c = _case(57, 1, 1, 4, 2, 1, 64, F32)
    want = ddt.ddt_qk_norm_rope(c["q"], c["k"], c["qw"], c["kw"], c["position"])[0].clone()
    c["q"][0, 0, 0] = 0.0
    c["q"][0, 0, 1, 0, 3] = float("nan")
    c["q"][0, 0, 2, 1, 5] = float("inf")
    got = ddt.ddt_qk_norm_rope(c["q"], c["k"], c["qw"], c["kw"], c["position"])[0]
    assert (got[0, 0, 0] == 0).all() and torch.isnan(got[0, 0, 1, 0]).all()
    assert torch.isnan(got[0, 0, 2, 1]).any()
    assert torch.equal(got[0, 0, 1, 1], want[0, 0, 1, 1]) and torch.equal(got[0, 0, 2, 0], want[0, 0, 2, 0])
    assert torch.equal(got[0, 0, 3], want[0, 0, 3])


def test_same_as_rope_tree_after_a_norm():
    """Rows of norm 1 already (weights 1, eps 0 over +-1 entries): what remains is ddt_rope_tree's rotation."""
    B, N, d = 2, 9, 128
    g = synth.gen(58, 1)
    q = (torch.randint(0, 2, (1, B, N, 4, d), generator=g) * 2.0 - 1).cuda()
    k = (torch.randint(0, 2, (1, B, N, 2, d), generator=g) * 2.0 - 1).cuda()
    pos = torch.randint(0, 40000, (B, N), generator=g).to(torch.int32).cuda()
    nn = torch.full((B,), N, dtype=torch.int32).cuda()
    one = torch.ones((1, d)).cuda()
    got = ddt.ddt_qk_norm_rope(q, k, one, one, pos, n_nodes=nn, rot_dim=64, eps=0.0)
    ddt.ddt_rope_tree(q, k, pos, nn, rot_dim=64)
    for a, b in zip(got, (q, k)):
        assert (a - b).abs().max() <= 2 * (2.0 ** -23 * 2 + 16 * Q.U)   # pairs of +-1: each call within its own bound
