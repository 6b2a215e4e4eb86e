"""What the binding of the 8-bit cache's calls refuses before the library is asked: types, shapes, layouts and
places of tensors."""
import pytest
import torch

from tree_speculative_decoding_02_gb300 import ddt

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _world():
    L, B, N, Hq, Hkv, d, page = 2, 2, 3, 4, 2, 64, 16
    z = lambda *s, dtype=BF: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    i = lambda *s: z(*s, dtype=torch.int32)  # noqa: E731
    k_pages, v_pages, k_scale, v_scale = ddt.quant_cache(L, 5, Hkv, page, d, block=8)
    return dict(k=z(L, B, N, Hkv, d), v=z(L, B, N, Hkv, d), k_pages=k_pages, v_pages=v_pages, k_scale=k_scale, v_scale=v_scale,
                table=i(B, 2), plen=i(B), count=i(B), node=i(B, 2), q=z(L, B, Hq, d), kn=z(L, B, Hkv, d), vn=z(L, B, Hkv, d),
                ko=z(L, B, Hkv, 32, d), vo=z(L, B, Hkv, 32, d), qx=z(L, B, N, Hq, d), w=z(L, d), pos=i(B, N))


def _append(w):
    return ddt.ddt_append_paged_quant(w["k"], w["v"], w["k_pages"], w["v_pages"], w["k_scale"], w["v_scale"], w["table"], w["plen"],
                                      w["count"], node=w["node"])


def _read(w):
    return ddt.ddt_read_paged_quant(w["k_pages"], w["v_pages"], w["k_scale"], w["v_scale"], w["table"], w["plen"], w["ko"], w["vo"])


def _decode(w):
    return ddt.ddt_decode_attn_paged_quant(w["q"], w["kn"], w["vn"], w["k_pages"], w["v_pages"], w["k_scale"], w["v_scale"],
                                           w["table"], w["plen"], scale=1.0)


def _norm(w):
    return ddt.ddt_qk_norm_rope(w["qx"], w["k"], w["w"], w["w"], w["pos"])


def test_the_calls_as_they_are():
    w = _world()
    for call in (_append, _read, _decode, _norm):
        call(w)
    # codes may be given as bytes
    w["k_pages"], w["v_pages"] = w["k_pages"].view(torch.uint8), w["v_pages"].view(torch.uint8)
    assert _append(w)["status"].tolist() == _read(w)["status"].tolist() == _decode(w)["status"].tolist() == [0, 0]


@pytest.mark.parametrize("call,names", [
    (_append, ("k", "v", "k_pages", "v_pages", "k_scale", "v_scale", "table", "plen", "count", "node")),
    (_read, ("k_pages", "v_pages", "k_scale", "v_scale", "table", "plen", "ko", "vo")),
    (_decode, ("q", "kn", "vn", "k_pages", "v_pages", "k_scale", "v_scale", "table", "plen")),
    (_norm, ("qx", "k", "w", "pos"))], ids=["append", "read", "decode", "norm"])
def test_refused(call, names):
    before = ddt.ddt_launch_count()
    for name in names:
        t = _world()[name]
        bad = [t.cpu(), t.to(torch.float16) if t.dtype != torch.float8_e4m3fn else t.float(), t[:1] if t.shape[0] > 1 else t[:, :1]]
        if not (call is _norm and name in ("qx", "k")):
            wide = torch.zeros((*t.shape[:-1], 2 * t.shape[-1]), dtype=torch.uint8 if t.dtype == torch.float8_e4m3fn else t.dtype,
                               device="cuda")[..., ::2]
            bad.append(wide)
        for x in bad:
            w = _world()
            w[name] = x
            with pytest.raises((ddt.DDTError, ValueError)):
                call(w)
    for name in ("kn", "vn"):
        if call is _decode:
            w = _world()
            w[name] = None
            with pytest.raises(ddt.DDTError):
                call(w)
    if call is _norm:   # channels apart
        w = _world()
        w["qx"] = torch.zeros((2, 2, 3, 4, 128), dtype=BF, device="cuda")[..., ::2]
        with pytest.raises(ddt.DDTError):
            call(w)
    assert ddt.ddt_launch_count() == before
