"""Plain 64-bit forms of the 8-bit cache's calls (quantised append, read back, single-token attention)
and of the norm and rotation of query and key heads, their inputs, and the tolerances the tests derive."""
from __future__ import annotations

import math

import numpy as np
import torch

from tree_speculative_decoding_02_gb300 import synth

U = 2.0 ** -24          # half a step of fp32, relative
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}
NAN_CODE = 0x7F


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


# ------------------------------------------------------------------------------- the format
def _table():
    """Values of the 256 codes: sign, 4 bits of exponent (bias 7), 3 of mantissa; 0x7f and 0xff are NaN."""
    v = np.zeros(256)
    for c in range(256):
        e, m = c >> 3 & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[c] = math.nan if c & 0x7F == NAN_CODE else (-x if c & 0x80 else x)
    return v


VALUE = _table()
_POS = VALUE[:NAN_CODE]                              # ascending: 0 .. 448


def encode(x):
    """Codes of values of at most 448 (or NaN), to the nearest, ties to the even code."""
    a = np.minimum(np.abs(np.nan_to_num(x)), 448.0)
    hi = np.clip(np.searchsorted(_POS, a), 1, len(_POS) - 1)
    lo = hi - 1
    up, down = _POS[hi] - a, a - _POS[lo]
    pick = np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))
    code = pick.astype(np.uint8) | np.where(np.signbit(x), 0x80, 0).astype(np.uint8)
    return np.where(np.isnan(x), NAN_CODE, code).astype(np.uint8)


def byte_of(amax):
    """The byte of the smallest e in [-100, 120] with amax <= 448 * 2^e; 0 for 0."""
    if amax == 0:
        return 0
    m, x = math.frexp(amax)                          # amax = m 2^x, m in [0.5, 1); 448 = 0.875 * 2^9
    return min(max(x - 9 + (m > 0.875), -100), 120) + 127


def same_codes(a, b):
    """Equal codes; every NaN code is one and the same value."""
    return (a == b) | ((a & 0x7F == NAN_CODE) & (b & 0x7F == NAN_CODE))


def values(codes, scale):
    """[..][Hkv][page][d] codes and [..][Hkv][page / block] bytes to fp64 values."""
    block = codes.shape[-2] // scale.shape[-1]
    s = np.where(scale > 0, np.exp2(scale.astype(np.float64) - 127), 0.0).repeat(block, axis=-1)
    with np.errstate(invalid="ignore"):
        return VALUE[codes] * s[..., None]


def append_ref(x, codes, scale, table, lens, count, node):
    """One of K and V, in place on numpy arrays: x [L][B][N][Hkv][d] fp64."""
    L, _, Hkv, page, _ = codes.shape
    S = page // scale.shape[3]
    for b, (P, n) in enumerate(zip(lens, count)):
        rows = x[:, b, :n] if node is None else x[:, b, node[b, :n]]
        for s0 in range(P // S * S, P + n if n else 0, S):
            pg, blk, at = table[b, s0 // page], s0 % page // S, s0 % page
            lo, hi = max(P, s0), min(P + n, s0 + S)
            for l in range(L):
                for g in range(Hkv):
                    r = rows[l, lo - P:hi - P, g]
                    fin = np.abs(r[np.isfinite(r)])
                    old = int(scale[l, pg, g, blk]) if lo > s0 else 0
                    new = max(old, byte_of(float(fin.max()) if fin.size else 0.0))
                    if old and new > old:
                        have = codes[l, pg, g, at:at + lo - s0]
                        codes[l, pg, g, at:at + lo - s0] = encode(VALUE[have] * 2.0 ** (old - new))
                    scale[l, pg, g, blk] = new
                    with np.errstate(invalid="ignore"):
                        q = np.where(np.isfinite(r), r * (2.0 ** (127 - new) if new else 0.0), math.nan)
                    codes[l, pg, g, at + lo - s0:at + hi - s0] = encode(q)


# --------------------------------------------------------------------------------- caches
def cache(workload, L, B, Hkv, d, lens, page, block, *, cap_rows=None, spread=0.0, poison=True):
    """Quantised pages of N(0,1) values (blocks scaled by 2^(spread N(0,1))) behind a shuffled block table over
    B * max_pages + 3 pages; rows that no request's prefix uses hold NaN codes.  numpy arrays."""
    g = synth.gen(workload, 80)
    mp = max(1, -(-max([cap_rows or 1, *lens]) // page))
    num = B * mp + 3
    table = torch.randperm(num, generator=g)[:B * mp].reshape(B, mp).numpy().astype(np.int32)
    live = np.zeros((num, page), bool)
    for b, n in enumerate(lens):
        for i in range(-(-n // page)):
            live[table[b, i], :min(page, n - i * page)] = True
    out = []
    for _ in range(2):
        x = torch.randn((L, num, Hkv, page // block, block * d), generator=g, dtype=torch.float64).numpy()
        x = x * np.exp2(np.round(spread * torch.randn(x.shape[:-1], generator=g, dtype=torch.float64).numpy()))[..., None]
        scale = np.vectorize(byte_of, otypes=[np.uint8])(np.abs(x).max(-1))
        codes = encode(x * np.exp2(127 - scale.astype(np.float64))[..., None]).reshape(L, num, Hkv, page, d)
        if poison:
            codes[np.broadcast_to(~live[None, :, None, :, None], codes.shape)] = NAN_CODE
            codes[:, ~live.any(1)] = NAN_CODE
        out += [codes, scale]
    return dict(k=out[0], ks=out[1], v=out[2], vs=out[3], table=table, lens=list(lens), page=page, block=block)


def to_gpu(c):
    """(k_pages, v_pages, k_scale, v_scale, block_table, prefix_len) of a cache() on the GPU."""
    t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    return (t(c["k"]).view(torch.float8_e4m3fn), t(c["v"]).view(torch.float8_e4m3fn), t(c["ks"]), t(c["vs"]), t(c["table"]),
            torch.tensor(c["lens"], dtype=torch.int32).cuda())


def rows_of(codes, scale, table, b, n):
    """Request b's first n rows as values, [L][Hkv][n][d]."""
    page = codes.shape[3]
    at = table[b, :-(-n // page)].astype(np.int64)
    x = values(codes[:, at], scale[:, at])
    L, p, Hkv, _, d = x.shape
    return x.transpose(0, 2, 1, 3, 4).reshape(L, Hkv, p * page, d)[:, :, :n]


# ------------------------------------------------------------------------------ attention
def decode_ref(q, k_new, v_new, c, scale, dtype):
    """o [L][B][Hq][d] and the bound on its error before the rounding to the output type.

    A score is a product of d terms on e4m3 operands with fp32 accumulation; an addition there may truncate, so
    it is off by at most 2 U, and q by 2^-21 (bf16; fp32: 2^-34) of its largest channel and 2^-24 of itself.  A weight
    has the score's error, 2^-22 from the exponential, and that of its parts: 2^-16 of it or 2^-26 of the largest
    (fp32: 2^-24, 2^-34).  Sums: over rows, 2 U for each MMA of 32 and for each row of a tile.  With every weight off by at
    most w_p r_p, sum and weighted sum move o by at most 2 max(r) sum_p w_p |v_p| (and second order)."""
    L, B, Hq, d = q.shape
    Hkv = c["k"].shape[2]
    G = Hq // Hkv
    bf = dtype == torch.bfloat16
    part, floor, q_floor = (2.0 ** -16, 2.0 ** -26, 2.0 ** -21) if bf else (U, 2.0 ** -34, 2.0 ** -34)
    o, bound = np.zeros(q.shape), np.zeros(q.shape)
    for b, n in enumerate(c["lens"]):
        K, V = rows_of(c["k"], c["ks"], c["table"], b, n), rows_of(c["v"], c["vs"], c["table"], b, n)
        if k_new is not None:
            K = np.concatenate([K, k_new[:, b][:, :, None]], axis=2)
            V = np.concatenate([V, v_new[:, b][:, :, None]], axis=2)
        m = K.shape[2]
        if not m:
            continue
        for l in range(L):
            for g in range(Hkv):
                at = slice(g * G, (g + 1) * G)
                qq = q[l, b, at]
                s = qq @ K[l, g].T * scale
                e = np.exp(s - s.max(axis=1, keepdims=True))
                p = e / e.sum(axis=1, keepdims=True)
                size = np.abs(qq) @ np.abs(K[l, g]).T * abs(scale)
                far = np.abs(qq).max(axis=1, keepdims=True) * np.abs(K[l, g]).sum(axis=1) * abs(scale)
                r = 2 * U * (d + 40) * size + U * size + q_floor * far + 8 * U * np.abs(s) + 2.0 ** -22 + part + 2 * U * (128 + m / 32)
                err = p * r.max(axis=1, keepdims=True) + floor * p.max(axis=1, keepdims=True)
                o[l, b, at] = p @ V[l, g]
                bound[l, b, at] = 2.2 * (err @ np.abs(V[l, g]) + err.sum(axis=1, keepdims=True) * (p @ np.abs(V[l, g])))
    return o, bound


# ------------------------------------------------------------------------- norm and rotation
def norm_ref(x, w, position, rot, theta, eps, offset):
    """fp64: rows [L][B][N][H][d]; and the bound on the error before the rounding to the output type: a sum of d
    squares over lanes of 16, a reciprocal root of 2 steps, three products; an angle of 2^-23, sine and cosine of 2
    steps, two products and a sum."""
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (offset + w)[:, None, None, None]
    d = x.shape[-1]
    a = position.astype(np.float64)[None, :, :, None, None] * theta ** (-2.0 * np.arange(rot // 2) / rot) if rot else None
    out, size = y.copy(), np.abs(y)
    if rot:
        u, v = y[..., :rot // 2], y[..., rot // 2:rot]
        out[..., :rot // 2], out[..., rot // 2:rot] = u * np.cos(a) - v * np.sin(a), v * np.cos(a) + u * np.sin(a)
        both = np.abs(u) + np.abs(v)
        size[..., :rot // 2] = size[..., rot // 2:rot] = both
    return out, size * ((d / 16 + 16) * U / 2 + 4 * U + 3 * U + 2.0 ** -23 + 4 * U + 4 * U)
