"""Plain 64-bit forms of the calls a server makes beside the verification round (single-token
attention over the paged cache, eviction by accumulated attention weight, token log
probabilities), their inputs, and the tolerances the tests derive."""
from __future__ import annotations

import math

import numpy as np
import torch

from tree_speculative_decoding_02_gb300 import synth

U = 2.0 ** -24          # half a step of fp32, relative
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def paged_cache(workload, L, B, Hkv, d, lens, page, *, dtype, cap_rows=None, poison=True):
    """Pages of N(0,1) values behind a shuffled block table over B * max_pages + 3 pages; rows
    that no request's prefix uses are NaN."""
    g = synth.gen(workload, 70)
    mp = max(1, -(-max([cap_rows or 1, *lens]) // page))
    num = B * mp + 3
    k = synth.normal((L, num, Hkv, page, d), g=g, dtype=dtype)
    v = synth.normal((L, num, Hkv, page, d), g=g, dtype=dtype)
    table = torch.randperm(num, generator=g)[:B * mp].reshape(B, mp).to(torch.int32)
    if poison:
        live = torch.zeros((num, page), dtype=torch.bool)
        for b, n in enumerate(lens):
            for i in range(-(-n // page)):
                live[int(table[b, i]), :min(page, n - i * page)] = True
        dead = ~live[None, :, None, :, None].expand_as(k)
        k[dead] = float("nan")
        v[dead] = float("nan")
    return k, v, table


def rows_of(pages, table, b, n):
    """Request b's first n rows, [L][Hkv][n][d]."""
    L, _, Hkv, page, d = pages.shape
    x = pages[:, table[b, :-(-n // page)].astype(np.int64)]          # [L][p][Hkv][page][d]
    return x.transpose(0, 2, 1, 3, 4).reshape(L, Hkv, -1, d)[:, :, :n]


def decode_ref(q, k_new, v_new, k_pages, v_pages, table, lens, scale):
    """o [L][B][Hq][d], per request the weights summed over each group [L][Hkv][n (+ 1)], and
    per (layer, request, kv head) the largest sum_i |q_i k_i| * scale (for the tolerance)."""
    L, B, Hq, d = q.shape
    Hkv = k_pages.shape[2]
    G = Hq // Hkv
    o = np.zeros((L, B, Hq, d))
    weights, size = [], np.zeros((L, B, Hkv))
    for b, n in enumerate(lens):
        K, V = rows_of(k_pages, table, b, n), rows_of(v_pages, table, b, n)
        if k_new is not None:
            K = np.concatenate([K, k_new[:, b][:, :, None]], axis=2)
            V = np.concatenate([V, v_new[:, b][:, :, None]], axis=2)
        w = np.zeros((L, Hkv, K.shape[2]))
        for l in range(L):
            for g in range(Hkv):
                if not K.shape[2]:
                    continue
                qq = q[l, b, g * G:(g + 1) * G]
                s = qq @ K[l, g].T * scale
                size[l, b, g] = (np.abs(qq) @ np.abs(K[l, g]).T).max() * abs(scale)
                e = np.exp(s - s.max(axis=1, keepdims=True))
                p = e / e.sum(axis=1, keepdims=True)
                o[l, b, g * G:(g + 1) * G] = p @ V[l, g]
                w[l, g] = p.sum(axis=0)
        weights.append(w)
    return o, weights, size


def decode_delta(d, n, size):
    """Bound on the relative error of one softmax weight before normalisation: an fp32 dot
    product of d terms is off by at most (d + 2) U sum |q_i k_i| in any order (and the score
    by two more roundings), the hardware exponential by 2^-22, a weight split into two bf16
    parts by 2^-16, and a sum of n weights taken 128 at a time by (128 + n / 128) U."""
    return (d + 8) * U * size + 2.0 ** -22 + 2.0 ** -16 + (128 + n / 128) * U


def evict_ref(k_pages, v_pages, table, lens, n_placed, seq_len, w, pos, keep, n_sink, n_recent):
    """In place on numpy arrays (any dtype of pages); returns the new (lens, n_placed)."""
    page = k_pages.shape[3]
    lens, n_placed = lens.copy(), n_placed.copy()
    for b in range(len(lens)):
        n = int(lens[b])
        if n <= keep:
            continue
        for l in range(k_pages.shape[0]):
            for g in range(k_pages.shape[2]):
                at = [int(pos[l, b, g, i]) if i < n_placed[b] else int(seq_len[b]) - n + i for i in range(n)]

                def rank(i):
                    x = float(w[l, b, g, i])
                    safe = at[i] < n_sink or at[i] >= seq_len[b] - n_recent
                    return (0 if safe else 1, 0 if safe else (1 if math.isnan(x) else 0),
                            0.0 if safe or math.isnan(x) else -x, i)
                kept = set(sorted(range(n), key=rank)[:keep])
                holes = [i for i in range(keep) if i not in kept]
                moved = [i for i in range(keep, n) if i in kept]
                assert len(holes) == len(moved)
                wn, an = w[l, b, g].copy(), list(at)
                for to, of in zip(holes, moved):
                    for x in (k_pages, v_pages):
                        x[l, table[b, to // page], g, to % page] = x[l, table[b, of // page], g, of % page]
                    wn[to], an[to] = w[l, b, g, of], at[of]
                wn[keep:n] = 0
                w[l, b, g] = wn
                pos[l, b, g, :keep] = an[:keep]
                pos[l, b, g, keep:n] = -1
        lens[b] = n_placed[b] = keep
    return lens, n_placed


def logprobs_ref(logits, node, token, top_n, T):
    """fp64 on finite or -inf rows: (logprob, entropy, top ids, top logprobs); padding as documented."""
    B, N, V = logits.shape
    A = token.shape[1]
    lp, en = np.zeros((B, A)), np.zeros((B, A))
    ids, tl = np.full((B, A, top_n), -1, np.int64), np.zeros((B, A, top_n))
    for b in range(B):
        for a in range(A):
            r = a if node is None else int(node[b, a])
            if r < 0 or r >= N or token[b, a] >= V:
                continue
            x = logits[b, r]
            u = (x - x.max()) / T
            e = np.exp(u)
            z = math.fsum(e)
            p = e / z
            lp[b, a] = u[token[b, a]] - math.log(z) if token[b, a] >= 0 else 0.0
            en[b, a] = math.log(z) - math.fsum(e[e > 0] * u[e > 0]) / z
            order = np.lexsort((np.arange(V), -x))[:top_n]
            ids[b, a], tl[b, a] = order, u[order] - math.log(z)
            assert p.sum() > 0
    return lp, en, ids, tl
