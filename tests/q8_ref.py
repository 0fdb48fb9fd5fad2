"""Plain 64-bit forms of the 8-bit indexer operators, on the CPU, for the
tests. They share no code with the library."""
from __future__ import annotations

import numpy as np
import torch

LIMIT = {"int8": 127.0, "e4m3": 448.0}
FMT = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


def e4m3_values():
    """The 127 non-negative e4m3 values, by the format's definition, in code order."""
    v = [m * 2.0 ** -9 for m in range(8)]
    v += [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8) if not (e == 15 and m == 7)]
    return np.array(v)


def e4m3_round(z):
    """Index of the nearest e4m3 value of |z| (ties to the even code), and the value with z's sign."""
    grid = e4m3_values()
    a = np.abs(z)
    hi = np.clip(np.searchsorted(grid, a), 0, len(grid) - 1)
    lo = np.maximum(hi - 1, 0)
    up, down = grid[hi] - a, a - grid[lo]
    pick = np.where(up < down, hi, np.where(down < up, lo, np.where(lo % 2 == 0, lo, hi)))
    return np.copysign(grid[pick], z)


def quantize(x, group, fmt):
    """(code values as float64 [...,D], scales float32 [...,D/group]) of a float32/16-bit torch tensor."""
    x = x.detach().cpu().to(torch.float64).numpy()
    g = x.reshape(x.shape[:-1] + (x.shape[-1] // group, group))
    bad = ~np.isfinite(g).all(-1)
    g = np.where(bad[..., None], 0.0, g)
    amax = np.abs(g).max(-1)
    safe = np.where(amax > 0, amax, 1.0)
    z = LIMIT[fmt] * g / safe[..., None]
    code = np.rint(z) if fmt == "int8" else e4m3_round(z)
    scale = amax.astype(np.float32) / np.float32(LIMIT[fmt])
    scale[bad] = np.nan
    return code.reshape(x.shape), scale


def code_values(codes):
    """8-bit codes (torch) as the numbers they hold."""
    return codes.detach().cpu().to(torch.float32).numpy().astype(np.float64)


def candidates(B, S, P, cr, q_start=None, k_len=None, doc_start=None):
    m = np.zeros((B, S, P), dtype=bool)
    j = np.arange(P, dtype=np.int64)
    for b in range(B):
        for t in range(S):
            pos = (0 if q_start is None else int(q_start[b])) + t
            d0 = 0 if doc_start is None else min(max(int(doc_start[b, t]), 0), pos)
            m[b, t] = ((j + 1) * cr - 1 <= pos) & (j * cr >= d0)
            if k_len is not None:
                m[b, t] &= j < int(k_len[b])
    return m


def scores(q8, qs, w, k8, ks, mask):
    """(scores [B,S,P], sum of the terms' magnitudes) from codes (numpy)."""
    dot = np.einsum("bthd,bjd->bthj", q8.astype(np.float64), k8.astype(np.float64))
    term = np.maximum(dot, 0) * (w.astype(np.float64) * qs)[..., None] * ks[:, None, None, :].astype(np.float64)
    return np.where(mask, term.sum(2), -np.inf), np.where(mask, np.abs(term).sum(2), 0.0)


def dense(ds, idx, mask):
    """dscores on every block: slots of one block added up, non-candidates 0."""
    B, S, P = mask.shape
    if idx is None:
        return np.where(mask, ds.astype(np.float64), 0.0)
    G = np.zeros((B, S, P))
    for b in range(B):
        for t in range(S):
            for k, j in enumerate(idx[b, t]):
                if 0 <= j < P and mask[b, t, j]:
                    G[b, t, j] += float(ds[b, t, k])
    return G


def scores_grad(G, q8, qs, w, k8, ks):
    """((dq, dk, dw), the same three with every term's magnitude)."""
    q8, k8, qs, w, ks = (a.astype(np.float64) for a in (q8, k8, qs, w, ks))
    dot = np.einsum("bthd,bjd->bthj", q8, k8)
    m = dot > 0
    gk = np.where(G != 0, G * ks[:, None, :], 0.0)[:, :, None, :]
    out = []
    for f in (lambda a: a, np.abs):
        a = np.where(m, f(gk), 0.0)
        c = np.where(m, f(G)[:, :, None, :], 0.0) * f(w * qs)[..., None]
        out.append((np.einsum("bthj,bjd->bthd", a, f(k8)) * f(w)[..., None],
                    np.einsum("bthj,bthd->bjd", c, f(q8)),
                    (a * np.where(m, dot, 0.0)).sum(-1) * qs))
    return out
