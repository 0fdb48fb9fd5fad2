"""The 8-bit indexer operators: measured cases, plain forms and 64-bit values.

Three operators around the distillation loss:

  cache   rows quantised as they are written into a cache and read back
          (q8_cache_write, q8_cache_read)
  scores  the lightning indexer's scores from 8-bit queries and 8-bit cached
          keys, for whole sequences and for single tokens (indexer_scores)
  grad    dscores back to the indexer's queries, keys and head weights, from
          the 8-bit codes the forward kept (indexer_scores_backward)

``run`` computes a case in elementary torch operations, or, with ``own`` true,
through the package's entry points. Codes of a group of values with largest
magnitude amax: int8 rint(127 x / amax) with scale amax / 127, e4m3
e4m3(448 x / amax) with scale amax / 448.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
CHUNK = 1 << 27            # elements of a [tokens, heads, keys] slab held at once


# ----------------------------------------------------------------- the cases
def listed():
    return [
        # one decoding step: 64 sequences append one compressed entry's indexer key to their pages and
        # read 32 selected ones back (latency)
        {"name": "cache-step", "op": "cache", "B": 64, "n": 1, "D": 128, "group": 128, "fmt": "int8", "dtype": "bf16",
         "page": 64, "pages": 16, "K": 32, "ragged": False},
        # a ragged prefill chunk of wide entries, e4m3 codes with a scale for every 128 values, an odd page size
        {"name": "cache-chunk", "op": "cache", "B": 5, "n": 777, "D": 512, "group": 128, "fmt": "e4m3",
         "dtype": "fp16", "page": 24, "pages": 40, "K": 801, "ragged": True},
        # the compressed pool of a packed training batch, written and read back whole
        {"name": "cache-pool", "op": "cache", "B": 8, "n": 8192, "D": 512, "group": 128, "fmt": "e4m3",
         "dtype": "bf16", "page": 8192, "pages": 1, "K": 0, "ragged": False},
        # a single decoded token of one short conversation (latency)
        {"name": "scores-token", "op": "scores", "B": 1, "S": 1, "H": 64, "D": 128, "cr": 4, "P": 1000, "page": 64,
         "docs": 1},
        # a decoding batch over long paged contexts of different lengths, two drafted tokens each
        {"name": "scores-decode", "op": "scores", "B": 32, "S": 2, "H": 64, "D": 128, "cr": 4, "P": 32768,
         "page": 64, "docs": 1},
        # the training forward at the flash width (S=4096, 1024 blocks)
        {"name": "scores-flash", "op": "scores", "B": 1, "S": 4096, "H": 64, "D": 128, "cr": 4, "P": 1024, "page": 0,
         "docs": 1},
        # a packed batch with few narrow heads and an odd length, two documents a row
        {"name": "scores-packed", "op": "scores", "B": 4, "S": 2020, "H": 24, "D": 64, "cr": 4, "P": 505, "page": 0,
         "docs": 2},
        # the long context (S=16384, 4096 blocks)
        {"name": "scores-long", "op": "scores", "B": 1, "S": 16384, "H": 64, "D": 128, "cr": 4, "P": 4096,
         "page": 0, "docs": 1},
        # a small odd problem, few heads
        {"name": "grad-small", "op": "grad", "B": 2, "S": 508, "H": 16, "D": 64, "cr": 4, "K": 61, "docs": 2},
        # the flash width's backward: K=512 selected of 1024
        {"name": "grad-flash", "op": "grad", "B": 1, "S": 4096, "H": 64, "D": 128, "cr": 4, "K": 512, "docs": 1},
        # the dense warm-up stage: every block is a slot
        {"name": "grad-dense", "op": "grad", "B": 2, "S": 2048, "H": 32, "D": 128, "cr": 4, "K": 0, "docs": 1},
        # the long context's backward: K=2048 of 4096
        {"name": "grad-long", "op": "grad", "B": 1, "S": 16384, "H": 64, "D": 128, "cr": 4, "K": 2048, "docs": 1},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["cache", "scores", "grad"])
    if op == "cache":
        D = rng.choice([64, 128, 256, 512])
        B = _log(rng, 1, 64)
        n = _log(rng, 1, max(2, min(8192, (1 << 25) // (B * D))))
        page = rng.choice([16, 24, 64, 128])
        pages = (n + page - 1) // page + rng.randint(0, 3)
        return {"op": op, "B": B, "n": n, "D": D, "group": rng.choice([g for g in (32, 64, 128, 256, 512) if g <= D]),
                "fmt": rng.choice(["int8", "e4m3"]), "dtype": rng.choice(["bf16", "fp16", "fp32"]), "page": page,
                "pages": pages, "K": rng.choice([0, _log(rng, 1, max(2, n))]), "ragged": rng.random() < 0.5}
    H, D, cr = rng.choice([8, 24, 32, 64]), rng.choice([64, 128]), rng.choice([2, 4, 8])
    if op == "scores" and rng.random() < 0.5:                          # single tokens over pages
        B = _log(rng, 1, 32)
        return {"op": op, "B": B, "S": rng.randint(1, 3), "H": H, "D": D, "cr": cr,
                "P": _log(rng, 100, min(32768, (1 << 20) // B)), "page": rng.choice([16, 32, 64, 128]), "docs": 1}
    S = _log(rng, 128, 8192) // cr * cr
    B = rng.randint(1, max(1, min(4, 8192 // S)))
    docs = rng.choice([1, 2])
    if op == "scores":
        return {"op": op, "B": B, "S": S, "H": H, "D": D, "cr": cr, "P": S // cr, "page": 0, "docs": docs}
    return {"op": op, "B": B, "S": S, "H": H, "D": D, "cr": cr,
            "K": rng.choice([0, _log(rng, 2, S // cr)]), "docs": docs}


def _pairs(case):
    """(token, candidate) pairs of a scores or grad case (documents left out)."""
    S, cr = case["S"], case["cr"]
    P = case.get("P", S // cr)
    if case.get("page"):
        return case["B"] * S * P * 3 / 4      # lengths are spread over P/2 .. P
    sel = case.get("K", 0) or P
    return case["B"] * sum(min(sel, P, (t + 1) // cr) for t in range(S))


def work(case):
    B = case["B"]
    if case["op"] == "cache":
        D, size = case["D"], 4 if case["dtype"] == "fp32" else 2
        row8 = D + 4 * (D // case["group"])
        rows, read = B * case["n"], B * (case["K"] or case["n"])
        return {"bytes": rows * (D * size + row8) + read * (row8 + D * size + (4 if case["K"] else 0)),
                "flops": 4 * rows * D + read * D}
    S, H, D, cr = case["S"], case["H"], case["D"], case["cr"]
    P = case.get("P", S // cr)
    pairs = _pairs(case)
    q, k = B * S * H * (D + 8), B * P * (D + 4) * (3 / 4 if case.get("page") else 1)
    if case["op"] == "scores":
        return {"bytes": q + k + B * S * P * 4, "flops": pairs * H * (2 * D + 3)}
    K = case["K"]
    return {"bytes": q + k + B * S * (8 * K if K else 4 * P) + B * S * H * (2 * D + 4) + B * P * 2 * D,
            "flops": pairs * H * (6 * D + 6)}


# ---------------------------------------------------------------- the inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _codes(x):
    """int8 codes and scale of each row: the form in which queries and keys are given."""
    amax = x.abs().amax(-1, keepdim=True)
    c = torch.where(amax > 0, torch.round(127.0 * x / amax), torch.zeros_like(x))
    return c.to(torch.int8), (amax / 127.0).squeeze(-1)


def _doc_start(g, B, S, docs):
    if docs == 1:
        return None
    split = torch.randint(1, S, (B, 1), generator=g, device=DEV, dtype=torch.int32)
    t = torch.arange(S, device=DEV, dtype=torch.int32)[None]
    return torch.where(t >= split, split, torch.zeros_like(split)).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    B = case["B"]

    def randn(*s):
        return torch.randn(*s, generator=g, device=DEV)

    if case["op"] == "cache":
        n, D, page, pages = case["n"], case["D"], case["page"], case["pages"]
        cap = page * pages
        # entries of different magnitude, as the rows of a pool have
        x = (randn(B, n, D) * torch.exp(randn(B, n, 1))).to(DTYPES[case["dtype"]])
        fmt = torch.int8 if case["fmt"] == "int8" else torch.float8_e4m3fn
        st = {"case": case, "x": x, "cache": torch.zeros(B * pages, page, D, device=DEV, dtype=torch.int8).view(fmt),
              "scales": torch.zeros(B * pages, page, D // case["group"], device=DEV)}
        st["table"] = torch.randperm(B * pages, generator=g, device=DEV).int().view(B, pages)
        st["start"] = torch.randint(0, cap - n + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
        st["n_new"] = (torch.randint(0, n + 1, (B,), generator=g, device=DEV, dtype=torch.int32) if case["ragged"]
                       else torch.full((B,), n, device=DEV, dtype=torch.int32))
        st["lens"] = st["start"] + st["n_new"]
        st["idx"] = None
        if case["K"]:
            # selected entries among the ones just written; a few slots unused
            r = torch.rand(B, case["K"], generator=g, device=DEV)
            idx = st["start"][:, None] + (r * st["n_new"][:, None]).int()
            drop = (torch.rand(B, case["K"], generator=g, device=DEV) < 0.05) | (st["n_new"] == 0)[:, None]
            st["idx"] = torch.where(drop, torch.full_like(idx, -1), idx)
        return st

    S, H, D, cr = case["S"], case["H"], case["D"], case["cr"]
    P = case.get("P", S // cr)
    st = {"case": case}
    st["q8"], st["qs"] = _codes(randn(B, S, H, D))
    st["w"] = randn(B, S, H) / math.sqrt(H * D)
    k8, ks = _codes(randn(B, P, D) + 0.3)
    if case.get("page"):
        page = case["page"]
        pages = (P + page - 1) // page
        table = torch.randperm(B * pages, generator=g, device=DEV)
        pad = pages * page - P
        cache = torch.zeros(B * pages, page, D, device=DEV, dtype=torch.int8)
        scales = torch.zeros(B * pages, page, device=DEV)
        cache[table] = torch.nn.functional.pad(k8, (0, 0, 0, pad)).view(B * pages, page, D)
        scales[table] = torch.nn.functional.pad(ks, (0, pad)).view(B * pages, page)
        st["k8"], st["ks"], st["table"] = cache, scales, table.int().view(B, pages)
        st["k_len"] = torch.randint(P // 2, P + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
        st["q_start"] = st["k_len"] * cr          # the new tokens follow the last whole block
    else:
        st["k8"], st["ks"], st["table"], st["k_len"], st["q_start"] = k8, ks, None, None, None
    st["doc"] = _doc_start(g, B, S, case["docs"])
    if case["op"] == "grad":
        K = case["K"]
        mask = _mask(st)
        if K:
            r = torch.rand(B, S, P, generator=g, device=DEV).masked_fill_(~mask, -1.0)
            v, idx = r.topk(K, dim=-1)
            idx = torch.where(v >= 0, idx, torch.full_like(idx, P)).sort(-1).values
            st["idx"] = torch.where(idx < P, idx, torch.full_like(idx, -1)).int()
            valid = st["idx"] >= 0
            del r, v, idx
        else:
            st["idx"], valid = None, mask
        # coeff/N (softmax(scores) - p), the loss's gradient
        a = randn(*valid.shape).mul_(math.sqrt(2.0)).masked_fill_(~valid, -math.inf).softmax(-1).nan_to_num_(0.0)
        p = randn(*valid.shape).exp_().masked_fill_(~valid, 0.0)
        p /= p.sum(-1, keepdim=True).clamp_min(1e-30)
        st["dscores"] = (a - p) * (1e-2 / (B * S))
    return st


# ------------------------------------------------------------ the plain form
def _mask(st):
    """[B,S,P]: block j is a candidate of token t."""
    c = st["case"]
    S, cr = c["S"], c["cr"]
    P = c.get("P", S // cr)
    t = torch.arange(S, device=DEV)[None, :, None]
    j = torch.arange(P, device=DEV)[None, None, :]
    if st["q_start"] is not None:
        t = t + st["q_start"].long()[:, None, None]
    m = (j + 1) * cr - 1 <= t
    if st["doc"] is not None:
        m = m & (j * cr >= st["doc"].long()[:, :, None])
    if st["k_len"] is not None:
        m = m & (j < st["k_len"].long()[:, None, None])
    return m.expand(c["B"], S, P)


def _keys(st):
    """The sequences' keys in order, codes and scales: [B,P,D], [B,P]."""
    if st["table"] is None:
        return st["k8"], st["ks"]
    c = st["case"]
    t = st["table"].long()
    return (st["k8"][t].reshape(c["B"], -1, c["D"])[:, :c["P"]], st["ks"][t].reshape(c["B"], -1)[:, :c["P"]])


def _cache_plain(st):
    c = st["case"]
    x = st["x"].float()
    B, n, D, grp, page = c["B"], c["n"], c["D"], c["group"], c["page"]
    xg = x.view(B, n, D // grp, grp)
    amax = xg.abs().amax(-1)
    lim = 127.0 if c["fmt"] == "int8" else 448.0
    # the code's border cases are decided in 64 bits
    v = torch.where(amax[..., None] > 0, lim * xg.double() / amax[..., None].double(), torch.zeros((), device=DEV,
                                                                                                   dtype=torch.float64))
    codes = (torch.round(v).to(torch.int8) if c["fmt"] == "int8" else _e4m3(v).float().to(torch.float8_e4m3fn))
    sc = amax / lim
    i = torch.arange(n, device=DEV)[None]
    pos = st["start"].long()[:, None] + i
    live = i < st["n_new"].long()[:, None]
    slot = st["table"].long().gather(1, (pos // page).clamp_max(c["pages"] - 1)) * page + pos % page
    flat, fsc = st["cache"].view(torch.int8).view(-1, D), st["scales"].view(-1, D // grp)
    flat[slot[live]] = codes.view(torch.int8).view(B, n, D)[live]
    fsc[slot[live]] = sc[live]
    # read back
    p = st["idx"].long() if st["idx"] is not None else torch.arange(n, device=DEV)[None] + st["start"].long()[:, None]
    ok = (p >= 0) & (p < st["lens"].long()[:, None])
    p = p.clamp(0, page * c["pages"] - 1)
    slot = st["table"].long().gather(1, p // page) * page + p % page
    got = flat.view(st["cache"].dtype)[slot].float().view(*slot.shape, D // grp, grp) * fsc[slot][..., None]
    got = torch.where(ok[..., None, None], got, torch.zeros((), device=DEV)).view(*slot.shape, D)
    return got.to(st["x"].dtype), st["scales"]


def _e4m3(v):
    """Nearest e4m3 value (64-bit in and out), ties to the even code."""
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6)))
    e = torch.where(torch.exp2(e) > v.abs().clamp_min(2.0 ** -6), e - 1, e)
    step = torch.exp2(e.clamp_min(-6.0) - 3.0)
    return torch.round(v / step) * step


def _scores_plain(st):
    c = st["case"]
    B, S, H = c["B"], c["S"], c["H"]
    k8, ks = _keys(st)
    P = k8.shape[1]
    ww = st["w"] * st["qs"]
    out = torch.empty(B, S, P, device=DEV)
    step = max(1, CHUNK // (H * P))
    for b in range(B):
        kt = k8[b].float().t()
        for t in range(0, S, step):
            q = st["q8"][b, t:t + step].float()
            dot = (q.reshape(-1, c["D"]) @ kt).view(-1, H, P)      # whole numbers, exact
            out[b, t:t + step] = (dot.relu_() * ww[b, t:t + step, :, None]).sum(1) * ks[b]
    return out.masked_fill_(~_mask(st), -math.inf)


def _dense_grad(st, dtype):
    """dscores on every block, zero where the token selected nothing."""
    c = st["case"]
    B, S, P = c["B"], c["S"], c["S"] // c["cr"]
    g = st["dscores"].to(dtype)
    if st["idx"] is not None:
        i = st["idx"].long()
        full = torch.zeros(B, S, P + 1, device=DEV, dtype=dtype)
        full.scatter_add_(2, torch.where(i >= 0, i, torch.full_like(i, P)), g)
        g = full[:, :, :P]
    return torch.where(_mask(st), g, torch.zeros((), device=DEV, dtype=dtype))


def _grad_plain(st):
    c = st["case"]
    B, S, H, D = c["B"], c["S"], c["H"], c["D"]
    k8, ks = st["k8"], st["ks"]
    P = k8.shape[1]
    G = _dense_grad(st, torch.float32)
    ww = st["w"] * st["qs"]
    dq = torch.empty(B, S, H, D, device=DEV)
    dk = torch.zeros(B, P, D, device=DEV)
    dw = torch.empty(B, S, H, device=DEV)
    step = max(1, CHUNK // (H * P))
    for b in range(B):
        kf = k8[b].float()
        for t in range(0, S, step):
            q = st["q8"][b, t:t + step].float().reshape(-1, D)
            dot = (q @ kf.t()).view(-1, H, P)                        # whole numbers, exact
            gt = G[b, t:t + step]
            gk = (gt * ks[b])[:, None]
            dw[b, t:t + step] = (gk * dot.clamp_min(0)).sum(-1) * st["qs"][b, t:t + step]
            on = (dot > 0).float()
            dq[b, t:t + step] = ((on * gk).view(-1, P) @ kf).view(-1, H, D) * st["w"][b, t:t + step, :, None]
            dk[b] += (on * gt[:, None] * ww[b, t:t + step, :, None]).view(-1, P).t() @ q
    return dq.to(torch.bfloat16), dk.to(torch.bfloat16), dw


def run(st):
    op = st["case"]["op"]
    if not own:
        return {"cache": _cache_plain, "scores": _scores_plain, "grad": _grad_plain}[op](st)
    import sparse_attention_indexer_window_b200 as sai
    c = st["case"]
    if op == "cache":
        sai.q8_cache_write(st["x"], st["cache"], st["scales"], start=st["start"], n_new=st["n_new"],
                           block_table=st["table"])
        got = sai.q8_cache_read(st["cache"], st["scales"], idx=st["idx"], n=None if c["K"] else c["n"],
                                start=None if c["K"] else st["start"], lens=st["lens"], block_table=st["table"],
                                dtype=st["x"].dtype)
        return got, st["scales"]
    if op == "scores":
        P = c["P"]
        return sai.indexer_scores(st["q8"], st["qs"], st["w"], st["k8"], st["ks"], c["cr"], P=P,
                                  block_table=st["table"], q_start=st["q_start"], k_len=st["k_len"],
                                  doc_start=st["doc"])
    return sai.indexer_scores_backward(st["dscores"], st["idx"], st["q8"], st["qs"], st["w"], st["k8"], st["ks"],
                                       c["cr"], doc_start=st["doc"])


# ------------------------------------------------------- the values in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "cache":
        return _cache_exact(st)
    B, S, H, cr = case["B"], case["S"], case["H"], case["cr"]
    P = case.get("P", S // cr)
    out = torch.full((B, S, P), -math.inf, device=DEV, dtype=torch.float64)
    grad = case["op"] == "grad"
    if grad:
        G = torch.zeros(B, S, P, device=DEV, dtype=torch.float64)
        dq = torch.zeros(B, S, H, case["D"], device=DEV, dtype=torch.float64)
        dk = torch.zeros(B, P, case["D"], device=DEV, dtype=torch.float64)
        dw = torch.zeros(B, S, H, device=DEV, dtype=torch.float64)
        if st["idx"] is None:
            G = st["dscores"].double()
        else:
            for b in range(B):
                row, slot = (st["idx"][b] >= 0).nonzero(as_tuple=True)
                G[b].index_put_((row, st["idx"][b][row, slot].long()), st["dscores"][b][row, slot].double(), True)
    for b in range(B):
        if st["table"] is None:
            k, ks = st["k8"][b].double(), st["ks"][b].double()
        else:
            r = torch.arange(P, device=DEV)
            pg = st["table"][b].long()[r // case["page"]]
            k, ks = st["k8"][pg, r % case["page"]].double(), st["ks"][pg, r % case["page"]].double()
        t0 = 0 if st["q_start"] is None else int(st["q_start"][b])
        n_k = P if st["k_len"] is None else int(st["k_len"][b])
        ends = (torch.arange(P, device=DEV) + 1) * cr - 1
        step = max(1, (1 << 25) // (H * P))
        for t in range(0, S, step):
            q, qs = st["q8"][b, t:t + step].double(), st["qs"][b, t:t + step].double()
            w = st["w"][b, t:t + step].double()
            pos = t0 + torch.arange(t, t + q.shape[0], device=DEV)
            see = ends[None] <= pos[:, None]
            see = see & (torch.arange(P, device=DEV) < n_k)[None]
            if st["doc"] is not None:
                see = see & (ends[None] - (cr - 1) >= st["doc"][b, t:t + step].long()[:, None])
            # products of the codes first: they are whole, so a product of zero is exactly zero
            s = torch.matmul(q, k.t()) * qs[..., None] * ks
            q = q * qs[..., None]
            if not grad:
                sc = torch.einsum("th,thj->tj", w, s.clamp(min=0))
                out[b, t:t + step] = torch.where(see, sc, out[b, t:t + step])
                continue
            g = torch.where(see, G[b, t:t + step], torch.zeros_like(G[b, t:t + step]))
            dw[b, t:t + step] = torch.matmul(s.clamp(min=0), g[..., None])[..., 0]
            ds = torch.where(s > 0, g[:, None] * w[..., None], torch.zeros_like(s))
            dq[b, t:t + step] = torch.matmul(ds, k * ks[:, None])
            dk[b] += torch.matmul(ds.flatten(0, 1).t(), q.flatten(0, 1))
    return (dq, dk, dw) if grad else out


def _cache_exact(st):
    c = st["case"]
    B, n, D, grp, page = c["B"], c["n"], c["D"], c["group"], c["page"]
    cap = page * c["pages"]
    lim = 127.0 if c["fmt"] == "int8" else 448.0
    x = st["x"].double().unflatten(-1, (D // grp, grp))
    top = x.abs().max(-1, keepdim=True).values
    unit = torch.where(top > 0, top, torch.ones_like(top))
    z = lim * x / unit
    if c["fmt"] == "int8":
        z = torch.round(z)
    else:
        _, e = torch.frexp(z)                                # |z| in [2^(e-1), 2^e)
        ulp = torch.ldexp(torch.ones_like(z), (e - 1).clamp(min=-6) - 3)
        z = torch.round(z / ulp) * ulp
    val = (z * top / lim).flatten(-2)
    sc = top[..., 0] / lim
    rows = torch.zeros(B, cap, D, device=DEV, dtype=torch.float64)
    scales = torch.zeros(B * c["pages"], page, D // grp, device=DEV, dtype=torch.float64)
    for b in range(B):
        s, m = int(st["start"][b]), int(st["n_new"][b])
        rows[b, s:s + m] = val[b, :m]
        full = torch.zeros(cap, D // grp, device=DEV, dtype=torch.float64)
        full[s:s + m] = sc[b, :m]
        scales[st["table"][b].long()] = full.view(c["pages"], page, D // grp)
    if st["idx"] is None:
        # positions start .. start+n-1, zero behind the sequence's length (already zero in rows)
        p = (torch.arange(n, device=DEV)[None] + st["start"].long()[:, None]).clamp(max=cap - 1)
        return rows.gather(1, p[..., None].expand(-1, -1, D)), scales
    p = st["idx"].long()
    got = rows.gather(1, p.clamp(min=0)[..., None].expand(-1, -1, D))
    return got * (p >= 0)[..., None], scales
