"""indexer_scores_backward against the formula in 64 bits and against
differences, and the whole step from the indexer's queries to its gradients.

Tolerances, A being the sum of the terms' magnitudes (tests/q8_ref.py):
  dq, dk  each term may be held in fp16 (2^-11 relative, and an absolute part
          below 2^-36 of the largest term: scaled so that the largest uses the
          type's range), products of scales are rounded in fp32 (a few 2^-24),
          n terms added in fp32 (n * 2^-24), one rounding to bf16 (2^-8). In dk
          both factors of a term are held in fp16, G and w q_scale q8: twice
          2^-11, and 2^-21 for the scale's own 22 bits
  dw      n terms in fp32 and three roundings of products: (n + 4) * 2^-24 * A
Below fp32's normal range (2^-126) a product G * k_scale, or G * w * q_scale, is
rounded to a multiple of 2^-149: off by up to 2^-150 however small it is. Each
of the n terms carries that into dq times 127 |w|, into dk times 127 (and 2^-150
times |G| where w * q_scale itself is that small), into dw times
127^2 D q_scale. A bf16 result below 2^-126 is off by up to 2^-134.
"""
import numpy as np
import pytest

from tests import q8_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def sai():
    import sparse_attention_indexer_window_b200 as m
    return m


def dev(*a):
    return [None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in a]


def inputs(seed, B, S, H, D, P):
    r = np.random.default_rng(seed)
    q8 = r.integers(-127, 128, (B, S, H, D)).astype(np.int8)
    k8 = r.integers(-127, 128, (B, P, D)).astype(np.int8)
    qs = (r.random((B, S, H)) * 0.05).astype(np.float32)
    ks = (r.random((B, P)) * 0.05).astype(np.float32)
    w = (r.standard_normal((B, S, H)) * 0.1).astype(np.float32)
    return q8, qs, w, k8, ks


def selection(seed, mask, K):
    """Distinct candidates, -1 padded, and gradients of very different size."""
    r = np.random.default_rng(seed)
    B, S, P = mask.shape
    idx = np.full((B, S, K), -1, np.int32)
    for b in range(B):
        for t in range(S):
            c = np.flatnonzero(mask[b, t])
            c = r.permutation(c)[:K]
            idx[b, t, :len(c)] = c
    ds = r.standard_normal((B, S, K)) * np.exp(r.standard_normal((B, S, 1)) * 2) * 1e-6
    return idx, ds.astype(np.float32)


def check(got, G, q8, qs, w, k8, ks):
    (want, mag) = ref.scores_grad(G, q8, qs, w, k8, ks)
    B, S, H, D = q8.shape
    P = k8.shape[1]
    top_k = float(np.nanmax(np.where(G != 0, np.abs(G) * ks[:, None, :], 0)))
    top_q = float(np.abs(G).max()) * float(np.abs(w * qs).max())
    for name, g, x, a, n, tiny in (("dq", got[0], want[0], mag[0], P, top_k * np.abs(w).max() * P),
                                   ("dk", got[1], want[1], mag[1], S * H, top_q * S * H)):
        g = g.cpu().double().numpy()
        held = 2.0 ** -11 if name == "dq" else 2.0 ** -10 + 2.0 ** -21
        tol = (held + (n + 4) * 2.0 ** -24) * a + 2.0 ** -8 * np.abs(x) + 2.0 ** -36 * 127 * tiny
        tol = tol + 2.0 ** -150 * 127 * n * (np.abs(w).max() if name == "dq" else 1 + np.abs(G).max()) + 2.0 ** -134
        # (the rounding to bf16 is of the computed value: 2^-8 of the error before it, too)
        d = np.abs(g - x)
        assert np.all(d <= tol * (1 + 2.0 ** -7)), (name, float((d / np.maximum(tol, 1e-300)).max()))
    d, tol = np.abs(got[2].cpu().double().numpy() - want[2]), (P + 4) * 2.0 ** -24 * mag[2]
    tol = tol + 2.0 ** -150 * P * 127 * 127 * D * qs + 2.0 ** -149
    assert np.all(d <= tol), ("dw", float((d - tol).max()))


def fresh(B, S, H, D, P):
    return (torch.full((B, S, H, D), float("nan"), dtype=torch.bfloat16, device="cuda"),
            torch.full((B, P, D), float("nan"), dtype=torch.bfloat16, device="cuda"),
            torch.full((B, S, H), float("nan"), device="cuda"))


@pytest.mark.parametrize("B,S,H,D,cr,K,docs", [
    (1, 64, 4, 32, 4, 8, False),     # the tiny workload
    (2, 256, 16, 128, 4, 20, True),
    (1, 516, 64, 128, 4, 60, False),  # P = 129: one block past a tile
    (2, 100, 24, 64, 2, 0, True),    # dense
    (1, 37, 1, 32, 1, 5, False),
    (1, 33, 3, 64, 1, 0, False),
    (1, 260, 128, 128, 2, 33, True),
    (1, 300, 100, 64, 1, 0, True),
    (1, 1100, 8, 32, 2, 100, False),  # more than four key tiles, many tokens a tile
    (3, 6, 64, 128, 4, 1, False),    # one candidate in all
    (1, 3, 8, 64, 4, 0, False),      # no candidate at all (P = 1 given)
])
def test_against_the_formula(sai, B, S, H, D, cr, K, docs):
    P = max(1, S // cr)
    q8, qs, w, k8, ks = inputs(S + D, B, S, H, D, P)
    doc = None
    if docs:
        doc = np.zeros((B, S), np.int32)
        doc[:, S // 3:] = S // 3
    mask = ref.candidates(B, S, P, cr, doc_start=doc)
    if K:
        idx, ds = selection(S, mask, K)
    else:
        idx, ds = None, (np.random.default_rng(S).standard_normal((B, S, P)) * 1e-5).astype(np.float32)
        ds[~mask] = np.nan                                   # masked entries are not used
    out = fresh(B, S, H, D, P)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    a = dev(ds, idx, q8, qs, w, k8, ks, doc)
    sai.indexer_scores_backward(*a[:7], cr, doc_start=a[7], dq=out[0], dk=out[1], dw=out[2], err=err)
    check(out, ref.dense(ds, idx, mask), q8, qs, w, k8, ks)
    assert int(err.item()) == 0


def test_repeated_masked_and_bad_slots(sai):
    """The same block in several slots adds up; future blocks and -1 slots give
    nothing (their gradients may be NaN); indices outside set the error word."""
    B, S, H, D, cr, K = 1, 96, 16, 64, 4, 12
    P = S // cr
    q8, qs, w, k8, ks = inputs(8, B, S, H, D, P)
    mask = ref.candidates(B, S, P, cr)
    idx, ds = selection(8, mask, K)
    idx[:, 60:, 1] = idx[:, 60:, 0]
    idx[:, 60:, 5] = idx[:, 60:, 0]
    idx[:, 20, :] = P - 1                                     # a block of the future, twelve times
    ds[:, 20, :] = np.nan
    ds[idx == -1] = np.nan
    out = fresh(B, S, H, D, P)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    sai.indexer_scores_backward(*dev(ds, idx, q8, qs, w, k8, ks), cr, dq=out[0], dk=out[1], dw=out[2], err=err)
    G = ref.dense(ds, idx, mask)
    check(out, G, q8, qs, w, k8, ks)
    assert int(err.item()) == 0
    bad = idx.copy()
    bad[:, 90, 3], bad[:, 91, 4] = P, -2
    err.zero_()
    got = sai.indexer_scores_backward(*dev(ds, bad, q8, qs, w, k8, ks), cr, err=err)
    check(got, ref.dense(ds, bad, mask), q8, qs, w, k8, ks)
    assert int(err.item()) == sai.SAI_ERR_INDEX


def test_unused_keys_may_hold_anything(sai):
    """Keys that no token selects: their scales (NaN, infinite, huge) change nothing."""
    B, S, H, D, cr = 1, 128, 16, 64, 4
    P = S // cr
    q8, qs, w, k8, ks = inputs(9, B, S, H, D, P)
    mask = ref.candidates(B, S, P, cr)
    mask[:, :, 7] = mask[:, :, 20] = mask[:, :, 21] = False
    idx, ds = selection(9, mask, 10)
    want = sai.indexer_scores_backward(*dev(ds, idx, q8, qs, w, k8, ks), cr)
    ks[:, 7], ks[:, 20], ks[:, 21] = np.nan, np.inf, 1e30
    got = sai.indexer_scores_backward(*dev(ds, idx, q8, qs, w, k8, ks), cr)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("factor", [1e-30, 1.0, 1e25])
def test_gradients_of_any_magnitude(sai, factor):
    B, S, H, D, cr = 1, 200, 16, 64, 4
    P = S // cr
    q8, qs, w, k8, ks = inputs(10, B, S, H, D, P)
    idx, ds = selection(10, ref.candidates(B, S, P, cr), 16)
    ds = (ds * factor).astype(np.float32)
    got = sai.indexer_scores_backward(*dev(ds, idx, q8, qs, w, k8, ks), cr)
    check(got, ref.dense(ds, idx, ref.candidates(B, S, P, cr)), q8, qs, w, k8, ks)


def test_all_zero_gradient(sai):
    q8, qs, w, k8, ks = inputs(12, 1, 40, 8, 32, 10)
    got = sai.indexer_scores_backward(torch.zeros(1, 40, 10, device="cuda"), None, *dev(q8, qs, w, k8, ks), 4)
    for g in got:
        assert int((g != 0).sum()) == 0


def test_token_ranges_add_up(sai):
    """Two calls over a split sequence: dq and dw are the whole call's rows, the
    dk add up to the whole call's (within their roundings)."""
    B, S, H, D, cr, K = 1, 320, 16, 128, 4, 30
    P = S // cr
    q8, qs, w, k8, ks = inputs(13, B, S, H, D, P)
    mask = ref.candidates(B, S, P, cr)
    idx, ds = selection(13, mask, K)
    G = ref.dense(ds, idx, mask)
    for lo, hi in ((0, 123), (123, 320)):
        r = slice(lo, hi)
        got = sai.indexer_scores_backward(*dev(ds[:, r], idx[:, r], q8[:, r], qs[:, r], w[:, r], k8, ks), cr,
                                          t_begin=lo)
        check(got, G[:, r], q8[:, r], qs[:, r], w[:, r], k8, ks)


def test_against_differences(sai):
    """dw and dq against central differences of indexer_scores itself: the
    scores are linear in w, and linear in q_scale (a direction of the query:
    d/dq_scale = <dq, q8>) and in k_scale (<dk, k8>)."""
    B, S, H, D, cr = 1, 120, 16, 64, 4
    P = S // cr
    q8, qs, w, k8, ks = inputs(14, B, S, H, D, P)
    mask = ref.candidates(B, S, P, cr)
    r = np.random.default_rng(14)
    g = np.where(mask, r.standard_normal(mask.shape), 0).astype(np.float32)
    dq, dk, dw = [x.cpu().double().numpy() for x in
                  sai.indexer_scores_backward(*dev(g), None, *dev(q8, qs, w, k8, ks), cr)]

    def loss(qs, w, ks):
        s = sai.indexer_scores(*dev(q8, qs, w, k8, ks), cr).cpu().double().numpy()
        return float((np.where(mask, s, 0) * g).sum()), float((np.where(mask, np.abs(s), 0) * np.abs(g)).sum())

    for name, base, grad in (("w", w, dw), ("qs", qs, (dq * q8).sum(-1)), ("ks", ks, (dk * k8).sum(-1))):
        step = np.abs(base) * r.random(base.shape).astype(np.float32)     # a whole direction at once
        up, down = (base + step).astype(np.float32), (base - step).astype(np.float32)
        args = {"qs": qs, "w": w, "ks": ks}
        (hi, m1), (lo, m2) = loss(**{**args, name: up}), loss(**{**args, name: down})
        want = (grad * (up.astype(np.float64) - down)).sum()
        # each score is off by at most (H + 3) 2^-24 of its terms' sizes, each
        # gradient value by 2^-8 of itself and 2^-11 of its terms
        tol = (m1 + m2) * 64 * (H + 3) * 2.0 ** -24 + 2.0 ** -7 * np.abs(grad * (up - down)).sum()
        assert abs((hi - lo) - want) <= tol, (name, hi - lo, want, tol)


def test_same_bits_again_and_in_a_graph(sai):
    B, S, H, D, cr, K = 2, 300, 64, 128, 4, 40
    P = S // cr
    q8, qs, w, k8, ks = inputs(15, B, S, H, D, P)
    idx, ds = selection(15, ref.candidates(B, S, P, cr), K)
    a = dev(ds, idx, q8, qs, w, k8, ks)
    first = sai.indexer_scores_backward(*a, cr)
    ws = torch.full((sai.scores_backward_workspace_bytes(B, S, H, D, P),), 255, dtype=torch.uint8, device="cuda")
    again = sai.indexer_scores_backward(*a, cr, workspace=ws)     # whatever the workspace holds
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [again]
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            outs.append(sai.indexer_scores_backward(*a, cr))
    for s in (s1, s2):
        torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = sai.indexer_scores_backward(*a, cr)
    g.replay()
    g.replay()
    for o in outs + [held]:
        for x, y in zip(o, first):
            assert torch.equal(x, y)


def test_the_whole_step(sai):
    """Queries and keys to 8 bits, scores, selection, loss and gradients in one
    run: each stage's output feeds the next, the gradients are the formula's
    on the selection that the step made."""
    import synth
    from tests.gpu_util import to_dev
    w_ = synth.make("flash", S=512, K=60)
    t = to_dev(w_)
    B, S, cr, K = w_.B, w_.S, w_.cr, w_.K
    H, D, P = 16, 128, S // cr
    gen = torch.Generator().manual_seed(4)
    qi = torch.randn(B, S, H, D, generator=gen).bfloat16().cuda()
    ki = torch.randn(B, P, D, generator=gen).bfloat16().cuda()
    w = (torch.randn(B, S, H, generator=gen) / H / D).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    loss, dq, dk, dw = sai.indexer_distill_step(qi, w, ki, t["Q"], t["Kw"], t["pool"], K=K, W=w_.W, cr=cr,
                                                scale=w_.scale, coeff=w_.coeff, sink=t["sink"], err=err)
    assert int(err.item()) == 0 and np.isfinite(float(loss.item()))
    q8, qs = sai.q8_quantize(qi)
    k8, ks = sai.q8_quantize(ki)
    mask = ref.candidates(B, S, P, cr)
    n = [x.cpu().numpy() for x in (q8, qs[..., 0], w, k8, ks[..., 0])]
    s = sai.indexer_scores(q8, qs, w, k8, ks, cr)
    want, mag = ref.scores(*n, mask)
    assert np.all(np.abs(np.where(mask, s.cpu().double().numpy() - np.where(mask, want, 0), 0))
                  <= (H + 3) * 2.0 ** -24 * mag)
    idx, sel, valid = sai.indexer_topk(s, cr, K)
    _, ds, _, _ = sai.distill_loss(t["Q"], t["Kw"], t["pool"], idx, sel, valid, W=w_.W, cr=cr, scale=w_.scale,
                                   coeff=w_.coeff, sink=t["sink"])
    G = ref.dense(ds.cpu().numpy(), idx.cpu().numpy(), mask)
    check((dq, dk, dw), G, *n)
    # the same through the paged cache: keys appended to pages, scored from there
    page = 16
    table = torch.randperm(P // page, generator=gen).int().view(1, -1).cuda()
    cache = torch.zeros(P // page, page, D, dtype=torch.int8, device="cuda")
    scl = torch.zeros(P // page, page, 1, device="cuda")
    half = P // 2
    sai.q8_cache_write(ki[:, :half], cache, scl, block_table=table)
    sai.q8_cache_write(ki[:, half:], cache, scl, block_table=table,
                       start=torch.full((1,), half, dtype=torch.int32, device="cuda"))
    assert torch.equal(sai.indexer_scores(q8, qs, w, cache, scl, cr, block_table=table), s)
    # and one token at its position, as decoding has it
    pos = 401
    one = sai.indexer_scores(q8[:, pos:pos + 1].contiguous(), qs[:, pos:pos + 1].contiguous(),
                             w[:, pos:pos + 1].contiguous(), cache, scl, cr, block_table=table,
                             q_start=torch.full((1,), pos, dtype=torch.int32, device="cuda"))
    assert torch.equal(one[:, 0], s[:, pos])


def test_padding_without_gradient_may_hold_anything(sai):
    """Tokens that select nothing: their weights and scales (NaN, huge) change
    nothing, and their own gradients are zero."""
    B, S, H, D, cr = 2, 150, 16, 64, 2
    P = S // cr
    q8, qs, w, k8, ks = inputs(16, B, S, H, D, P)
    idx, ds = selection(16, ref.candidates(B, S, P, cr), 20)
    idx[:, 100:] = -1
    idx[:, 40] = -1
    want = sai.indexer_scores_backward(*dev(ds, idx, q8, qs, w, k8, ks), cr)
    w[:, 100:], w[:, 40], qs[:, 120:] = np.nan, 1e30, np.inf
    got = sai.indexer_scores_backward(*dev(ds, idx, q8, qs, w, k8, ks), cr)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert int((got[0][:, 100:] != 0).sum()) == 0 and int((got[2][:, 40] != 0).sum()) == 0


def test_many_slots_of_one_block(sai):
    """A block named by 300 slots of a token, over more blocks than are gathered at once."""
    B, S, H, D, cr, P, K = 1, 40, 8, 32, 1, 9000, 300
    q8, qs, w, k8, ks = inputs(17, B, S, H, D, P)
    r = np.random.default_rng(17)
    idx = r.integers(0, P, (B, S, K)).astype(np.int32)
    idx[:, 3] = 5000
    idx[:, 9, ::3] = 4096
    ds = r.standard_normal((B, S, K)).astype(np.float32)
    mask = np.ones((B, S, P), bool)
    a = dev(ds, idx, q8, qs, w, k8, ks)
    got = sai.indexer_scores_backward(*a, cr, t_begin=20000)
    # G itself is a sum of up to 300 fp32 terms: its rounding is a part of every term's size
    G = ref.dense(ds, idx, mask)
    G32 = np.zeros((B, S, P), np.float32)
    for t in range(S):
        for k in range(K):
            G32[0, t, idx[0, t, k]] += ds[0, t, k]
    assert np.abs(G32 - G).max() < 1e-3
    check(got, G32.astype(np.float64), q8, qs, w, k8, ks)
    again = sai.indexer_scores_backward(*a, cr, t_begin=20000)
    for x, y in zip(got, again):
        assert torch.equal(x, y)


@pytest.mark.parametrize("S,H,D,cr,K", [(1500, 64, 64, 4, 60), (2600, 128, 32, 8, 0), (1400, 64, 32, 2, 100)])
def test_many_tiles_a_block_of_threads(sai, S, H, D, cr, K):
    """More token tiles than the GPU has SMs, from one key tile to several each:
    every SM works through a list of them, its last ones the shortest. Twenty
    runs give the same bits, and they are the formula's."""
    B, P = 1, S // cr
    q8, qs, w, k8, ks = inputs(S, B, S, H, D, P)
    mask = ref.candidates(B, S, P, cr)
    if K:
        idx, ds = selection(S, mask, K)
    else:
        idx, ds = None, (np.random.default_rng(S).standard_normal((B, S, P)) * 1e-5).astype(np.float32)
    a = dev(ds, idx, q8, qs, w, k8, ks)
    first = sai.indexer_scores_backward(*a, cr)
    check(first, ref.dense(ds, idx, mask), q8, qs, w, k8, ks)
    for _ in range(20):
        for x, y in zip(sai.indexer_scores_backward(*a, cr), first):
            assert torch.equal(x, y)
