"""indexer_scores against the formula in 64 bits.

Tolerance: the products of codes are exact, w * q_scale is rounded once, the
product with k_scale once, and H terms are added in fp32 in some order, each
with a rounding of at most 2^-24 (relative to the terms' magnitudes): at most
(H + 3) * 2^-24 * sum of magnitudes. Where a block is no candidate the score is
-inf exactly.
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


def inputs(seed, B, S, H, D, P):
    r = np.random.default_rng(seed)
    q8 = r.integers(-127, 128, (B, S, H, D)).astype(np.int8)
    k8 = r.integers(-127, 128, (B, P, D)).astype(np.int8)
    qs = (r.random((B, S, H)) * 0.05).astype(np.float32)
    ks = (r.random((B, P)) * 0.05).astype(np.float32)
    w = r.standard_normal((B, S, H)).astype(np.float32)
    return q8, qs, w, k8, ks


def dev(*a):
    return [None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in a]


def check(got, q8, qs, w, k8, ks, mask):
    got = got.cpu().double().numpy()
    want, mag = ref.scores(q8, qs, w, k8, ks, mask)
    assert np.array_equal(np.isneginf(got), ~mask)
    tol = (q8.shape[2] + 3) * 2.0 ** -24 * mag
    d = np.abs(np.where(mask, got, 0) - np.where(mask, want, 0))
    assert np.all(d <= tol), (float((d - tol).max()), np.argwhere(d > tol)[:3])


def documents(seed, B, S):
    r = np.random.default_rng(seed)
    d = np.zeros((B, S), np.int32)
    for b in range(B):
        s = int(r.integers(1, S))
        d[b, s:] = s
    return d


@pytest.mark.parametrize("B,S,H,D,cr,docs", [
    (1, 64, 4, 32, 4, False),       # the tiny workload's heads and width
    (2, 512, 16, 128, 4, True),     # the small workload's
    (1, 1028, 64, 128, 4, False),   # P = 257: one block past two tiles
    (2, 260, 24, 64, 2, True),
    (1, 36, 1, 32, 1, False),
    (3, 50, 3, 64, 5, True),
    (1, 516, 128, 128, 2, True),
    (1, 130, 100, 128, 1, False),
    (2, 4, 8, 128, 4, False),       # one candidate in all
])
def test_whole_sequences(sai, B, S, H, D, cr, docs):
    P = S // cr
    q8, qs, w, k8, ks = inputs(S + H, B, S, H, D, P)
    doc = documents(S, B, S) if docs else None
    out = torch.full((B, S, P), float("nan"), device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    a = dev(q8, qs, w, k8, ks)
    sai.indexer_scores(*a, cr, doc_start=dev(doc)[0], out=out, err=err)
    check(out, q8, qs, w, k8, ks, ref.candidates(B, S, P, cr, doc_start=doc))
    assert int(err.item()) == 0


@pytest.mark.parametrize("B,S,H,D,page,pages,P", [
    (3, 1, 64, 128, 64, 5, 320), (1, 1, 64, 128, 16, 70, 1111), (5, 2, 24, 64, 8, 33, 260),
    (2, 3, 8, 32, 32, 9, 288), (4, 1, 128, 128, 128, 4, 400), (2, 1, 16, 128, 384, 2, 700), (2, 5, 64, 128, 1000, 1, 1000),
])
def test_paged_cache_and_single_tokens(sai, B, S, H, D, page, pages, P):
    """Pages in any order, lengths that end inside a page or tile, an empty
    cache, entries behind the length (with NaN scales), positions that see
    only some of the entries."""
    q8, qs, w, k8, ks = inputs(P, B, S, H, D, P)
    r = np.random.default_rng(B * P)
    cr = 4
    k_len = r.integers(P // 3, P + 1, B).astype(np.int32)
    k_len[0] = P
    if B > 1:
        k_len[1] = 0
    q_start = (k_len * cr).astype(np.int32)
    if B > 2:
        q_start[2] = 2                                     # sees no entry or one
    n_pages = B * pages + 2
    table = r.permutation(n_pages)[:B * pages].astype(np.int32).reshape(B, pages)
    cache = r.integers(-127, 128, (n_pages, page, D)).astype(np.int8)
    scale = np.full((n_pages, page), np.nan, np.float32)
    for b in range(B):
        for j in range(k_len[b]):
            cache[table[b, j // page], j % page] = k8[b, j]
            scale[table[b, j // page], j % page] = ks[b, j]
        table[b, (k_len[b] + page - 1) // page:] = -1       # pages not yet given out
    out = torch.full((B, S, P), float("nan"), device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    a = dev(q8, qs, w, cache, scale, table, q_start, k_len)
    sai.indexer_scores(*a[:5], cr, P=P, block_table=a[5], q_start=a[6], k_len=a[7], out=out, err=err)
    check(out, q8, qs, w, k8, ks, ref.candidates(B, S, P, cr, q_start, k_len))
    assert int(err.item()) == 0


@pytest.mark.parametrize("B,S,H,D,page,pages,P,bad", [
    (4, 1, 64, 128, 64, 320, 20000, False), (5, 2, 8, 32, 8, 2600, 20800, True), (6, 1, 24, 64, 128, 150, 19111, True),
    (5, 1, 16, 64, 16, 1300, 20790, False), (5, 3, 64, 128, 20001, 1, 20001, False), (9, 1, 128, 32, 32, 640, 20480, True),
])
def test_long_caches_of_few_tokens(sai, B, S, H, D, page, pages, P, bad):
    """Few tokens over many entries, whose keys are split over the SMs: an empty
    cache between full ones, lengths inside a tile, a page id outside the cache."""
    q8, qs, w, k8, ks = inputs(P + B, B, S, H, D, P)
    r = np.random.default_rng(P - B)
    k_len = np.array([P, 0, P - 77, 129, P // 2 + 3, 1, P, 4000, P - 1][:B], np.int32)
    q_start = (k_len.astype(np.int64) * 4 + 8).astype(np.int32)
    n_pages = B * pages + 1
    table = r.permutation(n_pages)[:B * pages].astype(np.int32).reshape(B, pages)
    cache = r.integers(-127, 128, (n_pages, page, D)).astype(np.int8)
    scale = np.full((n_pages, page), np.nan, np.float32)
    for b in range(B):
        for i in range((k_len[b] + page - 1) // page):
            n = min(page, k_len[b] - i * page)
            cache[table[b, i], :n] = k8[b, i * page:i * page + n]
            scale[table[b, i], :n] = ks[b, i * page:i * page + n]
    mask = ref.candidates(B, S, P, 4, q_start, k_len)
    if bad:
        i = (P // 2) // page
        table[0, i] = n_pages
        mask[0, :, i * page:(i + 1) * page] = False
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    a = dev(q8, qs, w, cache, scale, table, q_start, k_len)
    outs = [torch.full((B, S, P), float("nan"), device="cuda") for _ in range(3)]
    for out in outs:
        sai.indexer_scores(*a[:5], 4, P=P, block_table=a[5], q_start=a[6], k_len=a[7], out=out, err=err)
    check(outs[0], q8, qs, w, k8, ks, mask)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    assert int(err.item()) == (sai.SAI_ERR_INDEX if bad else 0)


def test_page_ids_outside_the_cache(sai):
    B, S, H, D, page = 2, 1, 16, 64, 16
    q8, qs, w, k8, ks = inputs(5, B, S, H, D, 64)
    table = np.arange(8, dtype=np.int32).reshape(2, 4)
    bad = table.copy()
    bad[0, 1], bad[1, 3] = 8, -1
    a = dev(q8, qs, w, k8.reshape(8, page, D), ks.reshape(8, page), bad)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    start = torch.full((B,), 1000, dtype=torch.int32, device="cuda")
    out = sai.indexer_scores(*a[:5], 4, block_table=a[5], q_start=start, err=err)
    mask = np.ones((B, S, 64), bool)
    mask[0, :, 16:32] = False
    mask[1, :, 48:] = False
    check(out, q8, qs, w, k8, ks, mask)
    assert int(err.item()) == sai.SAI_ERR_INDEX


def test_extreme_codes_and_scales(sai):
    """Every code at its limit (the largest products), zero and NaN scales."""
    B, S, H, D = 1, 256, 64, 128
    q8 = np.full((B, S, H, D), 127, np.int8)
    k8 = np.full((B, 64, D), 127, np.int8)
    k8[:, ::2] = -127
    q8[:, ::3] = -128
    qs = np.full((B, S, H), 1e-3, np.float32)
    qs[:, 5] = 0
    ks = np.full((B, 64), 3e4, np.float32)
    ks[:, 4] = 0
    w = np.random.default_rng(0).standard_normal((B, S, H)).astype(np.float32)
    check(sai.indexer_scores(*dev(q8, qs, w, k8, ks), 4), q8, qs, w, k8, ks, ref.candidates(B, S, 64, 4))
    ks[:, 9] = np.nan
    out = sai.indexer_scores(*dev(q8, qs, w, k8, ks), 4).cpu().numpy()
    assert np.isnan(out[0, 39:, 9]).all() and np.isneginf(out[0, :39, 9]).all()
    assert not np.isnan(np.delete(out, 9, 2)).any()


def test_row_offsets_past_32_bits(sai):
    """An output of more than 2^31 scores: the last rows are right."""
    S, P, H, D = 34000, 65000, 8, 32
    q8, qs, w, k8, ks = inputs(1, 1, S, H, D, P)
    start = torch.tensor([10 * P], dtype=torch.int32, device="cuda")
    out = sai.indexer_scores(*dev(q8, qs, w, k8, ks), 1, q_start=start)
    assert out.numel() > 1 << 31
    tail = slice(S - 2, S)
    check(out[:, tail], q8[:, tail], qs[:, tail], w[:, tail], k8, ks, np.ones((1, 2, P), bool))


def test_streams_and_graph_give_the_same_bits(sai):
    B, S, H, D = 2, 200, 64, 128
    q8, qs, w, k8, ks = inputs(3, B, S, H, D, 50)
    a = dev(q8, qs, w, k8, ks)
    first = sai.indexer_scores(*a, 4)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for s in (s1, s2):                                       # two calls at once
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            outs.append(sai.indexer_scores(*a, 4))
    for s in (s1, s2):
        torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = sai.indexer_scores(*a, 4)
    g.replay()
    g.replay()
    for o in outs + [held]:
        assert torch.equal(o, first)
