"""indexer_scores_backward where gradients, weights and scales of one call span
far more than fp16's range: a token's dq depends on that token's own gradients
and a key's dk on that key's own terms, not on the largest of the batch.

Tolerances: as in test_gpu_indexer_backward.py, but the absolute part of a term
held in fp16 is taken from the token (dq) or the key (dk) itself. With a power of
two that brings the largest value to 2^14 at least, half of fp16's smallest step is
2^-25 * 2^-14 of it at most. dq: 2^-39 of the token's largest |G k_scale|, times
127 |w|, for each of n terms. dk: a term's two factors are G max_h|w q_scale|,
scaled by key (2^-38 of the key's largest, the power of two over the maximum being
twice it at most), and q8 w q_scale / max_h|w q_scale|, scaled by token to 2^7 at
least (127 half steps and two roundings of 2^-25: 129 * 2^-32).
"""
import numpy as np
import pytest

from tests import q8_ref as ref
from tests.test_gpu_indexer_backward import dev, fresh, inputs, selection

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def sai():
    import sparse_attention_indexer_window_b200 as m
    return m


def check_rows(got, G, q8, qs, w, k8, ks, parts=("dq", "dk", "dw")):
    want, mag = ref.scores_grad(G, q8, qs, w, k8, ks)
    B, S, H, D = q8.shape
    P = k8.shape[1]
    wmax = np.abs(w.astype(np.float64) * qs).max(-1)                          # [B,S]
    top_t = np.where(G != 0, np.abs(G) * ks[:, None, :], 0).max(-1)           # [B,S]
    n_t = (G != 0).sum(-1)
    gw = np.abs(G) * wmax[:, :, None]                                         # [B,S,P]
    top_j, n_j = gw.max(1), (G != 0).sum(1) * H
    lost = {"dq": (2.0 ** -39 * 127 * (top_t * n_t)[:, :, None] * np.abs(w))[..., None],
            "dk": (2.0 ** -38 * 127 * top_j * n_j + 129 * 2.0 ** -32 * H * gw.sum(1))[..., None]}
    for name, g, x, a, n in (("dq", got[0], want[0], mag[0], P), ("dk", got[1], want[1], mag[1], S * H)):
        if name not in parts:
            continue
        held = 2.0 ** -11 if name == "dq" else 2.0 ** -10 + 2.0 ** -21
        tol = (held + (n + 4) * 2.0 ** -24) * a + 2.0 ** -8 * np.abs(x) + lost[name]
        d = np.abs(g.cpu().double().numpy() - x)
        assert np.all(d <= tol * (1 + 2.0 ** -7)), (name, np.argwhere(d > tol * (1 + 2.0 ** -7))[:3],
                                                    float((d / np.maximum(tol, 1e-300)).max()))
    if "dw" in parts:
        d = np.abs(got[2].cpu().double().numpy() - want[2])
        assert np.all(d <= (P + 4) * 2.0 ** -24 * mag[2]), "dw"


def run(sai, ds, idx, q8, qs, w, k8, ks, cr, doc=None):
    out = fresh(*q8.shape, k8.shape[1])
    a = dev(ds, idx, q8, qs, w, k8, ks, doc)
    return sai.indexer_scores_backward(*a[:7], cr, doc_start=a[7], dq=out[0], dk=out[1], dw=out[2])


SHAPES = [(16, 64), (64, 128), (8, 32), (128, 128)]


@pytest.mark.parametrize("H,D", SHAPES)
@pytest.mark.parametrize("dense", [False, True])
def test_tokens_of_small_gradients_keep_their_dq(sai, H, D, dense):
    """Tokens whose gradients are 2^-35, 2^-60 and 2^-30 of the others', in the
    same sequence and in one of its own; and a key of a huge scale elsewhere."""
    B, S, cr = 2, 160, 4
    P = S // cr
    q8, qs, w, k8, ks = inputs(H + D, B, S, H, D, P)
    mask = ref.candidates(B, S, P, cr)
    if dense:
        idx, ds = None, np.where(mask, np.random.default_rng(D).standard_normal(mask.shape), 0).astype(np.float32)
    else:
        idx, ds = selection(H, mask, 12)
        ds = np.where(idx >= 0, ds * 1e6, 0).astype(np.float32)
    ds[0, 60:90] *= 2.0 ** -35
    ds[0, 131] *= 2.0 ** -60
    ds[1] *= 2.0 ** -30
    ks[0, 3] = 2.0 ** 20
    G = ref.dense(ds, idx, mask)
    check_rows(run(sai, ds, idx, q8, qs, w, k8, ks, cr), G, q8, qs, w, k8, ks, ("dq", "dw"))


@pytest.mark.parametrize("H,D", SHAPES)
@pytest.mark.parametrize("dense", [False, True])
def test_keys_of_small_gradients_keep_their_dk(sai, H, D, dense):
    """Two documents in a row and two rows: the gradients (or the head weights) of
    one are 2^-35 or 2^-45 of the other's."""
    B, S, cr = 2, 160, 4
    P = S // cr
    q8, qs, w, k8, ks = inputs(H + D + 1, B, S, H, D, P)
    doc = np.zeros((B, S), np.int32)
    doc[:, 80:] = 80
    mask = ref.candidates(B, S, P, cr, doc_start=doc)
    if dense:
        idx, ds = None, np.where(mask, np.random.default_rng(D).standard_normal(mask.shape), 0).astype(np.float32)
    else:
        idx, ds = selection(H, mask, 9)
        ds = np.where(idx >= 0, ds * 1e6, 0).astype(np.float32)
    ds[0, :80] *= 2.0 ** -35
    w[1, 80:] *= 2.0 ** -45
    ds[1] *= 2.0 ** -10
    G = ref.dense(ds, idx, mask)
    check_rows(run(sai, ds, idx, q8, qs, w, k8, ks, cr, doc), G, q8, qs, w, k8, ks)


def test_a_sequence_alone_and_in_a_batch(sai):
    """dq and dw of a sequence are the same bits whatever it is batched with."""
    B, S, H, D, cr = 3, 200, 24, 64, 2
    P = S // cr
    q8, qs, w, k8, ks = inputs(30, B, S, H, D, P)
    mask = ref.candidates(B, S, P, cr)
    idx, ds = selection(30, mask, 20)
    ds[1] *= np.float32(2.0 ** 40)
    ks[2, 5], qs[2, 7] = 2.0 ** 18, 2.0 ** 25
    whole = run(sai, ds, idx, q8, qs, w, k8, ks, cr)
    G = ref.dense(ds, idx, mask)
    for b in range(B):
        one = [x[b:b + 1] for x in (ds, idx, q8, qs, w, k8, ks)]
        alone = run(sai, *one, cr)
        assert torch.equal(alone[0], whole[0][b:b + 1]) and torch.equal(alone[2], whole[2][b:b + 1])
        check_rows(alone, G[b:b + 1], *one[2:])
        check_rows([x[b:b + 1] for x in whole], G[b:b + 1], *one[2:])


@pytest.mark.parametrize("S,H,D,cr,K", [(1500, 64, 128, 4, 60), (700, 128, 128, 2, 0), (5000, 8, 128, 20, 40)])
def test_lists_of_items_at_the_full_width(sai, S, H, D, cr, K):
    """D = 128, where tensor memory is full: more items than the GPU has SMs, of one
    key tile and of several, against the formula; ten runs give the same bits."""
    B, P = 1, S // cr
    q8, qs, w, k8, ks = inputs(S, B, S, H, D, P)
    mask = ref.candidates(B, S, P, cr)
    if K:
        idx, ds = selection(S, mask, K)
        ds = np.where(idx >= 0, ds, 0).astype(np.float32)
    else:
        idx, ds = None, np.where(mask, np.random.default_rng(S).standard_normal(mask.shape) * 1e-5, 0).astype(np.float32)
    first = run(sai, ds, idx, q8, qs, w, k8, ks, cr)
    check_rows(first, ref.dense(ds, idx, mask), q8, qs, w, k8, ks)
    a = dev(ds, idx, q8, qs, w, k8, ks)
    for _ in range(10):
        for x, y in zip(sai.indexer_scores_backward(*a, cr), first):
            assert torch.equal(x, y)
