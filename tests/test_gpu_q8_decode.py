"""Decoding with the 8-bit cache: new keys appended, scored for one token a sequence,
a selection made from the scores, its entries read back; against the formula
in 64 bits.

Scores are within (H + 3) 2^-24 of the sum of their terms' magnitudes
(test_gpu_indexer_scores.py), so every selected score is at least the exact K-th
best less two such errors. Entries read back equal fp32(code * scale) exactly.
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


@pytest.mark.parametrize("B,H,D,page,pages,K", [(3, 64, 128, 64, 6, 40), (1, 8, 32, 16, 9, 30), (4, 24, 64, 128, 2, 1)])
def test_append_score_select_read(sai, B, H, D, page, pages, K):
    g = torch.Generator().manual_seed(page)
    cap = page * pages
    keys = torch.randn(B, cap, D, generator=g).bfloat16()
    n_old = torch.tensor([cap - 5, 7, 0, cap // 2][:B], dtype=torch.int32)
    n_new = torch.tensor([5, 20, 0, 1][:B], dtype=torch.int32)
    n_now = n_old + n_new
    keys[0, 3] = float("nan")                                   # a spoiled entry is never selected
    table = torch.randperm(B * pages, generator=g).int().view(B, pages).cuda()
    cache = torch.zeros(B * pages, page, D, dtype=torch.int8, device="cuda")
    scales = torch.zeros(B * pages, page, 1, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    sai.q8_cache_write(keys.cuda(), cache, scales, n_new=n_old.cuda(), block_table=table, err=err)
    new = torch.stack([torch.nn.functional.pad(keys[b, int(n_old[b]):int(n_old[b]) + 20],
                                               (0, 0, 0, max(0, 20 - (cap - int(n_old[b]))))) for b in range(B)])
    sai.q8_cache_write(new.cuda(), cache, scales, start=n_old.cuda(), n_new=n_new.cuda(), block_table=table, err=err)
    q = torch.randn(B, 1, H, D, generator=g).bfloat16().cuda()
    w = torch.randn(B, 1, H, generator=g).cuda()
    q8, qs = sai.q8_quantize(q)
    pos = n_now * 4
    s = sai.indexer_scores(q8, qs, w, cache, scales, 4, block_table=table, q_start=pos.cuda(), k_len=n_now.cuda(),
                           err=err)[:, 0]
    best, chosen = s.masked_fill(s.isnan(), -torch.inf).topk(K)
    chosen = chosen.int().masked_fill(best == -torch.inf, -1)
    rows = sai.q8_cache_read(cache, scales, idx=chosen, lens=n_now.cuda(), block_table=table, dtype=torch.float32,
                             err=err)
    assert int(err.item()) == 0
    with pytest.raises(ValueError):                             # whole sequences only
        sai.indexer_topk(s[:, None].contiguous(), 4, K)

    code, scale = ref.quantize(keys, D, "int8")
    want, mag = ref.scores(ref.code_values(q8), qs[..., 0].cpu().numpy(), w.cpu().numpy(), code,
                           np.nan_to_num(scale[..., 0]), ref.candidates(B, 1, cap, 4, pos, n_now))
    want, tol = want[:, 0], (H + 3) * 2.0 ** -24 * mag[:, 0].max(-1)
    chosen, rows = chosen.cpu().numpy(), rows.cpu().numpy()
    for b in range(B):
        live = np.arange(cap) < int(n_now[b])
        if b == 0:
            live[3] = False
        sel = chosen[b][chosen[b] >= 0]
        assert len(set(sel)) == len(sel) == min(K, int(live.sum())) and live[sel].all()
        kth = np.sort(want[b][live])[::-1][len(sel) - 1] if len(sel) else 0.0
        assert np.all(want[b][sel] >= kth - 2 * tol[b])
        v = code[b, sel].astype(np.float32) * scale[b, sel]
        assert np.array_equal(rows[b][chosen[b] >= 0], v) and not rows[b][chosen[b] < 0].any()
