"""Refusals of the 8-bit indexer calls, before anything is launched: these run
without a GPU. (Addresses are never dereferenced.)"""
import ctypes

import numpy as np
import pytest

from tests import q8_ref as ref

FAKE = 1 << 20
MIS = FAKE + 4


@pytest.fixture(scope="module")
def sai():
    import sparse_attention_indexer_window_b200 as m
    return m


def test_cache_write_refusals(sai):
    f = sai.lib().sai_q8_cache_write

    def call(x=FAKE, ty=0, sb=512, sn=128, table=FAKE, B=2, n=4, D=128, group=128, code=0, np_=8, page=16, mp=4,
             cache=FAKE, scales=FAKE, start=None, n_new=None, err=None):
        return f(x, ty, sb, sn, start, n_new, table, B, n, D, group, code, np_, page, mp, cache, scales, err, None)

    assert call(x=None) == 1 and call(cache=None) == 1 and call(scales=None) == 1
    for kw in (dict(B=0), dict(n=0), dict(D=0), dict(D=160), dict(page=0), dict(mp=0), dict(np_=0),
               dict(mp=1 << 16, page=1 << 15), dict(table=None), dict(table=None, mp=1, np_=1), dict(sb=-1),
               dict(sn=-128), dict(B=1 << 16, n=1 << 15)):
        assert call(**kw) == 2, kw
    for kw in (dict(ty=3), dict(ty=-1), dict(code=2), dict(group=16), dict(group=96), dict(group=1024, D=1024)):
        assert call(**kw) == 3, kw
    for kw in (dict(x=FAKE + 1), dict(x=FAKE + 2, ty=2), dict(cache=MIS), dict(scales=FAKE + 2), dict(start=FAKE + 1),
               dict(n_new=FAKE + 2), dict(table=FAKE + 2), dict(err=FAKE + 1)):
        assert call(**kw) == 7, kw


def test_cache_read_refusals(sai):
    f = sai.lib().sai_q8_cache_read

    def call(cache=FAKE, scales=FAKE, idx=None, start=None, lens=None, table=FAKE, B=2, n=4, D=128, group=64, code=1,
             np_=8, page=16, mp=4, out=FAKE, ty=0):
        return f(cache, scales, idx, start, lens, table, B, n, D, group, code, np_, page, mp, out, ty, None, None)

    assert call(cache=None) == 1 and call(scales=None) == 1 and call(out=None) == 1
    assert call(idx=FAKE, start=FAKE) == 2 and call(n=0) == 2 and call(table=None) == 2
    assert call(ty=7) == 3 and call(code=-1) == 3 and call(group=8) == 3
    assert call(out=MIS) == 7 and call(cache=MIS) == 7 and call(lens=FAKE + 2) == 7 and call(idx=FAKE + 2) == 7


def test_scores_refusals(sai):
    f = sai.lib().sai_indexer_scores

    def call(q8=FAKE, qs=FAKE, w=FAKE, cache=FAKE, ks=FAKE, table=FAKE, q_start=None, k_len=None, doc=None, B=2, S=1,
             H=64, D=128, P=64, np_=8, page=16, mp=4, cr=4, out=FAKE):
        return f(q8, qs, w, cache, ks, table, q_start, k_len, doc, B, S, H, D, P, np_, page, mp, cr, out, None, None)

    for kw in (dict(q8=None), dict(qs=None), dict(w=None), dict(cache=None), dict(ks=None), dict(out=None)):
        assert call(**kw) == 1, kw
    for kw in (dict(B=0), dict(S=0), dict(H=0), dict(P=0), dict(cr=0), dict(P=65), dict(table=None),
               dict(B=1 << 12, S=1 << 13, H=64), dict(cr=1 << 26)):
        assert call(**kw) == 2, kw
    for kw in (dict(H=129), dict(D=96), dict(D=256), dict(page=24), dict(page=4, mp=16), dict(page=200, P=600)):
        assert call(**kw) == 3, kw
    for kw in (dict(q8=MIS), dict(cache=FAKE + 8), dict(ks=FAKE + 2), dict(out=FAKE + 1), dict(doc=FAKE + 2)):
        assert call(**kw) == 7, kw


def test_backward_refusals(sai):
    lib = sai.lib()
    f = lib.sai_indexer_scores_backward
    need = lib.sai_indexer_scores_backward_workspace_bytes(1, 64, 16, 64, 16)
    assert need > 0 and lib.sai_indexer_scores_backward_workspace_bytes(1, 64, 16, 48, 16) == 0

    def call(ds=FAKE, idx=FAKE, q8=FAKE, qs=FAKE, w=FAKE, k8=FAKE, ks=FAKE, B=1, S=64, H=16, D=64, P=16, K=8, cr=4,
             t0=0, dq=FAKE, dk=FAKE, dw=FAKE, ws=FAKE, nb=1 << 40):
        return f(ds, idx, q8, qs, w, k8, ks, None, B, S, H, D, P, K, cr, t0, dq, dk, dw, ws, nb, None, None)

    for kw in (dict(ds=None), dict(q8=None), dict(qs=None), dict(w=None), dict(k8=None), dict(ks=None), dict(dq=None),
               dict(dk=None), dict(dw=None)):
        assert call(**kw) == 1, kw
    for kw in (dict(K=0), dict(K=17), dict(idx=None), dict(t0=-1), dict(t0=(1 << 31) - 8), dict(cr=0), dict(P=0)):
        assert call(**kw) == 2, kw
    for kw in (dict(H=200), dict(D=80)):
        assert call(**kw) == 3, kw
    for kw in (dict(ws=None), dict(ws=MIS), dict(nb=need - 1)):
        assert call(**kw) == 6, kw
    for kw in (dict(ds=FAKE + 2), dict(q8=MIS), dict(dq=FAKE + 8), dict(dk=MIS), dict(dw=FAKE + 2)):
        assert call(**kw) == 7, kw


def test_binding_refusals(sai):
    import torch
    x = torch.zeros(2, 4, 64)
    with pytest.raises(ValueError):
        sai.q8_quantize(x)                                        # a CPU tensor
    with pytest.raises(ValueError):
        sai.q8_quantize(x, group=48)
    with pytest.raises(TypeError):
        sai.q8_quantize(x, fmt=torch.uint8)
    with pytest.raises(ValueError):
        sai.q8_quantize(torch.zeros(0, 64))
    with pytest.raises(TypeError):
        sai.q8_cache_write(x.double(), torch.zeros(2, 4, 64, dtype=torch.int8), torch.zeros(2, 4, 1))
    with pytest.raises(ValueError):
        sai.q8_cache_write(x[0], torch.zeros(2, 4, 64, dtype=torch.int8), torch.zeros(2, 4, 1))
    c, s = torch.zeros(2, 4, 64, dtype=torch.int8), torch.zeros(2, 4, 1)
    with pytest.raises(ValueError):
        sai.q8_cache_read(c, s, idx=torch.zeros(2, 3, dtype=torch.int32), start=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        sai.q8_cache_read(c, torch.zeros(2, 4, 5))
    with pytest.raises(TypeError):
        sai.q8_cache_read(c.to(torch.uint8), s)
    with pytest.raises(TypeError):
        sai.q8_cache_read(c, s, dtype=torch.float64)
    q8, qs, w = torch.zeros(2, 3, 4, 64, dtype=torch.int8), torch.zeros(2, 3, 4), torch.zeros(2, 3, 4)
    with pytest.raises(ValueError):
        sai.indexer_scores(q8[0], qs, w, c, s, 4)
    with pytest.raises(ValueError):
        sai.indexer_scores(q8, qs, w, c, s, 4)                    # CPU tensors
    with pytest.raises(ValueError):
        sai.indexer_scores_backward(torch.zeros(2, 3, 4), None, q8, qs, w, c, s, 4)


def test_reference_e4m3_grid():
    """The test's own e4m3 table against torch's type."""
    import torch
    v = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy().astype(np.float64)
    assert np.array_equal(v, ref.e4m3_values())
    z = np.linspace(-440, 440, 4001)
    assert np.array_equal(ref.e4m3_round(z), torch.from_numpy(z).float().to(torch.float8_e4m3fn).double().numpy())


@pytest.mark.parametrize("n", [0, 1, 127, 128, 255, 16383])
def test_lengths_next_to_the_last_number_of_31_bits(sai, n):
    """A key, row or block number may not run past 31 bits, in the last tile or in the plan."""
    big, lib = (1 << 31) - 1 - n, sai.lib()
    sizes = ((1, 1, 1, 32, big), (1, big, 1, 32, 4), (2, 1, 1, 32, big // 2), (2, big // 2, 1, 32, 4))
    for B, S, H, D, P in sizes:
        assert lib.sai_indexer_scores(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, None, None, B, S, H, D, P, 1, P, 1, 1,
                                      FAKE, None, None) == 2, (B, S, H, D, P)
        assert lib.sai_indexer_scores_backward_workspace_bytes(B, S, H, D, P) == 0, (B, S, H, D, P)
        assert lib.sai_indexer_scores_backward(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, B, S, H, D, P, 1, 1, 0,
                                               FAKE, FAKE, FAKE, FAKE, 1 << 60, None, None) == 2, (B, S, H, D, P)
    # tokens and key blocks together
    assert lib.sai_indexer_scores_backward(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, 1 << 10, (1 << 21) - 64, 1,
                                           128, 1 << 20, 1, 1, 0, FAKE, FAKE, FAKE, FAKE, 1 << 60, None, None) == 2


def test_import_without_cuda_in_torch():
    """A torch built without CUDA has no binding of streams and devices: the
    package imports there, and refuses on the host as before."""
    import os
    import subprocess
    import sys
    code = ("import torch\n"
            "for n in ('_cuda_getCurrentRawStream', '_cuda_getDevice'):\n"
            "    if hasattr(torch._C, n): delattr(torch._C, n)\n"
            "import sparse_attention_indexer_window_b200 as m\n"
            "assert m.lib().sai_indexer_scores(*[None] * 9, *[1] * 9, *[None] * 3) == 1\n"
            "assert m.version() > 0\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
