"""q8_cache_write / q8_cache_read / q8_quantize against the formula in 64 bits.

Codes and scales are equal to the formula's, and a value read back is equal to
code * scale rounded once: no tolerance is needed. The cases cover the element
types, both 8-bit formats, group and page sizes, strides, padded batches,
values on and next to the border between two codes, zero, subnormal, huge and
non-finite groups, entries outside the table, offsets past 32 bits, other
streams and captured graphs.
"""
import numpy as np
import pytest

from tests import q8_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def sai():
    import sparse_attention_indexer_window_b200 as m
    return m


def rows(seed, shape, dtype, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*shape, generator=g) * torch.exp(spread * torch.randn(*shape[:-1], 1, generator=g))
    return x.to(TYPES[dtype]).cuda()


def same(a, b):
    a, b = np.asarray(a, np.float64), np.asarray(b, np.float64)
    return a.shape == b.shape and np.array_equal(a, b, equal_nan=True)


def expect_read(code, scale, group, dtype):
    v = code.astype(np.float32) * np.repeat(scale, group, -1)
    return torch.from_numpy(v).to(TYPES[dtype]).double().numpy()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("D,group", [(32, 32), (192, 64), (128, 128), (512, 256), (1536, 512)])
def test_quantize_equals_the_formula(sai, fmt, dtype, D, group):
    x = rows(D + group, (3, 37, D), dtype)
    codes, scales = sai.q8_quantize(x, group=group, fmt=ref.FMT[fmt])
    rc, rs = ref.quantize(x, group, fmt)
    assert same(ref.code_values(codes), rc)
    assert same(scales.cpu().numpy(), rs)
    for out in ("bf16", "fp16", "fp32"):
        back = sai.q8_cache_read(codes, scales, dtype=TYPES[out])
        assert same(back.cpu().double().numpy(), expect_read(rc, rs, group, out))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_values_at_the_border_of_two_codes(sai, fmt, dtype):
    """Groups whose quotients are ties, or one unit in the last place off a tie."""
    lim = ref.LIMIT[fmt]
    grid = np.arange(128.0) if fmt == "int8" else ref.e4m3_values()
    ties = (grid[1:] + grid[:-1]) / 2
    x = []
    for amax in (lim, lim / 2, 3.0, 1.7, 0.3, 2.0 ** -100, lim * 2.0 ** 100 if dtype != "fp16" else 60000.0):
        t = torch.tensor(ties * amax / lim, dtype=torch.float64).to(TYPES[dtype])
        near = [t, torch.nextafter(t.float(), torch.tensor(0.0)).to(TYPES[dtype]),
                torch.nextafter(t.float(), torch.tensor(torch.inf)).to(TYPES[dtype]), -t]
        v = torch.cat(near)
        v = torch.cat([v, torch.zeros((-len(v)) % 31, dtype=v.dtype)]).view(-1, 31)
        a = torch.full((len(v), 1), amax, dtype=torch.float64).to(TYPES[dtype])
        x.append(torch.cat([v.clamp(-a, a), a], 1))
    x = torch.cat(x).cuda()
    codes, scales = sai.q8_quantize(x, fmt=ref.FMT[fmt])
    rc, rs = ref.quantize(x, 32, fmt)
    assert same(ref.code_values(codes), rc)
    assert same(scales.cpu().numpy(), rs)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_zero_subnormal_huge_and_non_finite_groups(sai, fmt, dtype):
    fi = torch.finfo(TYPES[dtype])
    x = torch.zeros(8, 64, dtype=TYPES[dtype])
    x[1] = torch.linspace(-1, 1, 64, dtype=torch.float64).mul(fi.max).to(x.dtype)
    x[2] = torch.linspace(-1, 1, 64, dtype=torch.float64).mul(fi.tiny).to(x.dtype)
    x[3, 5] = fi.tiny * fi.eps                         # the smallest subnormal alone
    x[4] = 1.0
    x[4, 40] = float("nan")                            # spoils the second group of 32 only
    x[5, 3] = float("inf")
    x[6, 63] = -float("inf")
    x[7] = -0.0
    x = x.cuda()
    codes, scales = sai.q8_quantize(x, group=32, fmt=ref.FMT[fmt])
    rc, rs = ref.quantize(x, 32, fmt)
    assert same(np.abs(ref.code_values(codes)), np.abs(rc))     # (the sign of a zero code is open)
    assert same(scales.cpu().numpy(), rs)
    assert torch.isnan(sai.q8_cache_read(codes[None], scales[None])[0, 4, 32:]).all()


@pytest.mark.parametrize("fmt,D,group,page,pages", [("int8", 128, 128, 64, 3), ("e4m3", 512, 128, 24, 5),
                                                    ("int8", 64, 32, 1, 90), ("e4m3", 32, 32, 100, 1)])
def test_paged_padded_batch(sai, fmt, D, group, page, pages):
    """Ragged new rows land in their entries, everything else stays as it was,
    and reads (by position and by index) see exactly that."""
    B, n, cap = 4, 60, page * pages
    g = torch.Generator().manual_seed(page)
    x = rows(page, (B, n, D), "bf16")
    start = torch.tensor([0, 17, cap - 60, 5], dtype=torch.int32)
    n_new = torch.tensor([60, 0, 60, 1], dtype=torch.int32)
    x[3, 1:] = float("nan")                            # padding is not read
    table = torch.randperm(B * pages + 3, generator=g)[:B * pages].int().view(B, pages)
    cache = torch.randint(0, 120, (B * pages + 3, page, D), generator=g, dtype=torch.int8)
    scales = torch.rand(B * pages + 3, page, D // group, generator=g)
    c, s = cache.cuda().view(ref.FMT[fmt]), scales.cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    sai.q8_cache_write(x, c, s, start=start.cuda(), n_new=n_new.cuda(), block_table=table.cuda(), err=err)
    want_c, want_s = ref.code_values(cache.view(ref.FMT[fmt])).copy(), scales.numpy().copy()
    rc, rs = ref.quantize(x, group, fmt)
    for b in range(B):
        for i in range(int(n_new[b])):
            pos = int(start[b]) + i
            want_c[int(table[b, pos // page]), pos % page] = rc[b, i]
            want_s[int(table[b, pos // page]), pos % page] = rs[b, i]
    assert same(ref.code_values(c), want_c)
    assert same(s.cpu().numpy(), want_s)

    lens = (start + n_new).clamp(max=cap)
    pos = torch.arange(cap)[None].expand(B, -1)
    live = pos < lens[:, None]
    slot = table.long().gather(1, pos // page), pos % page
    v = expect_read(want_c[slot], want_s[slot], group, "fp32")
    got = sai.q8_cache_read(c, s, lens=lens.cuda(), block_table=table.cuda(), dtype=torch.float32, err=err)
    assert same(got.cpu().numpy(), np.where(live.numpy()[..., None], v, 0.0))
    # by index, any order, the same entry twice, unused slots
    idx = torch.randint(0, cap, (B, 33), generator=g, dtype=torch.int32)
    idx[:, 7] = idx[:, 2]
    idx[:, 20:23] = -1
    got = sai.q8_cache_read(c, s, idx=idx.cuda(), lens=lens.cuda(), block_table=table.cuda(), dtype=torch.float32,
                            err=err)
    i = idx.long().clamp(min=0)
    keep = (idx >= 0) & (idx < lens[:, None])
    rows_ = np.take_along_axis(v, i.numpy()[..., None], 1)
    assert same(got.cpu().numpy(), np.where(keep.numpy()[..., None], rows_, 0.0))
    # from a start position
    first = torch.tensor([0, 3, cap - 9, 1], dtype=torch.int32)
    got = sai.q8_cache_read(c, s, n=9, start=first.cuda(), block_table=table.cuda(), dtype=torch.float32, err=err)
    i = (first.long()[:, None] + torch.arange(9)).numpy()[..., None]
    assert same(got.cpu().numpy(), np.take_along_axis(v, i, 1))
    torch.cuda.synchronize()
    assert int(err.item()) == 0


def test_entries_outside_the_cache_are_skipped_and_reported(sai):
    x = rows(1, (2, 4, 32), "fp32")
    table = torch.tensor([[0, 1], [-1, 7]], dtype=torch.int32, device="cuda")     # 2 pages exist
    for start, written in ((torch.tensor([6, 0]), [(0, 0, 1, 2), (0, 1, 1, 3)]),   # over the end; page -1
                           (torch.tensor([-2, 4]), [(0, 2, 0, 0), (0, 3, 0, 1)])):  # before the start; page 7
        cache = torch.zeros(2, 4, 32, dtype=torch.int8, device="cuda")
        scales = torch.zeros(2, 4, 1, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        sai.q8_cache_write(x, cache, scales, start=start.int().cuda(), block_table=table, err=err)
        rc, rs = ref.quantize(x, 32, "int8")
        want = np.zeros((2, 4, 32))
        for b, i, pg, off in written:
            want[pg, off] = rc[b, i]
        assert same(ref.code_values(cache), want)
        assert int(err.item()) == sai.SAI_ERR_INDEX
    cache.fill_(3)
    scales.fill_(1.0)
    idx = torch.tensor([[0, -2, 8, 7], [0, 4, -1, 1]], dtype=torch.int32, device="cuda")
    err.zero_()
    got = sai.q8_cache_read(cache, scales, idx=idx, block_table=table, dtype=torch.float32, err=err)
    assert same(got[:, :, 0].cpu().numpy(), [[3, 0, 0, 3], [0, 0, 0, 0]])
    assert int(err.item()) == sai.SAI_ERR_INDEX
    err.zero_()
    got = sai.q8_cache_read(cache, scales, idx=idx[:1, 2:], block_table=table[:1], dtype=torch.float32, err=err,
                            lens=torch.tensor([8], dtype=torch.int32, device="cuda"))
    assert same(got[:, :, 0].cpu().numpy(), [[0, 3]]) and int(err.item()) == 0    # behind the end: no error


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_strided_and_misaligned_rows(sai, dtype):
    base = rows(5, (6, 11, 3, 136), dtype)
    for x in (base[:, :, 1, :128], base[::2, 1::3, 2, 3:131], base[:, :, 0, 1:65], base[:1, :1, 0, 8:72].expand(4, 9, 64)):
        B, n, D = x.shape
        cache = torch.zeros(B, n + 2, D, dtype=torch.int8, device="cuda")
        scales = torch.zeros(B, n + 2, D // 32, device="cuda")
        sai.q8_cache_write(x, cache, scales, start=torch.full((B,), 2, dtype=torch.int32, device="cuda"))
        rc, rs = ref.quantize(x, 32, "int8")
        assert same(ref.code_values(cache[:, 2:]), rc) and same(scales[:, 2:].cpu().numpy(), rs)
        assert int(cache[:, :2].abs().max()) == 0
    q8, qs = sai.q8_quantize(base[..., :128][0])
    rc, rs = ref.quantize(base[..., :128][0], 128, "int8")
    assert same(ref.code_values(q8), rc) and same(qs.cpu().numpy(), rs)


def test_offsets_past_32_bits(sai):
    """The last pages of a cache of more than 2^32 bytes."""
    page, D = 4096, 512
    n_pages = (1 << 32) // (page * D) + 2
    cache = torch.empty(n_pages, page, D, dtype=torch.int8, device="cuda")
    scales = torch.empty(n_pages, page, 4, device="cuda")
    x = rows(9, (1, 50, D), "bf16")
    table = torch.tensor([[n_pages - 2, n_pages - 1]], dtype=torch.int32, device="cuda")
    start = torch.tensor([page - 25], dtype=torch.int32, device="cuda")
    sai.q8_cache_write(x, cache, scales, start=start, block_table=table)
    got = sai.q8_cache_read(cache, scales, n=50, start=start, block_table=table)
    rc, rs = ref.quantize(x, 128, "int8")
    assert same(got.cpu().double().numpy(), expect_read(rc, rs, 128, "bf16"))


def test_other_stream_and_captured_graph(sai):
    x = rows(11, (2, 300, 128), "bf16")
    cache = torch.zeros(2, 300, 128, dtype=torch.int8, device="cuda")
    scales = torch.zeros(2, 300, 1, device="cuda")
    out = torch.empty(2, 300, 128, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        sai.q8_cache_write(x, cache, scales)
        sai.q8_cache_read(cache, scales, out=out)
    torch.cuda.current_stream().wait_stream(side)
    want = out.clone()
    rc, rs = ref.quantize(x, 128, "int8")
    assert same(want.cpu().double().numpy(), expect_read(rc, rs, 128, "bf16"))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sai.q8_cache_write(x, cache, scales)
        sai.q8_cache_read(cache, scales, out=out)
    x.mul_(-2)
    for _ in range(2):
        cache.zero_()
        scales.zero_()
        out.zero_()
        g.replay()
        assert torch.equal(out, want * -2)
