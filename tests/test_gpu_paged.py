"""The paged cache on the GPU: decoding over pages, writing into them, and
reserve, fork, trim and compact, against plain implementations."""
import numpy as np
import pytest
import torch

import paged_ref as R
from exact_attention_04_gb300 import build as fabuild
from exact_attention_04_gb300 import fa, paged

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fabuild.build()
    fa.load()


def pools(layers, pages, h_kv, page, d, seed, layout="hnd", fill=None):
    """Two pools [layers, pages, h_kv, page, d] (views where the layout is not
    the contiguous one), random, or filled with a value."""
    g = torch.Generator().manual_seed(seed)
    shape = {"hnd": (layers, pages, h_kv, page, d), "nhd": (layers, pages, page, h_kv, d),
             "padded": (layers, pages, h_kv, page, d + 8)}[layout]
    out = []
    for _ in range(2):
        t = torch.randn(shape, generator=g).to(torch.bfloat16).cuda() if fill is None else \
            torch.full(shape, fill, dtype=torch.bfloat16, device="cuda")
        out.append(t.transpose(2, 3) if layout == "nhd" else t[..., :d])
    return out


def cuda(*arrays):
    return [torch.as_tensor(np.asarray(a, dtype=np.int32)).cuda() for a in arrays]


DECODE = [
    # H, h_kv, d, page, layout, lens, window, sinks
    (1, 1, 64, 1, "hnd", [1, 0, 2, 33], None, 0),
    (8, 2, 128, 16, "hnd", [1000, 1, 63, 64, 65, 0, 129], None, 0),
    (32, 8, 128, 64, "nhd", [777, 4096, 12], None, 0),
    (4, 4, 256, 48, "hnd", [500, 47, 48, 49], None, 0),
    (7, 1, 64, 16, "padded", [300, 16], None, 0),          # seven heads a group
    (40, 2, 128, 32, "hnd", [515, 90], None, 0),           # more than 16 heads a group
    (33, 1, 128, 16, "hnd", [700, 1, 64], None, 0),        # a second pass for one head
    (64, 1, 64, 24, "nhd", [3000, 129, 0], (500, 0), 7),   # 64 heads share one K/V head
    (34, 2, 256, 16, "hnd", [200, 65], None, 0),           # a pass a 16 heads
    (64, 1, 256, 100, "nhd", [1203, 100, 101], None, 0),
    (8, 8, 64, 16, "nhd", [2000, 100, 71, 70, 69], (69, 0), 4),
    (6, 3, 128, 24, "hnd", [1500, 64, 200, 1], (100, 0), 130),
    (4, 2, 256, 16, "padded", [900, 5], (0, 0), 0),        # the token itself alone
    (4, 2, 128, 16, "hnd", [900, 5], (0, 0), 1),
    (2, 1, 128, 8, "hnd", [20000, 3], (1 << 31 - 1, -1), 9),
]


@pytest.mark.parametrize("H,h_kv,d,page,layout,lens,window,sinks", DECODE)
def test_decode(H, h_kv, d, page, layout, lens, window, sinks):
    rng = np.random.default_rng(len(lens) * d + page)
    most = max(1, -(-max(lens) // page))
    pages = sum(-(-n // page) for n in lens) + 3
    table, kv_len, _ = cuda(*R.random_cache(rng, len(lens), most, page, pages, lens))
    k, v = pools(2, pages, h_kv, page, d, d + page, layout)
    q = torch.randn(len(lens), H, 1, d, generator=torch.Generator().manual_seed(3))
    q = q.to(torch.bfloat16).cuda()
    cache = paged.PagedKV(k, v)
    for layer in (0, 1):
        o, lse = paged.decode(q, cache, layer, table, kv_len, window=window, sinks=sinks)
        fa.fa_check()
        r = R.decode(q, k, v, layer, table, kv_len, None, window, sinks)
        R.check(r, "o", o)
        R.check(r, "lse", lse)


@pytest.mark.parametrize("d,layout", [(64, "nhd"), (128, "hnd"), (256, "hnd")])
def test_decode_reads_only_what_is_visible(d, layout):
    """Everything but the visible slots holds NaN or infinities: free pages,
    slots behind a row's end, tokens outside the window, missing pages."""
    rng = np.random.default_rng(d)
    page, lens, window, sinks = 16, [700, 31, 17, 200], (120, 0), 5
    most, pages = 60, 140
    table, kv_len, ref = R.random_cache(rng, 4, most, page, pages, lens, missing=0.2)
    clean = pools(1, pages, 2, page, d, 1, layout)
    dirty = [t.clone() for t in pools(1, pages, 2, page, d, 1, layout, float("nan"))]
    dirty[1].fill_(float("inf"))
    for r, n in enumerate(lens):
        for x in range(n):
            if (x >= n - 1 - window[0] or x < sinks) and table[r, x // page] >= 0:
                for a, b in zip(dirty, clean):
                    a[0, table[r, x // page], :, x % page] = b[0, table[r, x // page], :, x % page]
    table, kv_len = cuda(table, kv_len)
    table[0, 59] = 1 << 30                     # past the row, and no page
    table[1, 0] = -7
    q = torch.randn(4, 6, 1, d, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    o, lse = paged.decode(q, paged.PagedKV(*dirty), 0, table, kv_len, window=window, sinks=sinks)
    fa.fa_check()
    r = R.decode(q, *clean, 0, table, kv_len, None, window, sinks)
    R.check(r, "o", o)
    R.check(r, "lse", lse)


def test_decode_rows_without_a_key():
    """Empty rows, negative lengths, rows whose pages are all missing: O = 0,
    LSE = -inf, beside a long row that is split."""
    k, v = pools(1, 80, 1, 16, 128, 4)
    table = torch.full((5, 70), -1, dtype=torch.int32, device="cuda")
    table[2] = torch.arange(70, device="cuda")
    kv_len = torch.tensor([0, -5, 1100, 1100, 1 << 30], dtype=torch.int32, device="cuda")
    q = torch.randn(5, 4, 1, 128, device="cuda").to(torch.bfloat16)
    o, lse = paged.decode(q, paged.PagedKV(k, v), 0, table, kv_len)
    r = R.decode(q, k, v, 0, table, kv_len.cpu())
    R.check(r, "o", o)
    R.check(r, "lse", lse)
    for b in (0, 1, 3, 4):
        assert not o[b].any() and torch.isneginf(lse[b]).all()


def test_decode_many_rows_and_large_scores():
    """More rows than threads of a block, and scores of a standard deviation
    of 30 (the running maximum moves often)."""
    rng = np.random.default_rng(0)
    lens = rng.integers(0, 90, 700)
    most, page = 6, 16
    pages = int(sum(-(-n // page) for n in lens)) + 1
    table, kv_len, _ = cuda(*R.random_cache(rng, 700, most, page, pages, lens))
    k, v = pools(1, pages, 1, page, 64, 6)
    k *= 30
    q = torch.randn(700, 2, 1, 64, generator=torch.Generator().manual_seed(4))
    q = q.to(torch.bfloat16).cuda()
    o, lse = paged.decode(q, paged.PagedKV(k, v), 0, table, kv_len)
    r = R.decode(q, k, v, 0, table, kv_len)
    # scores up to 30 times the bound's: fp32 errors of the weights as well
    r["o_bound"] = r["o_bound"] + 30 * R.F32 * 4.5
    R.check(r, "o", o)
    assert ((R.f64(lse) - r["lse"]).abs()[torch.isfinite(r["lse"])] <= 3e-3).all()


def test_decode_is_a_contiguous_cache_s_and_repeats():
    """A contiguous cache as a pool of one page a row gives fa_decode's result
    (both within the bounds), repeats bit for bit, and ignores the workspace."""
    B, H, h_kv, N, d = 3, 8, 2, 3000, 128
    g = torch.Generator().manual_seed(8)
    k, v = (torch.randn(B, h_kv, N, d, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    q = torch.randn(B, H, 1, d, generator=g).to(torch.bfloat16).cuda()
    kv_len = torch.tensor([3000, 1, 1777], dtype=torch.int32, device="cuda")
    cache = paged.PagedKV(k, v)
    table = torch.arange(B, dtype=torch.int32, device="cuda")[:, None].contiguous()
    r = R.decode(q, k[None], v[None], 0, table, kv_len)
    ws = paged.decode_workspace(cache, H)
    first = None
    for fill in (0, 255):
        ws.fill_(fill)
        o, lse = paged.decode(q, cache, 0, table, kv_len, ws=ws)
        R.check(r, "o", o)
        R.check(r, "lse", lse)
        first = first or (o, lse)
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])
    o2, lse2 = fa.decode(q, k, v, causal=True, kv_len=kv_len)
    R.check(r, "o", o2)
    R.check(r, "lse", lse2)


@pytest.mark.parametrize("H,h_kv,d,width", [
    (8, 2, 128, 30), (8, 2, 128, 4000), (40, 2, 64, 30), (40, 2, 64, 4000),
    (4, 4, 256, 30), (4, 4, 256, 4000), (20, 1, 128, 250), (3, 1, 64, 4000)])
def test_decode_of_few_tiles(H, h_kv, d, width):
    """The same rows through a narrow and a wide table: the forms for few and
    for many tiles a row, a row's parts joined in both."""
    page = 16
    lens = [min(width * page, n) for n in (4000, 1, 0, 470, 64)]
    pages = sum(-(-n // page) for n in lens) + 3
    table, kv_len, ref = R.random_cache(np.random.default_rng(d), 5, width, page, pages, lens)
    table[3, 2] = -1                                     # a page that is not there
    k, v = pools(1, pages, h_kv, page, d, 7)
    table, kv_len = cuda(table, kv_len)
    q = torch.randn(5, H, 1, d, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16)
    q = q.cuda()
    for rows in (5, 1):
        for window, sinks in ((None, 0), ((100, 0), 3)):
            args = (table[:rows].contiguous(), kv_len[:rows].contiguous())
            o, lse = paged.decode(q[:rows].contiguous(), paged.PagedKV(k, v), 0, *args,
                                  window=window, sinks=sinks)
            r = R.decode(q[:rows], k, v, 0, *args, None, window, sinks)
            R.check(r, "o", o)
            R.check(r, "lse", lse)


def test_decode_pool_larger_than_2_31_elements():
    """Offsets past 2^31 elements: the last pages of a 5 GB pool."""
    pages, h_kv, page, d = 10300, 8, 256, 128
    k = torch.zeros(pages, h_kv, page, d, dtype=torch.bfloat16, device="cuda")
    assert k.numel() > 1 << 31
    k[-3:] = torch.randn(3, h_kv, page, d, device="cuda").to(torch.bfloat16)
    cache = paged.PagedKV(k, k)
    table = torch.tensor([[pages - 1, pages - 3, pages - 2]], dtype=torch.int32, device="cuda")
    kv_len = torch.tensor([600], dtype=torch.int32, device="cuda")
    q = torch.randn(1, 16, 1, d, device="cuda").to(torch.bfloat16)
    o, lse = paged.decode(q, cache, 0, table, kv_len)
    small = k[-3:].clone()[None]
    r = R.decode(q, small, small, 0, torch.tensor([[2, 0, 1]]), kv_len)
    R.check(r, "o", o)
    R.check(r, "lse", lse)
    new = torch.randn(1, h_kv, 5, d, device="cuda").to(torch.bfloat16)
    start = torch.tensor([700], dtype=torch.int32, device="cuda")
    paged.append(new, new, cache, 0, table, start, start + 5)
    assert torch.equal(k[pages - 2, :, 188:193], new[0])


@pytest.mark.parametrize("d,page,layout", [(64, 16, "hnd"), (128, 7, "nhd"), (256, 32, "padded")])
def test_reserve_and_append(d, page, layout):
    rng = np.random.default_rng(d)
    rows, h_kv, n, most = 9, 3, 50, 12
    lens = rng.integers(0, 40, rows)
    pages = 110
    table, kv_len, ref = R.random_cache(rng, rows, most, page, pages, lens)
    want = R.Cache(table, kv_len, ref, page)
    n_new = rng.integers(-2, n + 1, rows)
    n_new[0] = 10 ** 9                                   # up to the table's end
    info = want.reserve(n_new)
    k, v = pools(2, pages, h_kv, page, d, 1, layout)
    before = [k.clone(), v.clone()]
    cache = paged.PagedKV(k, v)
    table, kv_len, ref, n_new = cuda(table, kv_len, ref, n_new)
    new_len, new_ref, got = paged.reserve(cache, table, kv_len, ref, n_new)
    assert table.tolist() == want.table and new_len.tolist() == want.len
    assert new_ref.tolist() == want.ref and got.tolist() == info
    x = [torch.randn(rows, h_kv, n, d, device="cuda").to(torch.bfloat16) for _ in range(2)]
    paged.append(*x, cache, 1, table, kv_len, new_len)
    for pool, new, old in zip((k, v), x, before):
        for r in range(rows):
            for t in range(n):
                pos = int(kv_len[r]) + t
                if pos < want.len[r]:
                    old[1, want.table[r][pos // page], :, pos % page] = new[r, :, t]
        assert torch.equal(pool, old)
    # in place
    len2, ref2 = kv_len.clone(), ref.clone()
    info2 = torch.empty(2, dtype=torch.int32, device="cuda")
    ws = paged.workspace(cache, rows)
    st = fa.load().fa_pages_reserve(table.data_ptr(), most, page, len2.data_ptr(),
                                    n_new.data_ptr(), ref2.data_ptr(), pages, rows,
                                    len2.data_ptr(), ref2.data_ptr(), info2.data_ptr(),
                                    ws.data_ptr(), ws.numel(), None)
    assert st == fa.FA_OK
    torch.cuda.synchronize()
    assert torch.equal(len2, new_len) and torch.equal(ref2, new_ref) and torch.equal(info2, got)


@pytest.mark.parametrize("pages_left", [0, 1, 5])
def test_reserve_without_enough_pages(pages_left):
    page, rows, most = 4, 5, 8
    lens = np.array([3, 8, 0, 5, 32])
    pages = sum(-(-n // page) for n in lens) + pages_left
    rng = np.random.default_rng(pages_left)
    table, kv_len, ref = R.random_cache(rng, rows, most, page, pages, lens)
    want = R.Cache(table, kv_len, ref, page)
    n_new = np.array([1, 6, 9, 3, 4])
    info = want.reserve(n_new)
    assert info[1] == max(0, 5 - pages_left)          # five are asked for
    cache = paged.PagedKV(*pools(1, pages, 1, page, 64, 0))
    table, kv_len, ref, n_new = cuda(table, kv_len, ref, n_new)
    new_len, new_ref, got = paged.reserve(cache, table, kv_len, ref, n_new)
    assert table.tolist() == want.table and new_len.tolist() == want.len
    assert new_ref.tolist() == want.ref and got.tolist() == info


def test_append_leaves_the_rest():
    """Negative positions, positions past the table and rows without pages are
    not written."""
    k, v = pools(1, 6, 2, 8, 64, 0)
    old = k.clone()
    cache = paged.PagedKV(k, v)
    table = torch.tensor([[3, -1], [9, 1], [5, 2]], dtype=torch.int32, device="cuda")
    start = torch.tensor([4, 6, -3], dtype=torch.int32, device="cuda")
    end = torch.tensor([30, 1 << 30, 2], dtype=torch.int32, device="cuda")
    x = torch.randn(3, 2, 20, 64, device="cuda").to(torch.bfloat16)
    paged.append(x, x, cache, 0, table, start, end)
    old[0, 3, :, 4:8] = x[0, :, :4]
    old[0, 1] = x[1, :, 2:10]
    old[0, 5, :, :2] = x[2, :, 3:5]
    assert torch.equal(k, old)


FORK = [
    # rows, new rows, page, d, layout, spare pages, share, missing
    (1, 1, 4, 64, "hnd", 3, 0.0, 0.0),
    (6, 6, 8, 128, "nhd", 9, 0.5, 0.0),
    (5, 17, 16, 64, "padded", 30, 0.3, 0.1),
    (40, 23, 5, 256, "hnd", 20, 0.5, 0.1),
    (8, 30, 100, 128, "hnd", 4, 0.0, 0.0),         # the free pages run out
    (3, 8, 7, 64, "hnd", 0, 0.0, 0.3),
]


@pytest.mark.parametrize("rows,new_rows,page,d,layout,spare,share,missing", FORK)
def test_fork(rows, new_rows, page, d, layout, spare, share, missing):
    rng = np.random.default_rng(rows * 100 + new_rows)
    most = 9
    lens = rng.integers(0, most * page + 1, rows)
    pages = sum(-(-int(n) // page) for n in lens) + spare
    table, kv_len, ref = R.random_cache(rng, rows, most, page, pages, lens, share, missing)
    if spare > 4:
        ref[rng.integers(0, pages, 3)] += 1              # references of the caller's own
    parent = rng.integers(-1, rows, new_rows)
    parent[-1] = rows + 5 if new_rows > 3 else 0         # no row
    want = R.Cache(table, kv_len, ref, page)
    k, v = pools(2, pages, 2, page, d, 1, layout)
    expect = [k.clone(), v.clone()]
    info, copies = want.fork([p if p < rows else -1 for p in parent])
    for pool in expect:
        for s, x, n in copies:
            pool[:, x, :, :n] = pool[:, s, :, :n]
    cache = paged.PagedKV(k, v)
    ins = cuda(table, kv_len, ref, parent)
    kept = [t.clone() for t in ins]
    for _ in range(2):                                   # the inputs stay: it can run again
        t2, l2, r2, got = paged.fork(cache, *ins)
        assert t2.tolist() == want.table and l2.tolist() == want.len
        assert r2.tolist() == want.ref and got.tolist() == info
        assert torch.equal(k, expect[0]) and torch.equal(v, expect[1])
    assert all(torch.equal(a, b) for a, b in zip(ins, kept))


def test_fork_of_many_rows_over_a_large_pool():
    """More rows and pages than the cluster has threads."""
    rng = np.random.default_rng(5)
    rows, new_rows, page, most, pages = 9000, 12000, 2, 3, 30000
    lens = rng.integers(0, 6, rows)
    table, kv_len, ref = R.random_cache(rng, rows, most, page, pages, lens)
    parent = rng.integers(-1, rows, new_rows)
    want = R.Cache(table, kv_len, ref, page)
    k, v = pools(1, pages, 1, page, 64, 1)
    expect = k.clone()
    info, copies = want.fork(parent)
    src, dst = (torch.tensor([c[i] for c in copies]) for i in (0, 1))
    expect[0, dst, :, 0] = expect[0, src, :, 0]          # a partly filled page has one slot
    t2, l2, r2, got = paged.fork(paged.PagedKV(k, v), *cuda(table, kv_len, ref, parent))
    assert t2.tolist() == want.table and l2.tolist() == want.len
    assert r2.tolist() == want.ref and got.tolist() == info
    assert torch.equal(k, expect)


@pytest.mark.parametrize("page,d,layout,left,sinks", [
    (8, 64, "hnd", 20, 3), (16, 128, "nhd", 0, 0), (5, 256, "padded", 7, 11),
    (32, 64, "hnd", 10 ** 9, 4)])
def test_trim_and_compact(page, d, layout, left, sinks):
    rng = np.random.default_rng(page)
    rows, most = 7, 12
    lens = rng.integers(0, most * page + 1, rows)
    lens[1] = 0
    pages = sum(-(-int(n) // page) for n in lens) + 15
    table, kv_len, ref = R.random_cache(rng, rows, most, page, pages, lens, 0.4, 0.1)
    table[2, 0] = pages + 3                              # no page
    ref = np.bincount(table[(table >= 0) & (table < pages)], minlength=pages)
    want = R.Cache(table, kv_len, ref, page)
    k, v = pools(2, pages, 2, page, d, 1, layout)
    expect = [k.clone(), v.clone()]
    cache = paged.PagedKV(k, v)
    table, kv_len, ref = cuda(table, kv_len, ref)
    want.trim(left, sinks)
    t2, r2 = paged.trim(cache, table, kv_len, ref, left, sinks)
    assert t2.tolist() == want.table and r2.tolist() == want.ref
    st = fa.load().fa_pages_trim(table.data_ptr(), most, page, kv_len.data_ptr(), ref.data_ptr(),
                                 pages, rows, left, sinks, table.data_ptr(), ref.data_ptr(), None)
    torch.cuda.synchronize()
    assert st == fa.FA_OK and torch.equal(table, t2) and torch.equal(ref, r2)   # in place
    info, moves = want.compact()
    for pool in expect:
        for s, x in moves:
            pool[:, x] = pool[:, s]
    t3, r3, got = paged.compact(cache, t2, r2)
    assert t3.tolist() == want.table and r3.tolist() == want.ref and got.tolist() == info
    assert torch.equal(k, expect[0]) and torch.equal(v, expect[1])
    t4, r4, got = paged.compact(cache, t3, r3)           # nothing left to move
    assert torch.equal(t4, t3) and torch.equal(r4, r3) and got.tolist() == [info[0], 0]


def test_a_serving_run():
    """Prompts, decoding under a window with sinks, forking, trimming and
    compacting together: every step's attention is that of the row's whole
    history, kept beside the cache."""
    torch.manual_seed(0)
    layers, h_kv, H, d, page, window, sinks = 2, 2, 4, 64, 8, 40, 3
    k, v = pools(layers, 80, h_kv, page, d, 0, "nhd", float("nan"))
    cache = paged.PagedKV(k, v)
    table, kv_len, ref = cache.empty(3, 24)
    history = [[torch.zeros(2, h_kv, 0, d) for _ in range(layers)] for _ in range(3)]

    def step(n_new):
        nonlocal kv_len, ref
        n = torch.tensor(n_new, dtype=torch.int32, device="cuda")
        new_len, ref, info = paged.reserve(cache, table, kv_len, ref, n)
        assert int(info[1]) == 0
        for layer in range(layers):
            x = [torch.randn(len(n_new), h_kv, max(n_new), d).to(torch.bfloat16) for _ in range(2)]
            paged.append(x[0].cuda(), x[1].cuda(), cache, layer, table, kv_len, new_len)
            q = torch.randn(len(n_new), H, 1, d).to(torch.bfloat16)
            o, lse = paged.decode(q.cuda(), cache, layer, table, new_len, window=(window, 0),
                                  sinks=sinks)
            for r, c in enumerate(n_new):
                new = torch.stack([t[r, :, :c].float() for t in x])
                history[r][layer] = torch.cat([history[r][layer], new], 2)
                full = history[r][layer].to(torch.bfloat16)
                one = torch.zeros(1, 1, dtype=torch.int32)
                ref64 = R.decode(q[r:r + 1], full[0][None, None], full[1][None, None], 0, one,
                                 [full.shape[2]], None, (window, 0), sinks)
                R.check(ref64, "o", o[r:r + 1])
                R.check(ref64, "lse", lse[r:r + 1])
        kv_len = new_len

    step([50, 9, 1])
    for i in range(4):
        step([1, 1, 1])
        table, ref = paged.trim(cache, table, kv_len, ref, window, sinks)
    table, kv_len, ref, info = paged.fork(cache, table, kv_len, ref, *cuda([0, 0, 1, 2, 1]))
    assert int(info[1]) == 0
    history = [[t.clone() for t in history[p]] for p in (0, 0, 1, 2, 1)]
    step([1, 2, 1, 7, 1])
    table, ref, info = paged.compact(cache, table, ref)
    step([1, 1, 30, 1, 1])
    table, kv_len, ref, info = paged.fork(cache, table, kv_len, ref, *cuda([4, -1, 2]))
    history = [history[4], [torch.zeros(2, h_kv, 0, d) for _ in range(layers)], history[2]]
    step([3, 12, 1])
    table, ref, info = paged.compact(cache, table, ref)
    used = {int(x) for x in table.reshape(-1) if x >= 0}
    assert used == set(range(int(info[0])))
    fa.fa_check()


def test_a_captured_decode_step():
    """reserve, append and decode captured once and replayed as the cache
    grows; another graph with a workspace of its own on another stream."""
    torch.manual_seed(1)
    k, v = pools(1, 40, 2, 4, 128, 0)
    cache = paged.PagedKV(k, v)
    table, kv_len, ref = cache.empty(2, 16)
    one = torch.ones(2, dtype=torch.int32, device="cuda")
    q, kn, vn = (torch.zeros(2, h, 1, 128, dtype=torch.bfloat16, device="cuda") for h in (8, 2, 2))

    def step():
        new_len, new_ref, info = paged.reserve(cache, table, kv_len, ref, one)
        paged.append(kn, vn, cache, 0, table, kv_len, new_len)
        o, lse = paged.decode(q, cache, 0, table, new_len)
        kv_len.copy_(new_len)
        ref.copy_(new_ref)
        return o, lse
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    table.fill_(-1)
    kv_len.zero_()
    ref.zero_()
    graph, graph2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = step()
    with torch.cuda.graph(graph2):
        o2, lse2 = paged.decode(q, cache, 0, table, kv_len)
    ks, vs = torch.zeros(2, 2, 0, 128), torch.zeros(2, 2, 0, 128)
    for i in range(20):
        x = [torch.randn(t.shape).to(torch.bfloat16) for t in (q, kn, vn)]
        for t, y in zip((q, kn, vn), x):
            t.copy_(y)
        graph.replay()
        ks, vs = torch.cat([ks, x[1].float()], 2), torch.cat([vs, x[2].float()], 2)
        r = R.decode(x[0], ks[None].to(torch.bfloat16), vs[None].to(torch.bfloat16), 0,
                     torch.arange(2)[:, None], [i + 1, i + 1])
        R.check(r, "o", o)
        R.check(r, "lse", lse)
        with torch.cuda.stream(s):
            s.wait_stream(torch.cuda.default_stream())
            graph2.replay()
        s.synchronize()
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_calls_on_a_given_stream():
    """stream= runs there, outputs included, while the current stream is busy
    elsewhere."""
    k, v = pools(1, 30, 1, 16, 64, 2)
    cache = paged.PagedKV(k, v)
    rng = np.random.default_rng(1)
    table, kv_len, ref, parent = cuda(*R.random_cache(rng, 3, 6, 16, 30, [90, 7, 33]), [2, 2, 0, 1])
    q = torch.randn(3, 4, 1, 64, device="cuda").to(torch.bfloat16)
    torch.cuda.synchronize()
    here = paged.decode(q, cache, 0, table, kv_len), paged.fork(cache, table, kv_len, ref, parent)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    there = (paged.decode(q, cache, 0, table, kv_len, stream=s),
             paged.fork(cache, table, kv_len, ref, parent, stream=s))
    s.synchronize()
    for a, b in zip(here, there):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("rows,most,page", [(5, 9, 4), (700, 24, 3)])
def test_metadata_in_place(rows, most, page):
    """reserve, trim and compact with the outputs that may be the inputs."""
    rng = np.random.default_rng(rows)
    lens = rng.integers(0, (most - 3) * page, rows)
    pages = rows * most
    table, kv_len, ref = R.random_cache(rng, rows, most, page, pages, lens, 0.3)
    n_new = rng.integers(0, 3 * page, rows)
    k, v = pools(1, pages, 1, page, 64, 3)
    cache = paged.PagedKV(k, v)
    table, kv_len, ref, n_new = cuda(table, kv_len, ref, n_new)
    ws, info = paged.workspace(cache, rows), torch.zeros(2, dtype=torch.int32, device="cuda")
    lib = fa.load()

    def ptr(*tensors):
        return [t.data_ptr() for t in tensors]
    t1 = table.clone()
    want = paged.reserve(cache, t1, kv_len, ref, n_new)
    assert lib.fa_pages_reserve(*ptr(table), most, page, *ptr(kv_len, n_new, ref), pages, rows,
                                *ptr(kv_len, ref, info, ws), ws.numel(), None) == fa.FA_OK
    assert all(torch.equal(a, b) for a, b in zip((table, kv_len, ref, info), (t1, *want)))
    want = paged.trim(cache, table, kv_len, ref, 2 * page, 1)
    assert lib.fa_pages_trim(*ptr(table), most, page, *ptr(kv_len, ref), pages, rows, 2 * page, 1,
                             *ptr(table, ref), None) == fa.FA_OK
    assert torch.equal(table, want[0]) and torch.equal(ref, want[1])
    k2, v2 = k.clone(), v.clone()
    want = paged.compact(paged.PagedKV(k2, v2), table, ref)
    assert lib.fa_pages_compact(cache.ref, *ptr(table), most, *ptr(ref), rows,
                                *ptr(table, ref, info, ws), ws.numel(), None) == fa.FA_OK
    assert all(torch.equal(a, b) for a, b in zip((table, ref, info), want))
    assert torch.equal(k, k2) and torch.equal(v, v2)


def test_captured_maintenance():
    """fork, trim and compact captured once and replayed over other contents."""
    rows, most, page, pages = 6, 10, 8, 90
    k, v = pools(2, pages, 2, page, 64, 4)
    cache = paged.PagedKV(k, v)
    table, kv_len, ref = cache.empty(rows, most)
    parent = torch.zeros(rows, dtype=torch.int32, device="cuda")

    def step(c):
        t, n, r, info = paged.fork(c, table, kv_len, ref, parent)
        t, r = paged.trim(c, t, n, r, 19, 2)
        return (n, info) + paged.compact(c, t, r)
    step(cache)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(cache)
    for seed in range(5):
        rng = np.random.default_rng(seed)
        lens = rng.integers(0, most * page + 1, rows)
        for t, x in zip((table, kv_len, ref),
                        R.random_cache(rng, rows, most, page, pages, lens, 0.3)):
            t.copy_(torch.as_tensor(x))
        parent.copy_(torch.as_tensor(rng.integers(-1, rows, rows).astype(np.int32)))
        x = torch.randn(k.shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)
        k.copy_(x)
        v.copy_(-x)
        k2, v2 = k.clone(), v.clone()
        want = step(paged.PagedKV(k2, v2))
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert torch.equal(k, k2) and torch.equal(v, v2)


def test_two_calls_at_once():
    """Decoding two caches on two streams, each call with a workspace of its
    own, gives what it gives alone."""
    args = []
    for seed, (H, d) in enumerate(((32, 128), (40, 64))):
        k, v = pools(1, 600, 1, 16, d, seed)
        table = torch.randperm(600, generator=torch.Generator().manual_seed(seed))
        table = table.to(torch.int32).cuda().view(6, 100)
        kv_len, = cuda([1600, 3, 0, 911, 1599, 64])
        q = torch.randn(6, H, 1, d, device="cuda").to(torch.bfloat16)
        args.append((q, paged.PagedKV(k, v), 0, table, kv_len))
    alone = [paged.decode(*a) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in args]
    both = [paged.decode(*a, stream=s) for _ in range(50) for a, s in zip(args, streams)]
    torch.cuda.synchronize()
    for i, (o, lse) in enumerate(both):
        assert torch.equal(o, alone[i % 2][0]) and torch.equal(lse, alone[i % 2][1])


def test_a_window_past_32_bits():
    """A window or sinks beyond every position are none, however large."""
    k, v = pools(1, 8, 1, 16, 64, 5)
    cache = paged.PagedKV(k, v)
    table, kv_len, ref = cuda([[3, 1, 2, 7]], [60], [0, 1, 1, 1, 0, 0, 0, 1])
    q = torch.randn(1, 2, 1, 64, device="cuda").to(torch.bfloat16)
    want = paged.decode(q, cache, 0, table, kv_len)
    for window, sinks in (((1 << 32, 0), 0), ((3, 0), 1 << 32), ((1 << 40, 0), 1 << 40)):
        got = paged.decode(q, cache, 0, table, kv_len, window=window, sinks=sinks)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for window, sinks in ((1 << 32, 0), (3, 1 << 32)):
        t2, r2 = paged.trim(cache, table, kv_len, ref, window, sinks)
        assert torch.equal(t2, table) and torch.equal(r2, ref)


@pytest.mark.parametrize("B,H,h_kv,d", [(64, 8, 8, 64), (40, 32, 8, 128)])
def test_decode_through_a_very_wide_table(B, H, h_kv, d):
    """A table that could list 2^29 tokens a row (2^31 tiles and more in all)
    while the rows are short: the lengths count, not the width."""
    page, most = 1 << 14, 1 << 15
    k, v = pools(1, 3, h_kv, page, d, 11)
    table = torch.full((B, most), -1, dtype=torch.int32, device="cuda")
    table[:, 0] = torch.arange(B, device="cuda") % 3
    table[1, :3] = torch.tensor([2, 0, 1])
    lens = [(37 * b) % 300 for b in range(B)]
    lens[1] = 2 * page + 77
    kv_len, = cuda(lens)
    q = torch.randn(B, H, 1, d, generator=torch.Generator().manual_seed(5))
    q = q.to(torch.bfloat16).cuda()
    cache = paged.PagedKV(k, v)
    for window, sinks in ((None, 0), ((20000, 0), 9)):
        o, lse = paged.decode(q, cache, 0, table, kv_len, window=window, sinks=sinks)
        fa.fa_check()
        r = R.decode(q, k, v, 0, table[:, :3], kv_len, None, window, sinks)
        R.check(r, "o", o)
        R.check(r, "lse", lse)


@pytest.mark.parametrize("window,sinks", [
    (((1 << 31) - 1, -1), 9), (((1 << 30) + 1, -1), 9), ((1 << 30, -1), 0),
    (((1 << 31) - 1, -1), (1 << 31) - 1)])
def test_decode_under_the_largest_windows(window, sinks):
    """Windows at and past every position, over rows whose parts are joined."""
    lens, page = [20000, 3], 8
    table, kv_len, _ = cuda(*R.random_cache(np.random.default_rng(1), 2, 2500, page, 2510, lens))
    k, v = pools(1, 2510, 1, page, 128, 9)
    cache = paged.PagedKV(k, v)
    assert fa.load().fa_decode_paged_call_bytes(cache.ref, 2500, 2, 2, window[0], sinks) > 0
    q = torch.randn(2, 2, 1, 128, generator=torch.Generator().manual_seed(3))
    q = q.to(torch.bfloat16).cuda()
    o, lse = paged.decode(q, cache, 0, table, kv_len, window=window, sinks=sinks)
    fa.fa_check()
    r = R.decode(q, k, v, 0, table, kv_len, None, window, sinks)
    R.check(r, "o", o)
    R.check(r, "lse", lse)


@pytest.mark.parametrize("rows,most,page,pages", [
    (50, 40, 3, 3000),        # several CTAs of the cluster, a page a thread at most
    (300, 60, 2, 20000),      # several pages a thread
    (3000, 4, 5, 12000),      # and rows in several CTAs
])
def test_metadata_of_large_pools(rows, most, page, pages):
    """reserve, trim and compact over pools that all CTAs of the cluster share,
    against the plain implementation, the moved pages' contents included."""
    rng = np.random.default_rng(pages)
    lens = rng.integers(0, (most - 1) * page + 1, rows)
    table, kv_len, ref = R.random_cache(rng, rows, most, page, pages, lens, 0.2, 0.05)
    want = R.Cache(table, kv_len, ref, page)
    k, v = pools(1, pages, 1, page, 64, 3)
    expect = [k.clone(), v.clone()]
    cache = paged.PagedKV(k, v)
    n_new = rng.integers(-1, page + 2, rows)
    table, kv_len, ref, n_new = cuda(table, kv_len, ref, n_new)
    kv_len, ref, got = paged.reserve(cache, table, kv_len, ref, n_new)
    assert got.tolist() == want.reserve(n_new.tolist())
    assert table.tolist() == want.table and kv_len.tolist() == want.len
    assert ref.tolist() == want.ref
    want.trim(page, 1)
    table, ref = paged.trim(cache, table, kv_len, ref, page, 1)
    assert table.tolist() == want.table and ref.tolist() == want.ref
    info, moves = want.compact()
    assert len(moves) > 50
    src, dst = (torch.tensor([m[i] for m in moves]) for i in (0, 1))
    for pool in expect:
        pool[:, dst] = pool[:, src]
    table, ref, got = paged.compact(cache, table, ref)
    assert table.tolist() == want.table and ref.tolist() == want.ref and got.tolist() == info
    assert torch.equal(k, expect[0]) and torch.equal(v, expect[1])


@pytest.mark.parametrize("spare", [0, 1, 900, 2500])
def test_reserve_of_many_rows_that_runs_out(spare):
    """More rows than one CTA has threads, the pages running out inside a later
    CTA's."""
    rng = np.random.default_rng(spare)
    rows, most, page = 5000, 3, 2
    lens = rng.integers(0, 4, rows)
    pages = int(sum(-(-n // page) for n in lens)) + spare
    table, kv_len, ref = R.random_cache(rng, rows, most, page, pages, lens)
    want = R.Cache(table, kv_len, ref, page)
    n_new = rng.integers(0, 4, rows)
    info = want.reserve(n_new)
    assert info[1] > 0
    cache = paged.PagedKV(*pools(1, pages, 1, page, 64, 0))
    table, kv_len, ref, n_new = cuda(table, kv_len, ref, n_new)
    new_len, new_ref, got = paged.reserve(cache, table, kv_len, ref, n_new)
    assert table.tolist() == want.table and new_len.tolist() == want.len
    assert new_ref.tolist() == want.ref and got.tolist() == info
