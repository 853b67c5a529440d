"""Attention of a chunk of new tokens over the paged cache on the GPU, against
a plain implementation, and together with the cache's other calls."""
import ctypes

import numpy as np
import pytest
import torch

import paged_ref as R
import rope_ref as P
from exact_attention_04_gb300 import build as fabuild
from exact_attention_04_gb300 import fa, paged, rope
from test_gpu_paged import cuda, pools

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fabuild.build()
    fa.load()


def randn(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(
        torch.bfloat16).cuda()


def rows_of(have, new, page, seed=0, missing=0.0, extra=0):
    """(table, start, kv_len, pages): rows of have[r] + new[r] tokens (and
    `extra` more that no query is)."""
    rng = np.random.default_rng(seed)
    lens = np.add(have, new) + extra
    most = max(1, -(-int(max(lens)) // page)) + 1
    pages = int(sum(-(-int(n) // page) for n in lens)) + 3
    table, kv_len, _ = R.random_cache(rng, len(lens), most, page, pages, lens, missing=missing)
    return (*cuda(table, have, kv_len), pages)


def queries(B, H, N, d, how, seed=3):
    if how == "hnd":
        return randn(B, H, N, d, seed=seed)
    if how == "nhd":
        return randn(B, N, H, d, seed=seed).transpose(1, 2)
    return randn(B, N, H + 2, d + 8, seed=seed)[:, :, 2:, :d].transpose(1, 2)    # a slice


def check(r, o, lse, offsets=None):
    """Within the bounds wherever a row has a token."""
    end = o.shape[2] if offsets is None else int(offsets[-1])
    for name, got in (("o", o), ("lse", lse)):
        part = {k: x[:, :, :end] for k, x in r.items()}
        R.check(part, name, got[:, :, :end])


PREFILL = [
    # H, h_kv, d, page, layout, have, new, causal, window, sinks
    (1, 1, 64, 16, "hnd", [0], [1], True, None, 0),
    (2, 1, 64, 16, "hnd", [0, 5, 300, 0], [33, 1, 140, 0], True, None, 0),
    (8, 2, 128, 16, "nhd", [1000, 0, 63, 0], [5, 300, 64, 129], True, None, 0),
    (8, 8, 128, 64, "hnd", [200, 1], [257, 40], True, None, 0),
    (4, 2, 256, 32, "padded", [128, 17, 0], [129, 70, 3], True, None, 0),
    (7, 1, 64, 24, "hnd", [500, 3], [20, 90], True, None, 0),           # seven heads a group
    (12, 4, 128, 5, "hnd", [77, 0], [50, 131], True, None, 0),          # odd pages
    (4, 1, 128, 1, "nhd", [60, 200], [9, 70], True, None, 0),           # pages of one token
    (4, 4, 64, 3, "hnd", [100, 0], [64, 200], True, None, 0),
    (2, 2, 128, 100, "hnd", [250, 99], [101, 3], True, None, 0),
    (6, 2, 64, 128, "hnd", [1000, 127], [77, 2], True, None, 0),
    (6, 2, 128, 200, "nhd", [555, 0], [140, 260], True, None, 0),       # pages of two tiles
    (2, 1, 256, 129, "hnd", [300], [150], True, None, 0),
    (64, 1, 64, 16, "hnd", [150, 20], [3, 7], True, None, 0),
    (130, 1, 64, 16, "hnd", [70, 0], [3, 20], True, None, 0),           # a group of two tiles
    (150, 1, 128, 32, "hnd", [90], [2], True, None, 0),
    (8, 2, 128, 16, "hnd", [400, 0, 90], [150, 260, 1], True, (100, 0), 4),
    (4, 1, 64, 16, "nhd", [900, 129], [200, 30], True, (0, 0), 0),      # the token itself alone
    (4, 2, 64, 8, "hnd", [900, 60], [200, 90], True, (64, -1), 200),
    (4, 2, 256, 24, "hnd", [700], [300], True, (130, 5), 1),
    (4, 2, 128, 16, "hnd", [300], [100], True, (1 << 40, -1), 3),
    (4, 2, 128, 16, "hnd", [300, 10], [100, 40], False, None, 0),       # all of kv_len
    (4, 2, 64, 16, "hnd", [300, 10], [100, 40], False, (30, 20), 2),
    (2, 2, 256, 300, "hnd", [200], [180], False, (-1, 7), 0),
    # rows of very different lengths: the long pieces first, and more tiles than
    # are put in order
    (16, 4, 128, 16, "hnd", [3000, 0, 5, 900, 1500, 40, 0, 2200], [1, 90, 1, 64, 2, 1, 33, 30], True,
     None, 0),
    (32, 1, 64, 32, "hnd", [0, 700, 30], [700, 333, 120], True, None, 0),
]


@pytest.mark.parametrize("H,h_kv,d,page,layout,have,new,causal,window,sinks", PREFILL)
def test_prefill(H, h_kv, d, page, layout, have, new, causal, window, sinks):
    table, start, kv_len, pages = rows_of(have, new, page, d + page)
    k, v = pools(2, pages, h_kv, page, d, d + page, layout)
    cache = paged.PagedKV(k, v)
    rows, n = len(have), max(new)
    kw = dict(causal=causal, window=window, sinks=sinks)
    # padded: rows end early
    for how, layer in (("hnd", 0), ("slice", 1)):
        q = queries(rows, H, n, d, how)
        o, lse = paged.prefill(q, cache, layer, table, start, kv_len, **kw)
        fa.fa_check()
        check(P.prefill(q, k, v, layer, table, start, kv_len, **kw), o, lse)
    # packed, with tokens of no row behind
    offsets, = cuda(np.concatenate([[0], np.cumsum(new)]))
    q = queries(1, H, sum(new) + 7, d, "nhd")
    o, lse = paged.prefill(q, cache, 0, table, start, kv_len, offsets, **kw)
    fa.fa_check()
    check(P.prefill(q, k, v, 0, table, start, kv_len, offsets, **kw), o, lse, offsets)


@pytest.mark.parametrize("d,layout,page", [(64, "nhd", 16), (128, "hnd", 16), (128, "hnd", 24),
                                           (256, "hnd", 16), (64, "hnd", 160)])
def test_reads_only_what_is_visible(d, layout, page):
    """Everything but the slots that some token of the row sees holds NaN or
    infinities: free pages, slots behind a row's end, tokens outside the
    window, missing pages, pages that are none."""
    have, new, window, sinks = [700, 31, 0, 200], [40, 130, 17, 1], (120, 0), 5
    table, start, kv_len, pages = rows_of(have, new, page, d, missing=0.2, extra=6)
    clean = pools(1, pages, 2, page, d, 1, layout)
    dirty = pools(1, pages, 2, page, d, 1, layout, float("nan"))
    dirty[1].fill_(float("inf"))
    for r, (a, m) in enumerate(zip(have, new)):
        for x in range(a + m):
            if (x >= a - window[0] or x < sinks) and table[r, x // page] >= 0:
                for s, t in zip(dirty, clean):
                    s[0, table[r, x // page], :, x % page] = t[0, table[r, x // page], :, x % page]
    table[0, -1] = 1 << 30
    table[1, 0] = -7
    offsets, = cuda(np.concatenate([[0], np.cumsum(new)]))
    q = queries(1, 6, sum(new), d, "nhd")
    kw = dict(window=window, sinks=sinks)
    o, lse = paged.prefill(q, paged.PagedKV(*dirty), 0, table, start, kv_len, offsets, **kw)
    fa.fa_check()
    check(P.prefill(q, *clean, 0, table, start, kv_len, offsets, **kw), o, lse)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_rows_that_see_nothing(d):
    """Empty caches, negative lengths, rows whose pages are all missing, rows
    that lie before the first position or past the last: O = 0, LSE = -inf,
    beside a row that sees its keys."""
    k, v = pools(1, 80, 1, 16, d, 4)
    table = torch.full((6, 70), -1, dtype=torch.int32, device="cuda")
    table[2] = torch.arange(70, device="cuda")
    table[4] = table[2]
    table[5] = table[2]
    start, kv_len = cuda([0, 0, 1000, 1000, -500, 1 << 30], [0, -5, 1030, 1100, 1000, 1 << 30])
    q = randn(6, 4, 30, d)
    o, lse = paged.prefill(q, paged.PagedKV(k, v), 0, table, start, kv_len)
    r = P.prefill(q, k, v, 0, table, start, kv_len)
    check(r, o, lse)
    for b in (0, 1, 3, 4, 5):
        assert not o[b].any() and torch.isneginf(lse[b]).all()
    o, lse = paged.prefill(q, paged.PagedKV(k, v), 0, table, start, kv_len, causal=False,
                           window=(3, 3))
    check(P.prefill(q, k, v, 0, table, start, kv_len, causal=False, window=(3, 3)), o, lse)


@pytest.mark.parametrize("H,h_kv,d,have,new", [
    (4, 1, 128, [9000], [3]), (8, 2, 64, [9000, 100], [5, 200]), (2, 1, 256, [5000, 0], [1, 1]),
    (4, 2, 128, [4000, 10, 300], [129, 1, 40]), (32, 1, 64, [20000], [4])])
def test_few_rows_are_cut(H, h_kv, d, have, new):
    """Long rows of few queries: cut along the keys and joined; the same bit
    for bit whatever the workspace held."""
    page = 16
    table, start, kv_len, pages = rows_of(have, new, page, d)
    k, v = pools(1, pages, h_kv, page, d, 1)
    k *= 3                                               # the pieces' maxima differ
    cache = paged.PagedKV(k, v)
    offsets, = cuda(np.concatenate([[0], np.cumsum(new)]))
    q = queries(1, H, sum(new), d, "nhd")
    ws = paged.prefill_workspace(cache, len(have), H, sum(new), packed=True)
    first = None
    for fill in (0, 255):
        ws.fill_(fill)
        o, lse = paged.prefill(q, cache, 0, table, start, kv_len, offsets, ws=ws)
        first = first or (o, lse)
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])
    r = P.prefill(q, k, v, 0, table, start, kv_len, offsets)
    r["o_bound"] += 3 * R.F32 * 4.5                      # scores three times the bound's
    check(r, o, lse)


def test_many_rows_and_large_scores():
    """More rows than threads of a block, and scores of a standard deviation
    of 30 (the running maximum moves often)."""
    rng = np.random.default_rng(0)
    have, new = rng.integers(0, 200, 1300), rng.integers(0, 4, 1300)
    page = 16
    table, start, kv_len, pages = rows_of(have, new, page)
    k, v = pools(1, pages, 1, page, 64, 6)
    k *= 30
    offsets, = cuda(np.concatenate([[0], np.cumsum(new)]))
    q = queries(1, 2, int(new.sum()), 64, "nhd")
    o, lse = paged.prefill(q, paged.PagedKV(k, v), 0, table, start, kv_len, offsets)
    r = P.prefill(q, k, v, 0, table, start, kv_len, offsets)
    r["o_bound"] += 30 * R.F32 * 4.5
    R.check(r, "o", o)
    assert ((R.f64(lse) - r["lse"]).abs()[torch.isfinite(r["lse"])] <= 3e-3).all()


def test_values_that_are_not_numbers():
    """A NaN in a key or value that a token sees reaches that token (and its
    LSE, from a key) and no earlier tile's."""
    H, d, page, n = 2, 64, 16, 300
    table, start, kv_len, pages = rows_of([0], [n], page)
    k, v = pools(1, pages, 1, page, d, 1)
    k[0, table[0, 290 // page], :, 290 % page] = float("nan")
    q = queries(1, H, n, d, "hnd")
    o, lse = paged.prefill(q, paged.PagedKV(k, v), 0, table, start, kv_len)
    assert torch.isnan(lse[:, :, 290:]).all() and torch.isnan(o[:, :, 290:]).all()
    assert torch.isfinite(lse[:, :, :290]).all()
    # 64 tokens of two heads a tile, 128 keys: tokens up to 255 see no tile of it
    assert torch.isfinite(o[:, :, :256]).all()


def test_one_token_is_decode_s():
    rng = np.random.default_rng(5)
    have = rng.integers(0, 3000, 9)
    for d in (64, 128, 256):
        table, start, kv_len, pages = rows_of(have, [1] * 9, 16, d)
        k, v = pools(1, pages, 2, 16, d, 3)
        cache = paged.PagedKV(k, v)
        q = randn(9, 8, 1, d)
        for kw in (dict(), dict(window=(200, 0), sinks=4)):
            r = R.decode(q, k, v, 0, table, kv_len, None, kw.get("window"), kw.get("sinks", 0))
            for o, lse in (paged.prefill(q, cache, 0, table, start, kv_len, **kw),
                           paged.decode(q, cache, 0, table, kv_len, **kw)):
                R.check(r, "o", o)
                R.check(r, "lse", lse)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_whole_prompt_is_forward_s(d):
    """From an empty cache, in one piece or in chunks: the forward's result; a
    contiguous cache as a pool of one page a row."""
    B, H, h_kv, N = 2, 4, 2, 333
    q, k, v = (randn(B, h, N, d, seed=h + s) for s, h in enumerate((H, h_kv, h_kv)))
    cache = paged.PagedKV(k, v)
    table = torch.arange(B, dtype=torch.int32, device="cuda")[:, None].contiguous()
    o, lse = fa.forward(q, k, v, causal=True)
    r = R.attention(q, k, v)
    R.check(r, "o", o)
    at = 0
    for n in (200, 1, 132):
        start, kv_len = cuda([at] * B, [at + n] * B)
        oc, lc = paged.prefill(q[:, :, at:at + n], cache, 0, table, start, kv_len)
        part = {x: r[x][:, :, at:at + n] for x in ("o", "o_bound", "lse")}
        R.check(part, "o", oc)
        R.check(part, "lse", lc)
        at += n


@pytest.mark.parametrize("H,h_kv,N,d,page,new", [
    (32, 8, 8192, 128, 16, 2048), (32, 8, 5000, 128, 128, 1024), (16, 16, 6000, 64, 16, 2500),
    (16, 4, 4096, 256, 32, 4096), (16, 4, 9000, 256, 64, 512), (8, 1, 20000, 128, 24, 300)])
def test_large_chunks_are_forward_s(H, h_kv, N, d, page, new):
    """Chunks of many tiles, whole and cut in either way, against the forward
    of the whole sequence: both within their bounds of the exact output, whose
    sum over weights times |v| is the forward's of |v|."""
    q, k, v = (randn(1, h, N, d, seed=s) for s, h in ((1, H), (2, h_kv), (3, h_kv)))
    most = -(-N // page)
    pool = torch.zeros(2, 1, most, h_kv, page, d, dtype=torch.bfloat16, device="cuda")
    order = torch.randperm(most, generator=torch.Generator().manual_seed(0)).cuda()
    for i, t in enumerate((k, v)):
        padded = torch.zeros(1, h_kv, most * page, d, dtype=torch.bfloat16, device="cuda")
        padded[:, :, :N] = t
        pool[i, 0, order] = padded.view(h_kv, most, page, d).transpose(0, 1)
    table, start, kv_len = order.to(torch.int32)[None], *cuda([N - new], [N])
    cache = paged.PagedKV(pool[0], pool[1])
    o, lse = paged.prefill(q[:, :, N - new:], cache, 0, table, start, kv_len)
    fa.fa_check()
    want, want_lse = (t[:, :, N - new:] for t in fa.forward(q, k, v, causal=True))
    mean = fa.forward(q, k, v.abs(), causal=True)[0][:, :, N - new:].float() * 1.02
    bound = 2.02 * ((R.BF16 + R.F32) * mean + R.BF16 * want.float().abs()) + R.TINY
    assert ((o.float() - want.float()).abs() <= bound).all()
    assert (lse - want_lse).abs().max() <= 2e-4


def test_scale_and_streams():
    table, start, kv_len, pages = rows_of([100, 3], [40, 7], 16)
    k, v = pools(1, pages, 2, 16, 64, 1)
    cache = paged.PagedKV(k, v)
    q = queries(2, 4, 40, 64, "hnd")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o, lse = paged.prefill(q, cache, 0, table, start, kv_len, scale=0.5, stream=s)
    s.synchronize()
    r = P.prefill(q, k, v, 0, table, start, kv_len, scale=0.5)
    r["o_bound"] += 4 * R.F32 * 4.5                      # scores four times the bound's
    check(r, o, lse)


def test_tokens_of_no_row_stay():
    """Outputs behind the last row, and between an output's rows, are left."""
    H, d, page, T = 4, 64, 16, 90
    table, start, kv_len, pages = rows_of([30, 0], [20, 33], page)
    k, v = pools(1, pages, 2, page, d, 1)
    cache = paged.PagedKV(k, v)
    offsets, = cuda([3, 23, 56])                         # three tokens before the first row too
    q = queries(1, H, T, d, "nhd")
    buf = torch.full((T, H + 1, d + 8), 5.0, device="cuda").to(torch.bfloat16)
    lse = torch.full((1, H, T), 5.0, device="cuda")
    ws = paged.prefill_workspace(cache, 2, H, T, packed=True)
    ov = fa.FaStrided(buf.data_ptr(), 0, d + 8, (H + 1) * (d + 8))
    st = fa.load().fa_prefill_paged(
        rope.view("q", q, q.shape, 0), cache.ref, 0, table.data_ptr(), table.shape[1],
        start.data_ptr(), kv_len.data_ptr(), offsets.data_ptr(), ctypes.byref(ov), lse.data_ptr(), 2, H, T,
        d ** -0.5, 1, -1, -1, 0, ws.data_ptr(), ws.numel(), None)
    assert st == fa.FA_OK
    fa.fa_check()
    o = buf[:, :H, :d].transpose(0, 1)[None]
    r = P.prefill(q, k, v, 0, table, start, kv_len, offsets)
    part = {n: x[:, :, 3:56] for n, x in r.items()}
    R.check(part, "o", o[:, :, 3:56])
    R.check(part, "lse", lse[:, :, 3:56])
    for x in (o, lse[..., None]):
        assert (x[:, :, :3] == 5).all() and (x[:, :, 56:] == 5).all()
    assert (buf[:, H] == 5).all() and (buf[:, :, d:] == 5).all()


def test_offsets_that_are_none():
    """Offsets past the tokens or that fall: the call stays within its buffers
    (what it gives those rows is not said), other rows are right."""
    H, d, page, T = 2, 64, 16, 64
    table, start, kv_len, pages = rows_of([0, 0, 0], [40, 40, 40], page)
    k, v = pools(1, pages, 1, page, d, 1)
    cache = paged.PagedKV(k, v)
    q = queries(1, H, T, d, "nhd")
    offsets, = cuda([0, 40, 30, 1 << 30])
    o, lse = paged.prefill(q, cache, 0, table, start, kv_len, offsets)
    fa.fa_check()
    r = P.prefill(q, k, v, 0, table, start, kv_len, [0, 30, 30, 30])
    part = {n: x[:, :, :30] for n, x in r.items()}
    R.check(part, "o", o[:, :, :30])
    # many rows that name all tokens again and again: more than the list holds
    B = 600
    offsets, = cuda([0, T] * (B // 2) + [T])
    table = table[:1].expand(B, -1).contiguous()
    start, kv_len = cuda([0] * B, [40] * B)
    paged.prefill(q, cache, 0, table, start, kv_len, offsets)
    fa.fa_check()


def test_offsets_that_name_tokens_2_31_times():
    """More tiles than an int counts, by offsets that rise and fall: within the
    buffers, and the first row right."""
    H, d, page, T, B = 128, 64, 16, 1 << 17, 1 << 16
    table, start, kv_len, pages = rows_of([0], [20], page)
    k, v = pools(1, pages, 1, page, d, 1)
    q = torch.zeros(1, T, H, d, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    q[:, :, :20] = queries(1, H, 20, d, "nhd")
    offsets, = cuda([0, 20] + [0, T] * ((B - 2) // 2) + [0])
    assert offsets.numel() == B + 1
    lens = kv_len.expand(B).contiguous()
    o, lse = paged.prefill(q, paged.PagedKV(k, v), 0, table[:, :2].expand(B, -1).contiguous(),
                           torch.zeros_like(lens), lens, offsets)
    fa.fa_check()
    r = P.prefill(q[:, :, :20], k, v, 0, table[:, :2], start, kv_len, [0, 20])
    R.check(r, "o", o[:, :, :20])


def test_far_starts():
    """Without a window a start says nothing of what a token sees, next to 2^30
    and beyond either; under one it counts as documented."""
    have, new = [300, 40], [30, 30]
    table, start, kv_len, pages = rows_of(have, new, 16)
    k, v = pools(1, pages, 1, 16, 64, 1)
    q = queries(2, 2, 30, 64, "hnd")
    cache = paged.PagedKV(k, v)
    r = P.prefill(q, k, v, 0, table, start, kv_len, causal=False)
    for far in ([0, -5], [(1 << 30) - 1, (1 << 30) - 7], [1 << 30, (1 << 31) - 1],
                [-(1 << 31), -(1 << 30)]):
        o, lse = paged.prefill(q, cache, 0, table, cuda(far)[0], kv_len, causal=False)
        check(r, o, lse)
    for far, window in (([(1 << 30) - 3, (1 << 30) - 100], ((1 << 30) - 90, -1)),
                        ([-200, -20], (-1, 210)), ([-(1 << 30), -30], (-1, (1 << 30) + 50)),
                        ([(1 << 30) - 1, 700], ((1 << 31) - 2, 0))):
        far, = cuda(far)
        kw = dict(causal=False, window=window, sinks=3)
        o, lse = paged.prefill(q, cache, 0, table, far, kv_len, **kw)
        check(P.prefill(q, k, v, 0, table, far, kv_len, **kw), o, lse)


def test_captured_and_replayed():
    """A captured call follows the lengths, the table and the queries."""
    H, h_kv, d, page, rows, n = 8, 2, 128, 16, 3, 20
    k, v = pools(1, 300, h_kv, page, d, 2)
    cache = paged.PagedKV(k, v)
    table = torch.randperm(300, device="cuda").to(torch.int32)[:rows * 100].view(rows, 100)
    table = table.contiguous()
    start, kv_len = cuda([0, 0, 0], [0, 0, 0])
    q = queries(rows, H, n, d, "hnd")
    paged.prefill(q, cache, 0, table, start, kv_len)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse = paged.prefill(q, cache, 0, table, start, kv_len)
    for have in ([0, 5, 1500], [700, 0, 2], [1580, 1580, 1580]):
        start.copy_(torch.tensor(have))
        kv_len.copy_(torch.tensor(have) + n)
        table.copy_(table.flip(0))
        q.copy_(queries(rows, H, n, d, "hnd", seed=have[0]))
        g.replay()
        torch.cuda.synchronize()
        fa.fa_check()
        check(P.prefill(q, k, v, 0, table, start, kv_len), o, lse)


def test_two_calls_at_once():
    """Two streams, a workspace each, over and over."""
    H, h_kv, d, page = 8, 2, 64, 16
    table, start, kv_len, pages = rows_of([3000, 0], [9, 500], page)
    k, v = pools(1, pages, h_kv, page, d, 2)
    cache = paged.PagedKV(k, v)
    qs = [queries(2, H, 500, d, "hnd", seed=s) for s in (1, 2)]
    want = [paged.prefill(q, cache, 0, table, start, kv_len) for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for q, s in zip(qs, streams):
            got.append(paged.prefill(q, cache, 0, table, start, kv_len, stream=s))
    torch.cuda.synchronize()
    fa.fa_check()
    for i, (o, lse) in enumerate(got):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(lse, want[i % 2][1])


def test_pool_larger_than_2_31_elements():
    pages, h_kv, page, d = 10300, 8, 256, 128
    k = torch.zeros(pages, h_kv, page, d, dtype=torch.bfloat16, device="cuda")
    assert k.numel() > 1 << 31
    k[-3:] = torch.randn(3, h_kv, page, d, device="cuda").to(torch.bfloat16)
    cache = paged.PagedKV(k, k)
    table, start, kv_len = cuda([[pages - 1, pages - 3, pages - 2]], [590], [600])
    q = queries(1, 16, 10, d, "hnd")
    o, lse = paged.prefill(q, cache, 0, table, start, kv_len)
    small = k[-3:].clone()[None]
    check(P.prefill(q, small, small, 0, torch.tensor([[2, 0, 1]]), start, kv_len), o, lse)
    v = k.clone()                                        # (writes: pools of their own)
    new = torch.randn(1, 5, 3 * h_kv, d, device="cuda").to(torch.bfloat16).transpose(1, 2)
    at, to = cuda([700], [705])
    kn, vn = new[:, :h_kv], new[:, h_kv:2 * h_kv]
    rotary = rope.Rotary(d)
    paged.append_rotated(None, kn, vn, paged.PagedKV(k, v), 0, table, at, to, rotary)
    assert torch.equal(v[pages - 2, :, 188:193], vn[0])
    P.check(k[pages - 2, :, 188:193], *P.turn(kn[0], np.arange(700, 705)[None], rotary))


@pytest.mark.parametrize("d,page,window,sinks", [(64, 16, None, 0), (128, 16, (150, 0), 4),
                                                 (128, 100, None, 0), (256, 32, (90, 0), 2)])
def test_serving_steps(d, page, window, sinks):
    """Prompts in ragged chunks and single tokens through reserve,
    append_rotated, prefill, decode and trim, two layers: at each step the
    pages hold the tokens so far, turned at their positions, and the outputs
    are the attention over them."""
    H, h_kv, rows, layers, total = 4, 2, 3, 2, 420
    rotary = rope.Rotary(d, scaling=("linear", 2.0))
    x = [[randn(rows, h, total, d, seed=10 * layer + s) for s, h in enumerate((H, h_kv, h_kv))]
         for layer in range(layers)]
    most = -(-total // page)
    k, v = pools(layers, rows * most + 2, h_kv, page, d, 0, fill=float("nan"))
    cache = paged.PagedKV(k, v)
    table, kv_len, ref = cache.empty(rows, most)
    kw = dict(window=window, sinks=sinks)
    for step in ([200, 1, 33], [129, 0, 1], [1, 1, 1], [1, 1, 1], [7, 300, 2]):
        before = kv_len.clone()
        n_new, = cuda(step)
        new_len, ref, info = paged.reserve(cache, table, kv_len, ref, n_new)
        assert info[1] == 0
        offsets, = cuda(np.concatenate([[0], np.cumsum(step)]))
        for layer in range(layers):
            parts = [torch.cat([t[r, :, int(before[r]):int(before[r]) + m]
                                for r, m in enumerate(step)], 1)[None] for t in x[layer]]
            q = paged.append_rotated(*parts, cache, layer, table, before, new_len, rotary, offsets)
            o, lse = paged.prefill(q, cache, layer, table, before, new_len, offsets, **kw)
            fa.fa_check()
            at = np.concatenate([int(before[r]) + np.arange(m) for r, m in enumerate(step)])
            P.check(q, *P.turn(parts[0], at[None, None], rotary))
            for r in range(rows):
                kk, pos = R.gather(k, layer, table[r].cpu(), int(new_len[r]), page)
                vv, _ = R.gather(v, layer, table[r].cpu(), int(new_len[r]), page)
                assert window or pos == list(range(int(new_len[r])))
                P.check(kk.transpose(0, 1), *P.turn(x[layer][1][r][:, pos],
                                                    np.array(pos, dtype=np.int64)[None], rotary))
                assert torch.equal(vv.transpose(0, 1), x[layer][2][r][:, pos])
            check(P.prefill(q, k, v, layer, table, before, new_len, offsets, **kw), o, lse)
            if step == [1, 1, 1]:
                q1 = q[0].transpose(0, 1)[:, :, None].contiguous()
                o1, lse1 = paged.decode(q1, cache, layer, table, new_len, **kw)
                r1 = R.decode(q1, k, v, layer, table, new_len, None, window, sinks)
                R.check(r1, "o", o1)
                R.check(r1, "lse", lse1)
        kv_len = new_len
        if window is not None:
            table, ref = paged.trim(cache, table, kv_len, ref, window[0], sinks)


def test_a_walk_of_more_than_two_seconds():
    """A piece that takes longer than a single wait may (16.6 million keys in
    pages of one, a row of as many K/V heads as CTAs, so that none is cut): the
    epilogue's wait grows with its key tiles.  All keys are one and values are
    -1, 0, 1, so that every sum is a whole number below 2^24: O is V, and LSE
    the score and the logarithm of the keys."""
    n, d = 16_600_000, 256
    H = torch.cuda.get_device_properties(0).multi_processor_count
    g = torch.Generator().manual_seed(0)
    k = randn(1, 1, H, 1, d)
    v = torch.randint(-1, 2, (1, 1, H, 1, d), generator=g).to(torch.bfloat16).cuda()
    q = randn(1, H, 1, d, seed=1)
    table = torch.zeros(1, n, dtype=torch.int32, device="cuda")
    start, kv_len = cuda([n - 1], [n])
    o, lse = paged.prefill(q, paged.PagedKV(k, v), 0, table, start, kv_len)
    fa.fa_check()
    assert torch.equal(o[0, :, 0], v[0, 0, :, 0])
    s = (P.f64(q)[0, :, 0] * P.f64(k)[0, 0, :, 0]).sum(-1) * d ** -0.5
    # an LSE next to 17 has fp32 steps of 2^-19
    assert (P.f64(lse)[0, :, 0] - s - np.log(n)).abs().max() <= R.F32 + 2.0 ** -18
