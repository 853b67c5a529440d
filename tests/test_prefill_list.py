"""The list of pieces that a chunk's call makes on the device (fa_prefill.cu):
every place up to the list's end is written, and inside the list's room,
whatever the rows' offsets and lengths.

On the CPU: a model of the listing, under the room that the library gives it,
with every way to cut that the device may choose.  On the GPU: the list that a
call leaves in its workspace."""
import ctypes
import math
import random

import numpy as np
import pytest
import torch

import paged_ref as R
import rope_ref as P
from exact_attention_04_gb300 import build as fabuild
from exact_attention_04_gb300 import fa, paged
from test_gpu_paged import cuda, pools

SHAPE = "_ZN2fa13prefill_shapeEiiiibiPNS_12PrefillShapeE"  # fa::prefill_shape, Itanium ABI
ROUNDS, TAIL = 4, 8          # ways to cut: rounds of all CTAs, pieces behind the last whole one


class Shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("group", "gh", "parts", "units", "tpt", "slot_rows")] \
        + [(n, ctypes.c_longlong) for n in ("tiles", "entries", "slots")]


@pytest.fixture(scope="module")
def shape():
    fabuild.build()
    f = getattr(fa.load(), SHAPE)
    f.argtypes = [ctypes.c_int] * 4 + [ctypes.c_bool, ctypes.c_int, ctypes.POINTER(Shape)]
    f.restype = ctypes.c_bool

    def get(B, H, N, h_kv, packed, sms=152):
        s = Shape()
        assert f(B, H, N, h_kv, packed, sms, ctypes.byref(s))
        return s
    return get


def tiles_of(offsets, N, tpt, most):
    """The row of each tile that is listed: the rows' tiles in order, `most` of
    them."""
    rows = []
    for b, (begin, end) in enumerate(zip(offsets[:-1], offsets[1:])):
        begin = min(max(begin, 0), N)
        end = min(max(end, begin), N)
        rows += [b] * min(-(-(end - begin) // tpt), most - len(rows))
    return rows


def cuts(walks, units, grid):
    """(tiles from which on, the most key tiles of a piece) of every way to cut
    these walks."""
    ways = [(0, math.inf)]
    for k in range(1, ROUNDS + 1):
        ways.append((0, int(sum(walks) * units / (grid * k) * 1.000001 + 1)))
    whole = len(walks) * units // grid
    for c in range(2, TAIL + 1):
        ways.append((whole * grid // units, int(max(walks) / c * 1.000001) + 1))
    return ways


def pieces(walks, start, limit):
    return [-(-n // limit) if n > limit and i >= start else 1 for i, n in enumerate(walks)]


def unwritten(walks, room, start, limit):
    """Places before the list's end that no tile writes, where a tile writes
    its pieces only if all have room and the end is what the tiles take."""
    at, written = 0, 0
    for c in pieces(walks, start, limit):
        if at + c <= room:
            written += c
        at += c
    return min(at, room) - written


def fallen(B, T, long_row, keys):
    """Offsets that name T tokens again and again, and the keys of the rows'
    tokens: one row's are many."""
    offsets = [T * (b % 2) for b in range(B + 1)]
    return offsets, [keys if b == long_row else 100 for b in range(B)]


def test_fallen_offsets_leave_no_place_unwritten(shape):
    """Rows that fall, more tiles than any rising ones have: cut at the list's
    room instead, a long row next to its end would leave places unwritten."""
    B, T, tpt = 64, 4096, 64
    s = shape(B, 2, T, 1, True)
    assert s.tpt == tpt and s.tiles == T // tpt + B
    seen = 0
    for long_row in range(0, B, 2):
        offsets, keys = fallen(B, T, long_row, 64096)
        for most in (s.tiles, s.entries):
            walks = [-(-keys[r] // 128) for r in tiles_of(offsets, T, tpt, most)]
            lost = [unwritten(walks, s.entries, *way) for way in cuts(walks, s.units, 152)]
            if most == s.tiles:
                assert not any(lost)
            seen += max(lost) if most == s.entries else 0
    assert seen > 0


@pytest.mark.parametrize("seed", range(8))
def test_every_piece_has_room(shape, seed):
    """Any walks, of as many tiles as rising offsets make."""
    rng = random.Random(seed)
    for _ in range(60):
        h_kv, group = rng.choice([1, 2, 3, 8, 40]), rng.choice([1, 2, 7, 16, 130])
        B, N, sms = rng.randint(1, 300), rng.randint(1, 5000), rng.choice([1, 7, 132, 152])
        s = shape(B, h_kv * group, N, h_kv, True, sms)
        n = min(s.tiles, rng.choice([1, 5, 100, 400]))
        hi = rng.choice([1, 3, 40, 3000, 1 << 20])
        walks = [rng.choice([0, 1, rng.randint(0, hi), hi]) for _ in range(n)]
        for way in cuts(walks, s.units, sms):
            c = pieces(walks, *way)
            assert sum(c) <= s.entries, (walks, way)
            assert sum(x for x in c if x > 1) * s.units <= s.slots, (walks, way)
        # rows that rise, with borders anywhere, make at most `tiles`
        borders = sorted(rng.randint(0, N) for _ in range(B + 1))
        assert len(tiles_of(borders, N, s.tpt, 1 << 40)) <= s.tiles


ENTRY = ("row", "n0", "ntok", "pos0", "len", "s0", "s1", "slot", "jlo", "ns", "rlo", "rhi")


def left_list(ws, s, B):
    """(the pieces that a call left in its workspace, cut tiles, most pieces of
    one)."""
    raw = ws.cpu().numpy()
    items, _, joins, most = raw[:16].view(np.int32)
    assert items % s.units == 0 and 0 < items // s.units <= s.entries
    at = 256 + -(-(B + 1) * 4 // 256) * 256
    rows = raw[at:at + items // s.units * 48].view(np.int32).reshape(-1, 12)
    return [dict(zip(ENTRY, map(int, row))) for row in rows], joins, most


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.gpu
@pytest.mark.parametrize("fill", [0, 0x7f, 255])
@pytest.mark.parametrize("long_row", [1, 3, 17])
def test_the_list_of_fallen_offsets(shape, long_row, fill):
    """What a call leaves: each listed piece is one that the call wrote, the
    pieces of a tile follow one another, and the first row, which shares no
    token, is right."""
    B, H, d, page, T, first = 64, 2, 64, 16, 4096, 100
    rows = [r for r in range(1, B) if r % 2]             # first .. T again and again
    offsets = [0] + [first if r % 2 else T for r in range(1, B + 1)]
    keys = np.array([100 if r != long_row else 64096 for r in range(B)], np.int32)
    start = np.maximum(keys.astype(np.int64) - T + first, 0)
    start[0] = 0
    most = -(-64096 // page)
    rng = np.random.default_rng(0)
    table = rng.integers(0, 50, (B, most)).astype(np.int32)
    g = torch.Generator().manual_seed(long_row)
    k, v = (torch.randn(1, 50, 1, page, d, generator=g).to(torch.bfloat16).cuda()
            for _ in range(2))
    q = torch.randn(1, H, T, d, generator=g).to(torch.bfloat16).cuda()
    table, start, kv_len, off = (torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")
                                 for x in (table, start, keys, offsets))
    cache = paged.PagedKV(k, v)
    ws = paged.prefill_workspace(cache, B, H, T, packed=True)
    ws.fill_(fill)
    o, lse = paged.prefill(q, cache, 0, table, start, kv_len, off, ws=ws)
    fa.fa_check()
    s = shape(B, H, T, 1, True, sms())
    got, joins, most_of_one = left_list(ws, s, B)
    want = tiles_of(offsets, T, s.tpt, s.tiles)
    assert len(want) == s.tiles                          # (some tiles were left out)
    spans = {}
    for e in got:
        assert e["row"] in rows + [0] and 0 <= e["n0"] < T and 0 < e["ntok"] <= s.tpt
        assert e["n0"] + e["ntok"] <= T and e["len"] == keys[e["row"]]
        spans.setdefault((e["row"], e["n0"]), []).append((e["s0"], e["s1"]))
    assert len(spans) == len(want) and {r for r, _ in spans} == set(want)
    cut = 0
    for parts in spans.values():
        parts.sort()
        assert parts[0][0] == 0 and all(a[1] == b[0] for a, b in zip(parts, parts[1:]))
        cut += len(parts) > 1
    assert joins == cut and most_of_one == max([len(x) for x in spans.values() if len(x) > 1],
                                               default=0)
    assert (joins > 0) == (long_row in want)
    r = P.prefill(q[:, :, :first], k, v, 0, table[:1], start, kv_len, [0, first])
    R.check(r, "o", o[:, :, :first])
    R.check(r, "lse", lse[:, :, :first])


CUT = [
    # H, h_kv, d, page, layout, have, new, extra keys, causal, window, sinks, missing pages
    (4, 1, 64, 16, "hnd", [60000], [5], 0, True, (40000, 0), 9000, 0.0),
    (8, 2, 128, 16, "nhd", [30000, 40], [3, 2], 5, True, (20000, 0), 5000, 0.0),
    (4, 2, 256, 32, "hnd", [30000], [2], 0, True, (20000, -1), 6000, 0.0),
    (2, 1, 128, 24, "hnd", [50000], [9], 0, True, (40000, 0), 7000, 0.2),
    (4, 1, 128, 5, "hnd", [40000], [3], 0, True, (30000, 0), 5100, 0.1),
    (2, 1, 64, 160, "hnd", [50000], [4], 0, True, (35000, 0), 8400, 0.1),
    (4, 1, 256, 300, "nhd", [50000], [3], 40, True, (30000, 0), 9200, 0.2),
    (4, 4, 64, 16, "hnd", [6000, 3000], [7, 2], 0, False, None, 0, 0.0),
    (8, 2, 128, 200, "hnd", [5000], [6], 0, False, None, 0, 0.2),
    (4, 2, 256, 16, "nhd", [16000], [5], 0, False, None, 0, 0.0),
    (4, 2, 128, 16, "hnd", [30000], [5], 900, False, (20000, 700), 5000, 0.0),
    (2, 2, 64, 3, "hnd", [30000], [5], 500, False, (20000, 300), 4000, 0.1),
    (150, 1, 64, 16, "hnd", [5000], [2], 0, True, None, 0, 0.1),         # a group of two tiles
    (130, 1, 128, 32, "hnd", [30000], [1], 0, True, (22000, 0), 5000, 0.0),
    (4, 1, 128, 16, "hnd", [9000, 0, 5000], [200, 300, 1], 0, True, (6000, 0), 1700, 0.1),
    # few key tiles: a piece each
    (4, 1, 64, 16, "hnd", [2000, 900], [5, 40], 0, True, (600, 0), 500, 0.1),
]


@pytest.mark.gpu
@pytest.mark.parametrize("H,h_kv,d,page,layout,have,new,extra,causal,window,sinks,missing", CUT)
def test_cut_walks(shape, H, h_kv, d, page, layout, have, new, extra, causal, window, sinks,
                   missing):
    """Walks that are cut under every mask: pieces that begin among the sinks'
    tiles, that hold the step from these to the window, missing pages, and NaN
    or infinities in every slot that no token of the row sees."""
    rng = np.random.default_rng(d + page)
    B, T, lens = len(have), sum(new), np.add(have, new) + extra
    most = -(-int(max(lens)) // page)
    pages = int(sum(-(-int(n) // page) for n in lens)) + 3
    table, kv_len, _ = R.random_cache(rng, B, most, page, pages, lens, missing=missing)
    clean = pools(1, pages, h_kv, page, d, 1, layout)
    dirty = pools(1, pages, h_kv, page, d, 1, layout, float("nan"))
    dirty[1].fill_(float("inf"))
    left, right = (-1, -1) if window is None else window
    for r, (a, m) in enumerate(zip(have, new)):
        j, x = np.arange(lens[r])[None], a + np.arange(m)[:, None]
        ok = np.ones((m, lens[r]), bool)
        if causal:
            ok &= j <= x
        if right >= 0:
            ok &= j <= x + right
        if left >= 0:
            ok &= (j >= x - left) | (j < sinks)
        j = np.nonzero(ok.any(0))[0]
        j = j[table[r, j // page] >= 0]
        at, slot = (torch.from_numpy(y).long().cuda() for y in (table[r, j // page], j % page))
        for to, of in zip(dirty, clean):
            to[0, at, :, slot] = of[0, at, :, slot]
    offsets = np.concatenate([[0], np.cumsum(new)])
    q = torch.randn(1, H, T, d, generator=torch.Generator().manual_seed(5)).to(
        torch.bfloat16).cuda()
    table, start, kv_len, offsets = cuda(table, have, kv_len, offsets)
    cache = paged.PagedKV(*dirty)
    kw = dict(causal=causal, window=window, sinks=sinks)
    ws = paged.prefill_workspace(cache, B, H, T, packed=True)
    ws.fill_(255)
    o, lse = paged.prefill(q, cache, 0, table, start, kv_len, offsets, ws=ws, **kw)
    fa.fa_check()
    got, joins, _ = left_list(ws, shape(B, H, T, h_kv, True, sms()), B)
    assert joins > 0
    if sinks:
        assert any(0 < e["s0"] < e["ns"] for e in got)
    if sinks > 500 and sms() == 152:
        assert any(e["slot"] >= 0 and e["s0"] < e["ns"] < e["s1"] for e in got)
    r = P.prefill(q, *clean, 0, table, start, kv_len, offsets, **kw)
    R.check(r, "o", o)
    R.check(r, "lse", lse)


@pytest.mark.gpu
@pytest.mark.parametrize("H,h_kv,N,d,page,new,causal,window,sinks", [
    (16, 4, 9000, 128, 16, 2496, True, (6000, 0), 300),
    (16, 4, 8000, 256, 32, 2496, True, (4000, 0), 5),
    (16, 16, 6000, 64, 16, 1280, True, (1500, 0), 200),
    (16, 16, 5000, 64, 160, 1280, False, None, 0),
    (16, 4, 6000, 128, 24, 2496, False, (1500, 700), 0),
    (4, 4, 9000, 256, 16, 4992, False, None, 0)])
def test_cut_rounds_are_forward_s(shape, H, h_kv, N, d, page, new, causal, window, sinks):
    """Many tiles, of which those behind the last whole round are cut, under
    windows and without causality, against the forward of the whole sequence."""
    g = torch.Generator().manual_seed(N + d)
    q, k, v = (torch.randn(1, h, N, d, generator=g).to(torch.bfloat16).cuda()
               for h in (H, h_kv, h_kv))
    most = -(-N // page)
    pool = torch.zeros(2, 1, most, h_kv, page, d, dtype=torch.bfloat16, device="cuda")
    order = torch.randperm(most, generator=g).cuda()
    for i, t in enumerate((k, v)):
        padded = torch.zeros(1, h_kv, most * page, d, dtype=torch.bfloat16, device="cuda")
        padded[:, :, :N] = t
        pool[i, 0, order] = padded.view(h_kv, most, page, d).transpose(0, 1)
    table, start, kv_len = order.to(torch.int32)[None], *cuda([N - new], [N])
    cache = paged.PagedKV(pool[0], pool[1])
    ws = paged.prefill_workspace(cache, 1, H, new)
    ws.fill_(255)
    kw = dict(causal=causal, window=window, sinks=sinks)
    o, lse = paged.prefill(q[:, :, N - new:], cache, 0, table, start, kv_len, ws=ws, **kw)
    fa.fa_check()
    s = shape(1, H, new, h_kv, False, sms())
    got, joins, _ = left_list(ws, s, 1)
    if sms() == 152:
        assert joins > 0
    assert any(e["slot"] < 0 for e in got) or not joins
    want, want_lse = (t[:, :, N - new:] for t in fa.forward(q, k, v, **kw))
    mean = fa.forward(q, k, v.abs(), **kw)[0][:, :, N - new:].float() * 1.02
    bound = 2.02 * ((R.BF16 + R.F32) * mean + R.BF16 * want.float().abs()) + R.TINY
    assert ((o.float() - want.float()).abs() <= bound).all()
    assert (lse - want_lse).abs().max() <= 2e-4
