"""Rotary positions on the GPU: the turn and its gradient, and turned tokens
into the paged cache, against plain implementations."""
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


def heads(B, H, N, d, layout, seed=0):
    """[B, H, N, d] as the layout keeps it."""
    if layout == "hnd":
        return randn(B, H, N, d, seed=seed)
    if layout == "nhd":
        return randn(B, N, H, d, seed=seed).transpose(1, 2)
    return randn(B, N, H + 3, d + 8, seed=seed)[:, :, 1:H + 1, 8:].transpose(1, 2)   # a slice


ROTATE = [
    # B, H, h_kv, N, d, dims, interleaved, layout, scaling
    (1, 1, 1, 1, 64, 64, False, "hnd", None),
    (2, 5, 1, 17, 64, 64, False, "nhd", ("linear", 4.0)),
    (2, 3, 3, 33, 64, 2, False, "hnd", None),
    (1, 4, 2, 9, 64, 2, True, "slice", None),
    (1, 7, 1, 40, 64, 38, False, "slice", ("ntk", 8.0)),
    (2, 4, 2, 31, 128, 128, False, "slice", ("by_parts", 8.0, 4096)),
    (3, 2, 1, 50, 128, 128, True, "nhd", ("by_parts", 16.0, 2048, 20.0, 2.0)),
    (1, 9, 3, 65, 128, 64, False, "nhd", None),
    (1, 6, 2, 29, 128, 102, True, "hnd", None),
    (2, 2, 2, 20, 128, 126, False, "nhd", None),
    (2, 3, 1, 13, 256, 256, False, "nhd", None),
    (1, 2, 1, 70, 256, 256, True, "hnd", ("linear", 2.0)),
    (1, 3, 3, 11, 256, 80, False, "slice", None),
    (1, 2, 2, 12, 256, 90, False, "hnd", None),
    (1, 130, 2, 300, 64, 64, False, "nhd", None),          # several heads a walk
]


@pytest.mark.parametrize("B,H,h_kv,N,d,dims,interleaved,layout,scaling", ROTATE)
@pytest.mark.parametrize("back", [False, True])
def test_rotate(B, H, h_kv, N, d, dims, interleaved, layout, scaling, back):
    rotary = rope.Rotary(d, dims, interleaved=interleaved, scaling=scaling)
    q, k = heads(B, H, N, d, layout), heads(B, h_kv, N, d, layout, 1)
    rng = np.random.default_rng(N)
    start, = cuda(rng.integers(0, 200000, B))
    pos, = cuda(rng.integers(-1000, 1 << 20, (B, N)))
    t = np.arange(N)[None]
    call = rope.rotate_back if back else rope.rotate
    for kw, at in ((dict(), np.broadcast_to(t, (B, N))),
                   (dict(start=start), start.cpu().numpy()[:, None] + t),
                   (dict(pos=pos), pos.cpu().numpy())):
        before = q.clone(), k.clone()
        got = call(q, k, rotary, **kw)
        assert torch.equal(q, before[0]) and torch.equal(k, before[1])
        for x, y in zip((q, k), got):
            ref, bound = P.turn(x, at[:, None], rotary, back)
            P.check(y, ref, bound)
            assert torch.equal(y[..., dims:], x[..., dims:])
        alone, none = call(q, None, rotary, **kw)
        assert none is None and torch.equal(alone, got[0])
        # in place: the same, and nothing beside the views changes
        whole = [torch.full((B, N, H + 2, d + 16), 7.0, device="cuda").to(torch.bfloat16)
                 for _ in range(2)]
        views = [w[:, :, 1:1 + x.shape[1], 8:8 + d].transpose(1, 2) for w, x in zip(whole, (q, k))]
        for v, x in zip(views, (q, k)):
            v.copy_(x)
        out = call(*views, rotary, inplace=True, **kw)
        for v, o, y, w in zip(views, out, got, whole):
            assert o is v and torch.equal(v, y)
            v.fill_(7.0)
            assert (w == 7.0).all()


def test_rotate_far_positions():
    """Positions next to 32 bits' ends, and starts whose tokens pass them."""
    rotary = rope.Rotary(128)
    q = randn(4, 2, 6, 128)
    start, = cuda([(1 << 31) - 3, -(1 << 31), 1 << 30, -5])
    got, _ = rope.rotate(q, None, rotary, start=start)
    at = start.cpu().numpy().astype(np.int64)[:, None] + np.arange(6)
    P.check(got, *P.turn(q, at[:, None], rotary))


def test_rotate_by_whole_turns():
    """Frequencies of whole and half turns: the vector itself, and its
    negative; a magnitude scales it."""
    freqs = np.full(32, 2 * np.pi)
    q = randn(1, 2, 9, 64)
    got, _ = rope.rotate(q, None, rope.Rotary(64, freqs=freqs))
    # 2 pi in 64 bits is 2^-52 of a turn off: nothing at these positions
    assert torch.equal(got, q)
    got, _ = rope.rotate(q, None, rope.Rotary(64, freqs=freqs / 2, magnitude=4.0))
    sign = torch.tensor([1.0, -1.0], device="cuda").repeat(5)[:9, None]
    P.check(got, f64 := P.f64(q * sign) * 4, 2.0 ** -18 * 4 * (f64.abs().max() + 1))


@pytest.mark.parametrize("d,dims,interleaved", [(64, 64, False), (64, 30, False), (128, 64, True)])
def test_gradient(d, dims, interleaved):
    """The gradient of sum(g rotate(x)): by differences, which are exact for a
    linear map but for the roundings (unit vectors: the matrix itself, the
    transposed one's values rounded alike)."""
    rotary = rope.Rotary(d, dims, interleaved=interleaved, scaling=("by_parts", 4.0, 512))
    eye = torch.eye(d, device="cuda").to(torch.bfloat16)[None, None]
    pos = torch.full((1, d), 777, dtype=torch.int32, device="cuda")
    forth, _ = rope.rotate(eye, None, rotary, pos=pos)
    back, _ = rope.rotate_back(eye, None, rotary, pos=pos)
    assert torch.equal(forth[0, 0].T, back[0, 0])
    # differences of the loss along each coordinate, of a step of one
    x, g = randn(1, 1, 1, d), randn(1, 1, 1, d, seed=1)
    at = torch.full((1, 1), 777, dtype=torch.int32, device="cuda")
    dx = P.f64(rope.rotate_back(g, None, rotary, pos=at)[0])[0, 0, 0]
    steps = (P.f64(x)[0, 0] + torch.eye(d, dtype=torch.float64)).to(torch.bfloat16)[None, None]
    h = P.f64(steps)[0, 0] - P.f64(x)[0, 0]              # the steps after their rounding
    y = P.f64(rope.rotate(steps.cuda(), None, rotary, pos=pos)[0])[0, 0]
    y0 = P.f64(rope.rotate(x, None, rotary, pos=at)[0])[0, 0]
    gg = P.f64(g)[0, 0, 0]
    diff = ((y - y0) @ gg) / h.diagonal()
    # each value is rounded once in y and once in y0, and dx once; before that
    # 2^-20 of about eight a value, over d values of y, y0 and g
    tol = (R.BF16 * 1.01 * ((y.abs() + y0.abs()) @ gg.abs()) / h.diagonal().abs()
           + R.BF16 * 1.01 * dx.abs() + 2e-3)
    assert ((diff - dx).abs() <= tol).all()


def test_rotate_then_back_is_the_vector():
    rotary = rope.Rotary(128)
    q, k = randn(2, 4, 300, 128), randn(2, 2, 300, 128, seed=2)
    q2, k2 = rope.rotate_back(*rope.rotate(q, k, rotary), rotary)
    for x, y in ((q, q2), (k, k2)):
        # two roundings of a pair's values
        u, v = P.pairs(P.f64(x), 128, False)
        norm = torch.cat([torch.hypot(u, v)] * 2, -1)
        assert ((P.f64(y) - P.f64(x)).abs() <= norm * R.BF16 * 2.6).all()


def test_attention_sees_distances_alone():
    """Turned at positions that all lie further on, attention stays within its
    bounds of the same scores."""
    B, H, N, d = 1, 4, 200, 64
    rotary = rope.Rotary(d)
    q, k, v, do = (randn(B, H, N, d, seed=s) for s in range(4))
    outs = []
    for first in (0, 5000):
        start, = cuda([first])
        qr, kr = rope.rotate(q, k, rotary, start=start)
        r = R.attention(qr, kr, v, do)
        o, lse = fa.forward(qr, kr, v, causal=True)
        grads = fa.backward(qr, kr, v, o, lse, do, causal=True)
        dq, dk = rope.rotate_back(grads[0], grads[1], rotary, start=start)
        R.check(r, "o", o)
        for name, got, dt in (("dq", dq, grads[0]), ("dk", dk, grads[1])):
            ref, bound = P.turn(r[name], np.arange(first, first + N)[None, None], rotary, True)
            mag, _ = P.turn(r[name + "_bound"].abs(), np.zeros((1, 1, N)), rotary)
            u, w = P.pairs(mag, d, False)
            P.check(got, ref, bound + torch.cat([u + w] * 2, -1), name)
        outs.append((o, lse))
    # q and k are rounded once at either place: a score moves by 2^-8 of its
    # products' sum for each, an LSE by as much as its scores
    a, b = (P.f64(t).abs().amax((0, 1, 2)) for t in (q, k))
    u, w = (torch.cat([torch.hypot(*P.pairs(t, d, False))] * 2) for t in (a, b))
    moved = 2 * 2 * R.BF16 * 1.01 * float(u @ w) * d ** -0.5
    assert (outs[0][1] - outs[1][1]).abs().max() < moved


@pytest.mark.parametrize("H,h_kv,d,dims,interleaved,page,layout,packed", [
    (8, 2, 64, 64, False, 16, "hnd", True), (3, 3, 128, 128, False, 7, "nhd", False),
    (4, 1, 128, 64, True, 64, "padded", True), (2, 2, 256, 90, False, 100, "hnd", False),
    (5, 5, 64, 26, False, 1, "nhd", True), (0, 2, 128, 128, True, 32, "hnd", True)])
def test_append_rotated(H, h_kv, d, dims, interleaved, page, layout, packed):
    rng = np.random.default_rng(d + page)
    have, new = [0, 30, 5, 17, 64, 3], [9, 0, 1, 40, 2, 77]
    rows, n = 6, max(new)
    most = -(-(64 + 80) // page)
    ends = np.add(have, new)
    pages = sum(-(-int(x) // page) for x in ends) + 4
    table, kv_len, _ = R.random_cache(rng, rows, most, page, pages, ends)
    table[3, 20 // page] = -1                            # a page that is not there
    kv_len[5] -= 3                                       # tokens behind the row's end
    start = np.array(have)
    start[0] -= 4                                        # positions before the first
    table, kv_len, start = cuda(table, kv_len, start)
    k, v = pools(2, pages, h_kv, page, d, 1, layout)
    want = [k.clone(), v.clone()]
    rotary = rope.Rotary(d, dims, interleaved=interleaved)
    offsets, T = None, n
    if packed:
        offsets, = cuda(np.concatenate([[0], np.cumsum(new)]))
        T = sum(new) + 5                                 # tokens of no row
    B = 1 if packed else rows
    qkv = randn(B, T, H + 2 * h_kv, d).transpose(1, 2)
    q, kn, vn = qkv.split([H, h_kv, h_kv], 1)
    whole = qkv.clone()
    got = paged.append_rotated(q if H else None, kn, vn, paged.PagedKV(k, v), 1, table, start,
                               kv_len, rotary, offsets)
    assert torch.equal(qkv, whole)
    written = torch.zeros(pages, page, dtype=torch.bool)
    for r in range(rows):
        a, m = (int(offsets[r]), new[r]) if packed else (0, n)
        e = 0 if packed else r
        at = int(start[r]) + np.arange(m)
        if H and m:
            P.check(got[e, :, a:a + m], *P.turn(q[e, :, a:a + m], at[None], rotary))
        if not m:
            continue
        turned, bound = P.turn(kn[e, :, a:a + m], at[None], rotary)
        for t, x in enumerate(at):
            if x < 0 or x >= int(kv_len[r]) or x // page >= most or int(table[r, x // page]) < 0:
                continue
            pg, slot = int(table[r, x // page]), x % page
            written[pg, slot] = True
            P.check(k[1, pg, :, slot], turned[:, t], bound[:, t])
            assert torch.equal(v[1, pg, :, slot], vn[e, :, a + t])
    for pool, old in zip((k, v), want):
        assert torch.equal(pool[0], old[0])
        keep = ~written.cuda()[:, None, :, None].expand_as(pool[1])
        assert torch.equal(pool[1][keep], old[1][keep])
    if H:                                                # in place: other tokens stay
        paged.append_rotated(q, kn, vn, paged.PagedKV(k, v), 1, table, start, kv_len, rotary,
                             offsets, inplace=True)
        if packed:
            assert torch.equal(q[:, :, :sum(new)], got[:, :, :sum(new)])
            assert torch.equal(q[:, :, sum(new):], whole[:, :H, sum(new):])
        else:
            assert torch.equal(q, got)
        assert torch.equal(qkv[:, H:], whole[:, H:])


def test_append_rotated_is_rotate_and_append():
    rows, H, h_kv, n, d, page = 4, 8, 2, 33, 128, 16
    rotary = rope.Rotary(d, scaling=("ntk", 2.0))
    q, kn, vn = (randn(rows, h, n, d, seed=h) for h in (H, h_kv, h_kv + 1))
    vn = vn[:, :h_kv].contiguous()
    start, kv_len = cuda([0, 3, 40, 7], [33, 36, 73, 40])
    table = torch.arange(rows * 5, dtype=torch.int32, device="cuda").view(rows, 5)
    a, b = (pools(1, rows * 5, h_kv, page, d, 0) for _ in range(2))
    qa = paged.append_rotated(q, kn, vn, paged.PagedKV(*a), 0, table, start, kv_len, rotary)
    qb, kb = rope.rotate(q, kn, rotary, start=start)
    paged.append(kb, vn, paged.PagedKV(*b), 0, table, start, kv_len)
    assert torch.equal(qa, qb) and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_streams_and_graphs():
    """Another stream, and a captured call replayed over new inputs."""
    rotary = rope.Rotary(64)
    q, k = randn(2, 4, 50, 64), randn(2, 2, 50, 64, seed=1)
    start, = cuda([3, 9])
    want = rope.rotate(q, k, rotary, start=start)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = rope.rotate(q, k, rotary, start=start, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = rope.rotate(q, k, rotary, start=start)
    for shift in (0, 100):
        start += shift
        g.replay()
        torch.cuda.synchronize()
        want = rope.rotate(q, k, rotary, start=start)
        assert all(torch.equal(a, b) for a, b in zip(want, out))


# values of every kind: infinities, NaN (also with a payload), -0, the largest
# and the smallest
KINDS = [0x7f80, 0xff80, 0x7fc0, 0xffc1, 0x7fa5, 0x8000, 0x0000, 0x7f7f, 0xff7f, 0x0001, 0x8001,
         0x3f80]


@pytest.mark.parametrize("d,dims", [(64, 38), (64, 2), (64, 32), (64, 60), (128, 102), (128, 126),
                                    (128, 64), (256, 90), (256, 254)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_values_behind_the_pairs_stay(d, dims, interleaved):
    """Bit for bit, whatever they are and wherever the border falls, and they
    change no turned value: apart, in place, back, and on the way into the
    pages."""
    B, H, h_kv, N, page = 2, 3, 2, 13, 8
    rotary = rope.Rotary(d, dims, interleaved=interleaved)
    finite = [randn(B, h, N, d, seed=h) for h in (H, h_kv)]
    kinds = torch.tensor(KINDS, dtype=torch.int32).to(torch.int16).cuda()
    odd = []
    for i, x in enumerate(finite):
        y = x.clone()
        at = torch.arange(y[..., dims:].numel(), device="cuda") * 7 + i
        # (each value's place moves from token to token)
        at += torch.arange(N, device="cuda").repeat_interleave(d - dims).repeat(B * x.shape[1])
        y[..., dims:] = kinds[at % len(KINDS)].view(torch.bfloat16).view(y[..., dims:].shape)
        odd.append(y)

    def bits(x):
        return x.contiguous().view(torch.int16)

    for call in (rope.rotate, rope.rotate_back):
        want = call(*finite, rotary)
        got = call(*odd, rotary)
        same = call(*(x.clone() for x in odd), rotary, inplace=True)
        for x, w, g, s in zip(odd, want, got, same):
            assert torch.equal(bits(g)[..., :dims], bits(w)[..., :dims])
            assert torch.equal(bits(g)[..., dims:], bits(x)[..., dims:])
            assert torch.equal(bits(s), bits(g))
    q, k = rope.rotate(*odd, rotary)
    start, kv_len = cuda([0] * B, [N] * B)
    table = torch.arange(B * 2, dtype=torch.int32, device="cuda").view(B, 2)
    for inplace in (False, True):
        kp, vp = pools(1, B * 2, h_kv, page, d, 0)
        qa = paged.append_rotated(odd[0].clone(), odd[1], odd[1], paged.PagedKV(kp, vp), 0, table,
                                  start, kv_len, rotary, inplace=inplace)
        assert torch.equal(bits(qa), bits(q))
        for pool, x in ((kp, k), (vp, odd[1])):
            rows = pool[0].view(B, 2, h_kv, page, d).transpose(1, 2).reshape(B, h_kv, 16, d)
            assert torch.equal(bits(rows[:, :, :N]), bits(x))


@pytest.mark.parametrize("d,interleaved", [(64, False), (128, True), (256, False)])
def test_tokens_of_no_row_have_no_effect(d, interleaved):
    """Whatever they hold: the rows' results are the same, and nothing is
    written in their place."""
    H, h_kv, page, T = 6, 2, 16, 90
    rotary = rope.Rotary(d, interleaved=interleaved)
    qkv = randn(1, T, H + 2 * h_kv, d).transpose(1, 2)
    offsets, start, kv_len = cuda([3, 20, 20, 71], [5, 0, 30], [22, 4, 81])
    table = torch.arange(18, dtype=torch.int32, device="cuda").view(3, 6)
    outs = []
    for fill in (0.0, float("nan"), float("inf")):
        x = qkv.clone()
        x[:, :, :3], x[:, :, 71:] = fill, fill
        q, kn, vn = x.split([H, h_kv, h_kv], 1)
        kp, vp = pools(1, 18, h_kv, page, d, 0)
        got = paged.append_rotated(q, kn, vn, paged.PagedKV(kp, vp), 0, table, start, kv_len,
                                   rotary, offsets, inplace=True)
        outs.append((got[:, :, 3:71].clone(), kp, vp))
        for part in (got[:, :, :3], got[:, :, 71:]):
            assert part.isnan().all() if fill != fill else (part == fill).all()
    for other in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(outs[0], other))
