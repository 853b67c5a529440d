"""Plain 64-bit implementations of rotary positions and of attention of new
tokens over the paged cache, with the bounds that the GPU results are held to.

Turned values: rounded to bf16 once, 2^-8 of themselves at most.  Before that,
the angle is exact to 2^-25 of itself (at most pi), sine and cosine to 2^-23 (2
units), and the products and their sum add 3 2^-24: under 2^-20 of (|a| + |b|)
m.  Attention: paged_ref's bounds.
"""
import numpy as np
import torch

import paged_ref as R

f64 = R.f64


def pairs(x, dims, interleaved):
    return (x[..., 0:dims:2], x[..., 1:dims:2]) if interleaved else \
        (x[..., :dims // 2], x[..., dims // 2:dims])


def turn(x, pos, rotary, back=False):
    """(turned, bound): x [.., N, d], pos [.., N] (integers), in 64 bits.  The
    angle modulo a turn is taken in whole numbers where a product of doubles
    would lose it."""
    x, y = f64(x), f64(x).clone()
    pos = np.asarray(pos.cpu() if torch.is_tensor(pos) else pos).astype(object)
    turns = np.array([int(t) for t in rotary.turns.cpu().numpy().view(np.uint64)], dtype=object)
    frac = (pos[..., None] * turns) % (1 << 64)
    a = torch.from_numpy(frac.astype(np.float64) * (2 * np.pi / 2.0 ** 64))
    cos, sin, m = torch.cos(a), torch.sin(a), rotary.magnitude
    if back:
        sin = -sin
    u, v = pairs(x, rotary.dims, rotary.interleaved)
    p, q = pairs(y, rotary.dims, rotary.interleaved)
    bound = torch.zeros_like(y)
    bp, bq = pairs(bound, rotary.dims, rotary.interleaved)
    p.copy_((u * cos - v * sin) * m)
    q.copy_((u * sin + v * cos) * m)
    noise = (u.abs() + v.abs()) * abs(m) * 2.0 ** -20
    bp.copy_(noise + R.BF16 * p.abs())
    bq.copy_(noise + R.BF16 * q.abs())
    return y, bound * 1.01


def check(got, ref, bound, what=""):
    got = f64(got)
    assert torch.isfinite(got).all(), what
    over = (got - ref).abs() - bound
    assert over.max() <= 0, f"{what}: over by {over.max():.3e}"


def prefill(q, k, v, layer, table, start, kv_len, offsets=None, scale=None, causal=True,
            window=None, sinks=0):
    """Dict of o, lse (q's shape) with bounds: attention of each row's new
    tokens over the pages of k, v [layers, pages, h_kv, page, d].  Tokens of no
    row: NaN."""
    _, H, N, d = q.shape
    page, group = k.shape[3], H // k.shape[2]
    scale = d ** -0.5 if scale is None else scale
    left, right = (-1, -1) if window is None else window
    q, k, v, table = f64(q), f64(k), f64(v), table.cpu()
    nan = float("nan")
    r = {"o": torch.full_like(q, nan), "o_bound": torch.full_like(q, R.TINY),
         "lse": torch.full(q.shape[:3], nan, dtype=torch.float64)}
    for b in range(table.shape[0]):
        e, a, z = (b, 0, N) if offsets is None else (0, int(offsets[b]), int(offsets[b + 1]))
        n = max(0, min(int(kv_len[b]), table.shape[1] * page))
        pos = int(start[b]) + torch.arange(z - a)[:, None]
        kk, at = R.gather(k, layer, table[b], n, page)
        vv, _ = R.gather(v, layer, table[b], n, page)
        j = torch.tensor(at, dtype=torch.long)[None]
        ok = torch.ones(z - a, len(at), dtype=torch.bool)
        if causal:
            ok &= (j <= pos) & (pos < n)
        if right >= 0:
            ok &= j <= pos + right
        if left >= 0:
            ok &= (j >= pos - left) | (j < sinks)
        r["o"][e, :, a:z] = 0
        r["lse"][e, :, a:z] = -torch.inf
        if not ok.any():
            continue
        for h in range(H):
            P, lse = R.weights(q[e, h, a:z], kk[:, h // group], scale, ok)
            o = P @ vv[:, h // group]
            r["o"][e, h, a:z], r["lse"][e, h, a:z] = o, lse
            r["o_bound"][e, h, a:z] = ((R.BF16 + R.F32) * (P @ vv[:, h // group].abs())
                                       + R.BF16 * o.abs()) * 1.01 + R.TINY
    return r
