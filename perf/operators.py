"""Cases of the streaming-window and paged-cache operators: attention with a sliding window and
first tokens that stay visible (forward, forward and backward), decoding over a paged key/value
cache, writing tokens into pages, forking rows of a cache, and trimming and compacting it.

`run` computes a case in plain torch operations, or, where `own` is true, through the library's
own entry points.  `exact` is the same from the definitions, in 64 bits.
"""
import math

import numpy as np
import torch

own = False

NEG = float("-inf")


# ----------------------------------------------------------------------------- the cases
def listed():
    return [
        # one user's next token after a short prompt: a latency of a few microseconds
        dict(name="decode_one_short", op="decode", B=1, H=32, h_kv=8, d=128, page=16, lo=900,
             hi=1100, window=-1, sinks=0, layout="hnd"),
        # a serving batch of uneven lengths under a sliding window with four sinks
        dict(name="decode_window_ragged", op="decode", B=64, H=32, h_kv=8, d=64, page=16, lo=1,
             hi=16384, window=4095, sinks=4, layout="nhd"),
        # long contexts: the whole cache is read for each token
        dict(name="decode_long", op="decode", B=4, H=32, h_kv=8, d=128, page=128, lo=32768,
             hi=32768, window=-1, sinks=0, layout="hnd"),
        # a decode step's new tokens, one a row
        dict(name="append_step", op="append", B=128, h_kv=8, d=128, page=16, lo=0, hi=4096, n=1,
             layout="hnd"),
        # prompts of uneven lengths written into pages
        dict(name="append_prompts", op="append", B=8, h_kv=8, d=128, page=64, lo=0, hi=2000,
             n=8192, layout="hnd"),
        # beam search: eight searches of four beams choose their parents
        dict(name="fork_beams", op="fork", groups=8, width=4, fan=0, h_kv=8, d=128, page=16, lo=64,
             hi=2048, layers=4, layout="hnd"),
        # parallel sampling: each prompt becomes eight rows, over many layers
        dict(name="fork_samples", op="fork", groups=32, width=1, fan=8, h_kv=8, d=128, page=128,
             lo=256, hi=2048, layers=8, layout="hnd"),
        # a small cache after its rows have moved on under the window
        dict(name="compact_small", op="compact", B=4, h_kv=4, d=64, page=16, lo=100, hi=1500,
             window=511, sinks=4, layers=1, spare=0.5, layout="hnd"),
        # a large one, over several layers
        dict(name="compact_layers", op="compact", B=32, h_kv=8, d=128, page=64, lo=2000, hi=16384,
             window=4095, sinks=4, layers=2, spare=0.25, layout="nhd"),
        # training on short padded sequences of an odd length
        dict(name="sinks_train_padded", op="sinks", train=True, B=4, H=16, h_kv=16, N=1001, d=64,
             window=255, sinks=4, pad=True),
        # a prompt's forward pass with grouped heads
        dict(name="sinks_prompt", op="sinks", train=False, B=1, H=32, h_kv=8, N=8192, d=128,
             window=1023, sinks=16, pad=False),
        # training on long sequences with grouped heads
        dict(name="sinks_train_long", op="sinks", train=True, B=1, H=16, h_kv=4, N=16384, d=128,
             window=2047, sinks=4, pad=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "append", "fork", "compact", "sinks", "sinks"])
    d = rng.choice([64, 128, 128, 256])
    h_kv = rng.choice([1, 2, 4, 8])
    page = rng.choice([8, 16, 16, 24, 32, 64, 100, 128, 256])
    layout = rng.choice(["hnd", "nhd"])
    window = rng.choice([-1, -1, _log(rng, 16, 8000)])
    sinks = rng.choice([0, 1, 4, _log(rng, 1, 300)]) if window >= 0 else 0
    if op == "decode":
        hi = _log(rng, 1, 60000)
        most = max(1, min(200, (4 * 32768 * 8 * 128) // (hi * h_kv * d)))
        return dict(op=op, B=_log(rng, 1, most), H=h_kv * rng.choice([1, 2, 4, 7, 8, 16]),
                    h_kv=h_kv, d=d, page=page, lo=rng.choice([0, 1, hi // 2, hi]), hi=hi,
                    window=window, sinks=sinks, layout=layout)
    if op == "append":
        n = rng.choice([1, _log(rng, 2, 6000)])
        B = _log(rng, 1, max(1, min(200, (8 * 8192 * 8 * 128) // (n * h_kv * d) // 2)))
        return dict(op=op, B=B, h_kv=h_kv, d=d, page=page, lo=0, hi=_log(rng, 1, 2000), n=n,
                    layout=layout)
    if op == "fork":
        width = rng.choice([1, 2, 5, 8])
        return dict(op=op, groups=_log(rng, 1, 24), width=width,
                    fan=_log(rng, 2, 8) if width == 1 else 0, h_kv=h_kv, d=d, page=page,
                    lo=rng.choice([0, 17]), hi=_log(rng, 20, 2000), layers=rng.choice([1, 2, 3]),
                    layout=layout)
    if op == "compact":
        return dict(op=op, B=_log(rng, 1, 32), h_kv=h_kv, d=min(d, 128), page=page, lo=0,
                    hi=_log(rng, 50, 8000), window=_log(rng, 16, 4000), sinks=sinks,
                    layers=rng.choice([1, 2]), spare=rng.choice([0.1, 0.5, 1.0]), layout=layout)
    train = rng.choice([True, False])
    N = _log(rng, 33, 6000)
    H = h_kv * rng.choice([1, 2, 4])
    most = max(1, (16 * 12000 * 12000) // (H * N * N) // (2 if d == 256 else 1))
    return dict(op="sinks", train=train, B=_log(rng, 1, min(8, most)), H=H, h_kv=h_kv, N=N, d=d,
                window=max(1, _log(rng, 8, max(9, N - 1))), sinks=rng.choice([1, 4, 64, 130, 200]),
                pad=rng.choice([True, False]))


# ----------------------------------------------------------------------------- the inputs
def _pool(g, layers, pages, h_kv, page, d, layout):
    """[layers, pages, h_kv, page, d] as a view of memory laid out per head or per token."""
    shape = (layers, pages, h_kv, page, d) if layout == "hnd" else (layers, pages, page, h_kv, d)
    t = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    return t if layout == "hnd" else t.transpose(2, 3)


def _deal(counts, width, pages, g, most):
    """A table [rows, most] of pages dealt at random, rows of counts[r] pages."""
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    j = torch.arange(most, device="cuda")
    off = torch.cumsum(counts, 0) - counts
    at = (off[:, None] + j[None]).clamp(max=pages - 1)
    return torch.where(j[None] < counts[:, None], perm[at], -1).to(torch.int32)


def _refs(table, pages):
    t = table.reshape(-1).long()
    return torch.bincount(t[t >= 0], minlength=pages).to(torch.int32)


def _lens(g, n, lo, hi):
    return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda", dtype=torch.int32)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)

    if c["op"] == "sinks":
        B, H, h_kv, N, d = c["B"], c["H"], c["h_kv"], c["N"], c["d"]
        s.update(q=randn(B, H, N, d), k=randn(B, h_kv, N, d), v=randn(B, h_kv, N, d),
                 do=randn(B, H, N, d), kv_len=_lens(g, B, N // 2, N) if c["pad"] else None)
        return s
    page, h_kv, d = c["page"], c["h_kv"], c["d"]
    if c["op"] == "decode":
        B = c["B"]
        s["kv_len"] = _lens(g, B, c["lo"], c["hi"])
        most = max(1, -(-c["hi"] // page))
        counts = -(-s["kv_len"].long() // page)
        pages = B * most + 3
        s["table"] = _deal(counts, page, pages, g, most)
        s["k"], s["v"] = (_pool(g, 1, pages, h_kv, page, d, c["layout"]) for _ in range(2))
        s["q"] = randn(B, c["H"], 1, d)
    elif c["op"] == "append":
        B, n = c["B"], c["n"]
        s["kv_len"] = _lens(g, B, c["lo"], c["hi"])
        s["n_new"] = _lens(g, B, 1 if n > 1 else n, n)
        most = -(-(c["hi"] + n) // page)
        counts = -(-s["kv_len"].long() // page)
        pages = B * most + 3
        s["table"] = _deal(counts, page, pages, g, most)
        s["ref"] = _refs(s["table"], pages)
        s["k"], s["v"] = (_pool(g, 1, pages, h_kv, page, d, c["layout"]) for _ in range(2))
        s["k_new"], s["v_new"] = randn(B, h_kv, n, d), randn(B, h_kv, n, d)
    elif c["op"] == "fork":
        G, W, fan = c["groups"], c["width"], c["fan"]
        R = G * W
        s["kv_len"] = _lens(g, G, c["lo"], c["hi"]).repeat_interleave(W)
        most = max(1, -(-c["hi"] // page))
        counts = -(-s["kv_len"].long() // page)
        new = R * max(1, fan)
        pages = R * most + new + 5
        own_pages = _deal(counts, page, pages, g, most)
        # the rows of a group share the full pages of the first half of their tokens
        shared = (s["kv_len"].long() // 2 // page)[:, None] > torch.arange(most, device="cuda")
        first = own_pages.view(G, W, most)[:, :1].expand(G, W, most).reshape(R, most)
        s["table"] = torch.where(shared, first, own_pages)
        s["ref"] = _refs(s["table"], pages)
        if fan:
            s["parent"] = torch.arange(R, device="cuda").repeat_interleave(fan).to(torch.int32)
        else:
            pick = torch.randint(0, W, (R,), generator=g, device="cuda")
            s["parent"] = (torch.arange(R, device="cuda") // W * W + pick).to(torch.int32)
        s["k"], s["v"] = (_pool(g, c["layers"], pages, h_kv, page, d, c["layout"])
                          for _ in range(2))
    else:
        B = c["B"]
        s["kv_len"] = _lens(g, B, c["lo"], c["hi"])
        most = max(1, -(-c["hi"] // page))
        counts = -(-s["kv_len"].long() // page)
        pages = int(B * most * (1 + c["spare"])) + 2
        s["table"] = _deal(counts, page, pages, g, most)
        s["ref"] = _refs(s["table"], pages)
        s["k"], s["v"] = (_pool(g, c["layers"], pages, h_kv, page, d, c["layout"])
                          for _ in range(2))
    if own:
        from exact_attention_04_gb300 import paged
        s["cache"] = paged.PagedKV(s["k"], s["v"])
    return s


# ----------------------------------------------------------------------------- one pass
def run(s):
    c = s["case"]
    return {"sinks": _sinks, "decode": _decode, "append": _append, "fork": _fork,
            "compact": _compact}[c["op"]](s, c)


def _sinks(s, c):
    window = (c["window"], 0)
    if own:
        from exact_attention_04_gb300 import fa
        o, lse = fa.forward(s["q"], s["k"], s["v"], causal=True, kv_len=s["kv_len"], window=window,
                            sinks=c["sinks"])
        if not c["train"]:
            return {"o": o, "lse": lse}
        dq, dk, dv = fa.backward(s["q"], s["k"], s["v"], o, lse, s["do"], causal=True,
                                 kv_len=s["kv_len"], window=window, sinks=c["sinks"])
        return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}
    B, H, N, d = s["q"].shape
    h_kv = s["k"].shape[1]
    scale = 1.0 / math.sqrt(d)
    q = s["q"].float().view(B, h_kv, H // h_kv, N, d)
    k, v = s["k"].float()[:, :, None], s["v"].float()[:, :, None]
    i = torch.arange(N, device="cuda")[:, None]
    j = torch.arange(N, device="cuda")[None]
    hidden = (j > i) | ((j < i - c["window"]) & (j >= c["sinks"]))
    if s["kv_len"] is not None:
        hidden = hidden | (j >= s["kv_len"].view(B, 1, 1, 1, 1))
    p = (q * scale) @ k.transpose(-1, -2)
    p.masked_fill_(hidden, NEG)
    m = p.amax(-1, keepdim=True)
    base = torch.where(m == NEG, 0.0, m)
    p.sub_(base).exp_()
    total = p.sum(-1, keepdim=True)
    p.div_(torch.where(total > 0, total, 1.0))
    lse = (base + torch.log(total)).view(B, H, N)
    o = p @ v
    out = {"o": o.view(B, H, N, d).to(torch.bfloat16), "lse": lse}
    if not c["train"]:
        return out
    do = s["do"].float().view_as(q)
    dv = (p.transpose(-1, -2) @ do).sum(2)
    ds = do @ v.transpose(-1, -2)
    ds.sub_((do * o).sum(-1, keepdim=True)).mul_(p)
    dq = (ds @ k) * scale
    dk = (ds.transpose(-1, -2) @ q).sum(2) * scale
    out.update(dq=dq.view(B, H, N, d).to(torch.bfloat16), dk=dk.to(torch.bfloat16),
               dv=dv.to(torch.bfloat16))
    return out


def _decode(s, c):
    if own:
        from exact_attention_04_gb300 import paged
        window = None if c["window"] < 0 else (c["window"], 0)
        o, lse = paged.decode(s["q"], s["cache"], 0, s["table"], s["kv_len"], window=window,
                              sinks=c["sinks"])
        return {"o": o, "lse": lse}
    B, H, _, d = s["q"].shape
    h_kv, page = c["h_kv"], c["page"]
    at = s["table"].clamp(min=0).long()
    k, v = (s[n][0][at].permute(0, 2, 1, 3, 4).reshape(B, h_kv, 1, -1, d).float() for n in "kv")
    j = torch.arange(at.shape[1] * page, device="cuda")[None]
    last = s["kv_len"][:, None] - 1
    seen = (j <= last) & (s["table"] >= 0).repeat_interleave(page, 1)
    if c["window"] >= 0:
        seen = seen & ((j >= last - c["window"]) | (j < c["sinks"]))
    q = s["q"].float().view(B, h_kv, H // h_kv, 1, d) * (1.0 / math.sqrt(d))
    x = (q @ k.transpose(-1, -2)).masked_fill(~seen[:, None, None, None], NEG)
    m = x.amax(-1, keepdim=True)
    base = torch.where(m == NEG, 0.0, m)
    e = torch.exp(x - base)
    total = e.sum(-1, keepdim=True)
    o = (e @ v) / torch.where(total > 0, total, 1.0)
    return {"o": o.view(B, H, 1, d).to(torch.bfloat16),
            "lse": (base + torch.log(total)).view(B, H, 1)}


def _append(s, c):
    if own:
        from exact_attention_04_gb300 import paged
        kv_len, ref, info = paged.reserve(s["cache"], s["table"], s["kv_len"], s["ref"], s["n_new"])
        paged.append(s["k_new"], s["v_new"], s["cache"], 0, s["table"], s["kv_len"], kv_len)
        return {"k": s["k"], "v": s["v"], "table": s["table"], "kv_len": kv_len, "ref": ref,
                "info": info}
    page, table = c["page"], s["table"]
    R, most = table.shape
    have = s["kv_len"].long().clamp(0, most * page)
    want = (have + s["n_new"].long().clamp(min=0)).clamp(max=most * page)
    a, b = -(-have // page), -(-want // page)
    off = torch.cumsum(b - a, 0) - (b - a)
    total = int((b - a).sum())
    free = torch.nonzero(s["ref"] == 0).view(-1)
    served = min(total, free.numel())
    pad = torch.cat([free, free.new_full((1,), -1)])
    j = torch.arange(most, device="cuda")[None]
    rank = (off[:, None] + j - a[:, None]).clamp(0, free.numel())
    fresh = (j >= a[:, None]) & (j < b[:, None])
    table.copy_(torch.where(fresh, pad[rank].to(torch.int32), table))
    ref = s["ref"].clone()
    ref[free[:served]] = 1
    got = torch.minimum((free.numel() - off).clamp(min=0), b - a)
    kv_len = torch.minimum(want, (a + got) * page).to(torch.int32)
    t = torch.arange(c["n"], device="cuda")[None]
    pos = have[:, None] + t
    row, col = torch.nonzero(pos < kv_len[:, None], as_tuple=True)
    pos = pos[row, col]
    at = table[row, pos // page].long()
    s["k"][0][at, :, pos % page] = s["k_new"][row, :, col]
    s["v"][0][at, :, pos % page] = s["v_new"][row, :, col]
    info = torch.tensor([free.numel() - served, total - served], dtype=torch.int32, device="cuda")
    return {"k": s["k"], "v": s["v"], "table": table, "kv_len": kv_len, "ref": ref, "info": info}


def _count(pages, table):
    t = table.reshape(-1).long()
    return torch.bincount(t[(t >= 0) & (t < pages)], minlength=pages).to(torch.int32)


def _fork(s, c):
    if own:
        from exact_attention_04_gb300 import paged
        table, kv_len, ref, info = paged.fork(s["cache"], s["table"], s["kv_len"], s["ref"],
                                              s["parent"])
        return {"k": s["k"], "v": s["v"], "table": table, "kv_len": kv_len, "ref": ref,
                "info": info}
    page, table, parent = c["page"], s["table"], s["parent"].long()
    R, most = table.shape
    pages = s["ref"].numel()
    j = torch.arange(most, device="cuda")[None]
    old_len = s["kv_len"].long().clamp(0, most * page)
    held = torch.where(j < -(-old_len[:, None] // page), table, -1)
    valid = (parent >= 0) & (parent < R)
    par = parent.clamp(0, R - 1)
    length = torch.where(valid, old_len[par], 0)
    rows = torch.where(valid[:, None], held[par], -1)
    child = torch.arange(parent.numel(), device="cuda")
    first = torch.full((R,), parent.numel(), device="cuda").scatter_reduce(
        0, par, torch.where(valid, child, parent.numel()), "amin")
    tail = (length // page).clamp(max=most - 1)
    src = rows.gather(1, tail[:, None])[:, 0].long()
    need = valid & (length % page > 0) & (src >= 0) & (first[par] != child)
    at_tail = j == tail[:, None]
    kept = torch.where(need[:, None] & at_tail, -1, rows)
    ref = s["ref"] - _count(pages, held) + _count(pages, kept)
    free = torch.nonzero(ref == 0).view(-1)
    rank = (torch.cumsum(need, 0) - 1).clamp(0, free.numel())
    got = torch.cat([free, free.new_full((1,), -1)])[rank]
    done = need & (got >= 0)
    table = torch.where(need[:, None] & at_tail, got[:, None].to(torch.int32), rows)
    kv_len = torch.where(need & ~done, length // page * page, length).to(torch.int32)
    src, dst, fill = src[done], got[done], (length % page)[done]
    ref[dst] = 1
    live = torch.arange(page, device="cuda")[None] < fill[:, None]
    for pool in (s["k"], s["v"]):
        pool[:, dst] = torch.where(live[None, :, None, :, None], pool[:, src], pool[:, dst])
    asked = need.sum()
    given = done.sum()
    info = torch.stack([free.numel() - given, asked - given]).to(torch.int32)
    return {"k": s["k"], "v": s["v"], "table": table, "kv_len": kv_len, "ref": ref, "info": info}


def _compact(s, c):
    if own:
        from exact_attention_04_gb300 import paged
        table, ref = paged.trim(s["cache"], s["table"], s["kv_len"], s["ref"], c["window"],
                                c["sinks"])
        table, ref, info = paged.compact(s["cache"], table, ref)
        return {"k": s["k"], "v": s["v"], "table": table, "ref": ref, "info": info}
    page, table = c["page"], s["table"]
    R, most = table.shape
    pages = s["ref"].numel()
    j = torch.arange(most, device="cuda")[None]
    length = s["kv_len"].long().clamp(0, most * page)[:, None]
    drop = ((j + 1) * page <= length - c["window"]) & (j * page >= c["sinks"])
    ref = s["ref"] - _count(pages, torch.where(drop, table, -1))
    table = torch.where(drop, -1, table)
    live = ref > 0
    n = int(live.sum())
    holes = torch.nonzero(~live[:n]).view(-1)
    src = torch.nonzero(live[n:]).view(-1) + n
    to = torch.arange(pages + 1, device="cuda", dtype=torch.int32)
    to[src] = holes.to(torch.int32)
    to[pages] = -1
    table = to[torch.where((table >= 0) & (table < pages), table, pages).long()]
    ref[holes] = ref[src]
    ref[src] = 0
    for pool in (s["k"], s["v"]):
        pool[:, holes] = pool[:, src]
    info = torch.tensor([n, holes.numel()], dtype=torch.int32, device="cuda")
    return {"k": s["k"], "v": s["v"], "table": table, "ref": ref, "info": info}


# ----------------------------------------------------------------------------- what a pass needs
def _mean_seen(lo, hi, window, sinks):
    n = np.arange(lo, hi + 1, dtype=np.float64)
    if window >= 0:
        near = np.minimum(n, window + 1)
        n = near + np.minimum(n - near, sinks)
    return float(n.mean())


def work(case):
    c = case
    row = c["h_kv"] * c["d"] * 2 * 2        # K and V of one token
    if c["op"] == "sinks":
        N = c["N"]
        n = np.arange(1, N + 1, dtype=np.float64)
        near = np.minimum(n, c["window"] + 1)
        pairs = float((near + np.minimum(n - near, c["sinks"])).sum()) * c["B"] * c["H"]
        q = c["B"] * c["H"] * N * c["d"] * 2
        kv = c["B"] * N * row
        lse = c["B"] * c["H"] * N * 4
        if not c["train"]:
            return {"bytes": 2 * q + kv + lse, "flops": 4 * c["d"] * pairs}
        return {"bytes": 4 * q + 2 * kv + lse, "flops": 14 * c["d"] * pairs}
    if c["op"] == "decode":
        seen = c["B"] * _mean_seen(c["lo"], c["hi"], c["window"], c["sinks"])
        return {"bytes": seen * row + c["B"] * c["H"] * c["d"] * 4,
                "flops": 4 * c["d"] * c["H"] * seen}
    if c["op"] == "append":
        tokens = c["B"] * (1 + c["n"]) / 2
        return {"bytes": 2 * tokens * row + 4 * 4 * c["B"], "flops": 0}
    tail = c["page"] / 2
    mean = (c["lo"] + c["hi"]) / 2
    if c["op"] == "fork":
        rows = c["groups"] * c["width"] * max(1, c["fan"])
        w = c["width"]
        copies = rows * (1 - 1 / c["fan"] if c["fan"] else (1 - 1 / w) ** w if w > 1 else 0)
        return {"bytes": 2 * copies * tail * row * c["layers"] + 8 * rows * mean / c["page"],
                "flops": 0}
    pages = c["B"] * mean / c["page"]
    seen = c["B"] * _mean_seen(c["lo"], c["hi"], c["window"], c["sinks"]) / c["page"]
    total = pages * (1 + c["spare"]) * 2
    moved = seen * max(0.0, 1 - seen / total)
    return {"bytes": 2 * moved * c["page"] * row * c["layers"] + 8 * pages, "flops": 0}


# ----------------------------------------------------------------------------- the definitions
def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    return {"sinks": _exact_sinks, "decode": _exact_decode, "append": _exact_append,
            "fork": _exact_fork, "compact": _exact_compact}[c["op"]](s, c)


def _exact_sinks(s, c):
    B, H, N, d = s["q"].shape
    group = H // c["h_kv"]
    q, k, v, do = (s[n].double() for n in ("q", "k", "v", "do"))
    o, dq = torch.zeros_like(q), torch.zeros_like(q)
    dk, dv = torch.zeros_like(k), torch.zeros_like(v)
    lse = torch.full((B, H, N), NEG, dtype=torch.float64, device="cuda")
    step, keys = 1024, torch.arange(N, device="cuda")
    for b in range(B):
        length = N if s["kv_len"] is None else int(s["kv_len"][b])
        for r in range(0, N, step):
            at = torch.arange(r, min(N, r + step), device="cuda")[:, None]
            near = (keys <= at) & (keys >= at - c["window"])
            first = (keys < c["sinks"]) & (keys <= at)
            ok = (near | first) & (keys < length)
            used = torch.nonzero(ok.any(0)).view(-1)
            if not used.numel():
                continue
            ok = ok[:, used]
            for h in range(H):
                kk, vv, qq = k[b, h // group, used], v[b, h // group, used], q[b, h, r:r + step]
                x = torch.where(ok, qq @ kk.T / math.sqrt(d), NEG)
                z = torch.logsumexp(x, 1)
                w = torch.where(ok, torch.exp(x - torch.where(z == NEG, 0, z)[:, None]), 0)
                lse[b, h, r:r + step] = z
                o[b, h, r:r + step] = w @ vv
                if c["train"]:
                    g = do[b, h, r:r + step]
                    y = g @ vv.T
                    y = w * (y - (w * y).sum(1, keepdim=True)) / math.sqrt(d)
                    dq[b, h, r:r + step] = y @ kk
                    dk[b, h // group].index_add_(0, used, y.T @ qq)
                    dv[b, h // group].index_add_(0, used, w.T @ g)
    if not c["train"]:
        return {"o": o, "lse": lse}
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def _exact_decode(s, c):
    B, H, _, d = s["q"].shape
    group = H // c["h_kv"]
    o = torch.zeros(B, H, 1, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H, 1), NEG, dtype=torch.float64, device="cuda")
    for b in range(B):
        n = int(s["kv_len"][b])
        pos = torch.arange(n, device="cuda")
        if c["window"] >= 0:
            pos = pos[(pos >= n - 1 - c["window"]) | (pos < c["sinks"])]
        if not pos.numel():
            continue
        page = s["table"][b].long()[pos // c["page"]]
        for h in range(c["h_kv"]):
            kk, vv = (s[x][0][page, h, pos % c["page"]].double() for x in "kv")
            x = s["q"][b, h * group:(h + 1) * group, 0].double() @ kk.T / math.sqrt(d)
            lse[b, h * group:(h + 1) * group, 0] = torch.logsumexp(x, 1)
            o[b, h * group:(h + 1) * group, 0] = torch.softmax(x, 1) @ vv
    return {"o": o, "lse": lse}


def _gpu(x):
    return torch.from_numpy(np.asarray(x, dtype=np.int32)).cuda()


def _exact_append(s, c):
    table, kv_len, n_new, ref = (s[n].cpu().numpy().copy() for n in ("table", "kv_len", "n_new",
                                                                     "ref"))
    page, most = c["page"], table.shape[1]
    free = [p for p in range(ref.size) if ref[p] == 0]
    missing, out = 0, []
    for r in range(table.shape[0]):
        n, want = int(kv_len[r]), min(int(kv_len[r]) + int(n_new[r]), most * page)
        room = -(-n // page) * page
        for j in range(-(-n // page), -(-want // page)):
            if free:
                table[r, j] = free.pop(0)
                ref[table[r, j]] = 1
                room = (j + 1) * page
            else:
                table[r, j] = -1
                missing += 1
        out.append(min(want, room))
        pos = np.arange(n, out[-1])
        at = _gpu(table[r, pos // page]).long()
        for pool, new in ((s["k"], s["k_new"]), (s["v"], s["v_new"])):
            pool[0][at, :, _gpu(pos % page).long()] = new[r, :, :pos.size].transpose(0, 1)
    return {"k": s["k"].double(), "v": s["v"].double(), "table": _gpu(table), "kv_len": _gpu(out),
            "ref": _gpu(ref), "info": _gpu([len(free), missing])}


def _exact_fork(s, c):
    table, kv_len, ref, parent = (s[n].cpu().numpy() for n in ("table", "kv_len", "ref", "parent"))
    page, ref = c["page"], ref.copy()
    out = np.full((parent.size, table.shape[1]), -1, dtype=np.int64)
    lens, wait, seen = [], [], set()
    for r in range(table.shape[0]):
        for j in range(-(-int(kv_len[r]) // page)):
            if table[r, j] >= 0:
                ref[table[r, j]] -= 1
    for r, p in enumerate(parent):
        n = int(kv_len[p]) if 0 <= p < table.shape[0] else 0
        lens.append(n)
        for j in range(-(-n // page)):
            if table[p, j] < 0:
                continue
            if (j + 1) * page > n and p in seen:
                wait.append((r, j, int(table[p, j])))
                continue
            out[r, j] = table[p, j]
            ref[out[r, j]] += 1
        seen.add(p)
    free = [p for p in range(ref.size) if ref[p] == 0]
    missing = 0
    for r, j, src in wait:
        if not free:
            lens[r], missing = j * page, missing + 1
            continue
        out[r, j] = free.pop(0)
        ref[out[r, j]] = 1
        t = lens[r] % page
        for pool in (s["k"], s["v"]):
            pool[:, int(out[r, j]), :, :t] = pool[:, src, :, :t]
    return {"k": s["k"].double(), "v": s["v"].double(), "table": _gpu(out), "kv_len": _gpu(lens),
            "ref": _gpu(ref), "info": _gpu([len(free), missing])}


def _exact_compact(s, c):
    table, kv_len, ref = (s[n].cpu().numpy().copy() for n in ("table", "kv_len", "ref"))
    page = c["page"]
    for r in range(table.shape[0]):
        for j in range(-(-int(kv_len[r]) // page)):
            if table[r, j] >= 0 and j * page >= c["sinks"] \
                    and (j + 1) * page <= int(kv_len[r]) - c["window"]:
                ref[table[r, j]] -= 1
                table[r, j] = -1
    n = int((ref > 0).sum())
    holes = [p for p in range(n) if ref[p] <= 0]
    to = {}
    for p in range(n, ref.size):
        if ref[p] > 0:
            to[p] = holes[len(to)]
            ref[to[p]], ref[p] = ref[p], 0
    for r in range(table.shape[0]):
        for j in range(table.shape[1]):
            table[r, j] = to.get(int(table[r, j]), table[r, j])
    if to:
        src, dst = _gpu(list(to.keys())).long(), _gpu(list(to.values())).long()
        for pool in (s["k"], s["v"]):
            pool[:, dst] = pool[:, src]
    return {"k": s["k"].double(), "v": s["v"].double(), "table": _gpu(table), "ref": _gpu(ref),
            "info": _gpu([n, len(to)])}
