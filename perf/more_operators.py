"""Cases of rotary positions and of prompts over the paged cache: rotating queries and keys
(forward, and the gradients back), rotating new tokens on their way into the pages, and attention
of a chunk of new tokens over them.

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
        # one short sequence of an odd length, many small heads: a latency
        dict(name="rotate_short", op="rotate", back=False, B=1, H=16, h_kv=16, N=257, d=64, rot=64,
             inter=False, scaling="none", factor=1.0, layout="hnd", pos="start"),
        # a training step's queries and keys
        dict(name="rotate_train", op="rotate", back=False, B=2, H=16, h_kv=16, N=8192, d=128,
             rot=128, inter=False, scaling="none", factor=1.0, layout="hnd", pos="start"),
        # gradients of long packed documents with grouped heads: half of the head turned,
        # neighbouring pairs, positions of each token, frequencies scaled for long contexts
        dict(name="rotate_back_long", op="rotate", back=True, B=2, H=32, h_kv=8, N=16384, d=128,
             rot=64, inter=True, scaling="by_parts", factor=8.0, layout="nhd", pos="each"),
        # a decode step: one token a row from the fused projection into the cache
        dict(name="append_step", op="append", B=128, H=32, h_kv=8, d=128, page=16, lo=1, hi=4096,
             n=1, lens="even", rot=128, inter=False, scaling="linear", factor=4.0, layout="hnd"),
        # prompts of uneven lengths, one after the other
        dict(name="append_prompts", op="append", B=8, H=32, h_kv=8, d=128, page=64, lo=0, hi=2000,
             n=8192, lens="ramp", rot=64, inter=True, scaling="ntk", factor=2.0, layout="nhd"),
        # one user's five proposed tokens after a short prompt: a latency
        dict(name="prefill_few", op="prefill", B=1, H=32, h_kv=8, d=128, page=16, lo=900, hi=1100,
             n=5, lens="even", causal=True, window=-1, sinks=0, layout="hnd", packed=False),
        # proposals of a serving batch of uneven lengths: the cache is read once
        dict(name="prefill_verify", op="prefill", B=32, H=32, h_kv=8, d=128, page=16, lo=1,
             hi=16384, n=4, lens="even", causal=True, window=-1, sinks=0, layout="nhd",
             packed=False),
        # a chunk of a long prompt
        dict(name="prefill_chunk", op="prefill", B=1, H=32, h_kv=8, d=128, page=128, lo=30720,
             hi=30720, n=2048, lens="even", causal=True, window=-1, sinks=0, layout="hnd",
             packed=True),
        # whole prompts of uneven lengths, one after the other, small heads
        dict(name="prefill_prompts", op="prefill", B=4, H=16, h_kv=16, d=64, page=16, lo=0, hi=0,
             n=4096, lens="ramp", causal=True, window=-1, sinks=0, layout="nhd", packed=True),
        # a serving step that carries two chunks beside rows of one token
        dict(name="prefill_mixed", op="prefill", B=16, H=32, h_kv=8, d=128, page=32, lo=1, hi=6000,
             n=512, lens="mixed", causal=True, window=-1, sinks=0, layout="hnd", packed=True),
        # large heads under a sliding window with four sinks, odd lengths, padded rows
        dict(name="prefill_window", op="prefill", B=2, H=16, h_kv=4, d=256, page=64, lo=5000,
             hi=9000, n=3001, lens="even", causal=True, window=4095, sinks=4, layout="hnd",
             packed=False),
        # queries against an encoder's states of another length, each row's in one long page
        dict(name="prefill_cross", op="prefill", B=16, H=16, h_kv=16, d=64, page=1500, lo=400,
             hi=1500, n=200, lens="even", causal=False, window=-1, sinks=0, layout="hnd",
             packed=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "append", "prefill", "prefill", "prefill"])
    d = rng.choice([64, 128, 128, 256])
    h_kv = rng.choice([1, 2, 4, 8, 16])
    H = h_kv * rng.choice([1, 1, 2, 4, 7, 8])
    rot = d if rng.random() < 0.6 else 2 * rng.randint(1, d // 2)
    turn = dict(rot=rot, inter=rng.random() < 0.5,
                scaling=rng.choice(["none", "linear", "ntk", "by_parts"]),
                factor=rng.choice([2.0, 4.0, 8.0, 16.0]))
    layout = rng.choice(["hnd", "nhd"])
    if op == "rotate":
        N = _log(rng, 1, 32768)
        most = max(1, (2 * 40 * 16384 * 128) // ((H + h_kv) * N * d))
        return dict(op=op, back=rng.random() < 0.5, B=_log(rng, 1, min(64, most)), H=H, h_kv=h_kv,
                    N=N, d=d, layout=layout, pos=rng.choice(["start", "each"]), **turn)
    page = rng.choice([8, 16, 16, 24, 32, 64, 100, 128, 256])
    if op == "append":
        n = rng.choice([1, _log(rng, 2, 8192)])
        most = max(1, (36000 * 48 * 128) // (n * (H + 2 * h_kv) * d))
        return dict(op=op, B=_log(rng, 1, min(200, most)), H=H, h_kv=h_kv, d=d, page=page, lo=0,
                    hi=_log(rng, 1, 2000), n=n, lens=rng.choice(["even", "ramp", "mixed"]),
                    layout=layout, **turn)
    n, hi = rng.choice([_log(rng, 1, 16), _log(rng, 16, 4096)]), _log(rng, 1, 32000)
    # at most the scores and the keys of the largest listed cases
    most = max(1, min(64, int(2e9 / (H * n * (n + hi)) * 128 / d),
                      int(3e8 * 2 / (h_kv * d * (n + hi)))))
    window = rng.choice([-1, -1, _log(rng, 16, 8000)])
    return dict(op=op, B=_log(rng, 1, most), H=H, h_kv=h_kv, d=d, page=page,
                lo=rng.choice([0, hi // 2, hi]), hi=hi, n=n,
                lens=rng.choice(["even", "ramp", "mixed"]), causal=rng.random() < 0.8,
                window=window, sinks=rng.choice([0, 1, 4, _log(rng, 1, 300)]) if window >= 0 else 0,
                layout=layout, packed=rng.random() < 0.5)


# ----------------------------------------------------------------------------- the inputs
def _freqs(c):
    """(angles per position of the pairs, in 64 bits, and the factor of a turned vector)."""
    rot, base, f = c["rot"], 10000.0, c["factor"]
    i = np.arange(rot // 2, dtype=np.float64)
    if c["scaling"] == "ntk" and rot > 2:
        base *= f ** (rot / (rot - 2))
    w = base ** (-2 * i / rot)
    if c["scaling"] == "linear":
        return w / f, 1.0
    if c["scaling"] != "by_parts":
        return w, 1.0
    # pairs that turn often over the original length of 4096 keep their angles, slow ones are
    # stretched, a ramp lies between 32 turns and one
    at = [rot * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(base)) for turns in (32, 1)]
    lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
    ramp = np.clip((i - lo) / max(hi - lo, 1e-3), 0.0, 1.0)
    return w / f * ramp + w * (1 - ramp), 0.1 * math.log(f) + 1.0


def _lens(c, g):
    """New tokens of each row: all n, a ramp up to n, or a few of n and the others one."""
    B, n = c["B"], c["n"]
    i = torch.arange(B, device="cuda")
    if c["lens"] == "ramp":
        lens = (n * (i + 1) // B).clamp(min=1)
    elif c["lens"] == "mixed":
        lens = torch.where(i < (B + 7) // 8, n, 1)
    else:
        lens = torch.full((B,), n, device="cuda")
    return lens[torch.randperm(B, generator=g, device="cuda")]


def _total(c):
    """The sum of _lens."""
    B, n = c["B"], c["n"]
    if c["lens"] == "ramp":
        return sum(max(1, n * (i + 1) // B) for i in range(B))
    if c["lens"] == "mixed":
        return sum(n if i < (B + 7) // 8 else 1 for i in range(B))
    return B * n


def _cache(s, c, g, lens):
    """Pools, and a table of pages dealt at random, for rows of `lens` tokens."""
    B, page = c["B"], c["page"]
    most = max(1, -(-(c["hi"] + (c["n"] if c.get("causal", True) else 0)) // page))
    pages = B * most + 3
    counts = -(-lens // page)
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    j = torch.arange(most, device="cuda")
    off = torch.cumsum(counts, 0) - counts
    at = (off[:, None] + j[None]).clamp(max=pages - 1)
    s["table"] = torch.where(j[None] < counts[:, None], perm[at], -1).to(torch.int32)
    hnd = c["layout"] == "hnd"
    shape = (1, pages, c["h_kv"], page, c["d"]) if hnd else (1, pages, page, c["h_kv"], c["d"])
    for n in ("k", "v"):
        t = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
        s[n] = t if hnd else t.transpose(2, 3)
    if own:
        from exact_attention_04_gb300 import paged
        s["cache"] = paged.PagedKV(s["k"], s["v"])


def _offsets(lens):
    return torch.cat([lens.new_zeros(1), torch.cumsum(lens, 0)]).to(torch.int32)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    B, H, h_kv, d = c["B"], c["H"], c["h_kv"], c["d"]

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)

    if c["op"] != "prefill":
        w, s["magnitude"] = _freqs(c)
        s["freqs"] = torch.from_numpy(w).cuda()
        if own:
            from exact_attention_04_gb300 import rope
            scaling = {"none": None, "linear": ("linear", c["factor"]),
                       "ntk": ("ntk", c["factor"]),
                       "by_parts": ("by_parts", c["factor"], 4096)}[c["scaling"]]
            s["rotary"] = rope.Rotary(d, c["rot"], interleaved=c["inter"], scaling=scaling)
    if c["op"] == "rotate":
        N = c["N"]
        s["start"] = s["pos"] = None
        if c["pos"] == "start":     # sequences that go on, from the first token or a far one
            s["start"] = torch.randint(0, 100000, (B,), generator=g, device="cuda",
                                       dtype=torch.int32)
        else:                       # documents of N / 3 tokens, the first cut off
            first = torch.randint(0, N // 3 + 1, (B, 1), generator=g, device="cuda")
            s["pos"] = ((torch.arange(N, device="cuda")[None] + first) % (N // 3 + 1)
                        ).to(torch.int32)
        if c["layout"] == "hnd":
            s["q"], s["k"] = randn(B, H, N, d), randn(B, h_kv, N, d)
        else:
            s["q"], s["k"] = (randn(B, N, h, d).transpose(1, 2) for h in (H, h_kv))
        return s
    have = torch.randint(c["lo"], c["hi"] + 1, (B,), generator=g, device="cuda",
                         dtype=torch.int32)
    lens = _lens(c, g)
    T = _total(c)
    if c["op"] == "append":
        s["start"], s["kv_len"] = have, (have + lens).to(torch.int32)
        _cache(s, c, g, s["kv_len"].long())
        s["offsets"] = _offsets(lens)
        qkv = randn(1, T, H + 2 * h_kv, d).transpose(1, 2)
        s["q"], s["k_new"], s["v_new"] = qkv.split([H, h_kv, h_kv], 1)
        return s
    if c["causal"]:
        s["start"], s["kv_len"] = have, (have + lens).to(torch.int32)
    else:                       # another sequence's states: positions count from its first
        s["start"], s["kv_len"] = torch.zeros_like(have), have
    _cache(s, c, g, s["kv_len"].long())
    s["offsets"] = None
    if c["packed"]:
        s["offsets"] = _offsets(lens)
        s["q"] = randn(1, T, H, d).transpose(1, 2)
    else:
        s["q"] = randn(B, H, c["n"], d)
    return s


# ----------------------------------------------------------------------------- one pass
def run(s):
    c = s["case"]
    return {"rotate": _rotate, "append": _append, "prefill": _prefill}[c["op"]](s, c)


def _turn(x, cos, sin, rot, inter):
    """x [.., d] with its first `rot` values turned by the angles' cos, sin [.., rot / 2]."""
    y = x.float()
    if inter:
        a, b = y[..., :rot:2], y[..., 1:rot:2]
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
    a, b = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack([a, b], -1).flatten(-2) if inter else torch.cat([a, b], -1)
    return torch.cat([turned, y[..., rot:]], -1).to(torch.bfloat16)


def _angles(s, pos):
    """cos and sin, in 32 bits, of the angles at positions `pos`."""
    a = pos.double()[..., None] * s["freqs"]
    return (torch.cos(a) * s["magnitude"]).float(), (torch.sin(a) * s["magnitude"]).float()


def _rotate(s, c):
    if own:
        from exact_attention_04_gb300 import rope
        call = rope.rotate_back if c["back"] else rope.rotate
        q, k = call(s["q"], s["k"], s["rotary"], start=s["start"], pos=s["pos"])
        return {"q": q, "k": k}
    pos = s["pos"]
    if pos is None:
        pos = s["start"][:, None] + torch.arange(c["N"], device="cuda")[None]
    cos, sin = _angles(s, pos[:, None])
    if c["back"]:
        sin = -sin
    return {n: _turn(s[n], cos, sin, c["rot"], c["inter"]) for n in "qk"}


def _tokens(s, T):
    """(row, place in its row) of each of T packed tokens."""
    lens = (s["offsets"][1:] - s["offsets"][:-1]).long()
    row = torch.repeat_interleave(torch.arange(lens.numel(), device="cuda"), lens, output_size=T)
    return row, torch.arange(T, device="cuda") - s["offsets"].long()[row]


def _append(s, c):
    if own:
        from exact_attention_04_gb300 import paged
        q = paged.append_rotated(s["q"], s["k_new"], s["v_new"], s["cache"], 0, s["table"],
                                 s["start"], s["kv_len"], s["rotary"], offsets=s["offsets"])
        return {"q": q, "k": s["k"], "v": s["v"]}
    row, t = _tokens(s, s["q"].shape[2])
    pos = s["start"].long()[row] + t
    cos, sin = _angles(s, pos)
    q = _turn(s["q"], cos, sin, c["rot"], c["inter"])
    k = _turn(s["k_new"], cos, sin, c["rot"], c["inter"])
    at, slot = s["table"][row, pos // c["page"]].long(), pos % c["page"]
    s["k"][0][at, :, slot] = k[0].transpose(0, 1)
    s["v"][0][at, :, slot] = s["v_new"][0].transpose(0, 1)
    return {"q": q, "k": s["k"], "v": s["v"]}


def _prefill(s, c):
    window = None if c["window"] < 0 else (c["window"], -1)
    if own:
        from exact_attention_04_gb300 import paged
        o, lse = paged.prefill(s["q"], s["cache"], 0, s["table"], s["start"], s["kv_len"],
                               offsets=s["offsets"], causal=c["causal"], window=window,
                               sinks=c["sinks"])
        return {"o": o, "lse": lse}
    B, H, h_kv, d, n, page = (c[x] for x in ("B", "H", "h_kv", "d", "n", "page"))
    q, T = s["q"], s["q"].shape[2]
    if s["offsets"] is not None:        # packed rows to padded ones
        row, t = _tokens(s, T)
        at = (s["offsets"].long()[:-1, None] + torch.arange(n, device="cuda")).clamp(max=T - 1)
        q = q[0][:, at].transpose(0, 1)
    at = s["table"].clamp(min=0).long()
    L = at.shape[1] * page
    k, v = (s[x][0][at].permute(0, 2, 1, 3, 4).reshape(B, h_kv, 1, L, d).float() for x in "kv")
    j = torch.arange(L, device="cuda")[None, None]
    i = (s["start"][:, None] + torch.arange(n, device="cuda"))[..., None]
    length = s["kv_len"][:, None, None]
    seen = (j < length) & (s["table"] >= 0).repeat_interleave(page, 1)[:, None]
    if c["causal"]:
        seen = seen & (j <= i) & (i < length)
    if c["window"] >= 0:
        seen = seen & ((j >= i - c["window"]) | (j < c["sinks"]))
    x = (q.float().reshape(B, h_kv, H // h_kv, n, d) * (1.0 / math.sqrt(d))) @ k.transpose(-1, -2)
    x.masked_fill_(~seen[:, None, None], NEG)
    m = x.amax(-1, keepdim=True)
    base = torch.where(m == NEG, 0.0, m)
    x.sub_(base).exp_()
    total = x.sum(-1, keepdim=True)
    o = ((x @ v) / torch.where(total > 0, total, 1.0)).view(B, H, n, d).to(torch.bfloat16)
    lse = (base + torch.log(total)).view(B, H, n)
    if s["offsets"] is not None:
        o, lse = o[row, :, t].transpose(0, 1)[None], lse[row, :, t].transpose(0, 1)[None]
    return {"o": o, "lse": lse}


# ----------------------------------------------------------------------------- what a pass needs
def _row_lens(c):
    B, n = c["B"], c["n"]
    i = np.arange(B)
    if c["lens"] == "ramp":
        return np.maximum(1, n * (i + 1) // B)
    if c["lens"] == "mixed":
        return np.where(i < (B + 7) // 8, n, 1)
    return np.full(B, n)


def work(case):
    c = case
    H, h_kv, d = c["H"], c["h_kv"], c["d"]
    if c["op"] == "rotate":
        tokens = c["B"] * c["N"]
        return {"bytes": tokens * (2 * (H + h_kv) * d * 2 + (4 if c["pos"] == "each" else 0)),
                "flops": tokens * 3 * (H + h_kv) * c["rot"]}
    if c["op"] == "append":
        tokens = _total(c)
        return {"bytes": tokens * 2 * (H + 2 * h_kv) * d * 2,
                "flops": tokens * 3 * (H + h_kv) * c["rot"]}
    have = (c["lo"] + c["hi"]) / 2
    pairs = keys = 0.0
    for n in _row_lens(c):
        n = int(n)
        if not c["causal"]:
            pos, seen = np.arange(n), np.full(n, have)
            first = 0
        else:
            pos = have + np.arange(n)
            seen, first = pos + 1, have
        if c["window"] >= 0:
            near = np.clip(seen - np.maximum(pos - c["window"], 0), 0, None)
            seen = np.minimum(seen, near + np.minimum(c["sinks"], np.maximum(pos - c["window"], 0)))
        pairs += float(np.sum(seen))
        whole = have + (n if c["causal"] else 0)
        cut = max(0.0, min(whole, first - c["window"]) - c["sinks"]) if c["window"] >= 0 else 0.0
        keys += whole - cut
    return {"bytes": keys * h_kv * d * 4 + _total(c) * H * (4 * d + 4),
            "flops": 4 * d * H * pairs}


# ----------------------------------------------------------------------------- the definitions
def _wheel(x, pos, s, c):
    """x [.., N, d] in 64 bits, each pair a complex number times magnitude * e^(i angle)."""
    rot = c["rot"]
    x = x.double()
    w = torch.polar(torch.full_like(s["freqs"], s["magnitude"]).expand(pos.shape + (rot // 2,)),
                    pos.double()[..., None] * s["freqs"])
    if c.get("back"):
        w = w.conj()
    y = x.clone()
    if c["inter"]:
        z = torch.complex(x[..., 0:rot:2].contiguous(), x[..., 1:rot:2].contiguous()) * w
        y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
    else:
        z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * w
        y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
    return y


def _exact_rotate(s, c):
    out = {"q": [], "k": []}
    for b in range(c["B"]):
        pos = torch.arange(c["N"], device="cuda") + int(s["start"][b]) if s["pos"] is None \
            else s["pos"][b]
        for n in "qk":
            out[n].append(_wheel(s[n][b], pos, s, c))
    return {n: torch.stack(out[n]) for n in "qk"}


def _exact_append(s, c):
    page, off = c["page"], s["offsets"].tolist()
    k, v, q = s["k"].double(), s["v"].double(), []
    for b in range(c["B"]):
        a, e, first = off[b], off[b + 1], int(s["start"][b])
        pos = torch.arange(first, first + e - a, device="cuda")
        q.append(_wheel(s["q"][0, :, a:e], pos, s, c))
        kk, vv = _wheel(s["k_new"][0, :, a:e], pos, s, c), s["v_new"][0, :, a:e].double()
        at = s["table"][b].long()[pos // page]
        k[0][at, :, pos % page] = kk.transpose(0, 1)
        v[0][at, :, pos % page] = vv.transpose(0, 1)
    return {"q": torch.cat(q, 1)[None], "k": k, "v": v}


def _exact_prefill(s, c):
    q, page = s["q"], c["page"]
    group = c["H"] // c["h_kv"]
    o = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.full(q.shape[:3], NEG, dtype=torch.float64, device="cuda")
    for b in range(c["B"]):
        if s["offsets"] is None:
            qb, ob, lb = q[b], o[b], lse[b]
        else:
            a, e = (int(x) for x in s["offsets"][b:b + 2])
            qb, ob, lb = q[0, :, a:e], o[0, :, a:e], lse[0, :, a:e]
        n, first = int(s["kv_len"][b]), int(s["start"][b])
        if n == 0:
            continue
        key = torch.arange(n, device="cuda")
        at = s["table"][b].long()[key // page]
        for r in range(0, qb.shape[1], 1024):
            i = first + torch.arange(r, min(qb.shape[1], r + 1024), device="cuda")[:, None]
            ok = torch.ones(i.shape[0], n, dtype=torch.bool, device="cuda")
            if c["causal"]:
                ok &= (key <= i) & (i < n)
            if c["window"] >= 0:
                ok &= (key >= i - c["window"]) | (key < c["sinks"])
            for h in range(c["h_kv"]):
                kk, vv = (s[x][0][at, h, key % page].double() for x in "kv")
                for m in range(h * group, (h + 1) * group):
                    x = qb[m, r:r + 1024].double() @ kk.T / math.sqrt(c["d"])
                    x = torch.where(ok, x, NEG)
                    z = torch.logsumexp(x, 1)
                    lb[m, r:r + 1024] = z
                    w = torch.exp(x - torch.where(z == NEG, 0, z)[:, None])
                    ob[m, r:r + 1024] = w @ vv
    return {"o": o, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    return {"rotate": _exact_rotate, "append": _exact_append,
            "prefill": _exact_prefill}[c["op"]](s, c)
