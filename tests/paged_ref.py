"""Plain 64-bit implementations of attention with a sliding window and sinks
and of the paged cache's operations, from their definitions, with the bounds
that the GPU results are held to.

Rounding: a value rounded to bf16 moves by at most half a step, 2^-8 of
itself.  F32 covers the fp32 arithmetic between the roundings: a score is a
sum of d products, off by at most d 2^-24 sum |q||k| scale (1e-4 for the N(0,1)
inputs here: d = 256, sum |q||k| about 170, scale 1/16), which moves a weight
by that much relative to itself, twice (the score and the LSE); exponentials
and sums add 2^-20 or less.
"""
import numpy as np
import torch

BF16 = 2.0 ** -8
F32 = 5e-4
TINY = 1e-6


def f64(t):
    return t.detach().cpu().double()


def visible(N, length, window, sinks, causal=True):
    """[N, N] truth values: query i (row) sees key j; window (left, right), -1
    unbounded, or None."""
    i, j = torch.arange(N)[:, None], torch.arange(N)[None]
    left, right = (-1, -1) if window is None else window
    ok = torch.ones(N, N, dtype=torch.bool)
    if left >= 0:
        ok &= (j >= i - left) | (j < sinks)
    if right >= 0:
        ok &= j <= i + right
    if causal:
        ok &= j <= i
    return ok & (j < length)


def weights(q, k, scale, ok):
    """(P, LSE) of one head: q [n, d], k [m, d], ok [n, m] (float64)."""
    s = torch.where(ok, q @ k.T * scale, -torch.inf)
    m = s.amax(1, keepdim=True)
    m = torch.where(m == -torch.inf, 0.0, m)
    e = torch.exp(s - m)
    total = e.sum(1, keepdim=True)
    lse = (m + torch.log(total))[:, 0]
    return e / torch.where(total > 0, total, 1.0), lse


def attention(q, k, v, do=None, scale=None, causal=True, kv_len=None, window=None, sinks=0):
    """Dict of o, lse and, with do, dq, dk, dv (float64, the inputs' shapes),
    each with its bound under "<name>_bound".  K and V rows at or past kv_len
    count as zeros."""
    B, H, N, d = q.shape
    group = H // k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    q, k, v = f64(q), f64(k), f64(v)
    r = {n: torch.zeros_like(q) for n in ("o", "o_bound", "dq", "dq_bound")}
    r.update({n: torch.zeros_like(k) for n in ("dk", "dk_bound", "dv", "dv_bound")})
    r["lse"] = torch.zeros(B, H, N, dtype=torch.float64)
    do = None if do is None else f64(do)
    for b in range(B):
        length = N if kv_len is None else max(0, min(N, int(kv_len[b])))
        ok = visible(N, length, window, sinks, causal)
        for h in range(H):
            g = h // group
            kk, vv = k[b, g].clone(), v[b, g].clone()
            kk[length:] = 0
            vv[length:] = 0
            P, lse = weights(q[b, h], kk, scale, ok)
            o = P @ vv
            av = P @ vv.abs()
            r["o"][b, h], r["lse"][b, h] = o, lse
            o_err = (BF16 + F32) * av + BF16 * o.abs()
            r["o_bound"][b, h] = o_err * 1.01 + TINY
            if do is None:
                continue
            x = do[b, h]
            dP = x @ vv.T
            D = (x * o).sum(1, keepdim=True)
            dS = P * (dP - D)
            # D comes from the rounded O; dP and D are fp32 sums
            D_err = (x.abs() * o_err).sum(1, keepdim=True)
            noise = F32 * (x.abs() @ vv.abs().T + (x * o).abs().sum(1, keepdim=True))
            dS_err = (BF16 + F32) * dS.abs() + P * (D_err + noise)
            r["dq"][b, h] = dS @ kk * scale
            r["dq_bound"][b, h] = dS_err @ kk.abs() * scale
            r["dk"][b, g] += dS.T @ q[b, h] * scale
            r["dk_bound"][b, g] += dS_err.T @ q[b, h].abs() * scale
            r["dv"][b, g] += P.T @ x
            r["dv_bound"][b, g] += (BF16 + F32) * (P.T @ x.abs())
    for n in ("dq", "dk", "dv"):
        r[n + "_bound"] = r[n + "_bound"] * 1.01 + BF16 * r[n].abs() * 1.01 + TINY
    return r


def check(r, name, got):
    """got against r[name] within r["<name>_bound"] (the LSE: 1e-4 absolutely,
    a hundred times the fp32 sums' error, and equal infinities)."""
    got, ref = f64(got), r[name]
    if name == "lse":
        assert torch.equal(torch.isneginf(got), torch.isneginf(ref)), "rows that see no key"
        fin = torch.isfinite(ref)
        assert torch.isfinite(got[fin]).all()
        err = (got[fin] - ref[fin]).abs()
        assert err.numel() == 0 or err.max() <= 1e-4, f"lse off by {err.max():.3e}"
        return
    assert torch.isfinite(got).all(), f"{name}: not finite"
    over = (got - ref).abs() - r[name + "_bound"]
    worst = int(over.argmax())
    assert over.max() <= 0, (f"{name}: {got.reshape(-1)[worst]:.6f} and "
                             f"{ref.reshape(-1)[worst]:.6f}, bound "
                             f"{r[name + '_bound'].reshape(-1)[worst]:.3e}")


# ---------------------------------------------------------------- the cache
def gather(pool, layer, table_row, length, page_size):
    """(rows [n, h_kv, d], positions [n]) of a row's existing tokens."""
    pos = [x for x in range(length) if 0 <= int(table_row[x // page_size]) < pool.shape[1]]
    pages = [int(table_row[x // page_size]) for x in pos]
    slots = [x % page_size for x in pos]
    return pool[layer, pages, :, slots], pos


def decode(q, k, v, layer, table, kv_len, scale=None, window=None, sinks=0):
    """Dict of o [B, H, 1, d] and lse with bounds: attention of the newest
    token of each row over the pages of k, v [layers, pages, h_kv, page, d]."""
    B, H, _, d = q.shape
    page = k.shape[3]
    group = H // k.shape[2]
    scale = d ** -0.5 if scale is None else scale
    left = -1 if window is None else window[0]
    q, k, v, table = f64(q), f64(k), f64(v), table.cpu()
    r = {n: torch.zeros(B, H, 1, d, dtype=torch.float64) for n in ("o", "o_bound")}
    r["lse"] = torch.full((B, H, 1), -torch.inf, dtype=torch.float64)
    r["o_bound"] += TINY
    for b in range(B):
        n = max(0, min(int(kv_len[b]), table.shape[1] * page))
        kk, pos = gather(k, layer, table[b], n, page)
        vv, _ = gather(v, layer, table[b], n, page)
        keep = [i for i, x in enumerate(pos) if left < 0 or x >= n - 1 - left or x < sinks]
        if not keep:
            continue
        kk, vv = kk[keep], vv[keep]
        for h in range(H):
            P, lse = weights(q[b, h], kk[:, h // group], scale,
                             torch.ones(1, len(keep), dtype=torch.bool))
            o = P @ vv[:, h // group]
            r["o"][b, h], r["lse"][b, h] = o, lse
            r["o_bound"][b, h] = ((BF16 + F32) * (P @ vv[:, h // group].abs())
                                  + BF16 * o.abs()) * 1.01 + TINY
    return r


class Cache:
    """The cache's integers as Python lists, one step at a time."""

    def __init__(self, table, kv_len, ref, page):
        self.table = [[int(x) for x in row] for row in table]
        self.len = [int(x) for x in kv_len]
        self.ref = [int(x) for x in ref]
        self.page, self.most = page, len(self.table[0])

    def clamped(self, r):
        return max(0, min(self.len[r], self.most * self.page))

    def pages(self, n):
        return -(-n // self.page)

    def is_page(self, x):
        return 0 <= x < len(self.ref)

    def free(self):
        return [p for p, n in enumerate(self.ref) if n == 0]

    def reserve(self, n_new):
        free, missing = self.free(), 0
        for r, row in enumerate(self.table):
            n = self.clamped(r)
            want = min(n + max(0, int(n_new[r])), self.most * self.page)
            room = self.pages(n) * self.page
            for j in range(self.pages(n), self.pages(want)):
                row[j] = free.pop(0) if free else -1
                if row[j] < 0:
                    missing += 1
                else:
                    self.ref[row[j]] = 1
                    room = (j + 1) * self.page
            self.len[r] = min(want, room)
        return [len(free), missing]

    def fork(self, parent):
        """info and the copies (source, page, slots)."""
        old = [row[:] for row in self.table]
        old_len = [self.clamped(r) for r in range(len(old))]
        for r, row in enumerate(old):
            for j in range(self.pages(old_len[r])):
                if self.is_page(row[j]):
                    self.ref[row[j]] -= 1
        self.table, self.len, ask, seen = [], [], [], set()
        for r, par in enumerate(int(x) for x in parent):
            row = [-1] * self.most
            n = old_len[par] if 0 <= par < len(old) else 0
            for j in range(self.pages(n)):
                x = old[par][j]
                if not self.is_page(x):
                    continue
                if (j + 1) * self.page > n and par in seen:
                    ask.append((r, j, x))
                else:
                    row[j] = x
                    self.ref[x] += 1
            seen.add(par)
            self.table.append(row)
            self.len.append(n)
        free, copies, missing = self.free(), [], 0
        for r, j, x in ask:
            if not free:
                missing += 1
                self.len[r] = j * self.page
                continue
            self.table[r][j] = free.pop(0)
            self.ref[self.table[r][j]] = 1
            copies.append((x, self.table[r][j], self.len[r] % self.page))
        return [len(free), missing], copies

    def trim(self, left, sinks):
        for r, row in enumerate(self.table):
            n = self.clamped(r)
            for j in range(self.most):
                lo = j * self.page
                if lo >= sinks and lo + self.page <= n - left:
                    if self.is_page(row[j]):
                        self.ref[row[j]] -= 1
                    row[j] = -1

    def compact(self):
        """info and the moves (source, page)."""
        n = sum(x > 0 for x in self.ref)
        holes = [p for p in range(n) if self.ref[p] <= 0]
        moves = list(zip([p for p in range(n, len(self.ref)) if self.ref[p] > 0], holes))
        to = dict(moves)
        for s, h in moves:
            self.ref[h], self.ref[s] = self.ref[s], 0
        self.table = [[to.get(x, x) if self.is_page(x) else -1 for x in row]
                      for row in self.table]
        return [n, len(moves)], moves


def random_cache(rng, rows, most, page, pages, lens, share=0.0, missing=0.0):
    """(table, kv_len, ref) as int32 arrays: rows of the given lengths over
    distinct random pages; a share of the full pages is the first row's, and a
    share of the entries is missing."""
    free = list(rng.permutation(pages))
    table = np.full((rows, most), -1, dtype=np.int32)
    ref = np.zeros(pages, dtype=np.int32)
    for r in range(rows):
        for j in range(-(-int(lens[r]) // page)):
            full = (j + 1) * page <= min(int(lens[r]), int(lens[0]))
            if r and full and table[0, j] >= 0 and rng.random() < share:
                table[r, j] = table[0, j]
            elif rng.random() >= missing:
                table[r, j] = free.pop()
            if table[r, j] >= 0:
                ref[table[r, j]] += 1
    return table, np.asarray(lens, dtype=np.int32), ref
