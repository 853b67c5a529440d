"""The plain implementations that the GPU results are compared with: the
gradients against central differences, the masks against a count by hand, the
cache's operations against their invariants (CPU)."""
import numpy as np
import pytest
import torch

import paged_ref as R


@pytest.mark.parametrize("window,sinks,causal,kv", [
    ((3, 0), 2, True, None), ((2, 1), 1, False, None), ((4, -1), 3, False, [9]),
    (None, 0, True, [0]), ((0, 0), 0, True, None)])
def test_gradients_are_the_differences(window, sinks, causal, kv):
    g = torch.Generator().manual_seed(1)
    q = torch.randn(1, 2, 12, 4, generator=g, dtype=torch.float64)
    k, v = (torch.randn(1, 1, 12, 4, generator=g, dtype=torch.float64) for _ in range(2))
    do = torch.randn(1, 2, 12, 4, generator=g, dtype=torch.float64)

    def loss(q, k, v):
        return float((R.attention(q, k, v, None, None, causal, kv, window, sinks)["o"] * do).sum())
    r = R.attention(q, k, v, do, None, causal, kv, window, sinks)
    h = 1e-5
    for i, name in enumerate(("dq", "dk", "dv")):
        t = [q, k, v]
        for e in range(0, t[i].numel(), 5):
            up, down = ([x.clone() for x in t] for _ in range(2))
            up[i].view(-1)[e] += h
            down[i].view(-1)[e] -= h
            diff = (loss(*up) - loss(*down)) / (2 * h)
            # the second difference's error: h^2 times a third derivative of order 10
            assert abs(diff - float(r[name].reshape(-1)[e])) <= 1e-7


def test_visible_counts():
    ok = R.visible(10, 8, (2, 0), 3)
    assert [int(x) for x in ok.sum(1)] == [1, 2, 3, 4, 5, 6, 6, 6, 5, 4]
    assert bool(ok[9, 0]) and not bool(ok[9, 3]) and bool(ok[9, 7]) and not bool(ok[9, 8])


@pytest.mark.parametrize("seed", range(5))
def test_cache_operations_keep_the_references(seed):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, 60, 6)
    c = R.Cache(*R.random_cache(rng, 6, 9, 8, 70, lens, share=0.5, missing=0.1), page=8)

    def counted():
        n = [0] * len(c.ref)
        for r, row in enumerate(c.table):
            for j in range(c.pages(c.clamped(r))):
                if c.is_page(row[j]):
                    n[row[j]] += 1
        return n
    assert c.ref == counted()
    c.fork(rng.integers(-1, 6, 9))
    assert c.ref == counted()
    c.reserve(rng.integers(0, 20, 9))
    assert c.ref == counted()
    c.trim(10, 3)
    assert c.ref == counted()
    info, moves = c.compact()
    assert c.ref == counted() and all(x > 0 for x in c.ref[:info[0]]) \
        and not any(c.ref[info[0]:])
