"""Attention with a sliding window and sinks on the GPU (fa_fwd_sinks,
fa_bwd_sinks) against the plain 64-bit implementation and its bounds."""
import pytest
import torch

import paged_ref as R
from exact_attention_04_gb300 import build as fabuild
from exact_attention_04_gb300 import fa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fabuild.build()
    fa.load()


def inputs(B, H, h_kv, N, d, seed, kv=None):
    g = torch.Generator().manual_seed(seed)
    shapes = dict(q=(B, H, N, d), k=(B, h_kv, N, d), v=(B, h_kv, N, d), do=(B, H, N, d))
    x = {n: torch.randn(s, generator=g).to(torch.bfloat16).cuda() for n, s in shapes.items()}
    x["kv_len"] = None if kv is None else torch.tensor(kv, dtype=torch.int32).cuda()
    return x


def run(x, backward=True, **kw):
    o, lse = fa.forward(x["q"], x["k"], x["v"], kv_len=x["kv_len"], **kw)
    out = dict(o=o, lse=lse)
    if backward:
        out.update(zip(("dq", "dk", "dv"),
                       fa.backward(x["q"], x["k"], x["v"], o, lse, x["do"], kv_len=x["kv_len"],
                                   **kw)))
    fa.fa_check()
    return out


def compare(x, out, causal=True, window=None, sinks=0):
    kv = None if x["kv_len"] is None else x["kv_len"].tolist()
    r = R.attention(x["q"], x["k"], x["v"], x["do"], None, causal, kv, window, sinks)
    for name, t in out.items():
        R.check(r, name, t)


CASES = [
    # B, H, h_kv, N, d, causal, window, sinks, kv_len
    (1, 1, 1, 1, 64, True, (0, 0), 1, None),
    (1, 2, 1, 2, 128, True, (0, 0), 1, None),
    (2, 2, 2, 129, 64, True, (5, 0), 1, None),
    (1, 2, 1, 129, 128, True, (127, 0), 4, None),
    (1, 1, 1, 256, 128, True, (1, 0), 7, None),        # the last steps see sinks alone
    (1, 1, 1, 256, 64, True, (1, 0), 7, None),
    (1, 1, 1, 257, 256, True, (1, 0), 130, None),      # two blocks of sinks
    (2, 4, 2, 700, 64, True, (100, 0), 4, (700, 313)),
    (2, 4, 1, 700, 128, True, (63, 0), 200, (0, 451)),
    (1, 2, 2, 700, 256, True, (200, 0), 3, (640,)),
    (1, 2, 1, 2100, 64, True, (64, 0), 5, None),       # several far chunks
    (1, 2, 1, 2100, 128, True, (64, 0), 5, (2000,)),
    (1, 1, 1, 2100, 256, True, (130, 0), 140, None),
    (1, 2, 1, 1500, 128, True, (40, 0), 1500, None),   # every token a sink
    (2, 2, 2, 900, 64, False, (33, 20), 9, (900, 5)),  # both sides bounded, padding past the window
    (2, 2, 1, 900, 128, False, (33, 20), 9, (130, 1)),
    (1, 1, 1, 400, 128, False, (50, -1), 2, None),     # right side open
    (1, 2, 2, 300, 128, True, None, 4, (200,)),        # no window: sinks change nothing
    (1, 2, 2, 300, 64, True, (1 << 30, 0), 4, None),
    (3, 20, 20, 1000, 64, True, None, 4, None),        # more tiles than CTAs, no window
    (3, 20, 20, 1000, 64, True, None, 4, (1000, 999, 1)),
    (2, 4, 2, 500, 128, False, (-1, 70), 4, None),     # open to the left alone
    (2, 4, 2, 500, 128, False, (499, 1 << 30), 4, None),
    (3, 20, 10, 1000, 128, True, (700, 0), 9, (1000, 400, 77)),   # and a wide one
    (3, 20, 10, 1000, 64, True, (150, 0), 9, (1000, 400, 77)),
    (2, 6, 2, 1000, 256, False, (300, 90), 140, (900, 1000)),
    (5, 64, 64, 600, 128, True, (200, 0), 3, None),    # heads in several chunks
    (5, 64, 64, 600, 128, True, None, 3, None),        # no window, many blocks
    (5, 64, 64, 600, 64, False, (599, 40), 3, None),
]


@pytest.mark.parametrize("B,H,h_kv,N,d,causal,window,sinks,kv", CASES)
def test_matches_the_definition(B, H, h_kv, N, d, causal, window, sinks, kv):
    x = inputs(B, H, h_kv, N, d, N + d + sinks, kv)
    kw = dict(causal=causal, window=window, sinks=sinks)
    compare(x, run(x, **kw), **kw)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_rows_past_kv_len_may_hold_anything(d):
    """NaN and infinities in K and V at or past kv_len change nothing: not the
    outputs, not the gradients, and their own gradients are 0."""
    x = inputs(2, 4, 2, 500, d, 3, (131, 400))
    kw = dict(causal=True, window=(90, 0), sinks=6)
    clean = run(x, **kw)
    for b, n in enumerate((131, 400)):
        x["k"][b, :, n:] = float("nan")
        x["v"][b, :, n::2] = float("inf")
        x["v"][b, :, n + 1::2] = float("nan")
    dirty = run(x, **kw)
    for name in ("o", "lse", "dk", "dv"):
        assert torch.equal(clean[name], dirty[name]), name
    compare(x, dirty, **kw)
    for b, n in enumerate((131, 400)):
        assert not dirty["dk"][b, :, n:].any() and not dirty["dv"][b, :, n:].any()


@pytest.mark.parametrize("d", [64, 128, 256])
def test_without_sinks_the_window_alone(d):
    """No sinks through the same entry points: the window's attention (the
    kernels may cut a row's keys in other places than fa_fwd_v's, so both are
    held to the definition, not to each other's bits)."""
    x = inputs(1, 4, 2, 600, d, 5)
    kw = dict(causal=True, window=(255, 0))
    compare(x, run(x, **kw), **kw)
    B, H, N, _ = x["q"].shape
    o, lse = torch.empty_like(x["q"]), torch.empty(B, H, N, device="cuda")
    fa.fa_fwd_sinks(x["q"], x["k"], x["v"], o, lse, d ** -0.5, 0, True, None, (255, 0))
    dq, dk, dv = torch.empty_like(o), torch.empty_like(x["k"]), torch.empty_like(x["v"])
    ws = fa.sinks_workspace(B, H, N, d, "cuda")
    fa.fa_bwd_sinks(x["q"], x["k"], x["v"], o, x["do"], lse, dq, dk, dv, d ** -0.5, 0, True, None,
                    (255, 0), ws)
    fa.fa_check()
    compare(x, dict(o=o, lse=lse, dq=dq, dk=dk, dv=dv), **kw)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_repeats_and_ignores_the_workspace(d):
    """O, LSE, dK and dV repeat bit for bit whatever the workspace holds."""
    x = inputs(1, 4, 1, 1300, d, 7)
    kw = dict(causal=True, window=(70, 0), sinks=4)
    first = run(x, **kw)
    ws = fa.sinks_workspace(1, 4, 1300, d, "cuda")
    for fill in (0, 255):
        ws.fill_(fill)
        o, lse = fa.forward(x["q"], x["k"], x["v"], **kw)
        dq, dk, dv = fa.backward(x["q"], x["k"], x["v"], o, lse, x["do"], ws=ws, **kw)
        fa.fa_check()
        for name, t in dict(o=o, lse=lse, dk=dk, dv=dv).items():
            assert torch.equal(first[name], t), name
        assert torch.isfinite(dq).all()


def test_outputs_inside_guards():
    """Every output element is written and nothing beside it."""
    x = inputs(2, 2, 1, 333, 128, 9, (333, 0))
    scale, kw = 128 ** -0.5, dict(causal=True, kv_len=x["kv_len"], window=(20, 0))
    shapes = dict(o=(2, 2, 333, 128), dq=(2, 2, 333, 128), dk=(2, 1, 333, 128), dv=(2, 1, 333, 128))
    bufs, t = {}, {}
    for n, s in shapes.items():
        size = torch.Size(s).numel()
        bufs[n] = torch.full((size + 256,), float("nan"), dtype=torch.bfloat16, device="cuda")
        t[n] = bufs[n][128:128 + size].view(s)
    lse = torch.full((2, 2, 333), float("nan"), device="cuda")
    ws = fa.sinks_workspace(2, 2, 333, 128, "cuda")
    guarded = torch.full((ws.numel() + 512,), 255, dtype=torch.uint8, device="cuda")
    ws = guarded[256:256 + ws.numel()]
    fa.fa_fwd_sinks(x["q"], x["k"], x["v"], t["o"], lse, scale, 3, **kw)
    fa.fa_bwd_sinks(x["q"], x["k"], x["v"], t["o"], x["do"], lse, t["dq"], t["dk"], t["dv"], scale,
                    3, workspace=ws, **kw)
    fa.fa_check()
    assert not torch.isnan(lse).any()
    for n, b in bufs.items():
        assert torch.isnan(b[:128]).all() and torch.isnan(b[-128:]).all(), n
        assert not torch.isnan(t[n]).any(), n
    assert (guarded[:256] == 255).all() and (guarded[-256:] == 255).all()


def test_captured_and_replayed_on_another_stream():
    """Forward and backward captured into a graph follow new inputs."""
    x = inputs(1, 2, 1, 800, 64, 11)
    kw = dict(causal=True, window=(100, 0), sinks=4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run(x, **kw)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = fa.forward(x["q"], x["k"], x["v"], **kw)
        dq, dk, dv = fa.backward(x["q"], x["k"], x["v"], o, lse, x["do"], **kw)
    y = inputs(1, 2, 1, 800, 64, 12)
    for n in ("q", "k", "v", "do"):
        x[n].copy_(y[n])
    graph.replay()
    torch.cuda.synchronize()
    compare(x, dict(o=o, lse=lse, dq=dq, dk=dk, dv=dv), **kw)


def test_on_a_given_stream():
    """stream= runs there, with outputs and workspace allocated for it, while
    the current stream allocates and overwrites what was freed."""
    x = inputs(1, 4, 2, 900, 128, 13)
    kw = dict(causal=True, window=(100, 0), sinks=4)
    here = run(x, **kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        o, lse = fa.forward(x["q"], x["k"], x["v"], stream=s, **kw)
        grads = fa.backward(x["q"], x["k"], x["v"], o, lse, x["do"], stream=s, **kw)
        junk = torch.full((64 << 20,), 7, dtype=torch.uint8, device="cuda")
        del junk
    s.synchronize()
    assert torch.equal(o, here["o"]) and torch.equal(lse, here["lse"])
    assert torch.equal(grads[1], here["dk"]) and torch.equal(grads[2], here["dv"])


def test_sinks_past_the_sequence():
    """More sinks than tokens, at the largest count."""
    x = inputs(1, 2, 1, 200, 64, 14, (150,))
    kw = dict(causal=True, window=(10, 0), sinks=(1 << 31) - 1)
    compare(x, run(x, **kw), **kw)


def test_sinks_past_32_bits():
    q, k, v, do = (torch.randn(1, 2, 200, 64, device="cuda").to(torch.bfloat16) for _ in range(4))
    kw = dict(causal=True, window=(20, 0))
    o, lse = fa.forward(q, k, v, sinks=200, **kw)
    o2, lse2 = fa.forward(q, k, v, sinks=1 << 32, **kw)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    o2, lse2 = fa.forward(q, k, v, causal=True, window=((1 << 32) + 20, 0), sinks=4)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    a = fa.backward(q, k, v, o, lse, do, sinks=200, **kw)
    b = fa.backward(q, k, v, o, lse, do, sinks=1 << 32, **kw)
    assert torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])


def test_two_backwards_at_once():
    """On two streams, each with a workspace of its own: dK and dV as alone."""
    args = []
    for seed, (B, H, h_kv, N, d) in enumerate(((2, 8, 2, 1500, 128), (2, 8, 8, 1900, 64))):
        torch.manual_seed(seed)
        q, k, v, do = (torch.randn(B, h, N, d, device="cuda").to(torch.bfloat16)
                       for h in (H, h_kv, h_kv, H))
        kw = dict(causal=True, window=(200, 0), sinks=5)
        o, lse = fa.forward(q, k, v, **kw)
        args.append(((q, k, v, o, lse, do), kw))
    alone = [fa.backward(*a, **kw) for a, kw in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in args]
    both = [fa.backward(*a, stream=s, **kw) for _ in range(10)
            for (a, kw), s in zip(args, streams)]
    torch.cuda.synchronize()
    fa.fa_check()
    for i, grads in enumerate(both):
        assert torch.equal(grads[1], alone[i % 2][1]) and torch.equal(grads[2], alone[i % 2][2])


@pytest.mark.parametrize("B,H,h_kv,N,d,window,sinks,kv", [
    # (K/V heads times key blocks without sinks, twice that at d = 256, against
    # two rounds of 152 CTAs)
    (3, 16, 16, 1000, 64, (700, 0), 9, None),              # 336: the second round turned
    (3, 16, 16, 1000, 128, (700, 0), 9, (1000, 800, 977)),
    (2, 12, 12, 1000, 256, (700, 0), 9, None),             # 168 blocks, 336 items
    (4, 32, 16, 1500, 64, (90, 0), 4, None),               # 704, short windows: not turned
    (4, 32, 16, 1500, 128, (90, 0), 4, (1500, 1499, 700, 3)),
    (2, 24, 12, 2000, 256, (60, 0), 200, (2000, 1777)),    # 336 blocks behind two of sinks
    (1, 2, 1, 4500, 128, (1000, 0), 4, None),              # a long row, one K/V head
    (1, 2, 1, 4500, 64, (3000, 0), 130, None),
])
def test_several_rounds_under_a_window(B, H, h_kv, N, d, window, sinks, kv):
    """The backward's whole rounds of items, the turned ones among them, beside
    the pool of cut ones."""
    x = inputs(B, H, h_kv, N, d, N + d + sinks + 1, kv)
    kw = dict(causal=True, window=window, sinks=sinks)
    compare(x, run(x, **kw), **kw)
