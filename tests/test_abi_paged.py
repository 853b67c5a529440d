"""Host-side checks of the entry points for sinks and the paged cache (no GPU
needed): bad arguments get their status before the device is touched, the
binding's structure is the header's, the wrappers refuse what they document."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

from exact_attention_04_gb300 import build as fabuild
from exact_attention_04_gb300 import fa, paged

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK = 0x1000
WS = 0x100000
BIG = 1 << 40
BAD, UNSUPPORTED = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    fabuild.build()
    return fa.load()


def pool(**kw):
    f = dict(k=OK, v=OK, layer_stride=1 << 20, page_stride=4096, head_stride=1024,
             token_stride=64, num_layers=2, num_pages=50, page_size=16, h_kv=4, d=64)
    f.update(kw)
    return ctypes.byref(fa.FaPagedKV(**f))


def test_structure_layout_matches_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    names = [n for n, _ in fa.FaPagedKV._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "fa.h"\nint main(void) {\n'
                   'printf("%zu", sizeof(fa_paged_kv_t));\n'
                   + "".join(f'printf(" %zu", offsetof(fa_paged_kv_t, {n}));\n' for n in names)
                   + "return 0; }\n")
    exe = tmp_path / "layout"
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True,
                                          text=True).stdout.split()]
    assert got == [ctypes.sizeof(fa.FaPagedKV)] + [getattr(fa.FaPagedKV, n).offset for n in names]


POOL_ERRORS = [
    (dict(k=0), BAD), (dict(v=0), BAD), (dict(k=OK + 8), BAD), (dict(d=96), UNSUPPORTED),
    (dict(num_layers=0), BAD), (dict(num_pages=0), BAD), (dict(page_size=0), BAD),
    (dict(h_kv=0), BAD), (dict(page_stride=4), BAD), (dict(token_stride=-64), BAD),
    (dict(page_size=1 << 30), BAD),
]


@pytest.mark.parametrize("change,status", POOL_ERRORS)
def test_pool_errors(lib, change, status):
    p = pool(**change)
    assert lib.fa_decode_paged(OK, p, 0, OK, 4, OK, OK, OK, 2, 8, 0.1, -1, 0, WS, BIG,
                               None) == status
    assert lib.fa_paged_append(OK, OK, p, 0, OK, 4, OK, OK, 2, 1, None) == status
    assert lib.fa_pages_fork(p, OK, 4, OK, OK, 2, OK, 2, OK + 8, OK + 8, OK + 8, OK, WS, BIG,
                             None) == status
    assert lib.fa_pages_compact(p, OK, 4, OK, 2, OK, OK, OK, WS, BIG, None) == status


@pytest.mark.parametrize("change", [
    dict(head_stride=0), dict(token_stride=0), dict(page_stride=0), dict(layer_stride=0),
    dict(token_stride=56), dict(head_stride=1016), dict(page_stride=4096 - 8),
    dict(layer_stride=50 * 4096 - 8),
    dict(head_stride=64, token_stride=4 * 64 - 8),         # heads within a token
    dict(page_stride=64, token_stride=50 * 64 - 8, head_stride=1 << 16),
    dict(layer_stride=1 << 62), dict(page_stride=1 << 62), dict(layer_stride=(1 << 63) - 8)])
def test_pools_whose_values_share_a_place(lib, change):
    """Two pages, heads, slots or layers in one place (writing one would destroy
    the other), and strides past every address."""
    p = pool(**change)
    assert lib.fa_decode_paged(OK, p, 0, OK, 4, OK, OK, OK, 2, 8, 0.1, -1, 0, WS, BIG, None) == BAD
    assert lib.fa_paged_append(OK, OK, p, 0, OK, 4, OK, OK, 2, 1, None) == BAD
    assert lib.fa_pages_fork(p, OK, 4, OK, OK, 2, OK, 2, OK + 8, OK + 8, OK + 8, OK, WS, BIG,
                             None) == BAD
    assert lib.fa_pages_compact(p, OK, 4, OK, 2, OK, OK, OK, WS, BIG, None) == BAD


def test_which_pools_share_a_place():
    """PagedKV's own check: views of one pool keep apart, expanded and
    overlapping ones do not."""
    t = torch.zeros(2, 5, 4, 16, 64)                       # layers, pages, heads, slots, d
    both = torch.zeros(2, 5, 2, 16, 4, 64)                 # K and V of a page side by side
    for x in (t, t.transpose(2, 3), t[:, 1::2], t[:, :, 1:3, ::4], t[:1, :1, :1, :1],
              t.permute(1, 3, 0, 2, 4), both[:, :, 0].transpose(2, 3)):
        assert paged._apart(x.shape, x.stride())
    flat = torch.zeros(10000)
    for x in (t[:, :, :1].expand(2, 5, 4, 16, 64), t[:1].expand(2, 5, 4, 16, 64),
              flat.as_strided((1, 3, 2, 4, 64), (0, 504, 256, 64, 1)),
              flat.as_strided((1, 1, 2, 4, 64), (0, 0, 248, 64, 1)),
              flat.as_strided((1, 1, 1, 4, 64), (0, 0, 0, 32, 1))):
        assert not paged._apart(x.shape, x.stride())


def test_decode_errors(lib):
    def call(q=OK, layer=0, table=OK, most=4, kv=OK, o=OK, lse=OK, B=2, H=8, scale=0.1, left=-1,
             sinks=0, ws=WS, n=BIG, **kw):
        return lib.fa_decode_paged(q, pool(**kw), layer, table, most, kv, o, lse, B, H, scale,
                                   left, sinks, ws, n, None)
    for kw in (dict(q=0), dict(q=OK + 8), dict(table=0), dict(table=OK + 2), dict(kv=0),
               dict(kv=OK + 1), dict(o=0), dict(o=OK + 8), dict(lse=0), dict(lse=OK + 2),
               dict(layer=-1), dict(layer=2), dict(most=0), dict(most=1 << 27), dict(B=0),
               dict(H=0), dict(H=6), dict(scale=0.0), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(scale=-1.0), dict(left=-2), dict(sinks=-1),
               dict(ws=0, most=5000), dict(ws=WS + 16), dict(n=1000, most=5000),
               dict(B=1 << 30)):
        assert call(**kw) == BAD, kw
    assert lib.fa_decode_paged_workspace_bytes(6, 4, 64) == 0
    all_bytes = lib.fa_decode_paged_workspace_bytes(8, 4, 64)
    assert all_bytes > 0
    for args, want in (((4, 2, 8, -1, 0), 0), ((5000, 2, 8, -1, 0), all_bytes),
                       ((5000, 2, 8, 50, 3), 0), ((4, 1000, 8, -1, 0), all_bytes),
                       ((4, 2, 6, -1, 0), 0), ((0, 2, 8, -1, 0), 0)):
        assert lib.fa_decode_paged_call_bytes(pool(), *args) == want, args
    assert lib.fa_decode_paged_workspace_bytes(8, 4, 80) == 0
    assert lib.fa_decode_paged_workspace_bytes(8, 4, 64) % 256 == 0


def test_append_errors(lib):
    def call(k=OK, v=OK, layer=0, table=OK, most=4, start=OK, kv=OK, B=2, n=1):
        return lib.fa_paged_append(k, v, pool(), layer, table, most, start, kv, B, n, None)
    for kw in (dict(k=0), dict(v=OK + 4), dict(layer=-1), dict(layer=2), dict(table=0),
               dict(most=0), dict(start=0), dict(start=OK + 1), dict(kv=0), dict(B=0), dict(n=0),
               dict(n=1 << 30)):
        assert call(**kw) == BAD, kw


def test_metadata_errors(lib):
    def reserve(table=OK, most=4, page=16, kv=OK, n=OK, ref=OK, pages=50, rows=2, out=OK, info=OK,
                ws=WS, size=BIG):
        return lib.fa_pages_reserve(table, most, page, kv, n, ref, pages, rows, out, OK, info, ws,
                                    size, None)
    for kw in (dict(table=0), dict(most=0), dict(page=0), dict(kv=0), dict(n=0), dict(ref=OK + 1),
               dict(pages=0), dict(rows=0), dict(rows=1 << 25), dict(out=0), dict(info=0),
               dict(ws=0), dict(ws=WS + 4), dict(size=100), dict(most=1 << 27),
               dict(most=1 << 20, page=1, rows=1 << 12)):
        assert reserve(**kw) == BAD, kw

    def fork(table=OK, kv=OK, ref=OK, rows=2, parent=OK, new=2, t=OK + 8, n=OK + 8, r=OK + 8,
             info=OK, size=BIG):
        return lib.fa_pages_fork(pool(), table, 4, kv, ref, rows, parent, new, t, n, r, info, WS,
                                 size, None)
    for kw in (dict(table=0), dict(kv=0), dict(ref=0), dict(rows=0), dict(parent=0), dict(new=0),
               dict(t=OK), dict(n=OK), dict(r=OK), dict(info=0), dict(size=100),
               dict(new=1 << 25)):
        assert fork(**kw) == BAD, kw

    def trim(table=OK, most=4, page=16, kv=OK, ref=OK, pages=50, rows=2, left=5, sinks=0, t=OK,
             r=OK):
        return lib.fa_pages_trim(table, most, page, kv, ref, pages, rows, left, sinks, t, r, None)
    for kw in (dict(table=0), dict(most=0), dict(page=0), dict(kv=0), dict(ref=0), dict(pages=0),
               dict(rows=0), dict(left=-1), dict(sinks=-1), dict(t=0), dict(r=0)):
        assert trim(**kw) == BAD, kw

    def compact(table=OK, most=4, ref=OK, rows=2, t=OK, r=OK, info=OK, ws=WS, size=BIG):
        return lib.fa_pages_compact(pool(), table, most, ref, rows, t, r, info, ws, size, None)
    for kw in (dict(table=0), dict(most=0), dict(ref=0), dict(rows=0), dict(t=0), dict(r=0),
               dict(info=0), dict(ws=0), dict(size=100)):
        assert compact(**kw) == BAD, kw
    assert lib.fa_pages_workspace_bytes(0, 1) == 0 and lib.fa_pages_workspace_bytes(1, 0) == 0


def test_sinks_errors(lib):
    mask = fa.FaVariant(2, 5, 0, 0x2000)

    def fwd(q=OK, lse=OK, kv=None, N=128, d=64, scale=0.1, sinks=1, var=fa.FaVariant(2, 5, 0)):
        return lib.fa_fwd_sinks(q, OK, OK, OK, lse, 1, 4, N, d, scale, 1, kv, ctypes.byref(var),
                                sinks, None)

    def bwd(q=OK, lse=OK, kv=None, N=128, d=64, scale=0.1, sinks=1, var=fa.FaVariant(2, 5, 0),
            ws=WS, size=BIG):
        return lib.fa_bwd_sinks(q, OK, OK, OK, OK, lse, OK, OK, OK, 1, 4, N, d, scale, 1, kv,
                                ctypes.byref(var), sinks, ws, size, None)
    for call in (fwd, bwd):
        for kw in (dict(q=0), dict(q=OK + 8), dict(lse=OK + 2), dict(kv=OK + 1), dict(N=0),
                   dict(scale=0.0), dict(sinks=-1), dict(var=fa.FaVariant(3, 5, 0)),
                   dict(var=fa.FaVariant(2, -2, 0))):
            assert call(**kw) == BAD, kw
        assert call(d=96) == UNSUPPORTED
        assert call(var=mask) == UNSUPPORTED
    assert bwd(ws=WS + 16) == BAD and bwd(size=100) == BAD
    # the cut items' pieces count: what fa_bwd needs is too little
    need = lib.fa_bwd_sinks_workspace_bytes(1, 4, 4096, 64)
    assert need > fa.fa_bwd_workspace_bytes(1, 4, 4096, 64)
    assert bwd(N=4096, size=need - 1) == BAD
    for bad in ((1, 4, 64, 96), (1, 4, 0, 64), (0, 4, 64, 64)):
        assert lib.fa_bwd_sinks_workspace_bytes(*bad) == 0


def test_wrappers_refuse():
    """paged's Python checks need no device."""
    k = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        paged.PagedKV(k, k)                                # not on a GPU

    class Fake:                                            # a cache as the checks see it
        index, h_kv, d, num_pages, page_size = 0, 2, 64, 3, 16
    for bad in (torch.zeros(2, 3), torch.zeros(4, dtype=torch.int32)):
        with pytest.raises(ValueError):
            paged._ints("x", bad, torch.Size((2, 3)), 0)
    with pytest.raises(ValueError):
        paged._table(Fake, torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError):
        paged._bytes(torch.zeros(8, dtype=torch.uint8), 4, None)
    q = torch.zeros(1, 1, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fa.forward(q, q, q, window=(2, 0), sinks=1)        # not on a GPU
    with pytest.raises(ValueError):
        fa._check_sinks(q, object())


def test_a_cache_keeps_few_workspace_sizes(lib):
    """A long-lived cache called with ever other sizes holds a bounded number
    of them, and answers as the library does."""
    class Fake:
        ref, num_pages, _need = pool(), 50, {}
    for i in range(3000):
        sizes = (1 + i, 2, 8, i % 7 - 1, i % 5)
        assert paged._call_need(Fake, sizes) == lib.fa_decode_paged_call_bytes(Fake.ref, *sizes)
        assert paged._pages_need(Fake, 1 + i) == lib.fa_pages_workspace_bytes(50, 1 + i)
        assert len(Fake._need) <= 1024


def test_call_bytes_of_the_largest_windows(lib):
    """A window or sinks at the largest int hide nothing: a wide table's call
    needs the workspace that it needs without a window."""
    top = (1 << 31) - 1
    all_bytes = lib.fa_decode_paged_workspace_bytes(8, 4, 64)
    for left, sinks in ((-1, 0), (top, 0), (0, top), (top, top), (top, top - 100), (50, top - 1)):
        assert lib.fa_decode_paged_call_bytes(pool(), 5000, 2, 8, left, sinks) == all_bytes
        assert lib.fa_decode_paged_call_bytes(pool(), 4, 2, 8, left, sinks) == 0
