"""Host-side checks of rotary positions and of chunks over the paged cache (no
GPU needed): bad arguments get their status before the device is touched, the
binding's structures are the header's, the wrappers refuse what they
document."""
import ctypes
import math
import os
import shutil
import subprocess
from fractions import Fraction

import numpy as np
import pytest
import torch

import rope_ref as P
from exact_attention_04_gb300 import build as fabuild
from exact_attention_04_gb300 import fa, paged, rope
from test_abi_paged import BAD, BIG, OK, POOL_ERRORS, UNSUPPORTED, WS, pool

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    fabuild.build()
    return fa.load()


@pytest.mark.parametrize("struct,name", [(fa.FaStrided, "fa_strided_t"),
                                         (fa.FaRotary, "fa_rotary_t")])
def test_structure_layouts_match_the_header(tmp_path, struct, name):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    names = [n for n, _ in struct._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "fa.h"\nint main(void) {\n'
                   f'printf("%zu", sizeof({name}));\n'
                   + "".join(f'printf(" %zu", offsetof({name}, {n}));\n' for n in names)
                   + "return 0; }\n")
    exe = tmp_path / "layout"
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True,
                                          text=True).stdout.split()]
    assert got == [ctypes.sizeof(struct)] + [getattr(struct, n).offset for n in names]


APART = OK + (1 << 20)


def strided(p=OK, b=1 << 16, h=1 << 10, t=64):
    return ctypes.byref(fa.FaStrided(p, b, h, t))


def rotary(turns=OK, magnitude=1.0, dims=64, interleaved=0):
    return ctypes.byref(fa.FaRotary(turns, magnitude, dims, interleaved))


def rotate(lib, q=None, qo=None, H=4, k=None, ko=None, h_kv=2, B=2, N=16, d=64, start=0, pos=0,
           rot=None):
    return lib.fa_rotate(q or strided(), qo or strided(), H, k or strided(APART),
                         ko or strided(APART), h_kv, B, N, d, start or None, pos or None,
                         rot or rotary(), 0, None)


# views that a written tensor of [2, 4, 16, 64] may not have, and no tensor may
SHARED = [dict(b=0), dict(h=0), dict(t=0), dict(t=56), dict(h=1016), dict(b=4096 - 8)]
NO_VIEW = [dict(p=0), dict(p=OK + 8), dict(b=4), dict(h=1 << 10 | 4), dict(t=68), dict(t=-64),
           dict(b=1 << 62), dict(t=1 << 60)]


def test_rotate_errors(lib):
    for change in NO_VIEW:
        for name in ("q", "qo", "k", "ko"):
            assert rotate(lib, **{name: strided(**change)}) == BAD, (change, name)
    for change in SHARED:
        assert rotate(lib, qo=strided(**change)) == BAD, change
        # of two K/V heads
        assert rotate(lib, ko=strided(**{**change, **({"b": 2048 - 8} if change.get("b") else {})})
                      ) == BAD, change
    for d in (0, 32, 96, 512):
        assert rotate(lib, d=d) == UNSUPPORTED
    for bad in (dict(turns=0), dict(turns=OK + 4), dict(dims=0), dict(dims=63), dict(dims=66),
                dict(dims=-2), dict(magnitude=math.inf), dict(magnitude=math.nan)):
        assert rotate(lib, rot=rotary(**bad)) == BAD, bad
    for bad in (dict(B=0), dict(N=0), dict(H=0), dict(h_kv=-1), dict(H=65535), dict(N=1 << 30),
                dict(start=OK, pos=OK), dict(start=OK + 2), dict(pos=OK + 1)):
        assert rotate(lib, **bad) == BAD, bad
    # one tensor as queries and keys, turned in place, and other outputs on inputs
    assert rotate(lib, k=strided(), ko=strided()) == BAD
    assert rotate(lib, qo=strided(APART), ko=strided(APART + 4096)) == BAD
    assert rotate(lib, k=strided(), qo=strided(APART), ko=strided(APART)) == BAD
    assert rotate(lib, qo=strided(APART + 4096), ko=strided()) == BAD
    assert lib.fa_rotate(None, strided(), 4, None, None, 0, 2, 16, 64, None, None, rotary(), 0,
                         None) == BAD
    assert lib.fa_rotate(strided(), strided(), 4, None, None, 2, 2, 16, 64, None, None, rotary(),
                         0, None) == BAD
    assert lib.fa_rotate(strided(), strided(), 4, None, None, 0, 2, 16, 64, None, None, None, 0,
                         None) == BAD


def test_in_place_is_at_the_same_strides(lib):
    """An output at its input's address that sees it through other strides
    would overwrite what is still to be read; of axes of one strides do not
    count."""
    others = dict(b=1 << 17), dict(h=1 << 11), dict(h=64, t=256)
    for change in others:
        assert rotate(lib, qo=strided(**change)) == BAD, change
        assert rotate(lib, k=strided(APART), ko=strided(APART, **change)) == BAD, change
        assert append(lib, qo=strided(**change)) == BAD, change
    if torch.cuda.is_available():
        return
    # taken: without a GPU a call gets as far as the device
    for change in others:
        assert rotate(lib, qo=strided(3 * APART, **change)) not in (fa.FA_OK, BAD), change
        assert rotate(lib, ko=strided(3 * APART, **change)) not in (fa.FA_OK, BAD), change
        assert append(lib, qo=strided(3 * APART, **change)) not in (fa.FA_OK, BAD), change
    for call in (rotate, append):
        for kw in (dict(), dict(B=1, qo=strided(b=8)), dict(N=1, qo=strided(t=4))):
            assert call(lib, **kw) not in (fa.FA_OK, BAD), kw


def append(lib, cache=None, q=None, qo=None, H=4, k=None, v=None, layer=0, table=OK, most=4,
           start=OK, kv_len=OK, offsets=0, B=2, N=16, rot=None):
    return lib.fa_paged_append_rotated(
        q or strided(), qo or strided(), H, k or strided(APART), v or strided(2 * APART - OK),
        cache or pool(), layer,
        table, most, start, kv_len, offsets or None, B, N, rot or rotary(), None)


def test_append_rotated_errors(lib):
    for change, status in POOL_ERRORS:
        assert append(lib, cache=pool(**change)) == status, change
    for change in NO_VIEW:
        for name in ("q", "qo", "k", "v"):
            assert append(lib, **{name: strided(**change)}) == BAD, (change, name)
    for change in SHARED:
        assert append(lib, qo=strided(**change)) == BAD, change
    # queries on top of the keys or the values that are read
    assert append(lib, k=strided()) == BAD and append(lib, v=strided()) == BAD
    for bad in (dict(layer=-1), dict(layer=2), dict(table=0), dict(table=OK + 2), dict(most=0),
                dict(most=1 << 26), dict(start=0), dict(kv_len=0), dict(start=OK + 2),
                dict(kv_len=OK + 1), dict(offsets=OK + 2), dict(B=0), dict(N=0), dict(H=-1),
                dict(H=65535), dict(N=1 << 30), dict(rot=rotary(dims=65)), dict(rot=rotary(dims=66)),
                dict(B=1 << 20, N=1 << 12)):
        assert append(lib, **bad) == BAD, bad


def prefill(lib, q=None, cache=None, layer=0, table=OK, most=4, start=OK, kv_len=OK, offsets=0,
            o=None, lse=OK, B=2, H=4, N=16, scale=0.1, left=-1, right=-1, sinks=0, ws=WS,
            nbytes=BIG):
    return lib.fa_prefill_paged(q or strided(), cache or pool(), layer, table, most, start, kv_len,
                                offsets or None, o or strided(APART), lse, B, H, N, scale, 1, left,
                                right, sinks, ws, nbytes, None)


def test_prefill_errors(lib):
    for change, status in POOL_ERRORS:
        assert prefill(lib, cache=pool(**change)) == status, change
    assert prefill(lib, o=strided()) == BAD              # over the queries
    for change in NO_VIEW + SHARED:
        for name in ("q", "o"):
            assert prefill(lib, **{name: strided(**change)}) == BAD, (change, name)
    for bad in (dict(layer=-1), dict(layer=2), dict(table=0), dict(table=OK + 2), dict(most=0),
                dict(most=1 << 26), dict(start=0), dict(kv_len=0), dict(start=OK + 2),
                dict(kv_len=OK + 1), dict(offsets=OK + 2), dict(lse=0), dict(lse=OK + 2),
                dict(B=0), dict(N=0), dict(H=0), dict(H=6), dict(N=1 << 30), dict(scale=0.0),
                dict(scale=-1.0), dict(scale=math.inf), dict(scale=math.nan), dict(left=-2),
                dict(right=-2), dict(sinks=-1), dict(ws=0), dict(ws=WS + 128),
                dict(B=1 << 21, N=1 << 12), dict(B=1 << 30, offsets=OK)):
        assert prefill(lib, **bad) == BAD, bad


def test_workspace_sizes(lib):
    size = lib.fa_prefill_paged_workspace_bytes
    assert size(1, 8, 1, 2, 64, 0) > 0 and size(1, 8, 1, 2, 64, 1) > 0
    for bad in ((0, 8, 1, 2, 64, 0), (1, 0, 1, 2, 64, 0), (1, 8, 0, 2, 64, 0), (1, 8, 1, 3, 64, 0),
                (1, 8, 1, 0, 64, 0), (1, 8, 1, 2, 96, 0), (1, 8, 1 << 30, 2, 64, 1),
                (1 << 29, 8, 1, 2, 64, 0), (1 << 20, 8, 1 << 12, 2, 64, 0)):
        assert size(*bad) == 0, bad
    # a bounded number of partial outputs whatever the tokens
    assert size(1, 32, 1 << 20, 8, 128, 1) < 1 << 28


def test_frequencies():
    w, m = rope.frequencies(64)
    assert m == 1.0 and w[0] == 1.0 and np.allclose(w, [10000.0 ** (-i / 32) for i in range(32)],
                                                    rtol=1e-15)
    assert np.allclose(rope.frequencies(64, scaling=("linear", 8))[0], w / 8, rtol=1e-15)
    ntk = rope.frequencies(64, scaling=("ntk", 8))[0]
    assert ntk[0] == 1.0 and abs(ntk[-1] * 8 / w[-1] - 1) < 1e-12
    assert np.array_equal(rope.frequencies(2, scaling=("ntk", 8))[0], [1.0])
    parts, m = rope.frequencies(64, scaling=("by_parts", 8, 4096))
    turns = 4096 * w / (2 * np.pi)
    assert abs(m - (0.1 * math.log(8) + 1)) < 1e-15
    # pairs beyond the borders, which lie on whole pairs
    assert np.array_equal(parts[turns > 32 * 1.4], w[turns > 32 * 1.4])
    assert np.allclose(parts[turns < 1 / 1.4], w[turns < 1 / 1.4] / 8, rtol=1e-15)
    assert (np.diff(parts / w) <= 1e-15).all()
    assert rope.frequencies(64, scaling=("by_parts", 0.5, 4096))[1] == 1.0
    for bad in (dict(dims=0), dict(dims=7), dict(dims=64, base=1.0),
                dict(dims=64, scaling=("other", 2.0)), dict(dims=64, scaling=("linear",)),
                dict(dims=64, scaling=("linear", 0.0)), dict(dims=64, scaling=("linear", math.nan)),
                dict(dims=64, scaling=("by_parts", 2.0)),
                dict(dims=64, scaling=("by_parts", 2.0, 100.0, 32.0))):
        with pytest.raises(ValueError):
            rope.frequencies(**bad)


def test_turns():
    """Half a turn, a whole one, negative angles, and an angle in 64 bits."""
    got = [int(t) for t in rope.turns_of([0.0, math.pi, -math.pi / 2, 1.0])]
    eps = 2 ** 64 * 2 ** -52                              # of pi in double precision
    assert got[0] == 0 and abs(got[1] - 2 ** 63) < eps and abs(got[2] - 3 * 2 ** 62) < eps
    two_pi = 2 * Fraction("3.141592653589793238462643383279502884197")
    assert abs(Fraction(got[3], 2 ** 64) - 1 / two_pi) < Fraction(1, 2 ** 63)
    for bad in (math.inf, math.nan):
        with pytest.raises(ValueError):
            rope.turns_of([bad])


def test_the_angle_in_fp32():
    """A 64-bit fraction of a turn as the kernels take it, the upper 32 bits as
    a float of half turns: within 2^-26 + 2^-32 turns, at the borders between
    floats and next to half a turn above all, where it is more than 2^-32 off;
    and no more than the plain turn's bound leaves for it."""
    rng = np.random.default_rng(0)
    whole = rng.integers(0, 1 << 64, 200000, dtype=np.uint64)
    near = [(sign * (1 << b) + e) % (1 << 64) for b in range(32, 64) for sign in (1, -1)
            for e in (-(1 << 39), -(1 << 38) - 1, -(1 << 33), -1, 0, 1, (1 << 38) + 1, (1 << 39))]
    most = 0
    for a in [int(x) for x in whole] + near + [(1 << 63) - 1, 1 << 63, (1 << 64) - 1]:
        top = (a >> 32) - (1 << 32) * (a >> 63)          # the upper half as a signed int
        half_turns = Fraction(float(np.float32(top))) / (1 << 31)
        assert -1 <= half_turns <= 1
        off = abs(half_turns / 2 - Fraction(a - (1 << 64) * (a >> 63), 1 << 64))
        most = max(most, off)
        assert off < Fraction(1, 1 << 26) + Fraction(1, 1 << 32)
    assert most > Fraction(1, 1 << 32) * 32
    # rope_ref's 2^-20 of (|a| + |b|) m: this, 2 units of sine and cosine below
    # one, and 3 roundings of the products and their sum
    assert 2 * math.pi * (2.0 ** -26 + 2.0 ** -32) + 2 * 2.0 ** -24 + 3 * 2.0 ** -24 < 2.0 ** -21


def test_rotary_refuses():
    for bad in (dict(d=96), dict(d=64, dims=66), dict(d=64, dims=0), dict(d=64, dims=7),
                dict(d=64, freqs=np.ones(31)), dict(d=64, magnitude=math.inf),
                dict(d=64, freqs=np.ones(32), scaling=("linear", 2.0))):
        with pytest.raises(ValueError):
            rope.Rotary(device="cpu", **bad)
    r = rope.Rotary(128, 64, interleaved=True, scaling=("by_parts", 4.0, 2048), device="cpu")
    assert (r.struct.dims, r.struct.interleaved, r.turns.shape) == (64, 1, (32,))
    assert r.magnitude == rope.frequencies(64, scaling=("by_parts", 4.0, 2048))[1]


def test_wrappers_refuse_what_is_not_on_the_gpu():
    r = rope.Rotary(64, device="cpu")
    x = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        rope.rotate(x, x, r)
    with pytest.raises(ValueError):
        rope.view("q", x.float(), x.shape, -1)
    with pytest.raises(ValueError):
        rope.view("q", x, (1, 2, 4, 64), -1)
    with pytest.raises(ValueError):
        rope.view("q", torch.zeros(1, 2, 3, 72, dtype=torch.bfloat16)[..., 4:68], x.shape, -1)
    with pytest.raises(ValueError):
        rope.view("q", torch.zeros(1, 2, 3, 65, dtype=torch.bfloat16)[..., :64], x.shape, -1)
    with pytest.raises(ValueError):
        rope.view("q", x.transpose(2, 3).contiguous().transpose(2, 3), x.shape, -1)
    def unpacked(b):
        assert len(b) == ctypes.sizeof(fa.FaStrided)
        return fa.FaStrided.from_buffer_copy(b)

    v = unpacked(rope.view("q", x.transpose(1, 2).contiguous().transpose(1, 2), x.shape, -1))
    assert (v.batch_stride, v.head_stride, v.token_stride) == (384, 64, 128)
    o, v = rope.out_like(x.transpose(1, 2).contiguous().transpose(1, 2))
    v = unpacked(v)
    assert o.stride() == (384, 64, 128, 1) and v.p == o.data_ptr()
    assert (v.batch_stride, v.head_stride, v.token_stride) == (384, 64, 128)
    wide = torch.zeros(1, 3, 4, 72, dtype=torch.bfloat16)[:, :, :2, :64].transpose(1, 2)
    assert unpacked(rope.view("q", wide, wide.shape, -1)).token_stride == 288
    o, _ = rope.out_like(wide)
    assert o.transpose(1, 2).is_contiguous() or o.is_contiguous()
    with pytest.raises(ValueError):
        rope.view("q", torch.zeros(2, 2, 3 * 64 + 4, dtype=torch.bfloat16)[:, :, :192].view(
            2, 2, 3, 64), (2, 2, 3, 64), -1)
    with pytest.raises(ValueError):
        rope.ints("pos", torch.zeros(3), (3,), -1)
    assert rope.ints("pos", None, (3,), -1) is None


def test_the_plain_turn():
    """rope_ref against a product of complex numbers, a pair at a time."""
    r = rope.Rotary(64, 10, interleaved=True, scaling=("linear", 3.0), magnitude=1.5, device="cpu")
    h = rope.Rotary(64, 10, scaling=("linear", 3.0), magnitude=1.5, device="cpu")
    x = torch.randn(2, 3, 64, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16)
    pos = np.array([[0, 7, -3], [1000, 123456, 2]])
    for rot, at in ((r, lambda i: (2 * i, 2 * i + 1)), (h, lambda i: (i, i + 5))):
        for back in (False, True):
            y, bound = P.turn(x, pos, rot, back)
            for b in range(2):
                for t in range(3):
                    for i in range(5):
                        a, c = at(i)
                        w = 10000.0 ** (-i / 5) / 3 * pos[b, t] * (-1 if back else 1)
                        z = complex(float(x[b, t, a]), float(x[b, t, c])) * 1.5 * \
                            complex(math.cos(w), math.sin(w))
                        assert abs(complex(float(y[b, t, a]), float(y[b, t, c])) - z) < 1e-9
            assert torch.equal(y[..., 10:], x[..., 10:].double()) and not bound[..., 10:].any()


def test_the_plain_prefill_of_one_token_is_decode_s():
    import paged_ref as R
    rng = np.random.default_rng(1)
    table, kv_len, _ = R.random_cache(rng, 3, 9, 4, 30, [30, 1, 0], missing=0.1)
    table, kv_len = torch.from_numpy(table), torch.from_numpy(kv_len)
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(1, 30, 2, 4, 8, generator=g) for _ in range(2))
    q = torch.randn(3, 4, 1, 8, generator=g)
    for window, sinks in ((None, 0), ((5, 0), 2)):
        a = P.prefill(q, k, v, 0, table, kv_len - 1, kv_len, window=window, sinks=sinks)
        b = R.decode(q, k, v, 0, table, kv_len, None, window, sinks)
        for n in ("o", "lse"):
            assert torch.equal(torch.isneginf(a[n]), torch.isneginf(b[n]))
            assert (torch.nan_to_num(a[n]) - torch.nan_to_num(b[n])).abs().max() < 1e-12


def test_the_plain_prefill_of_a_prompt_is_attention_s():
    import paged_ref as R
    g = torch.Generator().manual_seed(2)
    q, k, v = (torch.randn(2, h, 20, 8, generator=g) for h in (4, 2, 2))
    for window, sinks, causal in ((None, 0, True), ((3, 0), 2, True), ((4, 2), 0, False)):
        a = R.attention(q, k, v, causal=causal, window=window, sinks=sinks)
        b = P.prefill(q, k[None], v[None], 0, torch.tensor([[0], [1]]), [0, 0], [20, 20],
                      causal=causal, window=window, sinks=sinks)
        for n in ("o", "lse"):
            assert (a[n] - b[n]).abs().max() < 1e-12
