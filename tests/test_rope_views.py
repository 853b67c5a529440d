"""Which tensors the binding of rotary positions and chunks takes, and the
outputs that it lays out like them."""
import random

import pytest
import torch

from exact_attention_04_gb300 import build as fabuild
from exact_attention_04_gb300 import fa, rope


def strides(packed):
    s = fa.FaStrided.from_buffer_copy(packed)
    return s.batch_stride, s.head_stride, s.token_stride


def zeros(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def test_an_expanded_last_axis_is_refused():
    """d values that are one, whatever the other strides: an axis of one may
    have a stride of one."""
    for x in (zeros(4, 1, 1, 1).expand(4, 2, 1, 64), zeros(4, 1, 64)[..., :1].unsqueeze(2).expand(
            4, 2, 1, 64), zeros(4, 16)[:, None, None, :1].expand(4, 2, 1, 64),
              zeros(1 << 12).as_strided((4, 2, 1, 64), (16, 8, 1, 0))):
        with pytest.raises(ValueError, match="contiguous"):
            rope.view("q", x, x.shape, -1)


@pytest.mark.parametrize("axis", [0, 1, 2])
@pytest.mark.parametrize("odd", [1, 2, 3, 7])
def test_strides_off_the_eights_are_refused(axis, odd):
    """Of axes that are longer than one; of others they do not count."""
    st = [4096, 1024, 64]
    st[axis] += odd
    x = zeros(1 << 15).as_strided((2, 2, 2, 64), (*st, 1))
    with pytest.raises(ValueError, match="multiples of 8"):
        rope.view("q", x, x.shape, -1)
    shape = [2, 2, 2, 64]
    shape[axis] = 1
    x = zeros(1 << 15).as_strided(shape, (*st, 1))
    assert strides(rope.view("q", x, x.shape, -1)) == tuple(st)


def test_outputs_are_dense_with_d_contiguous():
    """Whatever input is taken: expanded axes, slices, axes of one with any
    stride."""
    rng = random.Random(0)
    base, taken = zeros(1 << 14), 0
    for _ in range(20000):
        n = [rng.choice([1, 1, 2, 3]) for _ in range(3)]
        st = [rng.choice([0, 1, 2, 8, 16, 64, 64 * n[2], 64 * n[1], 64 * n[1] * n[2], 72, 72 * n[1],
                          72 * n[2]]) for _ in range(3)]
        x = base.as_strided((*n, 64), (*st, 1))
        try:
            rope.view("q", x, x.shape, -1)
        except ValueError:
            continue
        taken += 1
        o, packed = rope.out_like(x)
        assert o.shape == x.shape and o.dtype == x.dtype and o.stride(3) == 1, (x.shape, st)
        assert strides(packed) == o.stride()[:3]
        extent = 64
        for s, m in sorted((s, m) for s, m in zip(o.stride(), n) if m > 1):
            assert s == extent, (x.shape, st, o.stride())
            extent *= m
    assert taken > 5000


def test_expanded_tokens_of_one_head():
    """One token's queries for all, of a tensor whose head axis came last."""
    x = zeros(2, 64, 1).permute(0, 2, 1)[:, :, None].expand(2, 1, 5, 64)
    rope.view("q", x, x.shape, -1)
    o, _ = rope.out_like(x)
    assert o.is_contiguous()


@pytest.mark.gpu
def test_expanded_inputs_turn_as_their_copies():
    fabuild.build()
    rotary = rope.Rotary(64)
    g = torch.Generator().manual_seed(0)
    x = torch.randn(2, 64, 1, generator=g).to(torch.bfloat16).cuda().permute(0, 2, 1)
    k = torch.randn(2, 1, 5, 64, generator=g).to(torch.bfloat16).cuda()
    for q, kk in ((x[:, :, None].expand(2, 1, 5, 64), k.expand(2, 3, 5, 64)),
                  (k[:1].expand(2, 1, 5, 64), k[:, :, :1].expand(2, 1, 5, 64))):
        for call in (rope.rotate, rope.rotate_back):
            got = call(q, kk, rotary)
            want = call(q.contiguous(), kk.contiguous(), rotary)
            assert all(torch.equal(a, b) for a, b in zip(got, want))
