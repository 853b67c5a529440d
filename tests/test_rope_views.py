"""Which tensors the binding of rotary positions and chunks takes, and the
outputs that it lays out like them (no GPU needed)."""
import pytest
import torch

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
