"""Rotary positions of queries and keys: the turn before attention, and its
gradient after it.

``Rotary`` holds a head's frequencies as the library reads them; ``rotate``
turns q and k in one pass, ``rotate_back`` takes their gradients back::

    rotary = rope.Rotary(d)                               # base 10000, halves, the whole head
    q, k = rope.rotate(q, k, rotary)                      # positions 0, 1, ...
    o, lse = fa.forward(q, k, v, causal=True)
    dq, dk, dv = fa.backward(q, k, v, o, lse, do, causal=True)
    dq, dk = rope.rotate_back(dq, dk, rotary)

Tensors are bf16 [B, H, N, d] with any strides that are multiples of 8
([B, N, H, d] seen through transpose(1, 2), slices of a fused projection);
results are dense, and laid out like a dense input.
Nothing synchronises or copies to the host after the Rotary is made.
paged.append_rotated is the same turn on the way into the paged cache.
"""
import ctypes
import math
import struct
from fractions import Fraction

import numpy as np
import torch

from . import fa

_current_device = torch.cuda.current_device
_current_raw_stream = torch._C._cuda_getCurrentRawStream
_bf16, _int32, _empty_like, _load = torch.bfloat16, torch.int32, torch.empty_like, fa.load
_pack = struct.Struct("Pqqq").pack     # fa_strided_t


def frequencies(dims, base=10000.0, scaling=None):
    """(angles per position of dims / 2 pairs in 64 bits, magnitude).

    w_i = base^(-2 i / dims).  scaling, for contexts longer than the trained
    one:
      ("linear", factor)    w_i / factor
      ("ntk", factor)       base times factor^(dims / (dims - 2)): the slowest
                            pair is slowed by factor, the fastest stays
      ("by_parts", factor, length[, fast, slow])
                            pairs that turn more than `fast` (32) times over
                            the original length stay, those below `slow` (1)
                            turns become w_i / factor, a linear ramp over the
                            pairs lies between; the magnitude is 0.1 ln
                            factor + 1
    """
    if dims < 2 or dims % 2:
        raise ValueError("dims: expected an even number of values")
    if not base > 1:
        raise ValueError("base: expected a number above 1")
    i = np.arange(dims // 2, dtype=np.float64)
    kind = None if scaling is None else scaling[0]
    if kind is not None:
        args = [float(x) for x in scaling[1:]]
        if not args or not all(math.isfinite(x) and x > 0 for x in args) \
                or len(args) not in {"linear": (1,), "ntk": (1,), "by_parts": (2, 4)}.get(kind, ()):
            raise ValueError("scaling: expected ('linear', factor), ('ntk', factor) or "
                             "('by_parts', factor, length[, fast, slow])")
        factor = args[0]
    if kind == "ntk" and dims > 2:
        base = base * factor ** (dims / (dims - 2))
    w = base ** (-2.0 * i / dims)
    if kind == "linear":
        return w / factor, 1.0
    if kind != "by_parts":
        return w, 1.0
    length = args[1]
    fast, slow = args[2:] if len(args) == 4 else (32.0, 1.0)

    def pair_of(turns):     # the pair that turns so often over the length
        return dims * math.log(length / (turns * 2 * math.pi)) / (2 * math.log(base))

    lo = max(math.floor(pair_of(fast)), 0)
    hi = min(math.ceil(pair_of(slow)), dims - 1)
    ramp = np.clip((i - lo) / max(hi - lo, 1e-3), 0.0, 1.0)
    magnitude = 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
    return w / factor * ramp + w * (1 - ramp), magnitude


# 2^160 turns of one radian
_RADIAN = int(2 ** 160 / (2 * Fraction("3.14159265358979323846264338327950288419716939937510582")))


def turns_of(freqs):
    """Angles per position as 64-bit fractions of a turn (uint64)."""
    freqs = np.asarray(freqs, dtype=np.float64)
    if not np.isfinite(freqs).all():
        raise ValueError("freqs: expected finite angles")
    turns = []
    for w in freqs.tolist():
        n, d = w.as_integer_ratio()                   # d: a power of two
        turns.append((n * _RADIAN >> 96 + d.bit_length() - 1) % 2 ** 64)
    return np.array(turns, dtype=np.uint64)


class Rotary:
    """The turn of a head of d values: its first `dims` (all of them by
    default) in pairs of halves, or of neighbours when interleaved.  freqs:
    angles per position in 64 bits instead of base and scaling; magnitude: a
    factor on the turned values (default: the scaling's)."""

    def __init__(self, d, dims=None, base=10000.0, interleaved=False, scaling=None, freqs=None,
                 magnitude=None, device=None):
        dims = d if dims is None else int(dims)
        if d not in (64, 128, 256) or dims < 2 or dims > d or dims % 2:
            raise ValueError("d: expected 64, 128 or 256; dims: an even number up to d")
        if freqs is None:
            freqs, default = frequencies(dims, base, scaling)
        else:
            if scaling is not None:
                raise ValueError("freqs: not together with scaling")
            freqs, default = np.asarray(freqs, dtype=np.float64), 1.0
            if freqs.shape != (dims // 2,):
                raise ValueError(f"freqs: expected {dims // 2} angles")
        self.d, self.dims, self.interleaved = d, dims, bool(interleaved)
        self.freqs = freqs
        self.magnitude = float(default if magnitude is None else magnitude)
        if not math.isfinite(self.magnitude):
            raise ValueError("magnitude: expected a finite number")
        self.turns = torch.from_numpy(turns_of(freqs).view(np.int64)).to(
            "cuda" if device is None else device)
        self.index = self.turns.get_device()
        self.struct = fa.FaRotary(self.turns.data_ptr(), self.magnitude, dims,
                                  int(self.interleaved))
        self.address = ctypes.addressof(self.struct)


def view(name, t, shape, index):
    """The fa_strided_t, packed, of a bf16 tensor of this shape on device
    `index`."""
    if t.dtype is not _bf16 or t.shape != shape or t.get_device() != index:
        raise ValueError(f"{name}: expected a bf16 CUDA tensor {list(shape)} on the current device")
    b, h, n, c = t.stride()
    p = t.data_ptr()
    if c != 1 or p & 15 | (b | h | n) & 7:         # not d contiguous, 16 bytes, eights
        if (c != 1 and shape[3] > 1) or p % 16:
            raise ValueError(f"{name}: d must be contiguous and the tensor 16-byte aligned")
        for s, size in ((b, shape[0]), (h, shape[1]), (n, shape[2])):
            if s % 8 and size > 1:
                raise ValueError(f"{name}: strides must be multiples of 8")
    return _pack(p, b, h, n)


def out_like(t):
    """(a tensor like t, dense, its fa_strided_t)."""
    o = _empty_like(t)
    b, h, n, c = o.stride()
    if c != 1:             # (like an expanded input with an axis of one at stride one)
        o = torch.empty(t.shape, dtype=t.dtype, device=t.device)
        b, h, n, _ = o.stride()
    return o, _pack(o.data_ptr(), b, h, n)


def ints(name, t, shape, index):
    """The address of a contiguous int32 tensor, None for None."""
    if t is None:
        return None
    if t.dtype is not _int32 or t.shape != shape or t.get_device() != index \
            or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous int32 CUDA tensor {list(shape)} on the "
                         "current device")
    return t.data_ptr()


def _call(q, k, rotary, start, pos, inplace, back, stream):
    if stream is not None:
        with torch.cuda.stream(stream):
            return _call(q, k, rotary, start, pos, inplace, back, None)
    shape, index = q.shape, q.get_device()
    if len(shape) != 4 or index < 0 or index != _current_device():
        raise ValueError("q: expected a tensor [B, H, N, d] on the current CUDA device")
    B, H, N, d = shape
    if rotary.index != index or rotary.d != d:
        raise ValueError(f"rotary: made for d = {rotary.d} on device {rotary.index}")
    qs = view("q", q, shape, index)
    qo, qos = (q, qs) if inplace else out_like(q)
    h_kv, ko, ks, kos = 0, None, None, None
    if k is not None:
        kshape = k.shape
        if len(kshape) != 4:
            raise ValueError("k: expected a tensor [B, H_kv, N, d]")
        h_kv = kshape[1]
        ks = view("k", k, (B, h_kv, N, d), index)
        ko, kos = (k, ks) if inplace else out_like(k)
    status = _load().fa_rotate(
        qs, qos, H, ks, kos, h_kv, B, N, d,
        start if start is None else ints("start", start, (B,), index),
        pos if pos is None else ints("pos", pos, (B, N), index), rotary.address, back,
        _current_raw_stream(index))
    if status:
        raise fa.FAError(status, "fa_rotate")
    return qo, ko


def rotate(q, k, rotary, start=None, pos=None, inplace=False, stream=None):
    """(q, k) turned; q [B, H, N, d], k [B, H_kv, N, d] or None.  Token t is at
    position t, start[b] + t (start: int32 [B]) or pos[b, t] (int32 [B, N]).
    inplace: q and k themselves (not one tensor as both)."""
    return _call(q, k, rotary, start, pos, inplace, 0, stream)


def rotate_back(dq, dk, rotary, start=None, pos=None, inplace=False, stream=None):
    """The gradients (dq, dk) of the turned q and k as those of q and k."""
    return _call(dq, dk, rotary, start, pos, inplace, 1, stream)
