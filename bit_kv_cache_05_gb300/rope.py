"""Norm and rotation of query and key heads (vq_kivi_norm_rope): passes torch
tensor pointers, strides and the current CUDA stream to the CUDA library.

``Rope`` keeps the frequencies of a rotation on the device; ``norm_rope``
applies per-head RMS norms and the rotation to queries and keys in one kernel.
Its results go into ``KiviCache`` or, for the paged cache, the same happens
inside ``PagedKiviCache.append``.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import Optional, Sequence

import torch

from . import _lib

# the current stream's handle and the current device without the objects that
# torch.cuda builds
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(
    torch._C, "_cuda_getCurrentRawStream") else (
        lambda i: torch.cuda.current_stream(i).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device

# 2^320 / (2 pi)
_PER_RADIAN = 2 ** 320 * 10 ** 90 // int(
    "6283185307179586476925286766559005768394338798750211641949889184615632812572417997256069650")


def _turns(freq: float) -> int:
    """Radians per position as turns, times 2^64, rounded, modulo 2^64."""
    n, d = freq.as_integer_ratio()          # d is a power of two
    shift = 256 + d.bit_length() - 1
    return ((n * _PER_RADIAN + (1 << (shift - 1))) >> shift) % 2 ** 64


DTYPES = {torch.float16: _lib.F16, torch.bfloat16: _lib.BF16, torch.float32: _lib.F32}


class Rope:
    """A rotation by position on one to four axes.

    inv_freq   radians per position of each rotated pair (64 bits); or rot_dim
               and theta for theta ** (-2 j / rot_dim)
    axis       the axis of each pair (default: all 0); or sections, the number
               of neighbouring pairs on each axis
    interleaved  pairs (2 j, 2 j + 1) instead of (j, j + rot_dim / 2)
    scale      factor of cosine and sine
    """

    def __init__(self, inv_freq: Optional[Sequence[float]] = None, *,
                 rot_dim: Optional[int] = None, theta: float = 10000.0,
                 axis: Optional[Sequence[int]] = None,
                 sections: Optional[Sequence[int]] = None, interleaved: bool = False,
                 scale: float = 1.0, device=None):
        if inv_freq is None:
            if rot_dim is None or rot_dim < 0 or rot_dim % 2:
                raise ValueError("Rope needs inv_freq or an even rot_dim")
            inv_freq = [float(theta) ** (-2.0 * j / rot_dim) for j in range(rot_dim // 2)]
        freq = [float(f) for f in inv_freq]
        half = len(freq)
        if half % 8 or half > 128:
            raise ValueError(f"{half} rotated pairs: a multiple of 8, at most 128")
        if any(f != f or f in (float("inf"), float("-inf")) for f in freq):
            raise ValueError("inv_freq must be finite")
        if sections is not None:
            if axis is not None:
                raise ValueError("give axis or sections, not both")
            if any(int(n) < 0 for n in sections):
                raise ValueError("sections must not be negative")
            axis = [a for a, n in enumerate(sections) for _ in range(int(n))]
        axis = [0] * half if axis is None else [int(a) for a in axis]
        if len(axis) != half:
            raise ValueError(f"{len(axis)} axes for {half} rotated pairs")
        if any(a < 0 or a > 3 for a in axis):
            raise ValueError("an axis is 0, 1, 2 or 3")
        self.rot_dim, self.n_axes = 2 * half, max(axis, default=0) + 1
        if sections is not None:
            self.n_axes = max(self.n_axes, len(sections))
            if self.n_axes > 4:
                raise ValueError("at most 4 axes")
        self.interleaved, self.scale = bool(interleaved), float(scale)
        # turns per position in 64-bit fixed point, then the axes as bytes: one
        # copy to the device
        words = [_turns(f) for f in freq]
        words += [int.from_bytes(bytes(axis[j:j + 8]), "little") for j in range(0, half, 8)]
        words = [w - 2 ** 64 if w >= 2 ** 63 else w for w in words]
        device = torch.device("cuda" if device is None else device)
        self._words = torch.tensor(words, dtype=torch.int64).to(device)
        self.turns = self._words[:half]
        self.axis = self._words[half:].view(torch.uint8)
        self.device = self.turns.device
        self.spec = _lib.RopeSpec(self.rot_dim, int(self.interleaved), self.n_axes, self.scale,
                                  self.turns.data_ptr(), self.axis.data_ptr())


def _check_rows(t, heads, D, dtype, device, name, weight, out):
    """Say what is wrong with rows, or nothing."""
    if t.dim() != 3 or (heads is not None and t.shape[1] != heads) or (
            D is not None and t.shape[2] != D):
        raise ValueError(f"{name} must be [tokens][{heads or 'heads'}][{D or 'D'}], got "
                         f"{tuple(t.shape)}")
    T, H, D = t.shape
    for x, what in ((t, name), (out, name + "_out"), (weight, name + "_weight")):
        if x is None:
            continue
        if x.device != device:
            raise ValueError(f"{what} is on {x.device}, expected {device}")
        if x.dtype != dtype:
            raise ValueError(f"{what} must be {dtype}, got {x.dtype}")
        if x.requires_grad and torch.is_grad_enabled():
            raise ValueError(f"{what} requires a gradient: the cache's operators have none")
        if D > 1 and x.numel() and x.stride(-1) != 1:
            raise ValueError(f"{what}: the last dimension must be contiguous")
    if weight is not None and tuple(weight.shape) != (D,):
        raise ValueError(f"{name}_weight must be [{D}], got {tuple(weight.shape)}")
    if out is not None:
        if out.shape != t.shape:
            raise ValueError(f"{name}_out must be {tuple(t.shape)}, got {tuple(out.shape)}")
        o0, o1 = (out.stride(0) if T > 1 else 0), (out.stride(1) if H > 1 else 0)
        if out.numel() and ((T > 1 and o0 < D) or (H > 1 and o1 < D) or (
                T > 1 and H > 1 and o0 < (H - 1) * o1 + D and o1 < (T - 1) * o0 + D)):
            raise ValueError(f"{name}_out: rows overlap")


def _rows(t: torch.Tensor, heads: Optional[int], D: Optional[int], dtype, device, name: str,
          weight: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
          fresh: bool = False) -> _lib.Rows:
    """The C description of rows [tokens][heads][D] (last dimension
    contiguous).  fresh: `out` was just made for these rows."""
    shape, st = t.shape, t.stride()
    # what nearly every call passes, in few steps; anything else is looked at
    # one by one
    if not (len(shape) == 3 and (heads is None or shape[1] == heads) and
            (D is None or shape[2] == D) and t.dtype is dtype and t.device == device and
            not t.requires_grad and st[2] == 1 and (out is None or fresh) and
            (weight is None or (weight.dtype is dtype and weight.device == device and
                                weight.shape == shape[2:] and not weight.requires_grad and
                                weight.is_contiguous()))):
        _check_rows(t, heads, D, dtype, device, name, weight, out)
    T, H, _ = shape
    po, so = (0, (0, 0)) if out is None else (out.data_ptr(), out.stride())
    # the stride of a dimension of one element may be anything
    t1, h1 = T > 1, H > 1
    return _lib.Rows(t.data_ptr(), po, None if weight is None else weight.data_ptr(),
                     st[0] if t1 else 0, st[1] if h1 else 0, so[0] if t1 else 0,
                     so[1] if h1 else 0, H)


def _positions(p: torch.Tensor, n_axes: int, T: int, device):
    shape, st, dt = p.shape, p.stride(), p.dtype
    if not (shape == (n_axes, T) or (n_axes == 1 and shape == (T,))):
        raise ValueError(f"positions must be [{n_axes}][{T}], got {tuple(shape)}")
    if p.device != device or (dt is not torch.int64 and dt is not torch.int32):
        raise ValueError(f"positions must be int32 or int64 on {device}")
    if T > 1 and st[-1] != 1:
        raise ValueError("positions: the last dimension must be contiguous")
    return p.data_ptr() or None, int(dt is torch.int64), st[0] if n_axes > 1 else T


@contextlib.contextmanager
def _on(device: torch.device, stream):
    """The tensors' device current, and `stream` (so that what is allocated
    belongs to it)."""
    with torch.cuda.device(device):
        if stream is None:
            yield
        else:
            with torch.cuda.stream(stream):
                yield


def norm_rope(q: torch.Tensor, k: Optional[torch.Tensor], positions: Optional[torch.Tensor],
              rope: Optional[Rope], *, q_weight: Optional[torch.Tensor] = None,
              k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
              q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
              stream: Optional[torch.cuda.Stream] = None):
    """RMS norm over each head (with a weight) and the rotation by position,
    in one kernel: q [T][H_q][D] and k [T][H_kv][D] (or None), fp16, bf16 or
    fp32, any token and head strides -> (q_out, k_out).  positions: int32 or
    int64 [T], or [n_axes][T] (unused without a rope).  The outputs may be the
    inputs themselves."""
    dt, device = q.dtype, q.device
    if not q.is_cuda:
        raise ValueError("q must be a CUDA tensor")
    if dt not in DTYPES:
        raise ValueError(f"q must be fp16, bf16 or fp32, got {dt}")
    if stream is not None or device.index != _current_device():
        with _on(device, stream):
            return norm_rope(q, k, positions, rope, q_weight=q_weight, k_weight=k_weight,
                             eps=eps, q_out=q_out, k_out=k_out)
    if q.dim() != 3:
        raise ValueError(f"q must be [tokens][heads][D], got {tuple(q.shape)}")
    T, _, D = q.shape
    if k is not None and (k.dim() != 3 or k.shape[0] != T):
        raise ValueError(f"k must be [{T}][heads][{D}], got {tuple(k.shape)}")
    if k is None and (k_weight is not None or k_out is not None):
        raise ValueError("k_weight or k_out without k")
    fq = fk = False
    if q_out is None:
        q_out, fq = torch.empty(q.shape, dtype=dt, device=device), True
    rk = None
    if k is not None:
        if k_out is None:
            k_out, fk = torch.empty(k.shape, dtype=dt, device=device), True
        rk = _rows(k, None, D, dt, device, "k", k_weight, k_out, fk)
    rq = _rows(q, None, None, dt, device, "q", q_weight, q_out, fq)
    pos, pos64, pstride = None, 0, 0
    if rope is not None and rope.rot_dim > 0:
        if rope.device != device:
            raise ValueError(f"the rope is on {rope.device}, q on {device}")
        if positions is None:
            raise ValueError("positions are needed for the rotation")
        pos, pos64, pstride = _positions(positions, rope.n_axes, T, device)
    rc = _lib.load().vq_kivi_norm_rope(
        DTYPES[dt], T, D, rq, rk, None if rope is None else rope.spec, pos, pos64, pstride, eps,
        _raw_stream(device.index))
    if rc:
        _lib.check(rc)
    return q_out, k_out
