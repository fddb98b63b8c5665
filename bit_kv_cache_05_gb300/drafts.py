"""Verification of drafted tokens (vq_kivi_verify_drafts): passes torch tensor
pointers, strides and the current CUDA stream to the CUDA library.

One step of speculative decoding over a paged cache: append the drafted tokens
(``PagedKiviCache.append``), attend them (``attend``, with masks for a tree),
verify them here, and let the cache keep what stays (``keep``).
"""
from __future__ import annotations

from typing import Optional

import torch

from . import _lib
from .rope import DTYPES, _current_device, _on, _raw_stream


def _check(target, tokens, uniforms, cu_new, parents, draft, path, counts, after):
    """Say what is wrong with the arguments, or nothing."""
    device, dt = target.device, target.dtype
    if not target.is_cuda or dt not in DTYPES:
        raise ValueError("target must be an fp16, bf16 or fp32 CUDA tensor")
    if target.dim() != 2:
        raise ValueError(f"target must be [rows][V], got {tuple(target.shape)}")
    T, V = target.shape
    for t, name in ((target, "target"), (draft, "draft")):
        if t is None:
            continue
        if t.shape != target.shape or t.dtype is not dt or t.device != device or (
                V > 1 and t.stride(1) != 1):
            raise ValueError(f"{name} must be {dt} [{T}][{V}] with contiguous rows on {device}")
        if t.requires_grad and torch.is_grad_enabled():
            raise ValueError(f"{name} requires a gradient: the verification has none")
    tt, i32 = tokens.dtype, torch.int32
    if tt is not i32 and tt is not torch.int64:
        raise ValueError(f"tokens must be int32 or int64, got {tt}")
    if cu_new.dim() != 1 or cu_new.shape[0] < 1:
        raise ValueError("cu_new must be [B + 1]")
    B = cu_new.shape[0] - 1
    for t, n, want, name in ((tokens, T, tt, "tokens"), (uniforms, T, torch.float32, "uniforms"),
                             (cu_new, B + 1, i32, "cu_new"), (parents, T, i32, "parents"),
                             (path, T, i32, "path"), (counts, B, i32, "counts"),
                             (after, B, tt, "after")):
        if t is not None and (t.dtype is not want or t.device != device or t.shape != (n,) or
                              not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous {want} [{n}] on {device}")


def verify_drafts(target: torch.Tensor, tokens: torch.Tensor, uniforms: torch.Tensor,
                  cu_new: torch.Tensor, *, parents: Optional[torch.Tensor] = None,
                  draft: Optional[torch.Tensor] = None, path: Optional[torch.Tensor] = None,
                  counts: Optional[torch.Tensor] = None, after: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None):
    """Which drafted tokens stay and which token follows them, so that the
    results are distributed as the target's own samples.

    Row cu_new[b] + i of each array is node i of sequence b (64 at most), node
    0 the last known token.

    target    [rows][V] probabilities behind each node, fp16, bf16 or fp32 (rows
              may be strided)
    tokens    int32 or int64 [rows]: the nodes' tokens
    uniforms  fp32 [rows] in [0, 1): node i's decides on node i, node 0's draws
              the token behind the kept ones
    parents   int32 [rows]: a node's parent in its sequence, below it; None:
              chains
    draft     [rows][V], target's type: what the children of a node were drawn
              from, each independently of the others (torch.multinomial needs
              replacement=True for it); None: the drafts stand for themselves
              (the draft's best tokens, or tokens drawn without replacement)

    Returns (path, counts, after): int32 [rows] the nodes that stay, node 0
    first, -1 behind them; int32 [B] how many; [B] the token behind them in the
    tokens' type.  A sequence with offsets, parents or tokens outside their
    ranges has a count of -1.
    """
    device, dt, shape = target.device, target.dtype, target.shape
    index = device.index
    if target.is_cuda and (stream is not None or index != _current_device()):
        with _on(device, stream):
            return verify_drafts(target, tokens, uniforms, cu_new, parents=parents, draft=draft,
                                 path=path, counts=counts, after=after)
    i32, rows, tt, cs = torch.int32, shape[:1], tokens.dtype, cu_new.shape
    st = target.stride()
    sd = st if draft is None else draft.stride()
    # what nearly every call passes, in few steps; anything else is looked at
    # one by one
    if not (dt in DTYPES and target.is_cuda and len(shape) == 2 and st[1] == 1 and
            (draft is None or draft.shape == shape) and sd[1] == 1 and
            not target.requires_grad and
            (tt is torch.int64 or tt is i32) and tokens.shape == rows and
            tokens.get_device() == index and tokens.is_contiguous() and
            uniforms.dtype is torch.float32 and uniforms.shape == rows and
            uniforms.get_device() == index and uniforms.is_contiguous() and
            cu_new.dtype is i32 and len(cs) == 1 and cs[0] > 0 and
            cu_new.get_device() == index and cu_new.is_contiguous() and
            (parents is None or (parents.dtype is i32 and parents.shape == rows and
                                 parents.get_device() == index and parents.is_contiguous())) and
            (draft is None or (draft.dtype is dt and draft.get_device() == index and
                               not draft.requires_grad)) and
            path is None and counts is None and after is None):
        _check(target, tokens, uniforms, cu_new, parents, draft, path, counts, after)
    T, V = shape
    B = cs[0] - 1
    if path is None:
        path = torch.empty(T, dtype=i32, device=device)
    if counts is None:
        counts = torch.empty(B, dtype=i32, device=device)
    if after is None:
        after = torch.empty(B, dtype=tt, device=device)
    one = T <= 1                     # (the stride of one row may be anything)
    spec = _lib.Drafts(target.data_ptr() or None, None if draft is None else draft.data_ptr(),
                       V if one else st[0], V if one else sd[0], tokens.data_ptr() or None,
                       None if parents is None else parents.data_ptr(),
                       uniforms.data_ptr() or None, cu_new.data_ptr(), T, B, V,
                       int(tt is torch.int64))
    rc = _lib.load().vq_kivi_verify_drafts(spec, DTYPES[dt], path.data_ptr() or None,
                                           counts.data_ptr() or None, after.data_ptr() or None,
                                           _raw_stream(index))
    if rc:
        _lib.check(rc)
    return path, counts, after
