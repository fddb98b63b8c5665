"""Paged 4-bit cache over the C ABI (include/vq_kivi.h, "paged 4-bit cache"):
passes torch tensor pointers, strides and the current CUDA stream; holds no
arithmetic.

The pool and the status word are torch tensors; block tables and lengths are
int32 CUDA tensors that the caller keeps, so every call can be captured into a
CUDA graph and follows the tables and lengths that it finds when it runs.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _lib
from .rope import DTYPES, Rope, _current_device, _on, _positions, _raw_stream, _rows


class PagedKiviCache:
    """A pool of `n_pages` pages of `page` tokens in 4 bits.

    Keys and values are quantized per token, over `group` neighbouring
    channels, so that a token is complete when it is appended and a page
    stands by itself.  (``KiviCache`` quantizes keys per channel, over groups
    of tokens.)  A key channel that stands out therefore widens the code steps
    of its whole group: a smaller group keeps them to fewer channels.

    pool: an existing uint8 CUDA tensor of [n_pages][H_kv][page/16][block]
    (see `block_bytes`), else one is allocated (zeroed) on `device`.

    Every method takes `table` (int32 [B][max_pages], rows may be strided),
    `lens` (int32 [B], the new tokens included) and `cu_new` (int32 [B + 1]
    offsets of each sequence's new tokens in the token tensors, or None: one
    new token per sequence).
    """

    def __init__(self, n_pages: int, *, page: int, H_q: int, H_kv: int, D: int, group: int = 32,
                 pool: Optional[torch.Tensor] = None, device=None):
        L = _lib.load()
        self.n_pages, self.page, self.H_q, self.H_kv = int(n_pages), int(page), int(H_q), int(H_kv)
        self.D, self.group = int(D), int(group)
        self._spec = _lib.Paged(self.H_q, self.H_kv, self.D, self.group, self.page,
                                self.n_pages, None, None)
        nbytes = int(L.vq_kivi_paged_pool_bytes(ctypes.byref(self._spec)))
        if nbytes == 0:
            raise _lib.VqError(_lib.VQ_ERR_UNSUPPORTED, L.vq_kivi_last_error().decode())
        self.block_bytes = 16 * self.D + 128 * (self.D // self.group)
        shape = (self.n_pages, self.H_kv, self.page // 16, self.block_bytes)
        if pool is None:
            pool = torch.zeros(shape, dtype=torch.uint8,
                               device="cuda" if device is None else device)
        if not pool.is_cuda or pool.dtype != torch.uint8 or not pool.is_contiguous() or \
                tuple(pool.shape) != shape:
            raise ValueError(f"pool must be a contiguous uint8 CUDA tensor {list(shape)}")
        self.pool, self.device = pool, pool.device
        self._status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self._spec.pool, self._spec.status = pool.data_ptr(), self._status.data_ptr()
        self._lib, self._index = L, self.device.index
        self._ws = {}      # workspace bytes by (B, max_new)

    # -- arguments -------------------------------------------------------------

    def _check_batch(self, table, lens, cu_new):
        """Say what is wrong with a batch, or nothing."""
        for t, name in ((table, "table"), (lens, "lens"), (cu_new, "cu_new")):
            if t is not None and (t.dtype != torch.int32 or t.device != self.device):
                raise ValueError(f"{name} must be int32 on {self.device}")
        if lens.dim() != 1 or not lens.is_contiguous():
            raise ValueError("lens must be a contiguous [B]")
        B = lens.shape[0]
        if table.dim() != 2 or table.shape[0] != B or (table.shape[1] > 1 and
                                                       table.stride(1) != 1):
            raise ValueError(f"table must be [{B}][max_pages] with contiguous rows")
        if cu_new is not None and (tuple(cu_new.shape) != (B + 1,) or
                                   not cu_new.is_contiguous()):
            raise ValueError(f"cu_new must be a contiguous [{B + 1}]")

    def _batch(self, table, lens, cu_new, tokens: int) -> _lib.PagedBatch:
        dev, i32, ts, ls = self.device, torch.int32, table.shape, lens.shape
        B = ls[0] if len(ls) == 1 else -1
        if not (len(ts) == 2 and ts[0] == B and table.stride(1) == 1 and lens.is_contiguous() and
                table.dtype is i32 and lens.dtype is i32 and table.device == dev and
                lens.device == dev and
                (cu_new is None or (cu_new.dtype is i32 and cu_new.device == dev and
                                    cu_new.shape == (B + 1,) and cu_new.is_contiguous()))):
            self._check_batch(table, lens, cu_new)
        if cu_new is None and tokens != B:
            raise ValueError(f"without cu_new every sequence has one new token: {tokens} rows "
                             f"for {B} sequences")
        mp = ts[1]
        return _lib.PagedBatch(B, mp, table.data_ptr() or None,
                               table.stride(0) if B > 1 else max(mp, 1), lens.data_ptr() or None,
                               None if cu_new is None else cu_new.data_ptr(), tokens)

    def _dtype(self, t: torch.Tensor, name: str) -> int:
        if not t.is_cuda or t.device != self.device:
            raise ValueError(f"{name} must be a CUDA tensor on {self.device}")
        dt = t.dtype
        if dt is not torch.float16 and dt is not torch.bfloat16:
            raise ValueError(f"{name} must be fp16 or bf16, got {dt}")
        return DTYPES[dt]

    def _elsewhere(self, stream) -> bool:
        return stream is not None or self._index != _current_device()

    # -- steps -------------------------------------------------------------------

    def append(self, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor, lens: torch.Tensor,
               cu_new: Optional[torch.Tensor] = None, *, q: Optional[torch.Tensor] = None,
               rope: Optional[Rope] = None, positions: Optional[torch.Tensor] = None,
               q_weight: Optional[torch.Tensor] = None,
               k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
               q_out: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None) -> Optional[torch.Tensor]:
        """Quantize the new tokens k, v [tokens][H_kv][D] (fp16 or bf16, any
        token and head strides) into their pages, the keys normed (k_weight)
        and rotated (rope) on the way; with q [tokens][H_q][D], return the
        queries normed and rotated (rows of tokens that are not in the cache
        are left as allocated).  positions: [tokens] or [n_axes][tokens];
        None rotates by a token's place in its sequence."""
        if self._elsewhere(stream):
            with _on(self.device, stream):
                return self.append(k, v, table, lens, cu_new, q=q, rope=rope,
                                   positions=positions, q_weight=q_weight, k_weight=k_weight,
                                   eps=eps, q_out=q_out)
        dt, dtype, device = self._dtype(k, "k"), k.dtype, self.device
        if k.shape != v.shape:
            raise ValueError("k and v must have one shape")
        T = k.shape[0]
        rk = _rows(k, self.H_kv, self.D, dtype, device, "k", k_weight)
        rv = _rows(v, self.H_kv, self.D, dtype, device, "v")
        rq = None
        if q is not None:
            if q.shape[0] != T:
                raise ValueError(f"q has {q.shape[0]} tokens, k {T}")
            fresh = q_out is None
            if fresh:
                q_out = torch.empty(q.shape, dtype=dtype, device=device)
            rq = _rows(q, self.H_q, self.D, dtype, device, "q", q_weight, q_out, fresh)
        elif q_weight is not None or q_out is not None:
            raise ValueError("q_weight or q_out without q")
        batch = self._batch(table, lens, cu_new, T)
        pos, pos64, pstride = None, 0, 0
        if rope is not None:
            if rope.device != device:
                raise ValueError(f"the rope is on {rope.device}, the cache on {device}")
            if positions is not None:
                pos, pos64, pstride = _positions(positions, rope.n_axes, T, device)
        elif positions is not None:
            raise ValueError("positions without a rope")
        rc = self._lib.vq_kivi_paged_append(
            self._spec, batch, dt, rq, rk, rv, None if rope is None else rope.spec, pos, pos64,
            pstride, eps, _raw_stream(self._index))
        if rc:
            _lib.check(rc)
        return q_out

    def attend(self, q: torch.Tensor, table: torch.Tensor, lens: torch.Tensor,
               cu_new: Optional[torch.Tensor] = None, *, max_new: Optional[int] = None,
               scale: float = 0.0, out: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        """Attention of the new tokens' queries q [tokens][H_q][D] over their
        sequences, each seeing the positions up to its own -> [tokens][H_q][D]
        in q's type.  max_new: no sequence has more new tokens (default: 1
        without cu_new, else the rows of q)."""
        if self._elsewhere(stream):
            with _on(self.device, stream):
                return self.attend(q, table, lens, cu_new, max_new=max_new, scale=scale, out=out)
        dt, shape = self._dtype(q, "q"), q.shape
        fresh = out is None
        if fresh:
            out = torch.empty(shape, dtype=q.dtype, device=self.device)
        elif not out.is_contiguous():
            raise ValueError("out must be contiguous")
        rq = _rows(q, self.H_q, self.D, q.dtype, self.device, "q", None, out, fresh)
        rq.out_token, rq.out_head = self.H_q * self.D, self.D
        batch = self._batch(table, lens, cu_new, shape[0])
        if max_new is None:
            max_new = 1 if cu_new is None else max(shape[0], 1)
        key = (batch.B, max_new)
        nbytes = self._ws.get(key)
        if nbytes is None:
            nbytes = self._lib.vq_kivi_paged_workspace_bytes(self._spec, batch.B, int(max_new))
            if nbytes and len(self._ws) < 4096:
                self._ws[key] = nbytes
        ws = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        rc = self._lib.vq_kivi_paged_attend(
            self._spec, batch, dt, rq, int(max_new), scale, ws.data_ptr(), nbytes,
            _raw_stream(self._index))
        if rc:
            _lib.check(rc)
        return out

    def dequantize(self, table: torch.Tensor, lens: torch.Tensor,
                   cu_new: Optional[torch.Tensor] = None, *, n_tokens: Optional[int] = None,
                   out=None, stream: Optional[torch.cuda.Stream] = None):
        """The new tokens' rows as the values that the cache stands for: fp16
        K_hat, V_hat [n_tokens][H_kv][D] (n_tokens >= cu_new[B]; cu_new of the
        whole lengths reads whole sequences)."""
        if self._elsewhere(stream):
            with _on(self.device, stream):
                return self.dequantize(table, lens, cu_new, n_tokens=n_tokens, out=out)
        if n_tokens is None:
            if cu_new is not None:
                raise ValueError("n_tokens is needed with cu_new")
            n_tokens = lens.shape[0]
        shape = (int(n_tokens), self.H_kv, self.D)
        if out is None:
            out = (torch.empty(shape, dtype=torch.float16, device=self.device),
                   torch.empty(shape, dtype=torch.float16, device=self.device))
        else:
            for t in out:
                if tuple(t.shape) != shape or t.dtype != torch.float16 or \
                        t.device != self.device or not t.is_contiguous():
                    raise ValueError(f"outputs must be contiguous fp16 {list(shape)} on "
                                     f"{self.device}")
        K, V = out
        batch = self._batch(table, lens, cu_new, shape[0])
        rc = self._lib.vq_kivi_paged_dequantize(
            self._spec, batch, K.data_ptr() or None, V.data_ptr() or None,
            _raw_stream(self._index))
        if rc:
            _lib.check(rc)
        return K, V

    def status(self):
        """Raise if a kernel since the last check found a page or a length
        outside its range, or gave up a wait (synchronizes)."""
        with torch.cuda.device(self.device):
            _lib.check(self._lib.vq_kivi_paged_status(self._spec, _raw_stream(self._index)))
