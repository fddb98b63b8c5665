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
from .cache import _stream_handle
from .rope import DTYPES, Rope, _on, _positions, _rows


class PagedKiviCache:
    """A pool of `n_pages` pages of `page` tokens in 4 bits.

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

    # -- arguments -------------------------------------------------------------

    def _batch(self, table, lens, cu_new, tokens: int) -> _lib.PagedBatch:
        dev = self.device
        for t, name in ((table, "table"), (lens, "lens"), (cu_new, "cu_new")):
            if t is not None and (t.dtype != torch.int32 or t.device != dev):
                raise ValueError(f"{name} must be int32 on {dev}")
        if lens.dim() != 1 or not lens.is_contiguous():
            raise ValueError("lens must be a contiguous [B]")
        B = lens.shape[0]
        if table.dim() != 2 or table.shape[0] != B or (table.shape[1] > 1 and
                                                       table.stride(1) != 1):
            raise ValueError(f"table must be [{B}][max_pages] with contiguous rows")
        if cu_new is None:
            if tokens != B:
                raise ValueError(f"without cu_new every sequence has one new token: {tokens} "
                                 f"rows for {B} sequences")
        elif tuple(cu_new.shape) != (B + 1,) or not cu_new.is_contiguous():
            raise ValueError(f"cu_new must be a contiguous [{B + 1}]")
        mp = table.shape[1]
        return _lib.PagedBatch(B, mp, table.data_ptr() or None,
                               table.stride(0) if B > 1 else max(mp, 1), lens.data_ptr() or None,
                               None if cu_new is None else cu_new.data_ptr(), tokens)

    def _dtype(self, t: torch.Tensor, name: str) -> int:
        if not t.is_cuda or t.device != self.device:
            raise ValueError(f"{name} must be a CUDA tensor on {self.device}")
        if t.dtype not in (torch.float16, torch.bfloat16):
            raise ValueError(f"{name} must be fp16 or bf16, got {t.dtype}")
        return DTYPES[t.dtype]

    def _elsewhere(self, stream) -> bool:
        return stream is not None or self.device.index != torch.cuda.current_device()

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
        dt = self._dtype(k, "k")
        if k.shape != v.shape:
            raise ValueError("k and v must have one shape")
        T = k.shape[0]
        rk = _rows(k, self.H_kv, self.D, k.dtype, self.device, "k", k_weight)
        rv = _rows(v, self.H_kv, self.D, k.dtype, self.device, "v")
        rq = None
        if q is not None:
            if q.shape[0] != T:
                raise ValueError(f"q has {q.shape[0]} tokens, k {T}")
            if q_out is None:
                q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
            rq = _rows(q, self.H_q, self.D, k.dtype, self.device, "q", q_weight, q_out)
        elif q_weight is not None or q_out is not None:
            raise ValueError("q_weight or q_out without q")
        batch = self._batch(table, lens, cu_new, T)
        pos, pos64, pstride = 0, 0, 0
        if rope is not None:
            if rope.device != self.device:
                raise ValueError(f"the rope is on {rope.device}, the cache on {self.device}")
            if positions is not None:
                pos, pos64, pstride = _positions(positions, rope.n_axes, T, self.device)
        elif positions is not None:
            raise ValueError("positions without a rope")
        _lib.check(_lib.load().vq_kivi_paged_append(
            self._spec, batch, dt, rq, rk, rv, None if rope is None else rope.spec, pos or None,
            pos64, pstride, float(eps), _stream_handle(None, self.device.index)))
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
        dt = self._dtype(q, "q")
        T = q.shape[0]
        if out is None:
            out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        elif not out.is_contiguous():
            raise ValueError("out must be contiguous")
        rq = _rows(q, self.H_q, self.D, q.dtype, self.device, "q", None, out)
        rq.out_token, rq.out_head = self.H_q * self.D, self.D
        batch = self._batch(table, lens, cu_new, T)
        if max_new is None:
            max_new = 1 if cu_new is None else max(T, 1)
        L = _lib.load()
        nbytes = L.vq_kivi_paged_workspace_bytes(self._spec, batch.B, int(max_new))
        ws = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        _lib.check(L.vq_kivi_paged_attend(
            self._spec, batch, dt, rq, int(max_new), float(scale), ws.data_ptr(), nbytes,
            _stream_handle(None, self.device.index)))
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
        K, V = out
        for t in out:
            if tuple(t.shape) != shape or t.dtype != torch.float16 or \
                    t.device != self.device or not t.is_contiguous():
                raise ValueError(f"outputs must be contiguous fp16 {list(shape)} on "
                                 f"{self.device}")
        batch = self._batch(table, lens, cu_new, shape[0])
        _lib.check(_lib.load().vq_kivi_paged_dequantize(
            self._spec, batch, K.data_ptr() or None, V.data_ptr() or None,
            _stream_handle(None, self.device.index)))
        return K, V

    def status(self):
        """Raise if a kernel since the last check found a page or a length
        outside its range, or gave up a wait (synchronizes)."""
        with torch.cuda.device(self.device):
            _lib.check(_lib.load().vq_kivi_paged_status(
                self._spec, _stream_handle(None, self.device.index)))
