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


def _int32(x, name: str) -> int:
    """A number that the library takes in 32 bits (the call would cut others)."""
    x = int(x)
    if not -2 ** 31 <= x < 2 ** 31:
        raise ValueError(f"{name}={x} does not fit in 32 bits")
    return x


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
        # workspace bytes by (B, max_new), with weights (B, max_new, max_pages), of
        # evictions (B, max_pages, budget, recent)
        self._ws = {}

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

    def _weights(self, t: torch.Tensor, batch: _lib.PagedBatch, name: str) -> _lib.Weights:
        shape, st = t.shape, t.stride()
        if t.dtype is not torch.float32 or t.device != self.device or len(shape) != 3 or \
                shape[0] != batch.B or shape[1] != self.H_kv or (shape[2] > 1 and st[2] != 1):
            raise ValueError(f"{name} must be fp32 [{batch.B}][{self.H_kv}][places] with "
                             f"contiguous rows on {self.device}")
        if t.requires_grad and torch.is_grad_enabled():
            raise ValueError(f"{name} requires a gradient: the cache's operators have none")
        return _lib.Weights(t.data_ptr() or None, st[0], st[1], shape[2])

    def _lens_out(self, t: Optional[torch.Tensor], B: int) -> torch.Tensor:
        if t is None:
            return torch.empty(B, dtype=torch.int32, device=self.device)
        if t.dtype is not torch.int32 or t.device != self.device or t.shape != (B,) or \
                not t.is_contiguous():
            raise ValueError(f"lens_out must be a contiguous int32 [{B}] on {self.device}")
        return t

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
               tree: Optional[torch.Tensor] = None, weights: Optional[torch.Tensor] = None,
               scale: float = 0.0, out: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        """Attention of the new tokens' queries q [tokens][H_q][D] over their
        sequences, each seeing the positions up to its own -> [tokens][H_q][D]
        in q's type.  max_new: no sequence has more new tokens (default: 1
        without cu_new, else the rows of q, with a tree 64 at most).

        tree: int64 [tokens] masks.  A new token then sees the tokens before
        the new ones, and new token j of its sequence where bit j of its mask
        is set (its own bit among them); at most 64 new tokens a sequence.

        weights: fp32 [B][H_kv][>= max_pages * page] (rows may be strided):
        each stored token's softmax weights, summed over the new tokens and the
        query heads of its kv head, are added to its place.  At most 16 (new
        token, query head) pairs per kv head; not with a tree.  Such a call
        allocates 4 bytes for each of these pairs and each place that the tables
        have room for (64 sequences, 8 kv heads, 4 query heads each, tables of
        131072 places: 1 GiB), so cut the table to the pages in use."""
        if self._elsewhere(stream):
            with _on(self.device, stream):
                return self.attend(q, table, lens, cu_new, max_new=max_new, tree=tree,
                                   weights=weights, scale=scale, out=out)
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
            if tree is not None:
                max_new = min(max_new, 64)
        else:
            max_new = _int32(max_new, "max_new")
        w = None
        if tree is not None:
            if weights is not None:
                raise ValueError("weights are not added over a tree")
            if tree.dtype is not torch.int64 or tree.device != self.device or \
                    tree.shape != shape[:1] or not tree.is_contiguous():
                raise ValueError(f"tree must be a contiguous int64 [{shape[0]}] on {self.device}")
        elif weights is not None:
            w = self._weights(weights, batch, "weights")
        key = (batch.B, max_new) if w is None else (batch.B, max_new, batch.max_pages)
        nbytes = self._ws.get(key)
        if nbytes is None:
            L = self._lib
            nbytes = L.vq_kivi_paged_workspace_bytes(self._spec, batch.B, max_new) if w is None \
                else L.vq_kivi_paged_weights_workspace_bytes(self._spec, batch.B,
                                                             batch.max_pages, max_new)
            if nbytes and len(self._ws) < 4096:
                self._ws[key] = nbytes
        ws = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        tail = (max_new, scale, ws.data_ptr(), nbytes, _raw_stream(self._index))
        if tree is not None:
            rc = self._lib.vq_kivi_paged_attend_tree(self._spec, batch, dt, rq,
                                                     tree.data_ptr() or None, *tail)
        elif w is not None:
            rc = self._lib.vq_kivi_paged_attend_weights(self._spec, batch, dt, rq, w, *tail)
        else:
            rc = self._lib.vq_kivi_paged_attend(self._spec, batch, dt, rq, *tail)
        if rc:
            _lib.check(rc)
        return out

    def keep(self, table: torch.Tensor, lens: torch.Tensor, cu_new: torch.Tensor,
             path: torch.Tensor, counts: torch.Tensor, *,
             lens_out: Optional[torch.Tensor] = None,
             stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        """Of the new tokens of sequence b (64 at most) those stay that the
        first counts[b] entries of path (int32 [tokens], from row cu_new[b] on)
        name, in rising order: their codes move to the places of the first new
        tokens.  Returns the lengths without the others (lens_out, int32 [B];
        it may be lens).  path and counts are what verify_drafts gives."""
        if self._elsewhere(stream):
            with _on(self.device, stream):
                return self.keep(table, lens, cu_new, path, counts, lens_out=lens_out)
        if cu_new is None:
            raise ValueError("cu_new is needed")
        for t, name in ((path, "path"), (counts, "counts")):
            if t.dtype is not torch.int32 or t.device != self.device or t.dim() != 1 or \
                    not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous int32 vector on {self.device}")
        batch = self._batch(table, lens, cu_new, path.shape[0])
        if counts.shape[0] != batch.B:
            raise ValueError(f"counts must be [{batch.B}], got {tuple(counts.shape)}")
        lens_out = self._lens_out(lens_out, batch.B)
        rc = self._lib.vq_kivi_paged_keep(self._spec, batch, path.data_ptr() or None,
                                          counts.data_ptr() or None, lens_out.data_ptr() or None,
                                          _raw_stream(self._index))
        if rc:
            _lib.check(rc)
        return lens_out

    def evict(self, table: torch.Tensor, lens: torch.Tensor, weights: torch.Tensor, budget: int,
              *, recent: int, first: int = 0, lens_out: Optional[torch.Tensor] = None,
              weights_out: Optional[torch.Tensor] = None,
              stream: Optional[torch.cuda.Stream] = None):
        """Bring every sequence of more than `budget` tokens down to `budget`,
        each kv head by its own weights (what attend adds up): the `first`
        tokens in front and the `recent` newest stay, and of the others those
        of the largest weights.  Kept tokens in front of the newest stay in
        their places or fill those of the evicted ones, the newest follow in
        their order; places say no longer a token's position, so later appends
        give theirs.  Pages behind the budget are the caller's again; no other
        sequence may share the pages before it.

        Returns (lens_out, weights_out): the lengths (not lens itself) and the
        weights, moved with their tokens and zero behind (weights_out may be
        weights itself).  A sequence whose length is outside its range keeps
        both (and is reported by status)."""
        if self._elsewhere(stream):
            with _on(self.device, stream):
                return self.evict(table, lens, weights, budget, recent=recent, first=first,
                                  lens_out=lens_out, weights_out=weights_out)
        batch = self._batch(table, lens, None, lens.numel())
        w = self._weights(weights, batch, "weights")
        if weights_out is None:
            weights_out = torch.empty_like(weights)
        elif weights_out.shape != weights.shape:
            raise ValueError(f"weights_out must be {tuple(weights.shape)}")
        wo = self._weights(weights_out, batch, "weights_out")
        lens_out = self._lens_out(lens_out, batch.B)
        budget, recent, first = (_int32(budget, "budget"), _int32(recent, "recent"),
                                 _int32(first, "first"))
        key = (batch.B, batch.max_pages, budget, recent)
        nbytes = self._ws.get(key)
        if nbytes is None:
            nbytes = self._lib.vq_kivi_paged_evict_workspace_bytes(self._spec, *key)
            if nbytes and len(self._ws) < 4096:
                self._ws[key] = nbytes
        ws = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        rc = self._lib.vq_kivi_paged_evict(self._spec, batch, w, wo, budget, recent, first,
                                           lens_out.data_ptr() or None, ws.data_ptr() or None,
                                           nbytes, _raw_stream(self._index))
        if rc:
            _lib.check(rc)
        return lens_out, weights_out

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
        outside its range, or a path of kept tokens outside its tree, or gave up
        a wait (synchronizes)."""
        with torch.cuda.device(self.device):
            _lib.check(self._lib.vq_kivi_paged_status(self._spec, _raw_stream(self._index)))
