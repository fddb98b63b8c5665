"""Plain 64-bit implementations behind the tests of the rotation and of the
paged 4-bit cache, on the CPU, element by element from the documented layout;
and the bounds that their tests use.

Roundings: a value rounded to a type t is off by at most eps(t) / 2 of it
(plus half a subnormal step); every fp32 operation by 2^-24 of its result.
"""
import math
from fractions import Fraction

import numpy as np
import torch

U32 = 2.0 ** -24


def half_step(t):
    """Largest rounding error of the type relative to the value."""
    return torch.finfo(t).eps / 2


def sub_step(t):
    return torch.finfo(t).smallest_normal * torch.finfo(t).eps / 2


# ---- norm and rotation -------------------------------------------------------

def norm_rope64(x, weight, positions, inv_freq, axis, interleaved, scale=1.0, eps=1e-6):
    """x [T][H][D] -> (y, mag) in float64: the result and the magnitude that
    its fp32 errors scale with (|a| + |b| of a rotated pair, |x| behind)."""
    x = x.detach().cpu().double()
    if weight is not None:
        w = weight.detach().cpu().double()
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w
    y, mag = x.clone(), x.abs()
    half = len(inv_freq)
    for j in range(half):
        p = positions[axis[j]].cpu().tolist()
        # the angle reduced exactly (positions are whole numbers)
        turn = Fraction(float(inv_freq[j])) / Fraction("6.283185307179586476925286766559005768")
        ang = torch.tensor([2 * math.pi * float((turn * int(t)) % 1) for t in p],
                           dtype=torch.float64)[:, None]
        c, s = scale * torch.cos(ang), scale * torch.sin(ang)
        i0, i1 = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        a, b = x[..., i0], x[..., i1]
        y[..., i0], y[..., i1] = a * c - b * s, b * c + a * s
        mag[..., i0] = mag[..., i1] = (a.abs() + b.abs()) * max(1.0, abs(scale))
    return y, mag


def norm_rope_bound(y, mag, dtype, D):
    """|result - y|: one rounding to dtype and the fp32 arithmetic before it.
    The norm: D / 2 fused adds deep at most 16 + 4 in a lane's chain, a
    reciprocal root of 2 ulp, two products; cosine and sine: 2 ulp plus the
    angle's 2^-25 turns * 2 pi < 4 * 2^-24; the pair: three operations.  In
    all at most 32 units of 2^-24 of the magnitude."""
    return half_step(dtype) * y.abs() + 32 * U32 * mag + sub_step(dtype)


# ---- the quantizer and the pool ----------------------------------------------

def quantize32(x16, g):
    """fp16 [..., D] -> codes, scale, zero (fp16) in fp32 IEEE arithmetic."""
    x = x16.astype(np.float32).reshape(*x16.shape[:-1], x16.shape[-1] // g, g)
    lo, hi = x.min(-1), x.max(-1)
    lo = (lo + np.float32(0)).astype(np.float32)
    scale = ((hi - lo) / np.float32(15)).astype(np.float32)
    safe = np.where(scale > 0, scale, np.float32(1))
    code = np.rint(((x - lo[..., None]) / safe[..., None]).astype(np.float32))
    code = np.clip(code, 0, 15) * (scale > 0)[..., None]
    s = scale.astype(np.float16)
    over = np.float32(15) * s.astype(np.float32) + lo >= 65520
    s = np.where(over, (s.view(np.uint16) - 1).view(np.float16), s)
    return code.astype(np.uint8).reshape(x16.shape), s, lo.astype(np.float16)


def to_half_sat(x):
    return x.float().clamp(-65504, 65504).half()


def block_places(D, g, tl, c):
    """(key byte, value byte, key meta half, value meta half) of channel c of
    token tl of a block; a code sits in the byte's low nibble for even c."""
    I, ng = D // 32, D // g
    key = tl * (D // 2) + 4 * (c % 32 // 8 * I + c // 32) + c % 8 // 2
    val = 4 * (((8 * (tl // 8) + c % 32 // 4) * 4 + tl % 8 // 2) * I + c // 32) \
        + 2 * (tl % 2) + c % 4 // 2
    meta = ((tl // 2) * ng + c // g) * 4 + tl % 2
    return (key, 8 * D + 64 * ng + val, 4 * D + meta, 4 * D + 32 * ng + 4 * D + meta)


def cache_parts(pool, table_row, S, h, D, g):
    """Codes, scales, zeros of S tokens of kv head h: {"k", "v"} ->
    (code [S][D], scale [S][D], zero [S][D]) from the pool's bytes."""
    pool = pool.cpu().numpy()
    page = pool.shape[2] * 16
    c = np.arange(D)
    out = {"k": ([], [], []), "v": ([], [], [])}
    for t in range(S):
        blk = pool[int(table_row[t // page]), h, t % page // 16]
        f16 = blk.view(np.float16)
        kb, vb, km, vm = block_places(D, g, t % 16, c)
        for key, b, m in (("k", kb, km), ("v", vb, vm)):
            out[key][0].append((blk[b] >> (4 * (c % 2))) & 15)
            out[key][1].append(f16[m])
            out[key][2].append(f16[m + 2])
    return {k: tuple(np.array(x).reshape(S, D) for x in v) for k, v in out.items()}


def cache_rows64(pool, table_row, S, h, D, g):
    """Key and value rows [S][D] in float64 as the pool stands for them."""
    parts = cache_parts(pool, table_row, S, h, D, g)
    rows = []
    for k in ("k", "v"):
        code, s, z = parts[k]
        rows.append((code.astype(np.float64) * s.astype(np.float64) + z.astype(np.float64))
                    .astype(np.float16).astype(np.float64).reshape(S, D))
    return rows


# ---- attention ---------------------------------------------------------------

def attend64(q, pool, table, lens, cu, D, g, H_kv, scale=0.0, weight_step=2.0 ** -21):
    """(out, bound) [T][H_q][D] in float64.  The bound beside the rounding of
    the output: a weight's relative error is weight_step (its own rounding),
    2^-20 (the approximate exp2 and the fp32 scaling of its argument) and
    twice the score's error, at most (D + 4) 2^-23 of sum |q k| scale (fp32
    accumulation, possibly truncating, and the running maximum's subtraction
    of up to 2^-23 of the scores' size); the output sums add 2^-23 per step of
    16 tokens."""
    q = q.detach().cpu().double().numpy()
    T, H_q, _ = q.shape
    sc = scale if scale > 0 else D ** -0.5
    out, err = np.zeros((T, H_q, D)), np.zeros((T, H_q, D))
    lens = [int(x) for x in lens.cpu()]
    cu = list(range(len(lens) + 1)) if cu is None else [int(x) for x in cu.cpu()]
    tab = table.cpu().numpy()
    for b, S in enumerate(lens):
        n = cu[b + 1] - cu[b]
        if n == 0 or S == 0:
            continue
        for h in range(H_kv):
            K, V = cache_rows64(pool, tab[b], S, h, D, g)
            for i in range(n):
                seen = S - n + i + 1
                if seen <= 0:
                    continue
                for j in range(H_q // H_kv):
                    hq = h * (H_q // H_kv) + j
                    x = q[cu[b] + i, hq]
                    s = K[:seen] @ x * sc
                    p = np.exp(s - s.max())
                    p /= p.sum()
                    out[cu[b] + i, hq] = p @ V[:seen]
                    size = (np.abs(K[:seen]) @ np.abs(x)).max() * sc
                    rel = weight_step + 2.0 ** -20 + 2 * (D + 4) * 2.0 ** -23 * size \
                        + (seen / 16 + 4) * 2.0 ** -23
                    # the sum of the weights has the same relative error
                    err[cu[b] + i, hq] = 2 * rel * (p @ np.abs(V[:seen]))
    return out, err


def attend64_rows(q, K, V, seen, scale, weight_step=2.0 ** -21, floor=0.0):
    """As attend64 for rows q [R][D] over K, V [S][D] of one kv head, row r
    seeing the first seen[r] >= 1 tokens; all float64 tensors of one device.
    floor: what a weight is off by beside weight_step of itself, in units of
    the row's largest weight (fp16 has no steps below 2^-24)."""
    S, D = K.shape
    hidden = torch.arange(S, device=q.device) >= torch.as_tensor(seen, device=q.device)[:, None]
    s = (q @ K.T * scale).masked_fill(hidden, -math.inf)
    p = torch.softmax(s, -1)
    size = (q.abs() @ K.abs().T * scale).masked_fill(hidden, 0.0).amax(-1, keepdim=True)
    rel = weight_step + 2.0 ** -20 + 2 * (D + 4) * 2.0 ** -23 * size + (S / 16 + 4) * 2.0 ** -23
    sums = (~hidden).double() @ V.abs()
    err = 2 * rel * (p @ V.abs()) + floor * p.amax(-1, keepdim=True) * sums
    return (p @ V).cpu().numpy(), err.cpu().numpy()


def check_attend(got, want, err, dtype):
    got = got.detach().cpu().double().numpy()
    tol = err + half_step(dtype) * (np.abs(want) + err) + sub_step(dtype)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (f"{bad.sum()} of {bad.size} outside, worst "
                           f"{np.max(np.abs(got - want) / tol):.3g} of the bound")


def make_table(n_seq, lens, page, n_pages, device, seed=0, width=None):
    """Pages in a shuffled order; entries behind a sequence's last page are
    wild."""
    g = torch.Generator().manual_seed(seed)
    order = torch.randperm(n_pages, generator=g).tolist()
    need = [-(-int(s) // page) for s in lens]
    assert sum(need) <= n_pages
    width = max(max(need, default=0), 1) if width is None else width
    table = torch.full((n_seq, width), -7, dtype=torch.int32)
    for b, m in enumerate(need):
        for j in range(m):
            table[b, j] = order.pop()
    return table.to(device)
