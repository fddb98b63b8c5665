"""Plain implementations behind the tests of tree attention, draft verification,
kept paths, accumulated weights and eviction, on the CPU in 64 bits or in whole
numbers; and the bounds of the tests."""
import math

import numpy as np
import torch

import paged_ref as ref


# ---- trees -----------------------------------------------------------------------

def masks_of(parents):
    """Bit masks (int64) of one tree: each node sees itself and its ancestors."""
    m = []
    for i, p in enumerate(parents):
        m.append((m[p] if i else 0) | 1 << i)
    return [x - (1 << 64) if x >> 63 else x for x in m]


def depths_of(parents):
    d = []
    for i, p in enumerate(parents):
        d.append(d[p] + 1 if i else 0)
    return d


def random_tree(n, rng, chain=False):
    return [-1] + [i - 1 if chain else rng.randrange(i) for i in range(1, n)]


def seen_by(mask, i, n, S):
    """What new token i of n sees of S tokens."""
    base = S - n
    seen = np.zeros(S, dtype=bool)
    if base + i < 0:
        return seen
    seen[:max(base, 0)] = True
    for j in range(n):
        if mask >> j & 1 and base + j >= 0:
            seen[base + j] = True
    return seen


def attend_seen64(q, pool, table, lens, cu, seen, D, g, H_kv, weight_step, floor, scale=0.0):
    """paged_ref.attend64's outputs and bounds where row i sees seen[i]; and the
    sums of the weights per (sequence, kv head, token) with theirs.

    Weights: a weight's relative error is 2^-20 (exp2 and its argument's
    scaling), twice the score's error and the error of the sum, as for the
    outputs; sums over rows add 2^-23 of the sum per row."""
    q = q.detach().cpu().double().numpy()
    T, H_q, _ = q.shape
    sc = scale if scale > 0 else D ** -0.5
    GQ = H_q // H_kv
    out, err = np.zeros((T, H_q, D)), np.zeros((T, H_q, D))
    tab, sums = table.cpu().numpy(), []
    for b, S in enumerate(lens):
        w, we = np.zeros((H_kv, S)), np.zeros((H_kv, S))
        for h in range(H_kv if S else 0):
            K, V = ref.cache_rows64(pool, tab[b], S, h, D, g)
            for r in range(cu[b], cu[b + 1]):
                see = seen[r]
                if not see.any():
                    continue
                for j in range(GQ):
                    x = q[r, h * GQ + j]
                    s = np.where(see, K @ x * sc, -np.inf)
                    p = np.exp(s - s.max())
                    p /= p.sum()
                    size = (np.abs(K[see]) @ np.abs(x)).max() * sc
                    rel = 2.0 ** -20 + 2 * (D + 4) * 2.0 ** -23 * size + (S / 16 + 4) * 2.0 ** -23
                    a = p @ np.abs(V)
                    out[r, h * GQ + j] = p @ V
                    err[r, h * GQ + j] = 2 * (rel + weight_step) * a + \
                        floor * p.max() * np.abs(V[see]).sum(0)
                    w[h] += p
                    we[h] += 2 * rel * p
        n = (cu[b + 1] - cu[b]) * GQ
        sums.append((w, we + (n + 2) * 2.0 ** -23 * (w + we) + 1e-30))
    return out, err, sums


# ---- verification ------------------------------------------------------------------

UNIT = 2 ** 44


def units(w):
    """fp32 values as whole numbers of 2^-44 (exact in 64 bits)."""
    w = np.where(w > 0, np.minimum(w, 1), 0).astype(np.float64)     # NaN counts as 0
    return np.rint(w * UNIT).astype(np.int64)


def left32(p, q, c):
    """fp32 p - c q, rounded once: the product of two 24-bit numbers is exact in
    64 bits."""
    return (p.astype(np.float64) - np.float64(c) * q.astype(np.float64)).astype(np.float32)


def verify(p, q, tokens, parents, u):
    """One sequence: p, q fp32 [n][V] (q may be None) -> (path, token behind)."""
    n = len(tokens)
    at, path = 0, [0]
    c, mass, gone = np.float32(0), 1.0, []
    i = 0
    while i + 1 < n:
        i += 1
        if parents[i] != at:
            continue
        x, ui = tokens[i], np.float64(u[i])
        if q is not None:
            w = left32(p[at, x:x + 1], q[at, x:x + 1], c)[0] if c else p[at, x]
            good = mass > 0 and ui * np.float64(q[at, x]) * mass < w
        else:
            w = np.float32(0) if x in gone else p[at, x]
            good = mass > 0 and ui * mass < w
        if good:
            at, c, mass, gone = i, np.float32(0), 1.0, []
            path.append(i)
        elif q is not None:
            c = np.float32(np.float64(c) + mass)
            mass = int(units(left32(p[at], q[at], c)).sum()) / UNIT
        else:
            if x not in gone:
                mass = max(mass - int(units(np.array([w]))[0]) / UNIT, 0.0)
                gone.append(x)
    whole = units(left32(p[at], q[at], c) if q is not None and c else p[at])
    whole[gone] = 0
    if whole.sum() == 0:
        whole = units(p[at])
    total = int(whole.sum())
    if total == 0:
        return path, -1
    r = total * int(np.float64(u[0]) * 2 ** 31) >> 31
    return path, int(np.searchsorted(np.cumsum(whole), r, side="right"))


# ---- moved tokens ------------------------------------------------------------------

def move_tokens(pool, table, D, g, moves):
    """The pool (a copy) after moves (sequence, kv head, place, token): all read
    before any is written."""
    old = pool.cpu().numpy()
    new, tab, page = old.copy(), table.cpu().numpy(), old.shape[2] * 16
    c = np.arange(D)
    for b, h, to, src in moves:
        f, t = old[tab[b][src // page], h, src % page // 16], \
            new[tab[b][to // page], h, to % page // 16]
        pf, pt = ref.block_places(D, g, src % 16, c), ref.block_places(D, g, to % 16, c)
        for k in (0, 1):
            t[pt[k]] = f[pf[k]]                         # both codes of a byte are the token's
        f16, t16 = f.view(np.float16), t.view(np.float16)
        for k in (2, 3):
            for d in (0, 2):
                t16.view(np.uint16)[pt[k] + d] = f16.view(np.uint16)[pf[k] + d]
    return torch.from_numpy(new)


def evict_row(w, S, budget, recent, first):
    """The token of each place of one (sequence, kv head) after an eviction."""
    if S <= budget:
        return list(range(S))
    K, hi = budget - recent, S - recent
    w = [(-math.inf if math.isnan(x) else x, not math.isnan(x)) for x in w[:S].tolist()]
    order = sorted(range(first, hi), key=lambda t: (-w[t][0], not w[t][1], t))
    stay = set(order[:K - first]) | set(range(first))
    fill = iter(sorted(t for t in stay if t >= K))
    return [t if t in stay else next(fill) for t in range(K)] + list(range(hi, S))
