"""Trees of drafts over the paged cache, their verification, kept paths,
accumulated weights and eviction on the GPU, against 64-bit implementations
(drafts_ref.py, which also derives the bounds)."""
import math
import random

import numpy as np
import pytest
import torch

import drafts_ref as dref
import paged_ref as ref
from test_gpu_paged import (DT, FEW, FLOOR_FEW, FLOOR_MANY, MANY, filled, i32, lib,  # noqa: F401
                            new_cache, offsets, randn)

pytestmark = pytest.mark.gpu


def i64(x):
    return torch.tensor(list(x), dtype=torch.int64, device="cuda")


def steps_for(rows):
    return (FEW, FLOOR_FEW) if rows <= 8 else (MANY, FLOOR_MANY)


# ---- tree attention ----------------------------------------------------------------

def check_tree(c, table, lens, n, masks, dtype, H_q, H_kv, D, g, seed=7):
    cu = np.concatenate([[0], np.cumsum(n)]).tolist()
    T = cu[-1]
    q = randn(seed, T, H_q, D).to(DT[dtype])
    out = c.attend(q, table, i32(lens), i32(cu), max_new=max(n), tree=i64(masks))
    c.status()
    seen = [dref.seen_by(masks[r], r - cu[b], n[b], lens[b]) for b in range(len(n))
            for r in range(cu[b], cu[b + 1])]
    step, floor = steps_for(max(n) * (H_q // H_kv))
    want, err, _ = dref.attend_seen64(q, c.pool, table, lens, cu, seen, D, g, H_kv, step, floor)
    ref.check_attend(out, want, err, DT[dtype])
    return q, out


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("n,lens,H_q,H_kv,D,g,page", [
    ([4], [4], 2, 1, 64, 32, 16), ([8], [77], 2, 2, 128, 32, 64), ([1, 5], [1, 40], 6, 2, 64, 64, 32),
    ([4, 4], [300, 129], 8, 2, 128, 64, 16),                       # 16 rows of a kv head
    ([16], [16], 4, 1, 128, 128, 16), ([16, 9], [200, 9], 8, 2, 128, 32, 32),
    ([33], [160], 5, 1, 64, 32, 16),                               # rows that fill no tile
    ([64], [64], 2, 2, 64, 64, 64), ([64, 1, 40], [400, 130, 40], 8, 1, 128, 64, 16),
    ([64], [191], 8, 1, 64, 32, 128), ([17, 0, 20], [145, 12, 20], 3, 3, 128, 32, 16),
])
def test_tree_attention(dtype, n, lens, H_q, H_kv, D, g, page):
    rng = random.Random(3)
    c, table, _ = filled(lens, page, H_q, H_kv, D, g, DT[dtype])
    masks = [m for k in n for m in (dref.masks_of(dref.random_tree(k, rng)) if k else [])]
    check_tree(c, table, lens, n, masks, dtype, H_q, H_kv, D, g)


@pytest.mark.parametrize("H_q,n", [(2, 8), (4, 4), (8, 64), (3, 30)])
def test_masks_of_every_form(H_q, n):
    """Masks that are no trees: nothing, everything, later tokens, bits behind
    the last token, bit 63; and a sequence with nothing before its new tokens,
    whose rows without bits are zero."""
    rng = random.Random(5)
    lens, ns = [n, 150], [n, n]
    c, table, _ = filled(lens, 16, H_q, 1, 64, 32)
    masks = [rng.getrandbits(64) for _ in range(2 * n)]
    masks[0] = masks[n + 1] = 0
    masks[1] = masks[n] = (1 << 64) - 1
    masks[2] = masks[n + 2] = 1 << 63
    masks[3] = ((1 << 64) - 1) << n & ((1 << 64) - 1)
    signed = [m - (1 << 64) if m >> 63 else m for m in masks]
    _, out = check_tree(c, table, lens, ns, signed, "fp16", H_q, 1, 64, 32)
    assert (out[0] == 0).all() and (out[3] == 0).all()
    assert (out[1] != 0).any()


@pytest.mark.parametrize("dtype,gain", [("fp16", 6000.0), ("bf16", 1e30), ("bf16", 1e-30)])
@pytest.mark.parametrize("H_q,n", [(2, 8), (4, 16), (8, 20)])
def test_tree_scores_of_any_size(dtype, gain, H_q, n):
    """Queries of any finite size, in each of the three kernels: a row far from
    zero sees its largest score alone, one near it the mean; masks hold."""
    lens = [300 + n, n + 5]
    c, table, L = filled(lens, 16, H_q, 1, 64, 32)
    rng = random.Random(4)
    masks = [m for _ in lens for m in dref.masks_of(dref.random_tree(n, rng))]
    q = (randn(7, 2 * n, H_q, 64) * gain).to(DT[dtype])
    out = c.attend(q, table, L, offsets([n, n]), max_new=n, tree=i64(masks))
    c.status()
    assert torch.isfinite(out).all()
    small = gain < 1
    for b, S in enumerate(lens):
        K, V = (torch.as_tensor(x).cuda() for x in
                ref.cache_rows64(c.pool, table[b].cpu().numpy(), S, 0, 64, 32))
        for i in range(n):
            see = torch.as_tensor(dref.seen_by(masks[b * n + i], i, n, S)).cuda()
            for j in range(H_q):
                x = q[b * n + i, j].double()
                s = torch.where(see, K @ x / 8, -math.inf)
                top = torch.topk(s, 2).values
                got = out[b * n + i, j].double()
                if small:
                    want = V[see].mean(0)
                    tol = 2.0 ** -7 * want.abs() + 2.0 ** -7
                else:
                    # where no other token comes near the largest score
                    if top[0] - top[1] < 60 + 2.0 ** -12 * top[0].abs():
                        continue
                    want = V[int(s.argmax())]
                    tol = 2.0 ** -7 * want.abs() + 1e-6
                assert ((got - want).abs() <= tol).all()


@pytest.mark.parametrize("H_q,n", [(2, 8), (8, 20)])
def test_tree_padding_in_front(H_q, n):
    """New tokens before a sequence's first place see nothing and are seen by
    none."""
    S = n - 3
    c, table, L = filled([S, 40], 16, H_q, 1, 128, 32)
    masks = [(1 << n) - 1] * (2 * n)
    _, out = check_tree(c, table, [S, 40], [n, n], masks, "bf16", H_q, 1, 128, 32)
    assert (out[:3] == 0).all() and (out[3] != 0).any()


@pytest.mark.parametrize("H_q,n", [(4, 4), (4, 2), (4, 30), (8, 64)])
def test_chain_masks_are_the_causal_attention(H_q, n):
    c, table, L = filled([n, 333], 16, H_q, 1, 128, 64, torch.bfloat16)
    q = randn(1, 2 * n, H_q, 128).to(torch.bfloat16)
    masks = dref.masks_of(dref.random_tree(n, random.Random(0), chain=True)) * 2
    a = c.attend(q, table, L, offsets([n, n]), max_new=n, tree=i64(masks))
    b = c.attend(q, table, L, offsets([n, n]), max_new=n)
    # one rounding of the output apart at most (the line of work may be cut elsewhere)
    assert ((a.float() - b.float()).abs() <= 2.0 ** -7 * b.float().abs() + 2.0 ** -12).all()


@pytest.mark.parametrize("H_q,n", [(2, 6), (8, 24)])
def test_tree_nan_and_infinity_stay_where_they_are_seen(H_q, n):
    lens = [50, 60 + n]
    need = sum(-(-s // 16) for s in lens)
    c = new_cache(need + 1, 16, H_q, 1, 64, 32)
    table = ref.make_table(2, lens, 16, need + 1, "cuda", 1)
    T = sum(lens)
    k, v = randn(1, T, 1, 64).half(), randn(2, T, 1, 64).half()
    k[T - 2, 0, 5] = float("nan")
    v[T - 3, 0, 7] = float("nan")
    k[T - 4, 0, 1] = float("inf")
    c.append(k, v, table, i32(lens), offsets(lens))
    masks = [1 << i for i in range(n)] * 2          # each sees itself alone
    masks[n] |= 1 << (n - 1 - 1)                     # and the first also a NaN key
    out = c.attend(randn(3, 2 * n, H_q, 64).half(), table, i32(lens), offsets([n, n]), max_new=n,
                   tree=i64(masks))
    c.status()
    bad = torch.zeros(2 * n, dtype=torch.bool, device="cuda")
    bad[[n, 2 * n - 2, 2 * n - 3]] = True            # token T - 2 is row 2 n - 2
    assert torch.isnan(out[bad]).all() and torch.isfinite(out[~bad]).all()


def test_tree_of_a_long_sequence_and_many_sequences():
    for lens, n, H_q, H_kv, page in (([40000], [37], 8, 2, 128), ([40000], [4], 4, 2, 64),
                                     ([131] * 97, [5] * 97, 4, 1, 16)):
        c, table, L = filled(lens, page, H_q, H_kv, 64, 32)
        rng = random.Random(len(lens))
        masks = [m for k in n for m in dref.masks_of(dref.random_tree(k, rng))]
        q = randn(9, sum(n), H_q, 64).half()
        out = c.attend(q, table, L, offsets(n), max_new=max(n), tree=i64(masks))
        c.status()
        step, floor = steps_for(max(n) * H_q // H_kv)
        at = 0
        for b, S in enumerate(lens[:3]):
            pages = table[b].long()
            for h in range(H_kv):
                K, V = (torch.as_tensor(x).cuda() for x in
                        ref.cache_rows64(c.pool, table[b].cpu().numpy(), S, h, 64, 32)) \
                    if S < 1000 else [x.cuda().double()[:, h] for x in c.dequantize(
                        table, L, offsets([S]), n_tokens=S)]
                for i in range(n[b]):
                    see = torch.as_tensor(dref.seen_by(masks[at + i], i, n[b], S)).cuda()
                    GQ = H_q // H_kv
                    x = q[at + i, h * GQ:(h + 1) * GQ].double()
                    want, err = ref.attend64_rows(x, K[see], V[see], [int(see.sum())] * GQ,
                                                  64 ** -0.5, step, floor)
                    ref.check_attend(out[at + i, h * GQ:(h + 1) * GQ], want, err, torch.float16)
            del pages
            at += n[b]


# ---- verification --------------------------------------------------------------------

def draft_case(seed, n, V, dtype, chain, with_draft, spread=1.0, sharp=2.0):
    rng = random.Random(seed)
    g = torch.Generator().manual_seed(seed)
    T = sum(n)
    logits = sharp * torch.randn(T, V, generator=g)
    p = torch.softmax(logits, -1).to(DT[dtype])
    q = torch.softmax(logits + spread * torch.randn(T, V, generator=g), -1).to(DT[dtype])
    parents, tokens, at = [], [], 0
    for k in n:
        par = dref.random_tree(k, rng, chain) if k else []
        for i in range(k):
            row = q[at + max(par[i], 0)].float()
            tokens.append(int(torch.multinomial(row, 1, generator=g)))
        parents += par
        at += k
    u = torch.rand(T, generator=g)
    return p, q if with_draft else None, tokens, parents, u


def run_verify(p, q, tokens, parents, u, n, wide=True, **kw):
    from bit_kv_cache_05_gb300 import verify_drafts
    tok = torch.tensor(tokens, dtype=torch.int64 if wide else torch.int32, device="cuda")
    return verify_drafts(p.cuda(), tok, u.cuda(), offsets(n),
                         parents=None if parents is None else i32(parents),
                         draft=None if q is None else q.cuda(), **kw)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("with_draft", [True, False])
@pytest.mark.parametrize("n,V,chain,spread", [
    ([1], 1, True, 0.0), ([5], 7, True, 1.0), ([5, 1, 0, 9], 1000, True, 0.5),
    ([64], 31, False, 2.0), ([2, 64, 33, 17, 0, 50], 4099, False, 2.0),
    ([12] * 40, 333, False, 1.0), ([6] * 300, 64, False, 1.5),
])
def test_verify(dtype, with_draft, n, V, chain, spread):
    p, q, tokens, parents, u = draft_case(sum(n) + V, n, V, dtype, chain, with_draft, spread)
    path, counts, after = run_verify(p, q, tokens, parents, u, n)
    if chain:
        again = run_verify(p, q, tokens, None, u, n, wide=False)
        assert torch.equal(again[0], path) and torch.equal(again[1], counts)
        assert torch.equal(again[2].long(), after) and again[2].dtype == torch.int32
    P, Q = p.float().numpy(), None if q is None else q.float().numpy()
    at = 0
    for b, k in enumerate(n):
        s = slice(at, at + k)
        at += k
        if k == 0:
            assert counts[b] == 0 and after[b] == -1
            continue
        want, token = dref.verify(P[s], None if Q is None else Q[s], tokens[s], parents[s],
                                  u[s].numpy())
        assert path[s].tolist() == want + [-1] * (k - len(want)), b
        assert int(counts[b]) == len(want) and int(after[b]) == token, b


@pytest.mark.parametrize("with_draft", [True, False])
def test_verify_large_vocabulary_strided_rows(with_draft):
    """Rows of a wider tensor, on odd addresses; every cluster size."""
    for B, V in ((1, 131071), (40, 50021), (130, 9001)):
        n = [4 + b % 3 for b in range(B)]
        p, q, tokens, parents, u = draft_case(B, n, V, "fp32", False, with_draft, 1.0, 3.0)
        wide = torch.zeros(sum(n), 2, V + 3)
        wide[:, 0, 1:V + 1] = p
        if with_draft:
            wide[:, 1, 2:V + 2] = q
        w = wide.cuda()
        from bit_kv_cache_05_gb300 import verify_drafts
        got = verify_drafts(w[:, 0, 1:V + 1], i64(tokens), u.cuda(), offsets(n),
                            parents=i32(parents), draft=w[:, 1, 2:V + 2] if with_draft else None)
        at = 0
        for b, k in enumerate(n):
            s = slice(at, at + k)
            at += k
            want, token = dref.verify(p[s].numpy(), q[s].numpy() if with_draft else None,
                                      tokens[s], parents[s], u[s].numpy())
            assert got[0][s].tolist() == want + [-1] * (k - len(want))
            assert int(got[2][b]) == token


@pytest.mark.parametrize("dtype,B,n,V,with_draft,kids", [
    ("fp32", 1, 2, 2 ** 19, True, 1), ("fp32", 1, 3, 2 ** 19 - 3, False, 2),
    ("bf16", 1, 2, 2 ** 19, True, 1), ("fp16", 3, 3, 2 ** 19 - 5, True, 2),
    ("fp32", 320, 2, 40001, True, 1), ("fp16", 320, 2, 70001, False, 1),
])
def test_verify_large_slices(dtype, B, n, V, with_draft, kids):
    """Pieces of a warp of more than 16 steps (sums start anew there), and last
    draws in the second step of a warp's run and behind: the largest vocabulary
    over eight CTAs, and one CTA a sequence.  Rows start off a 16-byte boundary
    where V is odd."""
    from bit_kv_cache_05_gb300 import verify_drafts
    dt, T = DT[dtype], B * n
    p = torch.empty(T, V, dtype=dt, device="cuda")
    q = torch.empty_like(p) if with_draft else None
    for a in range(0, T, 64):
        logits = 2 * randn(100 + a, min(64, T - a), V)
        p[a:a + 64] = torch.softmax(logits, -1).to(dt)
        if with_draft:
            q[a:a + 64] = torch.softmax(logits + randn(900 + a, *logits.shape), -1).to(dt)
    rng = random.Random(V)
    parents = ([-1] + [0] * kids + [1])[:n] * B
    tokens = [rng.randrange(V) for _ in range(T)]
    u = torch.rand(T, generator=torch.Generator().manual_seed(V))
    u[1::n] = 0.999 if with_draft else 0.5             # most first children are rejected
    if B == 1:
        uniforms = [0.0, 0.03, 0.31, 0.77, 0.99999994]
    else:
        uniforms = [None]
    for u0 in uniforms:
        if u0 is not None:
            u[0] = u0
        path, counts, after = verify_drafts(p, i64(tokens), u.cuda(), offsets([n] * B),
                                            parents=i32(parents), draft=q)
        for b in range(B):
            s = slice(b * n, b * n + n)
            want, token = dref.verify(p[s].float().cpu().numpy(),
                                      q[s].float().cpu().numpy() if with_draft else None,
                                      tokens[s], parents[s], u[s].numpy())
            assert path[s].tolist() == want + [-1] * (n - len(want)), b
            assert int(counts[b]) == len(want) and int(after[b]) == token, b


def test_verify_rows_without_mass_and_odd_values():
    """Rows of zeros, NaN, infinities and values above one; drafts equal to the
    target (rejections leave nothing); uniforms at their ends."""
    V, n = 40, [3] * 8
    p, q, tokens, parents, u = draft_case(1, n, V, "fp32", False, True)
    p[0:3] = 0
    p[3:6] = float("nan")
    p[6, 5], q[6] = float("inf"), 1e-6
    p[9:12] = q[9:12]                                  # p == q
    u[9:12] = 0.99999994
    p[12, :20] = 3.0
    u[15:18] = 0.0
    q[18:21] = 0.0
    p[21:24] = 0
    p[21:24, V - 1] = 1.0
    got = run_verify(p, q, tokens, parents, u, n)
    for b in range(8):
        s = slice(3 * b, 3 * b + 3)
        want, token = dref.verify(p[s].numpy(), q[s].numpy(), tokens[s], parents[s], u[s].numpy())
        assert got[0][s].tolist() == want + [-1] * (3 - len(want)), b
        assert int(got[2][b]) == token, b
    assert got[2][:2].tolist() == [-1, -1] and got[2][7] in (V - 1,)


def test_verify_bad_sequences_are_left_out():
    from bit_kv_cache_05_gb300 import verify_drafts
    V, n = 50, [3, 3, 3, 3]
    p, q, tokens, parents, u = draft_case(2, n, V, "fp32", False, True)
    good = run_verify(p, q, tokens, parents, u, n)
    for row, what in ((4, "token"), (4, "negative"), (5, "parent"), (4, "root")):
        t, par = list(tokens), list(parents)
        if what == "token":
            t[row] = V
        elif what == "negative":
            t[row] = -1
        elif what == "parent":
            par[row] = 2                                # itself
        else:
            par[row] = -1
        got = run_verify(p, q, t, par, u, n)
        assert got[1].tolist()[1] == -1 and got[2].tolist()[1] == -1
        assert got[0][3:6].tolist() == [-1] * 3
        for x, y in zip(got[1:], good[1:]):
            assert x[[0, 2, 3]].tolist() == y[[0, 2, 3]].tolist()
    # a root's token and parent are not looked at
    t, par = list(tokens), list(parents)
    t[0], par[0] = V + 9, 77
    got = run_verify(p, q, t, par, u, n)
    assert all(torch.equal(x, y) for x, y in zip(got, good))
    # offsets: behind the rows, falling, more than 64 nodes
    big = draft_case(3, [70], V, "fp32", False, True)
    assert run_verify(*big, [70])[1].tolist() == [-1]
    cu = i32([0, 3, 2, 9, 13])
    got = verify_drafts(p.cuda(), i64(tokens), u.cuda(), cu, parents=i32(parents), draft=q.cuda())
    assert got[1].tolist()[1] == -1 and got[1].tolist()[3] == -1
    assert got[1].tolist()[0] == int(good[1][0])


def test_verify_arguments_of_other_shapes():
    """Every tensor with a dimension less or more: the argument is named."""
    from bit_kv_cache_05_gb300 import verify_drafts
    V, n = 50, [3, 2]
    p, q, tokens, parents, u = draft_case(3, n, V, "fp32", False, True)
    good = dict(target=p.cuda(), tokens=i64(tokens), uniforms=u.cuda(), cu_new=offsets(n),
                parents=i32(parents), draft=q.cuda(), path=i32([0] * 5), counts=i32([0, 0]),
                after=i64([0, 0]))
    verify_drafts(**good)
    for name, t in good.items():
        for bad in (t[0], t[:, 0] if t.dim() > 1 else t[:1], t[None], t.flatten()[0], t[:0]):
            if bad.shape == t.shape:
                continue
            with pytest.raises(ValueError):
                verify_drafts(**dict(good, **{name: bad}))


def test_verify_too_many_nodes_clear_their_path():
    """More nodes than a tree has, their rows in range: -1 in all of their path;
    rows behind the last sequence stay as they were."""
    n, V, extra = [3, 70, 2, 2000], 50, 4
    p, q, tokens, parents, u = draft_case(3, n, V, "fp32", False, True)
    T = sum(n)
    pad = lambda t: torch.cat((t, torch.zeros(extra, *t.shape[1:], dtype=t.dtype)))
    path = torch.full((T + extra,), 9, dtype=torch.int32, device="cuda")
    got = run_verify(pad(p), pad(q), tokens + [0] * extra, parents + [0] * extra, pad(u), n,
                     path=path)
    assert got[0] is path and got[1].tolist()[1::2] == [-1, -1]
    assert got[2].tolist()[1::2] == [-1, -1]
    assert (path[3:73] == -1).all() and (path[75:T] == -1).all() and (path[T:] == 9).all()
    # offsets behind the rows: nothing of them is written
    path.fill_(9)
    got = run_verify(p[:60], q[:60], tokens[:60], parents[:60], u[:60], [3, 70], path=path[:60])
    assert got[1].tolist()[1] == -1 and (path[3:] == 9).all()


@pytest.mark.parametrize("B,V", [(5, 40000), (50, 9000), (100, 5000), (200, 300)])
def test_verify_every_way_out_of_a_cluster(B, V):
    """Clusters of eight, four, two and one CTAs, whose sequences walk, have no
    nodes, too many of them, or a parent outside its range, side by side."""
    n = [(6, 0, 4, 70, 1)[b % 5] for b in range(B)]
    p, q, tokens, parents, u = draft_case(B, n, V, "fp32", False, True, 1.0, 3.0)
    at = np.cumsum([0] + n)
    bad = [b for b in range(B) if b % 10 == 2]
    for b in bad:
        parents[at[b] + 2] = 2
    for _ in range(3):
        path, counts, after = run_verify(p, q, tokens, parents, u, n)
        for b, k in enumerate(n):
            s = slice(at[b], at[b + 1])
            if k == 0 or k > 64 or b in bad:
                assert int(counts[b]) == (0 if k == 0 else -1) and int(after[b]) == -1
                continue
            want, token = dref.verify(p[s].numpy(), q[s].numpy(), tokens[s], parents[s],
                                      u[s].numpy())
            assert path[s].tolist() == want + [-1] * (k - len(want)), b
            assert int(counts[b]) == len(want) and int(after[b]) == token, b


@pytest.mark.parametrize("with_draft", [True, False])
@pytest.mark.parametrize("kids", [1, 3])
def test_verified_tokens_follow_the_target(with_draft, kids):
    """The first token behind the root is distributed as the target's row,
    whatever the draft: 60 batches of 1024 walks, each count within 5 standard
    deviations (the seeds are fixed)."""
    from bit_kv_cache_05_gb300 import verify_drafts
    V, B, rounds = 6, 1024, 60
    g = torch.Generator(device="cuda").manual_seed(4)
    p = torch.tensor([0.4, 0.05, 0.25, 0.0, 0.2, 0.1], device="cuda")
    q = torch.tensor([0.1, 0.4, 0.1, 0.2, 0.2, 0.0], device="cuda")
    n = 1 + kids
    rows_p, rows_q = p.repeat(B * n, 1), q.repeat(B * n, 1)
    cu = offsets([n] * B)
    parents = i32([-1] + [0] * kids).repeat(B)
    seen = torch.zeros(V, device="cuda")
    for _ in range(rounds):
        if with_draft:
            t = torch.multinomial(q.repeat(B, 1), n, replacement=True, generator=g)
        else:
            t = torch.tensor([0, 1, 4, 2], device="cuda")[:n].repeat(B, 1)
        u = torch.rand(B * n, generator=g, device="cuda")
        path, counts, after = verify_drafts(rows_p, t.flatten(), u, cu, parents=parents,
                                            draft=rows_q if with_draft else None)
        path = path.view(B, n)
        first = torch.where(counts > 1, t.gather(1, path[:, 1:2].clamp(min=0).long())[:, 0], after)
        seen += torch.bincount(first, minlength=V)
    N = B * rounds
    sigma = torch.sqrt(N * p * (1 - p))
    assert ((seen - N * p).abs() <= 5 * sigma).all(), (seen / N).tolist()
    assert seen[3] == 0


# ---- kept paths -----------------------------------------------------------------------

@pytest.mark.parametrize("D,g,page,H_kv", [(64, 32, 16, 3), (64, 64, 64, 1), (128, 32, 16, 2),
                                           (128, 64, 32, 40), (128, 128, 128, 1)])
def test_keep(D, g, page, H_kv):
    rng = random.Random(D + g)
    n = [1, 5, 64, 0, 33, 16, 20, 7]
    lens = [1, 5, 200, 9, 40, 16 + 7, 15, 90]          # the seventh: 5 tokens of padding
    paths = [[0], [0, 1, 4], sorted(rng.sample(range(64), 40)), [], list(range(33)), [15],
             [5, 9, 19], []]
    c, table, L = filled(lens, page, H_kv, H_kv, D, g)
    before = c.pool.clone()
    flat, moves, want = [], [], []
    for b, (k, S, p) in enumerate(zip(n, lens, paths)):
        flat += p + [-9] * (k - len(p))
        base = S - k
        start = max(base, 0)
        want.append(start + len(p) if k else S)
        moves += [(b, h, start + j, base + x) for h in range(H_kv) for j, x in enumerate(p)]
    out = c.keep(table, L, offsets(n), i32(flat), i32([len(p) for p in paths]))
    c.status()
    assert out.tolist() == want
    assert torch.equal(c.pool.cpu(), dref.move_tokens(before, table, D, g, moves))
    # in place
    c.pool.copy_(before)
    lens2 = L.clone()
    assert c.keep(table, lens2, offsets(n), i32(flat), i32([len(p) for p in paths]),
                  lens_out=lens2) is lens2
    assert lens2.tolist() == want
    assert torch.equal(c.pool.cpu(), dref.move_tokens(before, table, D, g, moves))


def test_keep_lengths_into_the_counts():
    """The counts' own array may take the lengths; neighbours of one buffer are
    apart."""
    c, table, L = filled([20, 30, 9], 16, 2, 2, 64, 32)
    n, path, counts = [4, 6, 5], [0, 2, -1, -1, 0, 1, 5, -1, -1, -1, 0, 4, -1, -1, -1], [2, 3, 2]
    before = c.pool.clone()
    want = c.keep(table, L, offsets(n), i32(path), i32(counts))
    pool = c.pool.clone()
    buffer = torch.cat((L, i32([0] * 3), i32(counts), offsets(n), i32(path)))
    lens, lens_out, k, cu, p = buffer.split([3, 3, 3, 4, 15])
    for out in (lens_out, k):
        c.pool.copy_(before)
        assert torch.equal(c.keep(table, lens, cu, p, k, lens_out=out), want)
        assert torch.equal(c.pool, pool)
    c.status()


@pytest.mark.parametrize("path,count", [
    ([0, 2, 2, 3], 4), ([0, 3, 1, 2], 3), ([0, 1, 2, 4], 4), ([-1, 0, 1, 2], 2), ([0, 1, 2, 3], 5),
    ([0, 1, 2, 3], -1),
])
def test_keep_leaves_bad_paths(path, count):
    from bit_kv_cache_05_gb300 import _lib
    c, table, L = filled([20, 30], 16, 2, 2, 64, 32)
    before = c.pool.clone()
    out = c.keep(table, L, offsets([4, 4]), i32(path + [1, 2, 3, 0]), i32([count, 2]))
    with pytest.raises(_lib.VqError, match="path"):
        c.status()
    assert out.tolist() == [20, 28]
    moves = [(1, h, 26 + j, 27 + j) for h in range(2) for j in range(2)]
    assert torch.equal(c.pool.cpu(), dref.move_tokens(before, table, 64, 32, moves))


def test_keep_bad_pages_and_lengths():
    from bit_kv_cache_05_gb300 import _lib
    c, table, L = filled([40, 40], 16, 1, 1, 64, 32)
    t2 = table.clone()
    t2[0, 2] = 99
    before = c.pool.clone()
    out = c.keep(t2, L, offsets([12, 12]), i32([0, 5] + [0] * 10 + [0, 5] + [0] * 10),
                 i32([2, 2]))
    with pytest.raises(_lib.VqError, match="page"):
        c.status()
    assert out.tolist() == [30, 30]
    # the first sequence's token lies on the bad page: not moved
    assert torch.equal(c.pool.cpu(), dref.move_tokens(before, table, 64, 32, [(1, 0, 29, 33)]))
    bad = i32([40, 49])
    c.pool.copy_(before)
    out = c.keep(table, bad, offsets([12, 12]), i32([0] * 24), i32([0, 0]))
    with pytest.raises(_lib.VqError, match="length"):
        c.status()
    assert out.tolist() == [28, 49] and torch.equal(c.pool, before)


# ---- accumulated weights ------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("n,lens,H_q,H_kv,D,g,page", [
    (None, [1], 1, 1, 64, 32, 16), (None, [0, 33, 500], 8, 2, 128, 32, 32),
    (None, [64, 31], 3, 3, 64, 64, 16), (None, [700], 8, 1, 128, 128, 64),
    ([4, 2, 0], [40, 2, 17], 4, 1, 64, 32, 16), ([2, 2], [2, 100], 10, 2, 128, 64, 16),
    ([3], [2], 2, 1, 64, 64, 16),
])
def test_weights(dtype, n, lens, H_q, H_kv, D, g, page):
    c, table, L = filled([max(s, 1) for s in lens], page, H_q, H_kv, D, g, DT[dtype])
    L = i32(lens)
    ns = [1] * len(lens) if n is None else n
    cu = np.concatenate([[0], np.cumsum(ns)]).tolist()
    q = randn(11, cu[-1], H_q, D).to(DT[dtype])
    places = table.shape[1] * page
    acc = torch.rand(len(lens), H_kv, places + 3, device="cuda")
    before = acc.clone()
    a = dict(max_new=max(ns)) if n else {}
    out = c.attend(q, table, L, None if n is None else i32(cu), weights=acc, **a)
    c.status()
    seen = [dref.seen_by((1 << i + 1) - 1, i, ns[b], lens[b]) for b in range(len(lens))
            for i in range(ns[b])]
    step, floor = steps_for(max(ns) * H_q // H_kv)
    want, err, sums = dref.attend_seen64(q, c.pool, table, lens, cu, seen, D, g, H_kv, step, floor)
    ref.check_attend(out, want, err, DT[dtype])
    assert torch.equal(out, c.attend(q, table, L, None if n is None else i32(cu), **a))
    got, old = acc.cpu().double().numpy(), before.cpu().double().numpy()
    for b, (w, we) in enumerate(sums):
        S = lens[b]
        assert (acc[b, :, S:] == before[b, :, S:]).all()
        tol = we + 2.0 ** -24 * (old[b, :, :S] + w + we)
        assert (np.abs(got[b, :, :S] - (old[b, :, :S] + w)) <= tol).all()
    # a second pass adds the same again, bit for bit the same way
    other = before.clone()
    c.attend(q, table, L, None if n is None else i32(cu), weights=other, **a)
    assert torch.equal(other, acc)


@pytest.mark.parametrize("dtype,gain", [("fp16", 6000.0), ("bf16", 1e30), ("bf16", 1e-30)])
@pytest.mark.parametrize("H_q,n", [(4, 1), (4, 2), (8, 2)])
def test_weights_of_scores_of_any_size(dtype, gain, H_q, n):
    """Queries of any finite size: the weights of a row still sum to one, all on
    the largest score where no other comes near it, equal ones near zero."""
    S = 700
    c, table, L = filled([S], 16, H_q, 1, 64, 32)
    q = (randn(3, n, H_q, 64) * gain).to(DT[dtype])
    acc = torch.zeros(1, 1, table.shape[1] * 16, device="cuda")
    c.attend(q, table, L, offsets([n]), max_new=n, weights=acc)
    c.status()
    # each weight is off by 2^-20 of itself, a row's sum by as much
    assert abs(float(acc.double().sum()) - n * H_q) <= n * H_q * 2.0 ** -18
    K = torch.as_tensor(ref.cache_rows64(c.pool, table[0].cpu().numpy(), S, 0, 64, 32)[0]).cuda()
    want, open_rows = torch.zeros(S, dtype=torch.float64, device="cuda"), 0
    for i in range(n):
        seen = S - n + i + 1
        for j in range(H_q):
            s = (K @ q[i, j].double() / 8)[:seen]
            if gain < 1:
                want[:seen] += 1 / seen
                continue
            top = torch.topk(s, 2).values
            if top[0] - top[1] < 60 + 2.0 ** -12 * top[0].abs():
                open_rows += 1
            else:
                want[int(s.argmax())] += 1
    off = (acc[0, 0, :S].double() - want).abs()
    if gain < 1:
        assert off.max() <= n * H_q * 2.0 ** -18 / (S - n)
    else:
        assert off.sum() <= 2 * open_rows + n * H_q * 2.0 ** -18


def test_weights_of_nan_tokens_bad_pages_and_strides():
    from bit_kv_cache_05_gb300 import _lib
    lens = [40, 50]
    c = new_cache(9, 16, 2, 1, 64, 32)
    table = ref.make_table(2, lens, 16, 9, "cuda", 1)
    k, v = randn(1, 90, 1, 64).half(), randn(2, 90, 1, 64).half()
    k[60, 0, 3] = float("nan")                      # place 20 of the second
    c.append(k, v, table, i32(lens), offsets(lens))
    big = torch.zeros(1, 2, 2 * 64 + 10, device="cuda")
    acc = big[0, :, 5:69][:, None]                  # [2][1][64], strided
    q = randn(3, 3, 2, 64).half()
    c.attend(q, table, i32(lens), offsets([1, 2]), max_new=2, weights=acc)
    c.status()
    # row 50 - 2 of the second sequence and the next see the NaN; nothing is
    # added where no row sees a token
    assert torch.isnan(acc[1, 0, :50]).all() and (acc[1, 0, 50:] == 0).all()
    assert torch.isfinite(acc[0]).all() and abs(float(acc[0].sum()) - 2) < 1e-4
    assert (big[0, :, :5] == 0).all() and (big[0, :, 69:] == 0).all()
    t2 = table.clone()
    t2[0, 1] = -5
    acc = torch.zeros(2, 1, 64, device="cuda")
    c.attend(q[:2], t2, i32([40, 20]), weights=acc)
    with pytest.raises(_lib.VqError, match="page"):
        c.status()
    assert torch.isfinite(acc).all() and abs(float(acc[1].sum()) - 2) < 1e-4
    # a length outside its range: left out
    acc = torch.zeros(2, 1, 64, device="cuda")
    c.attend(q[:2], table, i32([65, 20]), weights=acc)
    with pytest.raises(_lib.VqError, match="length"):
        c.status()
    assert (acc[0] == 0).all() and abs(float(acc[1].sum()) - 2) < 1e-4


# ---- eviction ---------------------------------------------------------------------------

def evict_weights(lens, H_kv, places, kind, seed=3):
    g = torch.Generator().manual_seed(seed)
    w = torch.exp(2 * torch.randn(len(lens), H_kv, places, generator=g))
    if kind == "ties":
        w = torch.randint(0, 3, w.shape, generator=g).float()
    elif kind == "equal":
        w = torch.full_like(w, 0.25)
    elif kind == "wild":
        pick = torch.randint(0, 8, w.shape, generator=g)
        for i, x in enumerate((float("nan"), float("inf"), -1.0, -0.0, 0.0, float("-inf"), 1e-42)):
            w[pick == i] = x
    return w.cuda()


def same_floats(a, b):
    return torch.equal(torch.nan_to_num(a, nan=123.5), torch.nan_to_num(b, nan=123.5)) and \
        torch.equal(torch.isnan(a), torch.isnan(b))


def check_evict(c, table, lens, w, budget, recent, first, D, g, in_place=False):
    H_kv, places = w.shape[1:]
    before, w0 = c.pool.clone(), w.clone()
    out, wo = c.evict(table, i32(lens), w, budget, recent=recent, first=first,
                      weights_out=w if in_place else None)
    c.status()
    assert out.tolist() == [min(s, budget) for s in lens]
    moves, want = [], torch.zeros_like(w0).cpu()
    cpu = w0.cpu()
    for b, S in enumerate(lens):
        for h in range(H_kv):
            take = dref.evict_row(cpu[b, h], S, budget, recent, first)
            want[b, h, :len(take)] = cpu[b, h, take]
            moves += [(b, h, i, t) for i, t in enumerate(take) if i != t]
    assert same_floats(wo.cpu(), want)
    if not in_place:
        assert same_floats(w, w0)
    assert torch.equal(c.pool.cpu(), dref.move_tokens(before, table, D, g, moves))
    return out, wo


@pytest.mark.parametrize("kind", ["plain", "ties", "equal", "wild"])
@pytest.mark.parametrize("lens,budget,recent,first,H_kv,D,g,page", [
    ([40], 20, 5, 2, 1, 64, 32, 16), ([41, 0, 20, 21, 100], 20, 0, 0, 2, 64, 64, 16),
    ([300, 17], 100, 100, 0, 3, 128, 32, 32), ([300, 280], 130, 60, 70, 1, 128, 64, 16),
    ([77], 1, 0, 0, 1, 64, 32, 16), ([77], 1, 1, 0, 2, 64, 32, 16), ([90], 89, 40, 4, 2, 128, 128, 64),
    ([700, 513], 512, 64, 4, 2, 64, 32, 16),
])
def test_evict(kind, lens, budget, recent, first, H_kv, D, g, page):
    c, table, _ = filled([max(s, 1) for s in lens], page, H_kv, H_kv, D, g)
    w = evict_weights(lens, H_kv, table.shape[1] * page, kind)
    check_evict(c, table, lens, w, budget, recent, first, D, g)
    c.pool.random_(0, 256)
    # (more places than the tables have room for: zero as well)
    w = torch.cat((w, torch.ones(len(lens), H_kv, 7, device="cuda")), -1)
    check_evict(c, table, lens, w, budget, recent, first, D, g)
    c.pool.random_(0, 256)
    check_evict(c, table, lens, w, budget, recent, first, D, g, in_place=True)


@pytest.mark.parametrize("lens,budget,recent,first,H_kv", [
    ([20000, 9000], 3001, 700, 4, 1), ([5000], 4800, 4000, 2, 2), ([2500] * 40, 1200, 100, 0, 4),
])
def test_evict_long_rows(lens, budget, recent, first, H_kv):
    """More tokens than one round of a cluster takes; every cluster size."""
    c, table, _ = filled(lens, 128, H_kv, H_kv, 64, 64)
    w = evict_weights(lens, H_kv, table.shape[1] * 128, "plain")
    before = c.pool.clone()
    K0, V0 = c.dequantize(table, i32(lens), offsets(lens), n_tokens=sum(lens))
    out, wo = c.evict(table, i32(lens), w, budget, recent=recent, first=first)
    c.status()
    stay = [min(s, budget) for s in lens]
    K1, V1 = c.dequantize(table, out, offsets(stay), n_tokens=sum(stay))
    a = o = 0
    for b, S in enumerate(lens):
        for h in range(H_kv):
            take = torch.tensor(dref.evict_row(w[b, h].cpu(), S, budget, recent, first)).cuda()
            assert torch.equal(K1[o:o + stay[b], h], K0[a:a + S, h][take])
            assert torch.equal(V1[o:o + stay[b], h], V0[a:a + S, h][take])
            assert torch.equal(wo[b, h, :stay[b]], w[b, h][take])
        assert (wo[b, :, stay[b]:] == 0).all()
        a, o = a + S, o + stay[b]
    # in place gives the same pool and weights
    first_pool = c.pool.clone()
    c.pool.copy_(before)
    c.evict(table, i32(lens), w, budget, recent=recent, first=first, weights_out=w)
    c.status()
    assert torch.equal(c.pool, first_pool) and torch.equal(w, wo)


def test_evict_strides_bad_pages_and_lengths():
    from bit_kv_cache_05_gb300 import _lib
    lens = [60, 60, 60]
    c, table, _ = filled(lens, 16, 2, 2, 64, 32)
    w = evict_weights(lens, 2, 64, "plain")
    wide = torch.full((2, 3, 70), 9.0, device="cuda")
    view = wide[:, :, 3:67].transpose(0, 1)            # [3][2][64], heads outermost
    view.copy_(w)
    check_evict(c, table, lens, view, 30, 8, 2, 64, 32, in_place=True)
    assert (wide[:, :, :3] == 9).all() and (wide[:, :, 67:] == 9).all()
    t2 = table.clone()
    t2[1, 3] = 99
    c.pool.random_(0, 256)
    before = c.pool.clone()
    L = i32([60, 60, 65])
    out, wo = c.evict(t2, L, w, 30, recent=8, first=2)
    with pytest.raises(_lib.VqError, match="page.*length"):
        c.status()
    assert out.tolist() == [30, 30, 65]
    moves = []
    for b in (0, 1):
        for h in (0, 1):
            take = dref.evict_row(w[b, h].cpu(), 60, 30, 8, 2)
            moves += [(b, h, i, t) for i, t in enumerate(take) if i != t and not (b == 1 and t >= 48)]
    assert torch.equal(c.pool.cpu(), dref.move_tokens(before, table, 64, 32, moves))


def evict_by_sorting(w, lens, budget, recent, first):
    """The token of each place of every row [B][H_kv][budget], by a stable sort
    (dref.evict_row says the same; a test compares them)."""
    K, t = budget - recent, torch.arange(w.shape[-1], device=w.device)
    hi = (lens.long() - recent)[:, None, None]
    candidate = (t >= first) & (t < hi)
    # NaN lowest, below -infinity; behind both what does not compete
    size = torch.where(torch.isnan(w), -math.inf, w.double() + 0.0)
    one = torch.sort(size, dim=-1, descending=True, stable=True)[1]
    group = torch.where(candidate, torch.isnan(w).long(), 2).gather(-1, one)
    order = one.gather(-1, torch.sort(group, dim=-1, stable=True)[1])
    rank = torch.empty_like(order).scatter_(-1, order, t.expand_as(order))
    stays = candidate & (rank < K - first) | (t < first)
    hole = ~stays & (t < K)
    source = torch.sort((~(stays & (t >= K))).to(torch.uint8), dim=-1, stable=True)[1]
    take = torch.where(hole, source.gather(-1, (hole.cumsum(-1) - 1).clamp(min=0)), t)
    return torch.where(t < K, take, hi - K + t)[..., :budget]


def test_evictions_of_the_references_agree():
    for kind in ("plain", "ties", "equal", "wild"):
        w = evict_weights([0, 0], 3, 90, kind)
        lens = [90, 71]
        got = evict_by_sorting(w, i32(lens), 50, 17, 3)
        for b, S in enumerate(lens):
            for h in range(3):
                assert got[b, h].tolist() == dref.evict_row(w[b, h].cpu(), S, 50, 17, 3)


# What a row is shared by: rows of up to 1536 places, and longer ones of at least
# eight per SM or of which few tokens go, take one CTA of 256 threads; others a
# cluster of at most eight CTAs of 512, as many as there are SMs for and 1024
# places each.
@pytest.mark.parametrize("kind", ["plain", "ties", "equal", "wild"])
@pytest.mark.parametrize("ctas,rows,S,budget,recent,first,D,g", [
    (2, 4, 2000, 900, 100, 4, 128, 32), (4, 4, 4000, 1500, 300, 0, 128, 64),
    (8, 2, 9000, 2500, 64, 4, 128, 32), (8, 2, 8100, 8000, 6000, 3, 128, 128),
    (2, "3/4", 5000, 600, 0, 0, 128, 32), (4, "3/8", 5000, 600, 77, 2, 64, 64),
    (1, "2", 1800, 500, 33, 1, 64, 32), (1, "9", 1700, 400, 20, 4, 64, 64),
    (1, 3, 5000, 4993, 64, 4, 128, 32),
])
def test_evict_over_clusters(kind, ctas, rows, S, budget, recent, first, D, g):
    """Clusters of two, four and eight and the forms of one CTA, at ties, equal
    weights, NaN and infinities: the order of equal weights crosses CTAs."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    H = 2
    if isinstance(rows, str):                          # rows by the number of SMs
        a, _, b = rows.partition("/")
        rows = int(sms * int(a) / int(b or 1)) // H * H
    B, page = rows // H if rows % H == 0 else rows, 128
    H = rows // B
    lens = [S - b % 7 for b in range(B)]
    need = sum(-(-s // page) for s in lens)
    c = new_cache(need + 2, page, H, H, D, g, 0)
    c.pool.view(-1)[:] = torch.randint(0, 256, (c.pool.numel(),), dtype=torch.uint8, device="cuda",
                                       generator=torch.Generator("cuda").manual_seed(S))
    # (random bytes: scales may be NaN, so compare the rows' bits)
    table, L = ref.make_table(B, lens, page, need + 2, "cuda", 1), i32(lens)
    w = evict_weights(lens, H, table.shape[1] * page, kind)
    before = c.pool.clone()

    def rows_of(pool, place):
        """The 16-bit parts of tokens place [B][H][n], in one order."""
        ng, I, t = D // g, D // 32, torch.arange(16, device="cuda")[:, None]
        x = torch.arange(D // 4, device="cuda")
        m = torch.arange(2 * ng, device="cuda")
        meta = 4 * D + (t // 2 * ng + m // 2) * 4 + 2 * (m % 2) + t % 2
        value = 2 * (((8 * (t // 8) + x // I) * 4 + t % 8 // 2) * I + x % I) + t % 2
        half = 4 * D + 32 * ng
        parts = torch.cat((t * (D // 4) + x, meta, half + value, half + meta), 1)
        b = torch.arange(B, device="cuda")[:, None, None]
        h = torch.arange(H, device="cuda")[:, None]
        blk = (table[b, place // page].long() * H + h) * (page // 16) + place % page // 16
        at = blk[..., None] * (pool.shape[-1] // 2) + parts[place % 16]
        return pool.view(torch.int16).view(-1)[at]

    take = evict_by_sorting(w, L, budget, recent, first)
    places = torch.arange(budget, device="cuda").expand_as(take)
    want = rows_of(before, take)
    for in_place in (False, True):
        c.pool.copy_(before)
        w0 = w.clone()
        lens_out, wo = c.evict(table, L, w, budget, recent=recent, first=first,
                               weights_out=w if in_place else None)
        c.status()
        assert (lens_out == budget).all()
        assert torch.equal(rows_of(c.pool, places), want)
        assert same_floats(wo[..., :budget], w0.gather(-1, take))
        assert (wo[..., budget:] == 0).all()


@pytest.mark.parametrize("budget", [30, 64])
def test_evict_keeps_the_weights_of_what_it_leaves_out(budget):
    """Lengths outside their range: their weights come out as they went in, in
    an array of its own and in place."""
    from bit_kv_cache_05_gb300 import _lib
    lens = [60] * 5
    c, table, _ = filled(lens, 16, 2, 2, 64, 32)
    w = evict_weights(lens, 2, 70, "wild")
    L = i32([60, 65, -1, 20, 2 ** 31 - 1])
    wo = torch.full_like(w, 9.0)
    for out in (wo, None, w):
        before, w0 = c.pool.clone(), w.clone()
        lens_out, got = c.evict(table, L, w, budget, recent=8, first=2, weights_out=out)
        with pytest.raises(_lib.VqError, match="length"):
            c.status()
        assert lens_out.tolist() == [min(60, budget), 65, -1, 20, 2 ** 31 - 1]
        for b in (1, 2, 4):
            assert same_floats(got[b], w0[b])
        assert same_floats(got[3, :, :20], w0[3, :, :20]) and (got[3, :, 20:] == 0).all()
        for b in (1, 2, 3, 4):
            pages = table[b].long()
            assert torch.equal(c.pool[pages], before[pages])


# ---- together ---------------------------------------------------------------------------

def test_speculative_steps_together():
    """Prompts, then steps as a server makes them: a tree of drafts appended
    with its depths' positions, attended, verified, and the kept path moved
    together.  The cache then is what appending the kept tokens alone gives."""
    from bit_kv_cache_05_gb300 import verify_drafts
    from bit_kv_cache_05_gb300.rope import Rope
    D, g, page, H_q, H_kv, dt, B, V = 128, 32, 16, 8, 2, torch.bfloat16, 3, 257
    rope, rng = Rope(rot_dim=D, theta=5e5), random.Random(8)
    table = ref.make_table(B, [192] * B, page, 40, "cuda", 2, width=12)
    c, plain = new_cache(40, page, H_q, H_kv, D, g), new_cache(40, page, H_q, H_kv, D, g)
    lens = [30, 7, 1]
    T = sum(lens)
    x = randn(1, T, 2 * H_kv, D).to(dt)
    for z in (c, plain):
        z.append(x[:, :H_kv], x[:, H_kv:], table, i32(lens), offsets(lens), rope=rope)
    L = i32(lens)
    for step in range(4):
        n = [rng.choice([3, 20, 9]) for _ in range(B)]
        p, q, tokens, parents, u = draft_case(50 + step, n, V, "fp32", False, step % 2 == 0, 0.3)
        cu, T = offsets(n), sum(n)
        trees, at = [], 0
        for k in n:
            trees.append(parents[at:at + k])
            at += k
        masks = i64(m for t in trees for m in dref.masks_of(t))
        depth = i32(d for t in trees for d in dref.depths_of(t))
        full = L + i32(n)
        x = randn(60 + step, T, H_q + 2 * H_kv, D).to(dt)
        qq, k, v = x[:, :H_q], x[:, H_q:H_q + H_kv], x[:, H_q + H_kv:]
        seq = torch.repeat_interleave(torch.arange(B, device="cuda"), i64(n))
        rotated = c.append(k, v, table, full, cu, q=qq, rope=rope, positions=L[seq] + depth)
        out = c.attend(rotated, table, full, cu, max_new=max(n), tree=masks)
        path, counts, after = run_verify(p, q, tokens, parents, u, n)
        L = c.keep(table, full, cu, path, counts)
        c.status()
        # the kept tokens alone
        kept = [int(x) for x in counts]
        rows = [int(cu[b]) + int(path[int(cu[b]) + j]) for b in range(B) for j in range(kept[b])]
        rq = plain.append(k[rows], v[rows], table, L, offsets(kept), q=qq[rows], rope=rope)
        assert torch.equal(rq, rotated[rows])
        a = plain.dequantize(table, L, torch.cat((i32([0]), L.cumsum(0).int())),
                             n_tokens=int(L.sum()))
        b_ = c.dequantize(table, L, torch.cat((i32([0]), L.cumsum(0).int())),
                          n_tokens=int(L.sum()))
        assert torch.equal(a[0], b_[0]) and torch.equal(a[1], b_[1])
        # a kept node's attention is the chain's
        chain = plain.attend(rq, table, L, offsets(kept), max_new=max(kept))
        plain.status()
        d = (out[rows].float() - chain.float()).abs()
        assert (d <= 2.0 ** -7 * chain.float().abs() + 2.0 ** -7 * chain.float().abs().mean()).all()


def test_captured_eviction_loop():
    """Decode steps with weights and an eviction, captured into one graph: the
    cache stays at its budget and follows tables and lengths of the replay."""
    B, H_q, H_kv, D, g, page, budget = 2, 4, 2, 64, 32, 16, 48
    c, table, L = filled([48, 48], page, H_q, H_kv, D, g, torch.float16, fill=0)
    free = sorted(set(range(c.n_pages)) - set(table.flatten().tolist()))
    table = torch.cat((table, i32(free[:2])[:, None]), 1)
    acc = torch.zeros(B, H_kv, table.shape[1] * page, device="cuda")
    k, v, q = randn(1, B, H_kv, D).half(), randn(2, B, H_kv, D).half(), randn(3, B, H_q, D).half()
    lens = L + 1
    out, lens_out = torch.empty_like(q), torch.empty_like(lens)

    def step():
        c.append(k, v, table, lens)
        c.attend(q, table, lens, weights=acc, out=out)
        c.evict(table, lens, acc, budget, recent=8, first=1, lens_out=lens_out, weights_out=acc)
        lens.copy_(lens_out + 1)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pool0, acc0, lens0 = c.pool.clone(), acc.clone(), lens.clone()
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        step()
    c.pool.copy_(pool0), acc.copy_(acc0), lens.copy_(lens0)
    results = []
    for _ in range(5):
        k.normal_(), v.normal_(), q.normal_()
        results.append((k.clone(), v.clone(), q.clone()))
        gr.replay()
    graph = (c.pool.clone(), acc.clone(), lens.clone(), out.clone())
    c.pool.copy_(pool0), acc.copy_(acc0), lens.copy_(lens0)
    for a, b, d in results:
        k.copy_(a), v.copy_(b), q.copy_(d)
        step()
    c.status()
    for x, y in zip(graph, (c.pool, acc, lens, out)):
        assert torch.equal(x, y)
    assert lens.tolist() == [49, 49] and (acc[:, :, 48:] == 0).all()
    # 5 steps, each sharing out a weight of 1 per query head; what left with
    # evicted tokens is missing
    assert 0 < float(acc.sum()) <= 5 * B * H_q + 1e-3


def test_captured_speculative_step():
    """Append, tree attention, verification and the kept path in one graph: replayed
    with other lengths, tables, trees, offsets and rows it gives what the calls
    give one by one."""
    from bit_kv_cache_05_gb300 import verify_drafts
    from bit_kv_cache_05_gb300.rope import Rope
    B, H_q, H_kv, D, page, V, T, most = 3, 8, 2, 64, 16, 501, 40, 24
    c, rope = new_cache(64, page, H_q, H_kv, D, 32, fill=0), Rope(rot_dim=D)
    rng = random.Random(12)
    pool0 = c.pool.random_(0, 256).clone() & 0x3f       # finite scales

    def inputs(seed):
        n = [rng.randrange(1, most) if seed else 13 for _ in range(B)]
        while sum(n) > T:
            n = [max(1, x - 1) for x in n]
        lens = [rng.randrange(0, 200) for _ in range(B)]
        pages = rng.sample(range(64), 3 * 14)
        p, q, tokens, parents, u = draft_case(70 + seed, n, V, "fp32", False, True)
        trees, at = [], 0
        for k in n:
            trees.append(parents[at:at + k])
            at += k
        pad = lambda x, v: list(x) + [v] * (T - len(x))
        rows = lambda x: torch.cat((x, torch.zeros(T - len(x), V))).cuda()
        x = randn(80 + seed, T, H_q + 2 * H_kv, D).half()
        seq = [b for b, k in enumerate(n) for _ in range(k)]
        return dict(table=i32(pages).view(B, 14), lens=i32([a + k for a, k in zip(lens, n)]),
                    cu=offsets(n), masks=i64(pad([m for t in trees for m in dref.masks_of(t)], 0)),
                    pos=i32(pad([lens[seq[i]] + d for i, d in enumerate(
                        d for t in trees for d in dref.depths_of(t))], 0)),
                    q=x[:, :H_q].contiguous(), k=x[:, H_q:H_q + H_kv].contiguous(),
                    v=x[:, H_q + H_kv:].contiguous(), p=rows(p), d=rows(q),
                    tokens=i64(pad(tokens, 0)), parents=i32(pad(parents, 0)),
                    u=torch.cat((u, torch.zeros(T - len(u)))).cuda())

    def step(s):
        q = c.append(s["k"], s["v"], s["table"], s["lens"], s["cu"], q=s["q"], rope=rope,
                     positions=s["pos"], q_out=torch.zeros_like(s["q"]))
        out = c.attend(q, s["table"], s["lens"], s["cu"], max_new=most, tree=s["masks"],
                       out=torch.zeros_like(q))
        path, counts, after = verify_drafts(s["p"], s["tokens"], s["u"], s["cu"],
                                            parents=s["parents"], draft=s["d"],
                                            path=torch.full_like(s["parents"], -1))
        return out, path, counts, after, c.keep(s["table"], s["lens"], s["cu"], path, counts)

    held = inputs(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(held)
    torch.cuda.current_stream().wait_stream(side)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        got = step(held)
    for seed in range(1, 6):
        new = inputs(seed)
        for k, t in new.items():
            held[k].copy_(t)
        c.pool.copy_(pool0)
        gr.replay()
        graph = [t.clone() for t in got] + [c.pool.clone()]
        c.pool.copy_(pool0)
        one = list(step(new)) + [c.pool.clone()]
        c.status()
        for x, y in zip(graph, one):
            assert torch.equal(x, y)
        assert torch.isfinite(one[0].float()).all()


def test_other_streams_and_repeatable():
    """On a stream given by argument, the same bits as on the current one."""
    c, table, L = filled([300, 200], 16, 8, 2, 128, 32)
    n = [20, 12]
    rng = random.Random(1)
    masks = i64(m for k in n for m in dref.masks_of(dref.random_tree(k, rng)))
    q = randn(4, 32, 8, 128).half()
    acc = torch.rand(2, 2, table.shape[1] * 16, device="cuda")
    p, dr, tokens, parents, u = draft_case(9, n, 777, "fp32", False, True)
    st = torch.cuda.Stream()

    def all_of(stream):
        w = acc.clone()
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        pool = c.pool.clone()
        a = c.attend(q, table, L, offsets(n), max_new=20, tree=masks, stream=stream)
        b = c.attend(q[:2], table, L, weights=w, stream=stream)
        v = run_verify(p, dr, tokens, parents, u, n, stream=stream)
        e = c.evict(table, L, w, 64, recent=9, stream=stream)
        kept = c.keep(table, L, offsets(n), v[0], v[1], stream=stream)
        torch.cuda.synchronize()
        moved = c.pool.clone()
        c.pool.copy_(pool)
        return [a, b, w, *v, *e, kept, moved]

    first = all_of(None)
    for stream in (None, st):
        for x, y in zip(first, all_of(stream)):
            assert torch.equal(x, y)
    c.status()


def test_empty_calls():
    from bit_kv_cache_05_gb300 import verify_drafts
    c, table, L = filled([20], 16, 4, 2, 64, 32)
    e = torch.zeros(0, 4, 64, dtype=torch.float16, device="cuda")
    assert c.attend(e, table, L, i32([0, 0]), tree=i64([])).shape == (0, 4, 64)
    assert c.keep(table, L, i32([0, 0]), i32([]), i32([0])).tolist() == [20]
    none = table[:0]
    assert c.keep(none, L[:0], i32([0]), i32([]), i32([])).shape == (0,)
    lo, wo = c.evict(none, L[:0], torch.zeros(0, 2, 32, device="cuda"), 4, recent=1)
    assert lo.shape == (0,) and wo.shape == (0, 2, 32)
    p, k, a = verify_drafts(torch.zeros(0, 9, device="cuda"), i64([]),
                            torch.zeros(0, device="cuda"), i32([0]))
    assert p.shape == (0,) and k.shape == (0,) and a.shape == (0,)
    p, k, a = verify_drafts(torch.zeros(0, 9, device="cuda"), i64([]),
                            torch.zeros(0, device="cuda"), i32([0, 0]))
    assert k.tolist() == [0] and a.tolist() == [-1]
    c.status()


def test_readme_samples_of_drafts_and_eviction():
    """The README's two samples as they stand."""
    import os
    from bit_kv_cache_05_gb300 import verify_drafts
    from bit_kv_cache_05_gb300.rope import Rope
    text = open(os.path.join(os.path.dirname(__file__), "..", "README.md")).read()
    code = [b.split("```")[0] for b in text.split("```python")[1:]]
    trees = [b for b in code if "verify_drafts(" in b]
    evict = [b for b in code if ".evict(" in b]
    assert len(trees) == len(evict) == 1
    B, H_q, H_kv, D, V, n, lens = 2, 8, 2, 128, 97, [9, 5], [700, 300]
    c, table, L = filled([s + 9 for s in lens], 16, H_q, H_kv, D, 32, torch.bfloat16)
    rng = random.Random(6)
    p, dr, tokens, parents, u = draft_case(31, n, V, "fp32", False, True)
    T = sum(n)
    x = randn(1, T, H_q + 2 * H_kv, D).to(torch.bfloat16)
    at = [0, n[0]]
    trees_of = [parents[a:a + k] for a, k in zip(at, n)]
    env = dict(cache=c, verify_drafts=verify_drafts, rope=Rope(rot_dim=D), table=table,
               lens=i32(lens), full=i32([a + b for a, b in zip(lens, n)]), cu=offsets(n),
               q=x[:, :H_q], k=x[:, H_q:H_q + H_kv], v=x[:, H_q + H_kv:], max_nodes=max(n),
               seq=i64([0] * n[0] + [1] * n[1]),
               depth=i32(d for t in trees_of for d in dref.depths_of(t)),
               masks=i64(m for t in trees_of for m in dref.masks_of(t)), parents=i32(parents),
               tokens=i64(tokens), uniforms=u.cuda(), target=p.cuda(), draft=dr.cuda())
    exec(trees[0], env)
    c.status()
    want = [dref.verify(p[a:a + k].numpy(), dr[a:a + k].numpy(), tokens[a:a + k],
                        parents[a:a + k], u[a:a + k].numpy()) for a, k in zip(at, n)]
    assert env["after"].tolist() == [w[1] for w in want]
    assert env["lens"].tolist() == [a + len(w[0]) for a, w in zip(lens, want)]
    kept = env["lens"].tolist()
    x = randn(2, B, H_q + 2 * H_kv, D).to(torch.bfloat16)
    env.update(q=x[:, :H_q], k=x[:, H_q:H_q + H_kv], v=x[:, H_q + H_kv:], budget=512,
               lens=i32([s + 1 for s in kept]), position=i32(kept),
               weights=torch.zeros(B, H_kv, table.shape[1] * 16, device="cuda"))
    exec(evict[0], env)
    c.status()
    assert env["lens"].tolist() == [512, kept[1] + 1]
    assert abs(float(env["weights"][1].sum()) - H_q) < 1e-3


def test_cache_arguments_of_other_shapes():
    """Every tensor of the tree attention, the weights, the kept paths and the
    eviction with a dimension less or more: the argument is named, and the cache
    stays as it is."""
    from bit_kv_cache_05_gb300 import _lib
    lens, n = [40, 30], [3, 2]
    c, table, L = filled(lens, 16, 4, 2, 64, 32)
    cu, T = offsets(n), sum(n)
    q, w = randn(1, T, 4, 64).half(), torch.zeros(2, 2, table.shape[1] * 16, device="cuda")
    base = dict(table=table, lens=L, cu_new=cu)
    calls = [(c.attend, dict(base, q=q, tree=i64([1, 3, 7, 1, 3]), out=torch.empty_like(q))),
             (c.attend, dict(base, q=q, weights=w, max_new=3)),
             (c.keep, dict(base, path=i32([0, 1, 2, 0, 1]), counts=i32([2, 1]),
                           lens_out=L.clone())),
             (c.evict, dict(table=table, lens=L, weights=w, budget=32, recent=4,
                            lens_out=L.clone(), weights_out=w.clone()))]
    before = c.pool.clone()
    for call, good in calls:
        for name, t in good.items():
            if not torch.is_tensor(t):
                continue
            for bad in (t[0], t[:, 0] if t.dim() > 1 else t[:1], t[None], t.flatten()[0], t[:0]):
                try:
                    call(**dict(good, **{name: bad}))
                except ValueError:
                    continue
                # fewer rows than the offsets say: found by the kernels
                assert name in ("q", "path") and bad.dim() == t.dim()
                if len(bad) or name == "path":
                    with pytest.raises(_lib.VqError, match="length"):
                        c.status()
        assert torch.equal(c.pool, before) and (w == 0).all()
    c.status()
    for call, good in calls:
        call(**good)
    c.status()


def test_numbers_beyond_32_bits():
    """Refused, not cut to their low bits."""
    c, table, L = filled([60], 16, 2, 2, 64, 32)
    w = evict_weights([60], 2, 64, "plain")
    q, before = randn(1, 1, 2, 64).half(), c.pool.clone()
    for a in (dict(budget=2 ** 32 + 20, recent=2), dict(budget=20, recent=2 ** 32 + 2),
              dict(budget=20, recent=2, first=2 ** 32), dict(budget=20 - 2 ** 32, recent=2),
              dict(budget=2 ** 31, recent=2)):
        with pytest.raises(ValueError, match="32 bits"):
            c.evict(table, L, w, **a)
    for n in (2 ** 32 + 1, 1 - 2 ** 32):
        for a in (dict(), dict(tree=i64([1])), dict(weights=w)):
            with pytest.raises(ValueError, match="32 bits"):
                c.attend(q, table, L, max_new=n, **a)
    assert torch.equal(c.pool, before)
    # the largest number is a budget that no sequence passes
    lens, _ = c.evict(table, L, w, 2 ** 31 - 1, recent=2)
    c.status()
    assert lens.tolist() == [60] and torch.equal(c.pool, before)


def test_rows_behind_the_last_sequence_stay():
    """Token tensors with more rows than the sequences have: the rows behind are
    neither read nor written."""
    from bit_kv_cache_05_gb300 import verify_drafts
    for n, H_q in (([4, 3], 4), ([20, 9], 4), ([40, 30], 8)):
        lens = [n[0] + 70, n[1] + 5]
        c, table, L = filled(lens, 16, H_q, 1, 64, 32)
        T, extra, cu = sum(n), 5, offsets(n)
        q = randn(3, T + extra, H_q, 64).half()
        q[T:] = float("nan")
        rng = random.Random(2)
        masks = [m for k in n for m in dref.masks_of(dref.random_tree(k, rng))]
        out = torch.full_like(q, 7.0)
        c.attend(q, table, L, cu, max_new=max(n), tree=i64(masks + [-1] * extra), out=out)
        want = c.attend(q[:T], table, L, cu, max_new=max(n), tree=i64(masks))
        assert torch.equal(out[:T], want) and (out[T:] == 7).all()
        p, dr, tokens, parents, u = draft_case(5, n, 50, "fp32", False, True)
        pad = lambda t, x: torch.cat((t, torch.full((extra, *t.shape[1:]), x, dtype=t.dtype)))
        path = torch.full((T + extra,), 9, dtype=torch.int32, device="cuda")
        verify_drafts(pad(p, 2.0).cuda(), pad(torch.tensor(tokens), -5).cuda(), pad(u, 3.0).cuda(),
                      cu, parents=pad(torch.tensor(parents, dtype=torch.int32), 99).cuda(),
                      draft=pad(dr, -1.0).cuda(), path=path)
        ref_path, counts, _ = run_verify(p, dr, tokens, parents, u, n)
        assert torch.equal(path[:T], ref_path) and (path[T:] == 9).all()
        kept = c.keep(table, L, cu, path, counts)
        assert kept.tolist() == [s - k + int(x) for s, k, x in zip(lens, n, counts)]
        c.status()


def test_offsets_past_32_bits_of_drafts_and_eviction():
    """Pages whose bytes lie past 2^32 of the pool."""
    D, g, page, H = 128, 32, 128, 8
    n_pages = 2 ** 32 // (H * 8 * 2560) + 5
    c = new_cache(n_pages, page, H, H, D, g, fill=0)
    table = i32([n_pages - 1, 1, n_pages - 3]).view(1, 3)
    S = 300
    k, v = randn(1, S, H, D).half(), randn(2, S, H, D).half()
    c.append(k, v, table, i32([S]), offsets([S]))
    rng = random.Random(1)
    for n in (4, 40):
        masks = dref.masks_of(dref.random_tree(n, rng))
        check_tree(c, table, [S], [n], masks, "fp16", H, H, D, g)
    K, V = c.dequantize(table, i32([S]), offsets([S]), n_tokens=S)
    path = [0, 3, 17, 31]
    L = c.keep(table, i32([S]), offsets([40]), i32(path + [0] * 36), i32([4]))
    order = list(range(260)) + [260 + x for x in path]
    K1, V1 = c.dequantize(table, L, offsets([264]), n_tokens=264)
    assert L.tolist() == [264] and torch.equal(K1, K[order]) and torch.equal(V1, V[order])
    w = evict_weights([264], H, 384, "plain")
    L2, w2 = c.evict(table, L, w, 150, recent=20, first=3)
    K2, V2 = c.dequantize(table, L2, offsets([150]), n_tokens=150)
    for h in range(H):
        take = dref.evict_row(w[0, h].cpu(), 264, 150, 20, 3)
        assert torch.equal(K2[:, h], K1[take, h]) and torch.equal(V2[:, h], V1[take, h])
        assert torch.equal(w2[0, h, :150], w[0, h][take]) and (w2[0, h, 150:] == 0).all()
    c.status()


def test_lengths_at_the_end_of_31_bits():
    """A table with room for 2^31 tokens: a length whose sums with a tile would
    pass 31 bits is outside its range for every operator; the others of the call
    are served."""
    from bit_kv_cache_05_gb300 import _lib
    page, S, n = 1024, 300, 3
    c = new_cache(1, page, 2, 1, 64, 64)
    table = torch.zeros(2, 2 ** 31 // page, dtype=torch.int32, device="cuda")
    k, v = randn(1, S, 1, 64).half(), randn(2, S, 1, 64).half()
    c.append(k, v, table[:1], i32([S]), offsets([S]))
    c.status()
    before, cu = c.pool.clone(), offsets([n, n])
    kv, q = randn(3, 2 * n, 1, 64).half(), randn(4, 2 * n, 2, 64).half()

    def reported():
        with pytest.raises(_lib.VqError, match="length"):
            c.status()

    for far in (2 ** 31 - 1, 2 ** 31 - 2 ** 16 + 1):
        L = i32([far, S])
        out = torch.full_like(q, 7.0)
        for a in (dict(), dict(tree=i64([1, 3, 7] * 2)), dict(max_new=40),
                  dict(max_new=40, tree=i64([1, 3, 7] * 2)), dict(max_new=20, tree=i64([1, 3, 7] * 2))):
            a.setdefault("max_new", n)
            c.attend(q, table, L, cu, out=out, **a)
            reported()
            assert (out[:n] == 7).all() and (out[n:] != 7).any()
        K = torch.full((2 * n, 1, 64), 7.0, dtype=torch.float16, device="cuda")
        V = K.clone()
        c.dequantize(table, L, cu, n_tokens=2 * n, out=(K, V))
        reported()
        assert (K[:n] == 7).all() and (V[:n] == 7).all() and (K[n:] != 7).any()
        out = c.keep(table, L, cu, i32([2, -1, -1] * 2), i32([1, 1]))
        reported()
        assert out.tolist() == [far, S - 2]
        c.pool.copy_(before)
        # the append leaves the far sequence out
        c.append(kv, kv, table[:1], L[:1], cu[:2])
        reported()
        assert torch.equal(c.pool, before)
        w = torch.zeros(1, 1, 2 ** 31, device="cuda")
        lens, _ = c.evict(table[:1], L[:1], w, 16, recent=4, weights_out=w)
        reported()
        assert lens.tolist() == [far] and torch.equal(c.pool, before)
        del w
    torch.cuda.empty_cache()


def test_most_sequences_of_a_call():
    """1024 sequences, as many as a call takes."""
    B, n = 1024, 3
    lens = [3 + b % 30 for b in range(B)]
    c, table, L = filled(lens, 16, 2, 1, 64, 32)
    q = randn(4, B * n, 2, 64).half()
    masks = [1, 3, 5] * B
    out = c.attend(q, table, L, offsets([n] * B), max_new=n, tree=i64(masks))
    big = c.attend(q, table, L, offsets([n] * B), max_new=40, tree=i64(masks))  # the other kernel
    assert ((out.float() - big.float()).abs() <= 2.0 ** -9 * big.float().abs() + 2.0 ** -9).all()
    acc = torch.zeros(B, 1, table.shape[1] * 16, device="cuda")
    c.attend(q[:B], table, L, weights=acc)
    assert ((acc.sum(-1) - 2).abs() < 1e-4).all()
    p, dr, tokens, parents, u = draft_case(8, [n] * B, 20, "fp32", False, True)
    path, counts, after = run_verify(p, dr, tokens, parents, u, [n] * B)
    for b in (0, 511, 1023):
        s = slice(n * b, n * b + n)
        want, token = dref.verify(p[s].numpy(), dr[s].numpy(), tokens[s], parents[s], u[s].numpy())
        assert path[s].tolist()[:len(want)] == want and int(after[b]) == token
    before = c.pool.clone()
    kept = c.keep(table, L, offsets([n] * B), path, counts)
    moves = [(b, 0, lens[b] - n + j, lens[b] - n + x) for b in range(B)
             for j, x in enumerate(path[n * b:n * b + int(counts[b])].tolist())]
    assert torch.equal(c.pool.cpu(), dref.move_tokens(before, table, 64, 32, moves))
    check_evict(c, table, kept.tolist(), acc, 12, 4, 1, 64, 32)


def test_two_streams_at_once():
    """Calls that run side by side on two streams share nothing: each gives what
    it gives alone."""
    jobs = []
    for seed in (1, 2):
        c, table, L = filled([900, 500], 16, 8, 2, 128, 32, seed=10 * seed)
        n = [24, 17]
        rng = random.Random(seed)
        masks = i64(m for k in n for m in dref.masks_of(dref.random_tree(k, rng)))
        jobs.append((c, table, L, n, masks, randn(seed, 41, 8, 128).half(),
                     torch.rand(2, 2, table.shape[1] * 16, device="cuda"),
                     draft_case(seed, n, 5000, "fp32", False, True), c.pool.clone()))

    def run(job, stream):
        c, table, L, n, masks, q, w, d, pool = job
        with torch.cuda.stream(stream):
            c.pool.copy_(pool)
            acc, got = w.clone(), []
            for _ in range(5):
                got.append(c.attend(q, table, L, offsets(n), max_new=24, tree=masks))
                got.append(c.attend(q[:2], table, L, weights=acc))
                got += run_verify(*d, n)
                got += c.evict(table, L, acc, 400, recent=30)
            return got + [acc, c.pool.clone()]

    alone = []
    for job in jobs:
        alone.append(run(job, torch.cuda.current_stream()))
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    both = [run(job, s) for job, s in zip(jobs, streams)]
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        assert len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b))
    for job in jobs:
        job[0].status()
