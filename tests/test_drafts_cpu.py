"""Refusals of the tree attention, the weights, the kept paths, the eviction and
the draft verification, and the facts behind their arithmetic, without a GPU."""
import ctypes
import os
import random
import re
from fractions import Fraction

import numpy as np
import pytest
import torch

import drafts_ref as dref
from test_paged_cpu import _batch, _paged, _rows

P = 1 << 20       # an aligned address that is never read


def _weights(**kw):
    from bit_kv_cache_05_gb300._lib import Weights
    d = dict(at=P, seq_stride=512, head_stride=256, capacity=256)
    d.update(kw)
    return Weights(**d)


def _drafts(**kw):
    from bit_kv_cache_05_gb300._lib import Drafts
    d = dict(target=P, draft=P, target_row=100, draft_row=100, token=P, parent=P, uniforms=P,
             cu_new=P, tokens=8, B=2, V=100, token_64=1)
    d.update(kw)
    return Drafts(**d)


@pytest.mark.parametrize("tree,max_new,batch,code", [
    (None, 4, {}, -1), (P + 4, 4, {}, -1), (P, 65, {}, -2), (P, 0, {}, -1),
    (P, 4, dict(cu_new=None), -1), (P, 4, dict(lens=None), -1),
])
def test_tree_refusals(vqlib, tree, max_new, batch, code):
    b = _batch(**dict(dict(cu_new=P, tokens=8), **batch))
    if b.cu_new is None:
        b.tokens = 2
    assert vqlib.vq_kivi_paged_attend_tree(_paged(), b, 0, _rows(8), tree, max_new, 0.0, P, 1 << 30,
                                           None) == code
    assert vqlib.vq_kivi_last_error()


def test_empty_calls_need_no_pointers(vqlib):
    b = _batch(B=0, tokens=0, table=None, lens=None, cu_new=P)
    assert vqlib.vq_kivi_paged_attend_tree(_paged(), b, 0, _rows(8, x=None, out=None), None, 4, 0.0,
                                           None, 0, None) == 0
    assert vqlib.vq_kivi_paged_keep(_paged(), b, None, None, None, None) == 0
    b.cu_new = None
    w = _weights(at=None)
    assert vqlib.vq_kivi_paged_evict(_paged(), b, w, w, 4, 1, 0, None, None, 0, None) == 0
    assert vqlib.vq_kivi_verify_drafts(_drafts(B=0, tokens=0, target=None, token=None), 2, None,
                                       None, None, None) == 0


@pytest.mark.parametrize("kw,max_new,code", [
    (dict(at=None), 1, -1), (dict(at=P + 2), 1, -1), (dict(capacity=255), 1, -1),
    (dict(seq_stride=511, head_stride=256), 1, -1), (dict(seq_stride=0), 1, -1),
    (dict(head_stride=0), 1, -1), (dict(head_stride=255), 1, -1), (dict(), 5, -2),
    (dict(seq_stride=256, head_stride=511), 1, -1),      # heads outermost, too near
])
def test_weights_refusals(vqlib, kw, max_new, code):
    b = _batch(cu_new=P, tokens=10)
    assert vqlib.vq_kivi_paged_attend_weights(_paged(), b, 0, _rows(8), _weights(**kw), max_new,
                                              0.0, P, 1 << 40, None) == code
    assert vqlib.vq_kivi_paged_attend_weights(_paged(), b, 0, _rows(8), None, 1, 0.0, P, 1 << 40,
                                              None) == -1
    assert vqlib.vq_kivi_paged_weights_workspace_bytes(_paged(), 2, 4, 5) == 0
    assert vqlib.vq_kivi_paged_weights_workspace_bytes(_paged(), 1 << 20, 1 << 20, 1) == 0


@pytest.mark.parametrize("kw", [dict(at=None), dict(at=P + 2), dict(seq_stride=0),
                                dict(head_stride=255), dict(capacity=-1), dict(at=None, capacity=-1)])
@pytest.mark.parametrize("B,max_pages", [(2, 0), (0, 4)])
def test_weights_without_room_in_the_table(vqlib, kw, B, max_pages):
    """Tables without a page: the places are cleared all the same, so that they
    are looked at; a call without sequences only looks at their number."""
    b = _batch(B=B, tokens=B, max_pages=max_pages, cu_new=None)
    w = _weights(**kw)
    code = -1 if B or w.capacity < 0 else 0
    assert vqlib.vq_kivi_paged_evict(_paged(), b, w, w, 4, 1, 0, 2 * P, 3 * P, 1 << 20,
                                     None) == code
    if code:
        assert vqlib.vq_kivi_last_error().startswith(b"weights")


@pytest.mark.parametrize("path,counts,after", [
    (P + 64, 2 * P, 3 * P), (2 * P, P, 3 * P), (2 * P, 3 * P, P + 56), (P - 28, 2 * P, 3 * P),
])
def test_verify_outputs_over_its_inputs(vqlib, path, counts, after):
    """The CTAs of a sequence read its nodes each for itself: what they read may
    not change under them."""
    far = 1 << 24
    d = _drafts(token=P, parent=P + 64, uniforms=P + 96, cu_new=P + 128, target=far, draft=far)
    rc = vqlib.vq_kivi_verify_drafts(d, 2, path, counts, after, None)
    assert rc == -1 and b"overlaps" in vqlib.vq_kivi_last_error()


def test_keep_lengths_half_over(vqlib):
    b = _batch(cu_new=P, tokens=8, lens=2 * P)
    assert vqlib.vq_kivi_paged_keep(_paged(), b, P, P, 2 * P + 4, None) == -1
    assert b"overlaps" in vqlib.vq_kivi_last_error()


@pytest.mark.parametrize("lens_out", ["path", "path end", "half counts", "cu_new", "table"])
def test_keep_lengths_over_what_others_read(vqlib, lens_out):
    """A sequence's CTA writes its length while others read theirs."""
    at = dict(path=4 * P, counts=5 * P, cu_new=6 * P, table=7 * P)
    at.update({"path end": at["path"] + 28, "half counts": at["counts"] + 4})
    b = _batch(cu_new=at["cu_new"], tokens=8, lens=2 * P, table=at["table"])
    out = at[lens_out] + (24 if lens_out == "table" else 0)
    assert vqlib.vq_kivi_paged_keep(_paged(), b, at["path"], at["counts"], out, None) == -1
    assert b"overlaps" in vqlib.vq_kivi_last_error()


@pytest.mark.parametrize("kw", [
    dict(lens_out=7 * P + 24), dict(lens_out=P + 1024), dict(lens_out=4 * P),
    dict(w_out=7 * P - 1000), dict(w_out=2 * P - 2048), dict(w_out=P, w=P, lens=P + 64),
])
def test_evict_outputs_over_the_batch(vqlib, kw):
    """The CTAs of other heads and sequences read the table, the lengths and their
    weights while one is done."""
    a = dict(lens_out=3 * P, w=P, w_out=4 * P, lens=2 * P)
    a.update(kw)
    b = _batch(table=7 * P, lens=a["lens"])
    rc = vqlib.vq_kivi_paged_evict(_paged(), b, _weights(at=a["w"]), _weights(at=a["w_out"]), 100, 8,
                                   2, a["lens_out"], 9 * P, 1 << 30, None)
    assert rc == -1 and b"overlaps" in vqlib.vq_kivi_last_error()


@pytest.mark.parametrize("path,counts,after", [
    (9 * P, 9 * P + 28, 4 * P), (9 * P, 4 * P, 9 * P + 24), (4 * P, 9 * P, 9 * P), # one another
    (11 * P, 2 * P, 3 * P), (2 * P, 12 * P + 4 * 250, 3 * P), (2 * P, 3 * P, 11 * P + 4 * 799 - 4),
])
def test_verify_outputs_over_rows_and_one_another(vqlib, path, counts, after):
    d = _drafts(token=P, parent=P + 64, uniforms=P + 96, cu_new=P + 128, target=11 * P, draft=12 * P)
    rc = vqlib.vq_kivi_verify_drafts(d, 2, path, counts, after, None)
    assert rc == -1 and (b"overlap" in vqlib.vq_kivi_last_error())


@pytest.mark.parametrize("which", ["path", "counts", "lens_out", "odd"])
def test_keep_refusals(vqlib, which):
    b = _batch(cu_new=P, tokens=8)
    a = dict(path=P, counts=P, lens_out=P)
    if which == "odd":
        a["path"] += 2
    else:
        a[which] = None
    assert vqlib.vq_kivi_paged_keep(_paged(), b, a["path"], a["counts"], a["lens_out"],
                                    None) == -1


@pytest.mark.parametrize("kw,code", [
    (dict(budget=0), -1), (dict(recent=-1), -1), (dict(first=-1), -1),
    (dict(budget=10, recent=8, first=3), -1), (dict(budget=2 ** 31 - 1, recent=2 ** 31 - 1, first=9), -1),
    (dict(lens_out=None), -1), (dict(lens_out=P + 2), -1), (dict(lens_out=P + 4), -1),
    (dict(ws=None), -1), (dict(ws=P + 8), -1), (dict(nbytes=10), -1), (dict(w=None), -1),
    (dict(w_out="shifted"), -1), (dict(w_out="other strides"), -1), (dict(cu=P), -1),
])
def test_evict_refusals(vqlib, kw, code):
    a = dict(budget=100, recent=8, first=2, lens_out=2 * P, ws=3 * P, nbytes=1 << 30,
             w=_weights(), w_out=_weights(at=4 * P), cu=None)
    a.update(kw)
    if a["w_out"] == "shifted":
        a["w_out"] = _weights(at=P + 400)
    if a["w_out"] == "other strides":
        a["w_out"] = _weights(seq_stride=1024)
    b = _batch(cu_new=a["cu"])
    assert vqlib.vq_kivi_paged_evict(_paged(), b, a["w"], a["w_out"], a["budget"], a["recent"],
                                     a["first"], a["lens_out"], a["ws"], a["nbytes"],
                                     None) == code
    assert vqlib.vq_kivi_last_error()


def test_evict_workspace(vqlib):
    f = vqlib.vq_kivi_paged_evict_workspace_bytes
    assert f(_paged(), 3, 4, 100, 40) == 3 * 2 * 60 * 8
    assert f(_paged(), 3, 4, 256, 40) == 256                  # no sequence can pass it
    assert f(_paged(), 3, 4, 2 ** 31 - 1, 0) == 256
    assert f(_paged(), 1, 4, 1, 1) == 256 and f(_paged(), 1, 4, 0, 0) == 0
    assert f(_paged(), 1, 4, 5, 6) == 0 and f(_paged(), 1, -1, 5, 1) == 0


@pytest.mark.parametrize("kw,dtype,code", [
    (dict(), 3, -2), (dict(B=-1), 2, -1), (dict(tokens=-1), 2, -1), (dict(V=0), 2, -1),
    (dict(B=1025), 2, -2), (dict(V=(1 << 19) + 1, target_row=1 << 20, draft_row=1 << 20), 2, -2),
    (dict(tokens=(1 << 24) + 1), 2, -2), (dict(target=None), 2, -1), (dict(token=None), 2, -1),
    (dict(uniforms=None), 2, -1), (dict(cu_new=None), 2, -1), (dict(target_row=99), 2, -1),
    (dict(draft_row=99), 2, -1), (dict(target=P + 2), 2, -1), (dict(target=P + 1), 0, -1),
    (dict(token=P + 4), 2, -1), (dict(parent=P + 2), 2, -1), (dict(uniforms=P + 1), 2, -1),
])
def test_verify_refusals(vqlib, kw, dtype, code):
    assert vqlib.vq_kivi_verify_drafts(_drafts(**kw), dtype, P, P, P, None) == code
    assert vqlib.vq_kivi_last_error()


@pytest.mark.parametrize("path,counts,after", [(None, P, P), (P, None, P), (P, P, None),
                                               (P + 2, P, P), (P, P + 1, P), (P, P, P + 4)])
def test_verify_outputs_refused(vqlib, path, counts, after):
    assert vqlib.vq_kivi_verify_drafts(_drafts(), 2, path, counts, after, None) == -1


def test_verify_drafts_arguments():
    from bit_kv_cache_05_gb300 import verify_drafts
    t, k, u, cu = torch.zeros(3, 5), torch.zeros(3).long(), torch.zeros(3), torch.zeros(2).int()
    with pytest.raises(ValueError, match="CUDA"):
        verify_drafts(t, k, u, cu)


def test_residuals_of_residuals_are_one_difference():
    """max(max(p - q, 0) / S1 - q, 0) = max(p - (1 + S1) q, 0) / S1, and so on:
    in exact fractions, each residual normed from the one before against p -
    c q with c the sum of the masses."""
    rng = random.Random(2)
    for _ in range(20):
        V = 7
        p = [Fraction(rng.randrange(0, 50)) for _ in range(V)]
        q = [Fraction(rng.randrange(0, 50)) for _ in range(V)]
        p, q = [x / sum(p) for x in p], [x / sum(q) for x in q]
        r, c, S = list(p), Fraction(0), Fraction(1)
        for _ in range(4):
            r = [max(a - b, 0) for a, b in zip(r, q)]
            if sum(r) == 0:
                break
            r = [x / sum(r) for x in r]
            c += S
            w = [max(a - c * b, 0) for a, b in zip(p, q)]
            S = sum(w)
            assert r == [x / S for x in w]


@pytest.mark.parametrize("kids", [1, 2, 3])
def test_independent_children_follow_the_target(kids):
    """The walk's rule over all draws of a root's children, in exact fractions:
    children drawn independently leave the target's distribution, children drawn
    without replacement do not (from the second on); without a draft any children
    leave it."""
    rng = random.Random(5)
    V = 4
    p, q = ([Fraction(rng.randrange(1, 30)) for _ in range(V)] for _ in range(2))
    p, q = [x / sum(p) for x in p], [x / sum(q) for x in q]

    def first(with_draft, replacement):
        out = [Fraction(0)] * V

        def walk(prob, k, drawn, c, S, gone):
            w = [max(a - c * b, 0) if with_draft else 0 if x in gone else a
                 for x, (a, b) in enumerate(zip(p, q))]
            if k == kids or sum(w) == 0:
                for x in range(V):
                    out[x] += prob * w[x] / sum(w) if sum(w) else prob * p[x]
                return
            rest = 1 if replacement else 1 - sum(q[x] for x in drawn)
            for x in range(V):
                if not replacement and x in drawn:
                    continue
                pick = prob * q[x] / rest
                # accepted if u q(x) S < w(x), or u S < w(x)
                yes = min(1, w[x] / (q[x] * S if with_draft else S))
                out[x] += pick * yes
                if yes == 1:
                    continue
                if with_draft:
                    c2 = c + S
                    S2 = sum(max(a - c2 * b, 0) for a, b in zip(p, q))
                    walk(pick * (1 - yes), k + 1, drawn | {x}, c2, S2, gone)
                else:
                    walk(pick * (1 - yes), k + 1, drawn | {x}, c, S - w[x], gone | {x})

        walk(Fraction(1), 0, frozenset(), Fraction(0), Fraction(1), frozenset())
        return out

    assert first(True, True) == p
    assert (first(True, False) == p) == (kids == 1)
    assert first(False, True) == p and first(False, False) == p


def test_whole_numbers_in_two_halves():
    """The kernel's way to a whole number of 2^-44, in steps of fp32: floor(w
    2^22) beside 2^23, then the rest rounded to 2^-22 of it, is the value
    rounded once."""
    g = np.random.default_rng(3)
    w = np.concatenate([g.random(20000), 2.0 ** -(50 * g.random(20000)),
                        [0.0, 1.0, 2.0 ** -45, 2.0 ** -44, 3 * 2.0 ** -45, 1 - 2.0 ** -24, 1e-45]])
    w = w.astype(np.float32)
    hi = np.floor(w.astype(np.float64) * 2 ** 22)
    t = (hi + 2 ** 23).astype(np.float32)                 # fma rounding down: exact
    assert (t == hi + 2 ** 23).all()
    rest = w.astype(np.float64) * 2 ** 22 - hi
    assert (rest.astype(np.float32) == rest).all()        # the second fma is exact
    lo = np.rint(rest * 2 ** 22)
    assert (lo <= 2 ** 22).all()
    assert (hi * 2 ** 22 + lo == dref.units(w)).all()
    # 1023 of the largest add up in 32 bits
    assert 1023 * 2 ** 22 < 2 ** 32


@pytest.mark.parametrize("name", ["drafts.cu", "paged_move.cu"])
def test_clusters_meet_before_they_touch_each_other(name):
    """A CTA may touch another one's shared memory once that one is known to run:
    in each kernel a barrier of the cluster stands before the first peer access,
    as every path to it passes them in the order of the source."""
    src = os.path.join(os.path.dirname(__file__), "..", "bit_kv_cache_05_gb300", "csrc", name)
    text = re.sub(r"//[^\n]*", "", open(src).read())
    kernels = re.split(r"(?=__global__)", text)[1:]
    touching = [k for k in kernels if re.search(r"\bpeer_(load|store)\(", k)]
    assert touching
    for k in touching:
        peer = re.search(r"\bpeer_(load|store)\(", k).start()
        waits = [m.start() for m in re.finditer(r"^\s*(cluster_sync|cluster_runs|all_sync)\(\);", k,
                                                re.M)]
        assert waits and waits[0] < peer


def test_masks_and_depths_of_a_tree():
    parents = [-1, 0, 0, 1, 3, 2]
    assert dref.masks_of(parents) == [1, 3, 5, 11, 27, 37]
    assert dref.depths_of(parents) == [0, 1, 1, 2, 3, 2]
    chain = dref.masks_of(dref.random_tree(64, random.Random(0), chain=True))
    assert chain[62] == 2 ** 63 - 1 and chain[63] == -1       # bit 63 is the sign


def test_weights_in_an_order_of_whole_numbers():
    """The eviction's order: fp32 bits, the negative ones turned over; -0 as 0
    (by adding 0), NaN below all."""
    x = np.array([-np.inf, -3e38, -1.0, -1e-45, -0.0, 0.0, 1e-45, 1.0, 3e38, np.inf], np.float32)
    u = (x + np.float32(0)).view(np.uint32)
    order = np.where(u & 0x80000000, ~u, u | np.uint32(0x80000000))
    assert (np.diff(order.astype(np.int64)) > 0).sum() == 8 and order[4] == order[5]
    assert (order > 0).all()                                  # NaN is 0


def test_evict_rows_of_the_reference():
    w = torch.tensor([5.0, 1, 7, 2, 9, 3, 8, 0, 0, 0])
    assert dref.evict_row(w, 10, 10, 2, 1) == list(range(10))
    # first 1, newest 3 (places 7 8 9); of the others (1 7 2 9 3 8) the 2 heaviest
    assert dref.evict_row(w, 10, 6, 3, 1) == [0, 4, 6, 7, 8, 9]
    assert dref.evict_row(w, 10, 5, 3, 0) == [4, 6, 7, 8, 9]
