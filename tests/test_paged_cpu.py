"""Refusals of the rotation and of the paged cache, and the facts behind their
arithmetic, without a GPU."""
import ctypes
import os
import shutil
import subprocess
from fractions import Fraction

import numpy as np
import pytest
import torch

import paged_ref as ref


def _paged(**kw):
    from bit_kv_cache_05_gb300._lib import Paged
    d = dict(H_q=8, H_kv=2, D=128, group=32, page=64, n_pages=4, pool=1 << 20, status=1 << 20)
    d.update(kw)
    return Paged(**d)


def _batch(**kw):
    from bit_kv_cache_05_gb300._lib import PagedBatch
    d = dict(B=2, max_pages=4, table=1 << 20, table_stride=4, lens=1 << 20, cu_new=None, tokens=2)
    d.update(kw)
    return PagedBatch(**d)


def _rows(heads, **kw):
    from bit_kv_cache_05_gb300._lib import Rows
    d = dict(x=1 << 20, out=1 << 21, weight=None, x_token=128 * heads, x_head=128,
             out_token=128 * heads, out_head=128, heads=heads)
    d.update(kw)
    return Rows(**d)


def _rope(**kw):
    from bit_kv_cache_05_gb300._lib import RopeSpec
    d = dict(rot_dim=128, interleaved=0, n_axes=1, scale=1.0, turns=1 << 20, axis=None)
    d.update(kw)
    return RopeSpec(**d)


@pytest.mark.parametrize("kw,code", [
    (dict(H_q=0), -1), (dict(n_pages=0), -1), (dict(H_q=9), -2), (dict(H_q=18), -2),
    (dict(D=256), -2), (dict(D=96), -2), (dict(group=16), -2), (dict(D=64, group=128), -2),
    (dict(page=24), -2), (dict(page=8), -2), (dict(page=2048), -2), (dict(pool=None), -1),
    (dict(pool=(1 << 20) + 8), -1), (dict(status=None), -1),
])
def test_pool_refusals(vqlib, kw, code):
    p, b = _paged(**kw), _batch()
    q = _rows(p.H_q)
    if p.H_q < 1:
        q = _rows(1)
    assert vqlib.vq_kivi_paged_attend(p, b, 0, q, 1, 0.0, 1 << 20, 1 << 30, None) == code
    assert vqlib.vq_kivi_paged_append(p, b, 0, None, _rows(2), _rows(2), None, None, 0, 0, 1e-6,
                                      None) == code
    assert vqlib.vq_kivi_paged_dequantize(p, b, 1 << 20, 1 << 20, None) == code
    assert len(vqlib.vq_kivi_last_error()) > 0
    if code == -2:
        assert vqlib.vq_kivi_paged_pool_bytes(p) == 0


def test_pool_bytes(vqlib):
    assert vqlib.vq_kivi_paged_pool_bytes(_paged(pool=None, status=None)) == 4 * 2 * 4 * 2560
    assert vqlib.vq_kivi_paged_pool_bytes(_paged(D=64, group=64, page=16)) == 4 * 2 * 1152


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), -1), (dict(tokens=-1), -1), (dict(B=1025, tokens=1025), -2),
    (dict(tokens=3), -1), (dict(tokens=(1 << 24) + 1, cu_new=1 << 20), -2),
    (dict(lens=None), -1), (dict(table=None), -1), (dict(table_stride=3), -1),
    (dict(max_pages=1 << 30, table_stride=1 << 30), -2), (dict(lens=(1 << 20) + 2), -1),
    (dict(cu_new=(1 << 20) + 1), -1),
])
def test_batch_refusals(vqlib, kw, code):
    p, b = _paged(), _batch(**kw)
    assert vqlib.vq_kivi_paged_attend(p, b, 0, _rows(8), 1, 0.0, 1 << 20, 1 << 30, None) == code
    assert vqlib.vq_kivi_paged_dequantize(p, b, 1 << 20, 1 << 20, None) == code


@pytest.mark.parametrize("q,dtype,max_new,scale,code", [
    (dict(heads=4), 0, 1, 0.0, -1), (dict(), 2, 1, 0.0, -2), (dict(), 7, 1, 0.0, -2),
    (dict(), 0, 0, 0.0, -1), (dict(), 0, 2, 0.0, -1), (dict(), 0, 1, float("nan"), -1),
    (dict(x=(1 << 20) + 8), 0, 1, 0.0, -1), (dict(x_token=1028), 0, 1, 0.0, -1),
    (dict(x=None), 0, 1, 0.0, -1), (dict(out=None), 0, 1, 0.0, -1),
    (dict(out_head=256), 0, 1, 0.0, -1), (dict(weight=1 << 20), 0, 1, 0.0, -1),
])
def test_attend_refusals(vqlib, q, dtype, max_new, scale, code):
    r = _rows(8)
    for k, v in q.items():
        setattr(r, k, v)
    assert vqlib.vq_kivi_paged_attend(_paged(), _batch(), dtype, r, max_new, scale, 1 << 20,
                                      1 << 30, None) == code


@pytest.mark.parametrize("q", [
    dict(out=1 << 20), dict(out=(1 << 20) + 2048), dict(out=(1 << 20) - 4080),
    dict(x_token=1 << 20, out=(1 << 21) + (1 << 20) + 2032),   # within the second token
    dict(x_token=-(1 << 19), out=(1 << 20) - 4096),              # rows in falling order
])
def test_attend_output_over_its_queries(vqlib, q):
    r = _rows(8)
    for k, v in q.items():
        setattr(r, k, v)
    args = (0, r, 1, 0.0, 1 << 20, 1 << 30, None)
    assert vqlib.vq_kivi_paged_attend(_paged(), _batch(), *args) == -1
    assert b"overlaps" in vqlib.vq_kivi_last_error()


@pytest.mark.parametrize("what,code", [
    ("k_null", -1), ("heads", -1), ("v_weight", -1), ("eps", -1), ("rot", -2), ("axes", -1),
    ("axis", -1), ("turns", -1), ("scale", -1), ("stride", -1), ("fp32", -2), ("q_out", -1),
])
def test_append_refusals(vqlib, what, code):
    k, v, q, rope, eps, pos, ps, dt = _rows(2), _rows(2), _rows(8), _rope(), 1e-6, 1 << 20, 2, 0
    if what == "k_null":
        k = None
    if what == "heads":
        k = _rows(4)
    if what == "v_weight":
        v.weight = 1 << 20
    if what == "eps":
        eps = -1.0
    if what == "rot":
        rope.rot_dim = 24
    if what == "axes":
        rope.n_axes = 5
    if what == "axis":
        rope.n_axes = 3
    if what == "turns":
        rope.turns = None
    if what == "scale":
        rope.scale = float("inf")
    if what == "stride":
        rope.n_axes, rope.axis, ps = 2, 1 << 20, 1
    if what == "fp32":
        dt = 2
    if what == "q_out":
        q.out = None
    assert vqlib.vq_kivi_paged_append(_paged(), _batch(), dt, q, k, v, rope, pos, 1, ps, eps,
                                      None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), -2), (dict(tokens=-1), -1), (dict(tokens=1 << 25), -2), (dict(D=24), -2),
    (dict(D=272), -2), (dict(q=None), -1), (dict(pos=None), -1), (dict(pos=(1 << 20) + 4), -1),
    (dict(eps=float("nan")), -1), (dict(heads=0), -1),
])
def test_norm_rope_refusals(vqlib, kw, code):
    a = dict(dtype=0, tokens=2, D=128, q=_rows(8), pos=1 << 20, eps=1e-6)
    heads = kw.pop("heads", None)
    a.update(kw)
    if heads is not None:
        a["q"].heads = heads
    assert vqlib.vq_kivi_norm_rope(a["dtype"], a["tokens"], a["D"], a["q"], None, _rope(),
                                   a["pos"], 1, 2, a["eps"], None) == code


def test_null_and_empty_calls(vqlib):
    assert vqlib.vq_kivi_paged_attend(None, _batch(), 0, _rows(8), 1, 0.0, None, 0, None) == -1
    assert vqlib.vq_kivi_paged_attend(_paged(), None, 0, _rows(8), 1, 0.0, None, 0, None) == -1
    assert vqlib.vq_kivi_paged_status(None, None) == -1
    empty = _batch(B=0, tokens=0, max_pages=0, table_stride=0, table=None, lens=None)
    assert vqlib.vq_kivi_paged_attend(_paged(), empty, 0, _rows(8), 1, 0.0, None, 0, None) == 0
    assert vqlib.vq_kivi_paged_append(_paged(), empty, 0, None, _rows(2), _rows(2), None, None,
                                      0, 0, 1e-6, None) == 0
    assert vqlib.vq_kivi_norm_rope(0, 0, 128, _rows(8), None, _rope(), 1 << 20, 1, 2, 1e-6,
                                   None) == 0


@pytest.mark.parametrize("kw", [
    dict(), dict(rot_dim=7), dict(rot_dim=24), dict(rot_dim=512), dict(inv_freq=[float("nan")] * 8),
    dict(rot_dim=32, axis=[0] * 8), dict(rot_dim=16, axis=[4] * 8),
    dict(rot_dim=16, axis=[0] * 8, sections=[8]), dict(rot_dim=16, sections=[4, -1, 5]),
    dict(rot_dim=16, sections=[2, 2, 2]),
])
def test_rope_refusals(kw):
    from bit_kv_cache_05_gb300.rope import Rope
    with pytest.raises(ValueError):
        Rope(device="cpu", **kw)


def test_rope_turns_are_the_frequencies():
    """Frequencies as fractions of a turn: position * turns mod 2^64 gives the
    angle of far positions."""
    from bit_kv_cache_05_gb300.rope import Rope
    r = Rope(rot_dim=64, theta=1e6, sections=[8, 12, 12], device="cpu")
    assert r.axis.tolist() == [0] * 8 + [1] * 12 + [2] * 12 and r.n_axes == 3
    two_pi = Fraction("6.283185307179586476925286766559005768")
    for j in (0, 5, 31):
        want = Fraction(1e6 ** (-2.0 * j / 64)) / two_pi
        turns = int(r.turns[j]) % 2 ** 64
        for p in (1, 131071, 2 ** 31 - 1):
            got = Fraction((p * turns) % 2 ** 64, 2 ** 64)
            d = abs(got - (want * p) % 1)
            assert min(d, 1 - d) <= Fraction(p, 2 ** 64)


def test_reference_layout_is_a_permutation():
    """Every byte of a block is used, each code nibble once."""
    for D, g in ((64, 32), (64, 64), (128, 32), (128, 64), (128, 128)):
        seen = {}
        n = 2 * (8 * D + 64 * (D // g))
        for tl in range(16):
            for c in range(D):
                kb, vb, km, vm = ref.block_places(D, g, tl, c)
                for byte in (kb, vb):
                    assert (byte, c % 2) not in seen
                    seen[byte, c % 2] = 1
                for m in (km, km + 2, vm, vm + 2):
                    seen[2 * m, "m"] = seen[2 * m + 1, "m"] = 1
        assert {b for b, _ in seen} == set(range(n))


def test_python_refusals_without_a_device():
    from bit_kv_cache_05_gb300 import rope
    q = torch.zeros(2, 2, 16, dtype=torch.float16)
    with pytest.raises(ValueError):
        rope.norm_rope(q, None, None, None)
    with pytest.raises(ValueError):
        rope._rows(q, 3, 16, q.dtype, q.device, "q")
    with pytest.raises(ValueError):
        rope._rows(q, 2, 16, torch.bfloat16, q.device, "q")
    with pytest.raises(ValueError):
        rope._rows(q.transpose(0, 2), None, None, q.dtype, q.device, "q")
    with pytest.raises(ValueError):                       # a gradient would be lost
        rope._rows(q.clone().requires_grad_(), 2, 16, q.dtype, q.device, "q")
    with pytest.raises(ValueError):                       # rows of the output overlap
        rope._rows(q, 2, 16, q.dtype, q.device, "q", None,
                   torch.zeros(16, dtype=q.dtype).expand(2, 2, 16))
    with pytest.raises(ValueError):
        rope._positions(torch.zeros(2, dtype=torch.int64), 3, 2, q.device)
    with pytest.raises(ValueError):
        rope._positions(torch.zeros(2, dtype=torch.int16), 1, 2, q.device)
    r = rope._rows(q[:, :1], 1, 16, q.dtype, q.device, "q")
    assert (r.x_token, r.x_head, r.heads) == (32, 0, 1)


def test_quantizer_reference_worked():
    """Hand-worked groups: unit scale, a constant group, the full range (its
    scale goes to the next smaller fp16, so that code 15 stays finite)."""
    x = np.zeros((3, 32), dtype=np.float16)
    x[0] = np.arange(32) % 16
    x[1] = 2.5
    x[2, 0], x[2, 1] = -65504, 65504
    code, s, z = ref.quantize32(x, 32)
    assert (code[0] == np.arange(32) % 16).all() and s[0, 0] == 1 and z[0, 0] == 0
    assert (code[1] == 0).all() and s[1, 0] == 0 and z[1, 0] == 2.5
    top = np.float16(15 * float(s[2, 0]) + float(z[2, 0]))
    assert code[2, 1] == 15 and np.isfinite(top) and s[2, 0] == 8728


RING = r"""
#include <cstdio>
#include <cstdlib>
#include "stage_ring.h"
// A ring of ST stages under random copies, landings and one wait that gives
// up; a barrier counts its completed phases, and a wait for parity p ends when
// the phase under way has the other one.
int main() {
  srand(1);
  for (int run = 0; run < 200000; ++run) {
    const int ST = 3 + rand() % 2, steps = 1 + rand() % 12, fail = rand() % steps;
    vqk::StageRing ring;
    int done[4] = {}, copies[4] = {};        // completed phases; copies not landed
    int issued = 0;
    auto issue = [&](int s) {
      const unsigned which = rand() % 4;
      if (ring.blocks(s)) return false;
      ring.issued(s, which);
      copies[s] = which != 0;
      ++issued;
      return true;
    };
    auto land = [&](int s) { if (copies[s]) { copies[s] = 0; ++done[s]; } };
    auto over = [&](int s) { return (unsigned)(done[s] & 1) != ring.parity(s); };
    for (int s = 0; s < ST && issued < steps; ++s) if (!issue(s)) return 1;
    bool dead = false;
    for (int u = 0; u < steps && !dead; ++u) {
      const int s = u % ST;
      for (int i = 0; i < ST; ++i) if (rand() % 3 == 0 && !(u == fail && i == s)) land(i);
      if (ring.blocks(s)) {
        if (u == fail && copies[s]) { dead = true; break; }   // gives up
        land(s);
        if (!over(s)) return 2;
        ring.landed(s);
      }
      if (issued < steps && !issue(s)) return 3;
    }
    // what is left: a wait for every stage with copies, ended by their landing
    // and not before, and none for the others
    for (int i = 0; i < ST; ++i) {
      if (copies[i]) {
        if (!ring.blocks(i) || over(i)) return 4;
        land(i);
      }
      if (ring.blocks(i) && !over(i)) return 5;
    }
  }
  return 0;
}
"""


def test_a_warp_that_gives_up_waits_for_its_copies(tmp_path):
    """The decode's bookkeeping of its shared-memory stages, run on the host:
    after a wait that gave up, the copies under way, that one's among them, are
    waited for, and no stage whose copies were used."""
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    import bit_kv_cache_05_gb300
    src = tmp_path / "ring.cc"
    src.write_text(RING)
    inc = os.path.join(os.path.dirname(bit_kv_cache_05_gb300.__file__), "csrc")
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", inc, str(src), "-o", str(tmp_path / "ring")],
                   check=True)
    assert subprocess.run([str(tmp_path / "ring")]).returncode == 0


def test_attend_scale_beyond_fp32_in_base_two(vqlib):
    args = (_paged(), _batch(), 0, _rows(8), 1)
    assert vqlib.vq_kivi_paged_attend(*args, 3e38, 1 << 20, 1 << 30, None) == -1
    assert b"softmax_scale" in vqlib.vq_kivi_last_error()
