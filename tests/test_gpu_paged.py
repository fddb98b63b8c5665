"""The rotation and the paged 4-bit cache on the GPU against 64-bit
implementations (paged_ref.py, which also derives the bounds)."""
import numpy as np
import pytest
import torch

import paged_ref as ref

pytestmark = pytest.mark.gpu
DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
# the split-KV kernel keeps the weights of up to 8 rows in 32 bits (hi + lo);
# with more rows, and in the tensor-memory kernel, a weight is rounded to fp16
# once (2^-11)
FEW, MANY = 2.0 ** -21, 2.0 ** -11


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_kv_cache_05_gb300 import _lib, build
    build.build()
    return _lib.load()


def randn(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).cuda()


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def offsets(n):
    return i32(np.concatenate([[0], np.cumsum(n)]))


def new_cache(n_pages, page, H_q, H_kv, D, group, fill=0xff):
    """A cache whose free slots hold NaN scales (0xff) or whatever `fill` says."""
    from bit_kv_cache_05_gb300.paged import PagedKiviCache
    c = PagedKiviCache(n_pages, page=page, H_q=H_q, H_kv=H_kv, D=D, group=group)
    c.pool.fill_(fill)
    return c


def filled(lens, page, H_q, H_kv, D, group, dtype=torch.float16, seed=0, fill=0xff, gain=1.0):
    """A cache holding whole sequences of random tokens; (cache, table, lens)."""
    need = sum(-(-s // page) for s in lens)
    c = new_cache(need + 2, page, H_q, H_kv, D, group, fill)
    table = ref.make_table(len(lens), lens, page, need + 2, "cuda", seed)
    T = sum(lens)
    k, v = (randn(seed + 1, T, H_kv, D) * gain).to(dtype), randn(seed + 2, T, H_kv, D).to(dtype)
    if T:
        c.append(k, v, table, i32(lens), offsets(lens))
    c.status()
    return c, table, i32(lens)


# ---- norm_rope -----------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("T,H_q,H_kv,D,rot,axes,inter,norm", [
    (1, 1, 1, 16, 16, 1, False, True), (3, 5, 2, 64, 64, 1, False, True),
    (33, 8, 2, 128, 128, 3, True, False), (7, 3, 3, 96, 48, 2, False, True),
    (130, 4, 1, 256, 256, 1, True, True), (9, 7, 1, 128, 32, 4, True, True),
    (5, 2, 1, 112, 0, 1, False, True),
])
def test_norm_rope(dtype, T, H_q, H_kv, D, rot, axes, inter, norm):
    from bit_kv_cache_05_gb300.rope import Rope, norm_rope
    dt = DT[dtype]
    x = (randn(1, T, H_q + 2 * H_kv, D) * 3).to(dt)      # heads as strided views
    q, k = x[:, :H_q], x[:, H_q:H_q + H_kv]
    qw, kw = ((1 + 0.2 * randn(2, D)).to(dt), (1 + 0.2 * randn(3, D)).to(dt)) if norm \
        else (None, None)
    axis = [j % axes for j in range(rot // 2)]
    rope = Rope(rot_dim=rot, theta=1e5, axis=axis, interleaved=inter, scale=1.25) if rot else None
    pos = torch.randint(-5, 2 ** 31 - 1, (axes, T), generator=torch.Generator().manual_seed(4))
    pos[0, 0] = 0
    pos = pos.cuda()
    before = x.clone()
    got = norm_rope(q, k, pos if rot else None, rope, q_weight=qw, k_weight=kw)
    assert torch.equal(x, before)
    inv = [1e5 ** (-2.0 * j / rot) for j in range(rot // 2)]
    for y, src, w in ((got[0], q, qw), (got[1], k, kw)):
        want, mag = ref.norm_rope64(src, w, pos, inv, axis, inter, 1.25)
        err = (y.cpu().double() - want).abs()
        assert (err <= ref.norm_rope_bound(want, mag, dt, D)).all(), err.max()
    # int32 positions, in place, queries alone
    q2 = q.clone()
    out, none = norm_rope(q2, None, pos.int() if rot else None, rope, q_weight=qw, q_out=q2)
    assert none is None and out is q2 and torch.equal(q2, got[0])


def test_norm_rope_empty_nan_and_stream():
    from bit_kv_cache_05_gb300.rope import Rope, norm_rope
    rope = Rope(rot_dim=64)
    q = randn(1, 6, 4, 64).half()
    e, _ = norm_rope(q[:0], None, torch.zeros(0, dtype=torch.int64, device="cuda"), rope)
    assert e.shape == (0, 4, 64)
    pos = torch.arange(6, device="cuda")
    q[2, 1, 3] = float("nan")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    out, _ = norm_rope(q, None, pos, rope, stream=st)
    st.synchronize()
    bad = torch.isnan(out)
    assert bad[2, 1, 3] and bad[2, 1, 35] and bad.sum() == 2     # its pair and nothing else


# ---- append ----------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("D,g,page,H_kv", [(64, 32, 16, 3), (64, 64, 32, 1), (128, 32, 64, 2),
                                           (128, 64, 16, 5), (128, 128, 128, 1)])
def test_append_is_the_quantizer_bit_for_bit(dtype, D, g, page, H_kv):
    """Without a norm or a rotation codes, scales and zeros equal the fp32
    IEEE quantizer's, token by token, and nothing else in the pool changes."""
    n, before = [1, 0, 17, 40], [0, 9, 15, 3]
    lens = [a + b for a, b in zip(n, before)]
    need = sum(-(-s // page) for s in lens)
    c = new_cache(need + 1, page, H_kv, H_kv, D, g)
    table = ref.make_table(4, lens, page, need + 1, "cuda", 3)
    T = sum(n)
    x = randn(5, T + 2, 2 * H_kv, D) * 2
    x[3] *= 1e6                      # beyond fp16: saturates
    x[4] = 0.25                      # constant groups
    x[5] *= 1e-6                     # subnormal
    x[6, :, ::2] = -0.0
    x[7, 0, 0], x[7, 0, 1] = -70000.0, 70000.0
    x = x.to(DT[dtype])
    k, v = x[:, :H_kv], x[:, H_kv:]
    c.append(k, v, table, i32(lens), offsets(n))
    c.status()
    tab, at = table.cpu().numpy(), 0
    touched = np.zeros(c.pool.shape, dtype=bool)
    for b in range(4):
        for h in range(H_kv):
            parts = ref.cache_parts(c.pool, tab[b], lens[b], h, D, g)
            for name, src in (("k", k), ("v", v)):
                want = ref.quantize32(ref.to_half_sat(src[at:at + n[b], h]).cpu().numpy(), g)
                code, s, z = (p[before[b]:] for p in parts[name])
                assert np.array_equal(code, want[0])
                assert np.array_equal(s.view(np.uint16)[:, ::g], want[1].view(np.uint16))
                assert np.array_equal(z.view(np.uint16)[:, ::g], want[2].view(np.uint16))
        for p in range(before[b], lens[b]):
            pg, blk = tab[b, p // page], p % page // 16
            for ch in range(D):
                kb, vb, km, vm = ref.block_places(D, g, p % 16, ch)
                for y in (kb, vb, 2 * km, 2 * km + 1, 2 * km + 4, 2 * km + 5, 2 * vm, 2 * vm + 1,
                          2 * vm + 4, 2 * vm + 5):
                    touched[pg, :, blk, y] = True
        at += n[b]
    assert (c.pool.cpu().numpy()[~touched] == 0xff).all()
    # read back: one rounding of code * scale + zero
    K, V = c.dequantize(table, i32(lens), offsets(lens), n_tokens=sum(lens))
    at = 0
    for b in range(4):
        for h in range(H_kv):
            rows = ref.cache_rows64(c.pool, tab[b], lens[b], h, D, g)
            for got, want in zip((K, V), rows):
                assert np.array_equal(got[at:at + lens[b], h].cpu().numpy()[before[b]:],
                                      want.astype(np.float16)[before[b]:])
        at += lens[b]


@pytest.mark.parametrize("dtype,axes,explicit,norm", [
    ("fp16", 1, False, True), ("bf16", 3, True, True), ("fp16", 2, True, False),
    ("bf16", 1, False, False),
])
def test_append_norms_and_rotates(dtype, axes, explicit, norm):
    from bit_kv_cache_05_gb300.rope import Rope
    dt, D, g, page, H_q, H_kv = DT[dtype], 128, 32, 16, 6, 3
    n, lens = [5, 33, 1], [100005, 33, 20]
    # a far sequence needs a table wide enough, with pages where it is written
    need = [-(-s // page) for s in lens]
    table = torch.full((3, max(need)), -1, dtype=torch.int32)
    table[0, need[0] - 1] = 0
    table[1, :3], table[2, :2] = torch.tensor([5, 2, 1]), torch.tensor([4, 3])
    table = table.cuda()
    c = new_cache(7, page, H_q, H_kv, D, g)
    T = sum(n)
    x = (randn(7, T, (H_q + 2 * H_kv) * D) * 2).to(dt).view(T, -1, D)
    q, k, v = x[:, :H_q], x[:, H_q:H_q + H_kv], x[:, H_q + H_kv:]
    qw, kw = ((1 + 0.1 * randn(8, D)).to(dt), (1 + 0.1 * randn(9, D)).to(dt)) if norm \
        else (None, None)
    axis = [j % axes for j in range(D // 2)]
    place = torch.cat([torch.arange(s - m, s) for s, m in zip(lens, n)])
    pos = torch.randint(0, 50000, (axes, T), generator=torch.Generator().manual_seed(4)) \
        if explicit else place.repeat(axes, 1)
    rope = Rope(rot_dim=D, axis=axis)
    got = c.append(k, v, table, i32(lens), offsets(n), q=q, rope=rope, q_weight=qw, k_weight=kw,
                   positions=pos.cuda() if explicit else None)
    c.status()
    inv = [1e4 ** (-2.0 * j / D) for j in range(D // 2)]
    want, mag = ref.norm_rope64(q, qw, pos, inv, axis, False)
    assert ((got.cpu().double() - want).abs() <= ref.norm_rope_bound(want, mag, dt, D)).all()
    K, V = c.dequantize(table, i32(lens), offsets(n), n_tokens=T)
    c.status()
    want, mag = ref.norm_rope64(k, kw, pos, inv, axis, False)
    # the stored key: half a code step of the group (its scale from the exact
    # rows, both ends off by at most the rotated keys' own error), the scale's
    # and the zero's roundings to fp16 and the one of the value read back
    e0 = ref.norm_rope_bound(want, mag, torch.float16, D)
    grp = want.view(T, H_kv, -1, g)
    e0g = e0.view(T, H_kv, -1, g)
    width = grp.amax(-1) - grp.amin(-1) + 2 * e0g.amax(-1)
    half = ref.half_step(torch.float16)
    tol = e0g + (width / 30 * (1 + 2.0 ** -20) + width * (half + 2.0 ** -20))[..., None] \
        + (half * (grp.abs() + width[..., None])) + e0g.amax(-1, keepdim=True)
    err = (K.cpu().double().view(T, H_kv, -1, g) - grp).abs()
    assert (err <= tol).all(), (err / tol).max()
    vq = ref.quantize32(ref.to_half_sat(v).cpu().numpy(), g)
    vals = (vq[0].astype(np.float64) * np.repeat(vq[1], g, -1).astype(np.float64)
            + np.repeat(vq[2], g, -1).astype(np.float64)).astype(np.float16)
    assert np.array_equal(V.cpu().numpy(), vals)


def test_append_padding_and_bad_pages():
    """Rows behind the last sequence, padded sequences, tokens on pages outside
    the pool: left out, the rest stored, the fault reported once."""
    from bit_kv_cache_05_gb300 import _lib
    D, g, page, H = 64, 32, 16, 2
    c = new_cache(3, page, H, H, D, g)
    table = torch.tensor([[0, 1], [-1, -1], [9, 2]], dtype=torch.int32, device="cuda")
    n, lens = [18, 2, 17], [18, 0, 32]          # the second: padding, lens < n
    T = sum(n)
    k, v, q = (randn(i, T + 3, H, D).half() for i in (1, 2, 3))
    q_out = torch.full_like(q, 7.0)
    c.append(k, v, table, i32(lens), offsets(n), q=q, q_out=q_out)
    with pytest.raises(_lib.VqError):
        c.status()                               # page 9 of 3
    c.status()                                   # reported once
    assert (q_out[T:] == 7).all() and (q_out[18:20] == 7).all()
    assert torch.equal(q_out[:18], q[:18]) and torch.equal(q_out[20:T], q[20:T])
    K, V = c.dequantize(table[:1], i32([18]), offsets([18]), n_tokens=18)
    ends = ref.quantize32(k[:18].cpu().numpy(), g)
    assert np.array_equal(K.cpu().numpy().view(np.uint16),
                          (ends[0] * np.repeat(ends[1], g, -1).astype(np.float64)
                           + np.repeat(ends[2], g, -1).astype(np.float64))
                          .astype(np.float16).view(np.uint16))
    # a length beyond the table, and a negative one
    c.append(k[:2], v[:2], table[:2], i32([33, -4]))
    with pytest.raises(_lib.VqError):
        c.status()


# ---- attention -------------------------------------------------------------------

DECODE = [
    # lens, H_q, H_kv, D, g, page
    ([1], 1, 1, 64, 32, 16), ([0, 1, 15, 16, 17], 2, 1, 128, 32, 16),
    ([513, 0, 64, 63], 8, 1, 128, 64, 32), ([300, 2000], 12, 4, 64, 64, 64),
    ([129, 1025, 1, 700], 10, 2, 128, 128, 128), ([4097], 5, 5, 128, 32, 64),
    ([31] * 40, 6, 2, 64, 32, 16),
]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("lens,H_q,H_kv,D,g,page", DECODE)
def test_decode(dtype, lens, H_q, H_kv, D, g, page):
    c, table, L = filled(lens, page, H_q, H_kv, D, g, seed=len(lens))
    q = (randn(11, len(lens), H_q, D) * 2).to(DT[dtype])
    out = c.attend(q, table, L)
    c.status()
    want, err = ref.attend64(q, c.pool, table, L, None, D, g, H_kv, weight_step=FEW)
    ref.check_attend(out, want, err, q.dtype)
    assert (out[L == 0] == 0).all()


CHUNK = [
    # n, lens, H_q, H_kv, D, g, page: up to 8 rows of a kv head, up to 16, more
    ([2, 1, 0, 4], [2, 70, 33, 400], 2, 1, 128, 32, 16),
    ([3, 2], [300, 2], 4, 2, 64, 64, 32),
    ([3, 2, 0], [300, 2, 9], 8, 2, 128, 32, 16),
    ([4, 1, 2], [61, 800, 1], 4, 1, 64, 32, 64),
    ([2, 2], [2049, 33], 16, 2, 128, 128, 32),
    ([3, 2], [40, 1200], 5, 1, 128, 64, 16),
    ([16, 9], [700, 31], 2, 2, 128, 64, 128),
    ([5, 3], [900, 131], 8, 2, 128, 32, 16),
    ([1, 200, 0, 17], [1, 200, 50, 150], 4, 2, 64, 32, 32),
    ([129, 64], [129, 700], 3, 3, 128, 64, 64),
    ([40, 9], [1500, 9], 16, 2, 128, 128, 128),
    ([33], [65], 5, 1, 128, 32, 16),
    ([300], [300], 7, 1, 64, 64, 16),
]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("n,lens,H_q,H_kv,D,g,page", CHUNK)
def test_chunk(dtype, n, lens, H_q, H_kv, D, g, page):
    c, table, L = filled(lens, page, H_q, H_kv, D, g, seed=sum(n))
    T = sum(n)
    x = (randn(11, T + 2, H_q + 1, D) * 2).to(DT[dtype])
    q = x[:, 1:]                                  # strided rows
    out = torch.full(q.shape, 5.0, dtype=q.dtype, device="cuda")
    c.attend(q, table, L, offsets(n), max_new=max(n), out=out)
    c.status()
    few = max(n) * (H_q // H_kv) <= 8
    want, err = ref.attend64(q, c.pool, table, L, offsets(n), D, g, H_kv,
                             weight_step=FEW if few else MANY)
    ref.check_attend(out[:T], want[:T], err[:T], q.dtype)
    assert (out[T:] == 5).all()                   # rows behind the last sequence


def test_scores_of_any_size_and_equal_keys():
    """Scores near 1e4 (no overflow), queries of one large value among tiny
    ones in bf16, all keys equal (the mean of the values), a given scale."""
    c, table, L = filled([200, 37], 16, 4, 2, 128, 32, gain=30.0)
    q = randn(3, 2, 4, 128) * 30
    q[1, 2] = 1e-20
    q[1, 3] = 0
    q[0, 1, 5] = 3e4
    for dt in (torch.float16, torch.bfloat16):
        for scale in (0.0, 0.5):
            out = c.attend(q.to(dt), table, L, scale=scale)
            want, err = ref.attend64(q.to(dt), c.pool, table, L, None, 128, 32, 2, scale, FEW)
            ref.check_attend(out, want, err, dt)
    big = torch.full((2, 4, 128), 1e30, dtype=torch.bfloat16, device="cuda")
    assert torch.isfinite(c.attend(big * 1e-30, table, L)).all()


@pytest.mark.parametrize("H_q,n", [(2, [1, 3]), (8, [1, 40])])
def test_nan_and_infinity_stay_where_they_are_seen(H_q, n):
    """A NaN in a token's key or value reaches exactly the rows that see it;
    an infinity is stored as the largest fp16 value."""
    D, g, page, H_kv = 128, 32, 16, 1
    lens = [50, 60]
    need = 8
    c = new_cache(need + 1, page, H_q, H_kv, D, g)
    table = ref.make_table(2, lens, page, need + 1, "cuda", 1)
    k, v = randn(1, 110, 1, D).half(), randn(2, 110, 1, D).half()
    k[20, 0, 5] = float("inf")
    v[21, 0, 7] = float("-inf")
    bad = 50 + 60 - 2                              # the last token but one
    for src in (k, v):
        x = src.clone()
        x[bad, 0, 9] = float("nan")
        c.append(x if src is k else k, x if src is v else v, table, i32(lens), offsets(lens))
        T = sum(n)
        q = randn(3, T, H_q, D).half()
        out = c.attend(q, table, i32(lens), offsets(n), max_new=max(n))
        c.status()
        sees = torch.zeros(T, dtype=torch.bool, device="cuda")
        sees[T - 2:] = True
        assert torch.isnan(out[sees]).all()
        assert torch.isfinite(out[~sees]).all()


def test_attend_bad_arguments():
    from bit_kv_cache_05_gb300 import _lib
    c, table, L = filled([20, 5], 16, 4, 2, 64, 32)
    q = randn(1, 2, 4, 64).half()
    with pytest.raises(ValueError):
        c.attend(q.float(), table, L)
    with pytest.raises(ValueError):
        c.attend(q[:, :2], table, L)
    with pytest.raises(ValueError):
        c.attend(q, table.long(), L)
    with pytest.raises(ValueError):
        c.attend(q, table.cpu(), L)
    with pytest.raises(ValueError):
        c.attend(q[:1], table, L)
    with pytest.raises(_lib.VqError):
        c.attend(q, table, L, max_new=3)
    with pytest.raises(_lib.VqError):
        c.attend(q, table, L, scale=float("inf"))
    wide = torch.zeros(2 * 4 * 64 + 4, dtype=torch.float16, device="cuda")
    with pytest.raises(_lib.VqError):              # 8-byte aligned rows
        c.attend(wide[4:].view(2, 4, 64), table, L)
    # more new tokens than said: reported, the sequence left out
    big = randn(1, 4, 4, 64).half()
    c.attend(big, table, L, offsets([3, 1]), max_new=2)
    with pytest.raises(_lib.VqError):
        c.status()
    t2 = table.clone()
    t2[0, 1] = 99
    out = c.attend(q, t2, L)
    with pytest.raises(_lib.VqError):
        c.status()
    want = c.attend(q, table, L)
    assert torch.equal(out[1], want[1]) and torch.isfinite(out).all()


# ---- together --------------------------------------------------------------------

def test_serving_run_prompt_drafts_and_steps():
    """A run as a server makes it: ragged prompts appended and attended, drafts
    of three tokens, single steps, each checked; a prompt in two chunks gives
    the same pool as in one."""
    from bit_kv_cache_05_gb300.rope import Rope
    D, g, page, H_q, H_kv, dt = 128, 32, 32, 8, 2, torch.bfloat16
    rope, B = Rope(rot_dim=D, theta=5e5), 3
    kw = (1 + 0.1 * randn(9, D)).to(dt)
    table = ref.make_table(B, [160] * B, page, 16, "cuda", 2, width=5)
    c = new_cache(16, page, H_q, H_kv, D, g)
    two = new_cache(16, page, H_q, H_kv, D, g)
    lens = [0] * B
    for step, n in enumerate([[70, 9, 33], [3, 3, 3], [1, 1, 1], [1, 1, 1], [0, 40, 2]]):
        lens = [a + b for a, b in zip(lens, n)]
        cu, T = (None if set(n) == {1} else offsets(n)), sum(n)
        x = randn(20 + step, T, (H_q + 2 * H_kv) * D).to(dt).view(T, -1, D)
        q, k, v = x[:, :H_q], x[:, H_q:H_q + H_kv], x[:, H_q + H_kv:]
        qr = c.append(k, v, table, i32(lens), cu, q=q, rope=rope, q_weight=kw, k_weight=kw)
        out = c.attend(qr, table, i32(lens), cu, max_new=max(n))
        c.status()
        want, err = ref.attend64(qr, c.pool, table, i32(lens), cu, D, g, H_kv, weight_step=MANY)
        ref.check_attend(out, want, err, dt)
        if step == 0:
            first = [40, 0, 33]
            pick = list(range(40)) + list(range(79, 112))
            two.append(k[pick], v[pick], table, i32(first), offsets(first), rope=rope,
                       k_weight=kw)
            rest = list(range(40, 79))
            two.append(k[rest], v[rest], table, i32(lens), offsets([30, 9, 0]), rope=rope,
                       k_weight=kw)
            assert torch.equal(two.pool, c.pool)
    # a chunk's last row is the decode of the same token
    qs = randn(50, B, H_q, D).to(dt)
    a = c.attend(qs, table, i32(lens))
    wide = torch.zeros(3 * 20, H_q, D, dtype=dt, device="cuda")
    wide[19::20] = qs
    b = c.attend(wide, table, i32(lens), offsets([20] * 3), max_new=20)
    want, err = ref.attend64(qs, c.pool, table, i32(lens), None, D, g, H_kv, weight_step=MANY)
    ref.check_attend(a, want, err, dt)
    ref.check_attend(b[19::20], want, err, dt)


def test_rotated_rows_feed_the_contiguous_cache():
    """norm_rope before KiviCache: append and decode over rotated keys."""
    from bit_kv_cache_05_gb300.cache import KiviCache
    from bit_kv_cache_05_gb300.rope import Rope, norm_rope
    S, H_q, H_kv, D = 100, 4, 2, 64
    rope, w = Rope(rot_dim=D), (1 + 0.1 * randn(5, D)).half()
    k, v = randn(1, S + 1, H_kv, D).half(), randn(2, S + 1, H_kv, D).half()
    q = randn(3, S + 1, H_q, D).half()
    qr, kr = norm_rope(q, k, torch.arange(S + 1, device="cuda"), rope, q_weight=w, k_weight=w)
    rows = lambda x: x.transpose(0, 1).contiguous()[None]     # [1][H_kv][S][D]
    with KiviCache(rows(kr[:S]), rows(v[:S]), [S], H_q=H_q, bits=4, group=32, residual=32,
                   max_seq=S + 1) as c:
        c.append(rows(kr[S:]), rows(v[S:]), [1])
        out = c.decode_attend(qr[S:].contiguous())
        K, V = (x.double().cpu().numpy()[0] for x in c.dequantize())
    for hq in range(H_q):
        s = K[hq // 2] @ qr[S, hq].double().cpu().numpy() / 8
        p = np.exp(s - s.max())
        want = (p / p.sum()) @ V[hq // 2]
        assert np.abs(out[0, hq].cpu().numpy() - want).max() <= 1e-3 * (1 + np.abs(want).max())


@pytest.mark.parametrize("n", [1, 24])
def test_captured_step_follows_lengths_and_tables(n):
    """A captured append and attend, replayed after lengths, tables, offsets
    and inputs changed (longer and shorter sequences, padding)."""
    from bit_kv_cache_05_gb300.rope import Rope
    D, g, page, H_q, H_kv, B = 128, 64, 16, 8, 2, 3
    rope = Rope(rot_dim=D)
    c = new_cache(120, page, H_q, H_kv, D, g, fill=0)
    table = ref.make_table(B, [600] * B, page, 120, "cuda", 4, width=38)
    lens, T = i32([n] * B), n * B
    cu = None if n == 1 else offsets([n] * B)
    x = randn(1, T, H_q + 2 * H_kv, D).half()

    def step():
        q = c.append(x[:, H_q:H_q + H_kv], x[:, H_q + H_kv:], table, lens, cu, q=x[:, :H_q],
                     rope=rope)
        return c.attend(q, table, lens, cu, max_new=n)

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step()
    torch.cuda.current_stream().wait_stream(st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    tabs = ref.make_table(B, [600] * B, page, 120, "cuda", 5, width=38)
    for new_lens in ([n, 300, n + 7], [512, 0, 33 + n], [100, 100, 599]):
        table.copy_(tabs)
        lens.copy_(i32(new_lens))
        x.copy_(randn(sum(new_lens), T, H_q + 2 * H_kv, D).half())
        if cu is not None:
            cu.copy_(i32([0, n, n + n // 2, n + n // 2]))
        graph.replay()
        got, pool = out.clone(), c.pool.clone()
        want = step()
        torch.cuda.synchronize()
        end = T if cu is None else int(cu[-1])
        assert torch.equal(pool, c.pool)
        live = torch.ones(T, dtype=torch.bool)
        live[end:] = False
        if cu is None:
            live = torch.tensor([s > 0 for s in new_lens])
        assert torch.equal(got[live], want[live])
    c.status()


def test_two_streams_and_repeatable():
    """Calls of one cache that overlap on two streams have workspaces of their
    own; equal calls give equal bits."""
    c, table, L = filled([3000, 1000, 2000], 64, 8, 2, 128, 32)
    qa, qb = randn(1, 3, 8, 128).half(), randn(2, 3, 8, 128).half()
    qc = randn(3, 96, 8, 128).half()
    cu = offsets([32] * 3)
    a, b, m = c.attend(qa, table, L), c.attend(qb, table, L), c.attend(qc, table, L, cu,
                                                                       max_new=32)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        x = c.attend(qa, table, L, stream=s1)
        y = c.attend(qb, table, L, stream=s2)
        z = c.attend(qc, table, L, cu, max_new=32, stream=s1)
        w = c.attend(qc, table, L, cu, max_new=32, stream=s2)
        torch.cuda.synchronize()
        assert torch.equal(x, a) and torch.equal(y, b)
        assert torch.equal(z, m) and torch.equal(w, m)


@pytest.mark.parametrize("n,H_q", [(4, 2), (6, 4), (40, 4)])
def test_rows_before_the_first_token_are_zero(n, H_q):
    """Sequences shorter than their new tokens (padding in front): those rows
    see nothing."""
    c, table, L = filled([2, 13, 1], 16, H_q, 2, 64, 32)
    q = randn(5, 3 * n, H_q, 64).half()
    cu = offsets([n] * 3)
    out = c.attend(q, table, L, cu, max_new=n)
    c.status()
    want, err = ref.attend64(q, c.pool, table, L, cu, 64, 32, 2, weight_step=MANY)
    ref.check_attend(out, want, err, q.dtype)
    for b, s in enumerate([2, 13, 1]):
        assert (out[b * n:b * n + max(0, n - s)] == 0).all()


@pytest.mark.parametrize("B,n", [(1024, 1), (300, 3), (130, 12)])
def test_many_sequences(B, n):
    """Batches up to the largest, many of them empty, all three kernels."""
    D, g, page, H_q, H_kv = 64, 64, 16, 4, 2
    lens = [(7 * b) % 53 for b in range(B)]
    news = [min(n, s) if n > 1 else 1 for s in lens]
    c, table, L = filled(lens, page, H_q, H_kv, D, g, seed=B)
    q = randn(5, sum(news), H_q, D).half()
    cu = None if n == 1 else offsets(news)
    out = c.attend(q, table, L, cu, max_new=n)
    c.status()
    want, err = ref.attend64(q, c.pool, table, L, cu, D, g, H_kv,
                             weight_step=FEW if 2 * n <= 8 else MANY)
    ref.check_attend(out, want, err, q.dtype)


def test_large_pages_and_few_heads_of_many():
    c, table, L = filled([1500, 1024, 1], 1024, 8, 8, 128, 64)
    for n in (1, 20):
        q = randn(5, 3 * n, 8, 128).bfloat16()
        cu = offsets([n, n, n])
        out = c.attend(q, table, L, cu, max_new=n)
        c.status()
        want, err = ref.attend64(q, c.pool, table, L, cu, 128, 64, 8,
                                 weight_step=FEW if n == 1 else MANY)
        ref.check_attend(out, want, err, q.dtype)


def test_bad_page_of_one_sequence_in_a_chunk():
    from bit_kv_cache_05_gb300 import _lib
    c, table, L = filled([200, 150], 16, 8, 2, 128, 32)
    q = randn(5, 80, 8, 128).half()
    want = c.attend(q, table, L, offsets([40, 40]), max_new=40)
    bad = table.clone()
    bad[0, 3] = 1 << 20
    out = c.attend(q, bad, L, offsets([40, 40]), max_new=40)
    with pytest.raises(_lib.VqError):
        c.status()
    assert torch.equal(out[40:], want[40:])


def test_offsets_past_32_bits():
    """Pages whose bytes lie past 2^32 of the pool."""
    D, g, page, H = 128, 32, 128, 8
    n_pages = 2 ** 32 // (H * 8 * 2560) + 5
    c = new_cache(n_pages, page, H, H, D, g, fill=0)
    table = i32([n_pages - 1, n_pages - 3, 1]).view(1, 3)
    S = 300
    k, v = randn(1, S, H, D).half(), randn(2, S, H, D).half()
    c.append(k, v, table, i32([S]), offsets([S]))
    for n in (1, 4):
        q = randn(3, n, H, D).half()
        out = c.attend(q, table, i32([S]), offsets([n]), max_new=n if n == 1 else 40)
        want, err = ref.attend64(q, c.pool, table, i32([S]), offsets([n]), D, g, H,
                                 weight_step=MANY)
        ref.check_attend(out, want, err, q.dtype)
    c.status()


# ---- weights far apart, and walks of many steps -----------------------------------

# a weight's error beside weight_step of itself, relative to the row's largest
# weight: fp16's half step 2^-25 of weights whose largest is 2^9 or more,
# twice (written, and brought to a new maximum); with hi + lo (up to 8 rows)
# the half step of the remainders times 2^12
FLOOR_FEW, FLOOR_MANY = 2.0 ** -43, 2.0 ** -33


def levels_cache(levels, page, H_q, H_kv, D, g, seed):
    """One sequence whose token t has the key levels[t] in every channel (so a
    query of ones scores it D levels[t]) and values that are constant over a
    group: 1 in the first group, but 0 for the token of the largest level;
    some multiple of 1/8 in the others.  All exact in 4 bits."""
    S = len(levels)
    c = new_cache(-(-S // page) + 1, page, H_q, H_kv, D, g)
    table = ref.make_table(1, [S], page, c.n_pages, "cuda", seed)
    lv = torch.tensor(levels, dtype=torch.float64, device="cuda")
    assert torch.equal(lv.half().double(), lv)
    v = torch.randint(-16, 17, (S, D // g), generator=torch.Generator().manual_seed(seed)) / 8.0
    v[:, 0] = 1.0
    v[lv.argmax().item(), 0] = 0.0
    K = lv[:, None].expand(S, D).contiguous()
    V = v.double().cuda().repeat_interleave(g, -1)
    rows = lambda x: x.half()[:, None].expand(S, H_kv, D)
    c.append(rows(K), rows(V), table, i32([S]), offsets([S]))
    c.status()
    return c, table, K, V


def _sink(S, at, gap):
    x = [0.0] * S
    x[at] = gap
    return x


def _stairs(S):
    """Nothing for a tile, then half a tile 10.25 nats higher, then one token
    17.75 nats up: what was weighed against the first maximum is brought far
    down inside the tile."""
    x = [0.0] * S
    x[128:192] = [10.25] * 64
    x[200] = 17.75
    return x


LEVELS = {
    "sink 14": lambda S: _sink(S, 3, 14.0), "sink 16": lambda S: _sink(S, 0, 16.0),
    "sink 17.5": lambda S: _sink(S, 70, 17.5), "sink 20": lambda S: _sink(S, 2001, 20.0),
    "stairs": _stairs,
    "rising": lambda S: [round(64 * 24 * t / S) / 64 for t in range(S)],
}


@pytest.mark.parametrize("name", list(LEVELS))
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("H_q,H_kv,n,D,g", [
    (8, 8, 1, 128, 32), (32, 8, 1, 64, 64), (32, 8, 4, 128, 64), (16, 8, 8, 64, 32),
    (8, 8, 33, 128, 32), (8, 8, 200, 64, 32), (32, 8, 50, 128, 128),
])
def test_one_large_weight_before_a_long_tail(name, dtype, H_q, H_kv, n, D, g):
    """Weights far below a row's largest still count in sum (an attention sink
    of value 0 before a flat tail; maxima that rise late).  As many sequences,
    all of the same pages, as give every resident warp or CTA whole sequences
    to walk."""
    S = 4100
    c, table, K, V = levels_cache(LEVELS[name](S), 64, H_q, H_kv, D, g, 3)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    few = n * (H_q // H_kv) <= 16
    B = -(-sms * 16 // H_kv) + 1 if few else -(-2 * sms // H_kv)
    q = torch.ones(B * n, H_q, D, dtype=DT[dtype], device="cuda")
    cu = None if n == 1 else offsets([n] * B)
    out = c.attend(q, table.repeat(B, 1), i32([S] * B), cu, max_new=n, scale=1.0 / D)
    c.status()
    hi_lo = n * (H_q // H_kv) <= 8
    want, err = ref.attend64_rows(torch.ones(n, D, dtype=torch.float64, device="cuda"), K, V,
                                  range(S - n + 1, S + 1), 1.0 / D, FEW if hi_lo else MANY,
                                  FLOOR_FEW if hi_lo else FLOOR_MANY)
    for b in range(0, B, max(B // 8, 1)):
        for h in range(0, H_q, 3):
            ref.check_attend(out[b * n:(b + 1) * n, h], want, err, q.dtype)


@pytest.mark.parametrize("dtype,size,step", [("fp16", 2.0 ** 15, 32.0), ("bf16", 2.0 ** 120, 1.0),
                                             ("bf16", -(2.0 ** 118), 1.0), ("fp16", -60000.0, 8.0),
                                             ("bf16", 2.0 ** 15, 32.0)])
@pytest.mark.parametrize("H_q,H_kv,n,D", [(4, 2, 1, 128), (8, 2, 4, 64), (2, 2, 33, 128),
                                          (4, 2, 80, 64)])
def test_finite_rows_of_any_size_give_finite_outputs(dtype, size, step, H_q, H_kv, n, D):
    """Scores far beyond 2^24, whose fp32 steps are whole bits, and bf16 rows
    near the type's largest values.  Keys are constant over the channels and
    climb by `step` with the token, three equal ones in front: the softmax is
    one token's, or the mean of the equal ones.  2^120 times 304 times 128
    channels is no fp32 number by any way of adding up, so that the bf16 rows'
    scale is 2^-16."""
    S = 300
    lv = torch.arange(S, dtype=torch.float64) * step - 2048 * step * (size == 2.0 ** 15)
    lv[:3] = lv[-1] + 5 * step if size > 0 else lv[0] - 5 * step
    assert torch.equal(lv.half().double(), lv)
    c = new_cache(20, 16, H_q, H_kv, D, 32)
    table = ref.make_table(1, [S], 16, 20, "cuda", 3)
    v = (torch.randint(-16, 17, (S, D // 32), generator=torch.Generator().manual_seed(1)) / 8.0)
    V = v.repeat_interleave(32, -1)
    rows = lambda x: x.half().cuda()[:, None].expand(S, H_kv, D)
    c.append(rows(lv[:, None].expand(S, D)), rows(V), table, i32([S]), offsets([S]))
    q = torch.full((n, H_q, D), size, dtype=DT[dtype], device="cuda")
    scale = 2.0 ** -16 if abs(size) > 1e30 else 0.0
    out = c.attend(q, table, i32([S]), offsets([n]), max_new=n, scale=scale)
    c.status()
    want = V[:3].double().mean(0).numpy()
    err = 4 * 2.0 ** -11 * V[:3].double().abs().mean(0).numpy()
    ref.check_attend(out, np.broadcast_to(want, out.shape), np.broadcast_to(err, out.shape), q.dtype)
    # and the climbing tokens alone: the newest that a row sees
    if size > 0:
        lv2 = lv.clone()
        lv2[:3] = lv[3]
        c.append(rows(lv2[:, None].expand(S, D)), rows(V), table, i32([S]), offsets([S]))
        out = c.attend(q, table, i32([S]), offsets([n]), max_new=n, scale=scale)
        want = np.repeat(V[S - n:].double().numpy()[:, None], H_q, 1)
        ref.check_attend(out, want, 4 * 2.0 ** -11 * np.abs(want), q.dtype)


@pytest.mark.parametrize("size,scale", [(2.0 ** -125, 1e-10), (2.0 ** -130, 1e-3), (1.0, 1e-42),
                                        (2.0 ** 100, 1e20)])
@pytest.mark.parametrize("H_q,H_kv,n", [(4, 2, 1), (8, 2, 4), (2, 2, 40)])
def test_factors_at_the_ends_of_fp32(size, scale, H_q, H_kv, n):
    """Tiny rows under a tiny scale, whose factors multiply to less than fp32
    holds, and large ones whose factors pass it, over keys of 0: every seen
    token weighs the same, masked ones (lengths inside a block) nothing."""
    c, table, L = filled([45], 16, H_q, H_kv, 64, 32, gain=0.0 if size > 2 else 1.0)
    q = torch.full((n, H_q, 64), size, dtype=torch.bfloat16, device="cuda")
    out = c.attend(q, table, L, offsets([n]), max_new=n, scale=scale)
    c.status()
    V = c.dequantize(table, L, offsets([45]), n_tokens=45)[1].double().cpu()
    for i in range(n):
        v = V[:45 - n + i + 1].repeat_interleave(H_q // H_kv, 1)
        ref.check_attend(out[i], v.mean(0).numpy(),
                         (4 * 2.0 ** -11 * v.abs().mean(0)).numpy(), q.dtype)


def test_status_keeps_what_another_stream_finds_meanwhile():
    """A fault set by a kernel of another stream at any moment around a check
    that has another fault to report is reported by this check or the next."""
    from bit_kv_cache_05_gb300 import _lib
    c = new_cache(2, 16, 1, 1, 64, 32)
    k = randn(1, 1, 1, 64).half()
    far, here = i32([7]).view(1, 1), i32([0]).view(1, 1)
    one, long = i32([1]), i32([17])
    other = torch.cuda.Stream()
    c.append(k, k, here, one, stream=other)
    torch.cuda.synchronize()

    def found():
        try:
            c.status()
        except _lib.VqError as e:
            return str(e)
        return ""

    for i in range(600):
        c.append(k, k, far, one)                      # a page outside the pool
        torch.cuda.synchronize()
        with torch.cuda.stream(other):
            torch.cuda._sleep(400 * i)                # up to about 120 us
            c.append(k, k, here, long)                # a length outside its range
        first = found()
        assert "page" in first
        torch.cuda.synchronize()
        assert "length" in first + found()
        assert found() == ""


@pytest.mark.parametrize("cu,lens,left", [
    ([0, 3, 5, 11], [3, 20, 30], [2]),            # more new tokens than rows
    ([0, 3, 1, 9], [3, 20, 30], [1]),             # falling
    ([-2, 3, 5, 9], [30, 20, 30], [0]),           # a row before the first
    ([0, 3, 3, 9], [3, 999, 30], [1]),            # too long, nothing new
    ([0, 3, 3, 9], [3, -1, 30], [1]),
    ([0, 3, 5, 9], [3, 999, 30], [1]),
])
def test_all_operators_leave_out_and_report_the_same_sequences(cu, lens, left):
    """A sequence whose length or new tokens lie outside their ranges: append,
    read-back and attention each report it, leave its pages and rows as they
    were and serve the others."""
    from bit_kv_cache_05_gb300 import _lib
    H, D, T = 2, 64, 9
    k, v, q = (randn(i, T, H, D).half() for i in (1, 2, 3))
    table = i32([0, 1, 2, 3, 4, 5]).view(3, 2)
    c = new_cache(6, 16, H, H, D, 32)
    good = [b for b in range(3) if b not in left and cu[b + 1] > cu[b]]

    def faulty(f):
        r = f()
        with pytest.raises(_lib.VqError, match="length"):
            c.status()
        c.status()
        return r

    qo = torch.full_like(q, 7.0)
    faulty(lambda: c.append(k, v, table, i32(lens), i32(cu), q=q, q_out=qo))
    out = (torch.full_like(k, 7.0), torch.full_like(v, 7.0))
    faulty(lambda: c.dequantize(table, i32(lens), i32(cu), n_tokens=T, out=out))
    n = [cu[b + 1] - cu[b] for b in range(3)]
    for b in left:
        assert (c.pool[table[b].long()] == 0xff).all()
    mine = torch.zeros(T, dtype=torch.bool)
    want = new_cache(6, 16, H, H, D, 32)
    for b in good:
        r = slice(cu[b], cu[b + 1])
        mine[r] = True
        want.append(k[r], v[r], table[b:b + 1], i32([lens[b]]), offsets([n[b]]))
        K, V = want.dequantize(table[b:b + 1], i32([lens[b]]), offsets([n[b]]), n_tokens=n[b])
        if cu != [0, 3, 1, 9]:                    # there rows belong to two sequences
            assert torch.equal(c.pool[table[b].long()], want.pool[table[b].long()])
            assert torch.equal(qo[r], q[r])
            assert torch.equal(out[0][r].view(torch.int16), K.view(torch.int16))
            assert torch.equal(out[1][r].view(torch.int16), V.view(torch.int16))
    assert (qo[~mine] == 7).all() and (out[0][~mine] == 7).all() and (out[1][~mine] == 7).all()
    # whole caches for the attention
    c.pool.fill_(0)
    for max_new in (4, 20):
        o = torch.full_like(q, 7.0)
        faulty(lambda: c.attend(q, table, i32(lens), i32(cu),
                                max_new=max(max_new, max(n)), out=o))
        assert (o[~mine] == 7).all() and (o[mine] == 0).all()


@pytest.mark.parametrize("dtype", [torch.int64, torch.int32])
def test_positions_broadcast_over_the_axes(dtype):
    """One row of positions for all axes, as text has them: expanded, not
    copied."""
    from bit_kv_cache_05_gb300.rope import Rope, norm_rope
    T, H, D = 37, 2, 64
    rope = Rope(rot_dim=D, sections=[8, 12, 12])
    q, k, v = (randn(i, T, H, D).half() for i in (1, 2, 3))
    pos = torch.randint(0, 100000, (T,), generator=torch.Generator().manual_seed(4)).to(dtype).cuda()
    many = pos[None].expand(3, -1)
    assert many.stride(0) == 0
    a, b = norm_rope(q, k, many, rope), norm_rope(q, k, many.contiguous(), rope)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    inv = [1e4 ** (-2.0 * j / D) for j in range(D // 2)]
    want, mag = ref.norm_rope64(q, None, many, inv, [0] * 8 + [1] * 12 + [2] * 12, False)
    assert ((a[0].cpu().double() - want).abs()
            <= ref.norm_rope_bound(want, mag, torch.float16, D)).all()
    pools = []
    for p in (many, many.contiguous()):
        c = new_cache(3, 16, H, H, D, 32)
        out = c.append(k, v, i32([0, 1, 2]).view(1, 3), i32([T]), offsets([T]), q=q, rope=rope,
                       positions=p)
        assert torch.equal(out, a[0])
        pools.append(c.pool)
    assert torch.equal(pools[0], pools[1])


def test_readme_sample():
    """The README's paged sample as it stands: a prompt chunk, then one token
    more per sequence, which must see the whole prompt."""
    import os
    text = open(os.path.join(os.path.dirname(__file__), "..", "README.md")).read()
    code = [b.split("```")[0] for b in text.split("```python")[1:] if "PagedKiviCache(" in b]
    assert len(code) == 1
    n, B, H_q, H_kv, D, dt = [300, 128], 2, 32, 8, 128, torch.bfloat16
    T = sum(n)
    x = randn(1, T + B, H_q + 2 * H_kv, D).to(dt)
    w = (1 + 0.1 * randn(2, D)).to(dt)
    part = lambda r: (x[r, :H_q], x[r, H_q:H_q + H_kv], x[r, H_q + H_kv:])
    q, k, v = part(slice(0, T))
    q1, k1, v1 = part(slice(T, T + B))
    env = dict(q=q, k=k, v=v, q1=q1, k1=k1, v1=v1, wk=w, wq=w, lens=i32(n), cu_new=offsets(n),
               table=ref.make_table(B, [a + 1 for a in n], 64, 1024, "cuda", 3),
               positions=torch.arange(T, device="cuda"))
    exec(code[0], env)
    c, table = env["cache"], env["table"]
    lens = i32([a + 1 for a in n])
    assert torch.equal(env["lens"], lens)
    want, err = ref.attend64(env["q1"], c.pool, table, lens, None, D, 32, H_kv, weight_step=FEW)
    ref.check_attend(env["out1"], want, err, dt)
    # the prompt's tokens and the new ones as they would be stored at once
    from bit_kv_cache_05_gb300.rope import Rope
    one = new_cache(1024, 64, H_q, H_kv, D, 32)
    order = list(range(300)) + [T] + list(range(300, T)) + [T + 1]
    one.append(x[order, H_q:H_q + H_kv], x[order, H_q + H_kv:], table, lens, offsets([301, 129]),
               rope=Rope(rot_dim=128, theta=5e5), k_weight=w)
    a = c.dequantize(table, lens, offsets([301, 129]), n_tokens=T + B)
    b = one.dequantize(table, lens, offsets([301, 129]), n_tokens=T + B)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# decode (one row, few rows, drafts), chunks of one query tile and of two,
# mixed: heads, D, group, page, new tokens of a sequence
LONG = [
    (32, 8, 128, 32, 64, (1, 1)), (8, 8, 64, 64, 16, (1, 1)), (12, 4, 128, 64, 32, (1, 2)),
    (32, 8, 128, 128, 128, (2, 4)), (16, 8, 64, 32, 16, (1, 8)),
    (16, 4, 128, 64, 64, (17, 32)), (8, 4, 64, 32, 16, (20, 64)), (20, 4, 128, 32, 32, (4, 25)),
    (8, 4, 128, 32, 64, (100, 300)), (16, 4, 64, 64, 32, (1, 150)),
]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("H_q,H_kv,D,g,page,new", LONG)
def test_long_walks(dtype, H_q, H_kv, D, g, page, new):
    """More work than resident warps and CTAs: 40 steps a warp, 10 key tiles a
    CTA at least, so that every stage and barrier phase is used many times and
    pieces of the work line end inside sequences and span whole ones.  The
    sequences (empty and short ones among them) share a pool's pages in orders
    of their own; keys grow with the page, so that maxima rise late, early or
    at random."""
    gen = torch.Generator().manual_seed(7)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    few = new[1] * (H_q // H_kv) <= 16
    S = 8192
    n_pages = S // page
    c = new_cache(n_pages + 1, page, H_q, H_kv, D, g)
    gain = (0.2 + 2.0 * torch.arange(S) / S).cuda()[:, None, None]
    whole = torch.arange(n_pages, dtype=torch.int32, device="cuda")[None]
    c.append((randn(1, S, H_kv, D) * gain).half(), randn(2, S, H_kv, D).half(), whole, i32([S]),
             offsets([S]))
    # 32-token steps of 16 warps an SM, or 128-token tiles of a CTA an SM
    need = 40 * 16 * sms * 32 if few else 12 * sms * 128
    B = min(-(-need // (H_kv * 7000)) + 4, 200)
    lens = [int(x) for x in torch.randint(6000, S + 1, (B,), generator=gen)]
    lens[1], lens[B // 2], lens[B - 2] = 0, 1, 33
    news = [int(x) for x in torch.randint(new[0], new[1] + 1, (B,), generator=gen)]
    news[B // 3] = news[B // 3] if new == (1, 1) else 0
    table = torch.stack([torch.arange(n_pages) if b % 3 == 0 else
                         torch.arange(n_pages).flip(0) if b % 3 == 1 else
                         torch.randperm(n_pages, generator=gen) for b in range(B)]).int().cuda()
    T = sum(news)
    q = (randn(3, T, H_q, D) * 2).to(DT[dtype])
    cu = None if new == (1, 1) else offsets(news)
    out = c.attend(q, table, i32(lens), cu, max_new=new[1])
    c.status()
    at = np.concatenate([[0], np.cumsum(news)])
    hi_lo = new[1] * (H_q // H_kv) <= 8
    for b in sorted({0, 1, 2, B // 3, B // 2, B - 2, B - 1, *range(4, B, max(1, B // 6))}):
        rows = out[at[b]:at[b + 1]]
        seen = [lens[b] - news[b] + i + 1 for i in range(news[b])]
        off = sum(s <= 0 for s in seen)
        assert (rows[:off] == 0).all()
        if off == news[b]:
            continue
        K, V = c.dequantize(table[b:b + 1], i32(lens[b:b + 1]), offsets([lens[b]]),
                            n_tokens=lens[b])
        for h in {0, b % H_kv, H_kv - 1}:
            for hq in (h * (H_q // H_kv), (h + 1) * (H_q // H_kv) - 1):
                want, err = ref.attend64_rows(q[at[b] + off:at[b + 1], hq].double(),
                                              K[:, h].double(), V[:, h].double(), seen[off:],
                                              D ** -0.5, FEW if hi_lo else MANY,
                                              FLOOR_FEW if hi_lo else FLOOR_MANY)
                ref.check_attend(rows[off:, hq], want, err, q.dtype)


@pytest.mark.parametrize("dtype,D,g,rot,inter,scale,axes,H_kv", [
    ("fp16", 128, 32, 128, True, 1.0, 1, 3), ("bf16", 128, 64, 64, False, 1.25, 3, 2),
    ("fp16", 128, 128, 96, True, 0.75, 2, 1), ("bf16", 64, 32, 64, False, 1.0, 1, 5),
    ("fp16", 64, 64, 64, True, 1.0, 3, 2), ("bf16", 64, 32, 32, False, 2.0, 1, 8),
    ("fp16", 64, 64, 16, True, 1.0, 1, 1), ("fp16", 128, 64, 128, False, 1.0, 4, 4),
])
def test_append_of_every_rotation(dtype, D, g, rot, inter, scale, axes, H_kv):
    """Interleaved pairs, a partial rotation, a factor, D = 64 and groups
    longer than a lane's channels: the stored keys' scales, zeros and codes are
    those of the 64-bit rotation, up to its roundings."""
    from bit_kv_cache_05_gb300.rope import Rope
    dt, n, H_q = DT[dtype], [5, 40, 1], 2 * H_kv
    T = sum(n)
    x = (randn(7, T, H_q + 2 * H_kv, D) * 2).to(dt)
    q, k, v = x[:, :H_q], x[:, H_q:H_q + H_kv], x[:, H_q + H_kv:]
    w = (1 + 0.1 * randn(9, D)).to(dt)
    axis = [j % axes for j in range(rot // 2)]
    inv = [1e4 ** (-2.0 * j / rot) for j in range(rot // 2)]
    rope = Rope(inv, axis=axis, interleaved=inter, scale=scale)
    pos = torch.randint(0, 50000, (axes, T), generator=torch.Generator().manual_seed(4))
    table = ref.make_table(3, n, 16, 8, "cuda", 3)
    c = new_cache(8, 16, H_q, H_kv, D, g)
    got = c.append(k, v, table, i32(n), offsets(n), q=q, rope=rope, q_weight=w, k_weight=w,
                   positions=pos.cuda())
    c.status()
    want, mag = ref.norm_rope64(q, w, pos, inv, axis, inter, scale)
    assert ((got.cpu().double() - want).abs() <= ref.norm_rope_bound(want, mag, dt, D)).all()
    # the keys: norm and rotation of fp32 rows, rounded to fp16 as the append does
    want, mag = ref.norm_rope64(k, w, pos, inv, axis, inter, scale)
    err = ref.norm_rope_bound(want, mag, torch.float32, D)
    tab, at = table.cpu().numpy(), 0
    for b, m in enumerate(n):
        for h in range(H_kv):
            code, s, z = ref.cache_parts(c.pool, tab[b], m, h, D, g)["k"]
            for i in range(m):
                y, e = want[at + i, h].numpy(), err[at + i, h].numpy()
                lo = y.reshape(-1, g).min(-1).repeat(g)
                span = y.reshape(-1, g).max(-1).repeat(g) - lo
                # an fp16 rounding (half a step) of the row's values on top of
                # their fp32 errors, for the group's ends and the value itself
                d = (e + 2.0 ** -11 * np.abs(y) + 2.0 ** -25).reshape(-1, g).max(-1).repeat(g)
                zz, ss = z[i].astype(np.float64), s[i].astype(np.float64)
                assert (np.abs(zz - lo) <= d).all()
                assert (np.abs(ss - span / 15) <= 2 * d / 15 + 2.0 ** -11 * (span + 2 * d) / 15
                        + 2.0 ** -25).all()
                # the value's place between the ends, in steps of the scale:
                # half a step, and the errors of both ends
                step = np.maximum(span / 15, 1e-30)
                place = (y - lo) / step
                assert (np.abs(code[i] - place) <= 0.5 + 4 * d / step + 2.0 ** -20).all()
        at += m


@pytest.mark.parametrize("n", [1, 4, 40])
def test_one_sequence_of_131089_tokens(n):
    """A table of 1025 pages, each of the pool's 64 many times."""
    H_q, H_kv, D, g, page, S = 8, 2, 128, 64, 128, 131072 + 17
    c = new_cache(64, page, H_q, H_kv, D, g)
    whole = torch.arange(64, dtype=torch.int32, device="cuda")[None]
    c.append(randn(1, 8192, H_kv, D).half(), randn(2, 8192, H_kv, D).half(), whole, i32([8192]),
             offsets([8192]))
    gen = torch.Generator().manual_seed(5)
    table = torch.randint(0, 64, (1, 1025), generator=gen).int().cuda()
    q = (randn(3, n, H_q, D) * 2).bfloat16()
    out = c.attend(q, table, i32([S]), offsets([n]), max_new=n)
    c.status()
    K, V = c.dequantize(table, i32([S]), offsets([S]), n_tokens=S)
    for hq in (0, 3, 4, 7):
        want, err = ref.attend64_rows(q[:, hq].double(), K[:, hq // 4].double(),
                                      V[:, hq // 4].double(), range(S - n + 1, S + 1), D ** -0.5,
                                      FEW if n == 1 else MANY,
                                      FLOOR_FEW if n == 1 else FLOOR_MANY)
        ref.check_attend(out[:, hq], want, err, q.dtype)
