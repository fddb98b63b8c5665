"""Measured cases of the paged 4-bit cache's operators and of the per-head norm
with rotation that feeds it.

Four kinds of pass, each as a serving program makes it:

  norm_rope   queries and keys of a packed projection: RMS norm over each head
              (optional), then the position rotation on one or several axes
  append      new tokens enter the paged 4-bit cache: keys normed and rotated
              on the way, keys and values quantized, the queries normed and
              rotated in the same pass; the tokens' rows are read back as the
              values that the cache now stands for
  decode      attention of one new token per sequence over the paged cache
  chunk       causal attention of several new tokens per sequence

`own` chooses between the plain form (elementary torch operations in 32 bits,
angles in 64) and the framework's kernels.  Both work on the same state.

The pool is uint8 [n_pages][H_kv][page / 16][block]; a block holds 16 tokens of
one kv head: key codes, key (scale, zero), value codes, value (scale, zero).
  key codes     per token D/8 words; word (D/32) t + i holds channels
                32 i + 8 t ... + 7, the lowest nibble first (t < 4)
  value codes   word ((8 h + g) 4 + t) (D/32) + i holds channels
                32 i + 4 g ... + 3 of token 8 h + 2 t in its low half and of
                the next token in its high half, the lowest nibble first
  scale, zero   fp16, per token pair and group: s, s', z, z'
A value stands for code * scale + zero, rounded to fp16.
"""
import math
import random

import torch

own = False

EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---- cases ---------------------------------------------------------------

def listed():
    return [
        # a decode step of 16 sequences: one token each, latency counts
        dict(name="norm_rope step B16", op="norm_rope", T=16, H_q=32, H_kv=8, D=128, rot=128,
             axes=1, interleaved=False, norm=True, dtype="bf16", far=131072),
        # a whole prompt in one go, positions far into a long context
        dict(name="norm_rope prompt 16384", op="norm_rope", T=16384, H_q=32, H_kv=8, D=128,
             rot=128, axes=1, interleaved=False, norm=True, dtype="bf16", far=1048576),
        # image tokens: time, height and width positions, no norm, an odd count
        dict(name="norm_rope image 4099", op="norm_rope", T=4099, H_q=32, H_kv=32, D=64, rot=64,
             axes=3, interleaved=True, norm=False, dtype="fp16", far=4096),
        # the append of one decode step, 64 running sequences, small pages
        dict(name="append step B64", op="append", B=64, n_lo=1, n_hi=1, s_lo=1, s_hi=8192,
             H_q=32, H_kv=8, D=128, group=32, page=16, axes=1, norm=True, dtype="bf16"),
        # ragged prompt chunks of four sequences, the context already long
        dict(name="append prompt 4x8192", op="append", B=4, n_lo=2048, n_hi=8192, s_lo=8192,
             s_hi=32768, H_q=32, H_kv=8, D=128, group=64, page=64, axes=1, norm=False,
             dtype="fp16"),
        # one short sequence, every head with its own keys: latency counts
        dict(name="decode S512", op="decode", B=1, s_lo=512, s_hi=512, H_q=32, H_kv=32, D=128,
             group=32, page=64, dtype="fp16", outliers=0),
        # one long sequence, every head with its own keys
        dict(name="decode S65536", op="decode", B=1, s_lo=65536, s_hi=65536, H_q=32, H_kv=32,
             D=128, group=32, page=64, dtype="fp16", outliers=0),
        # a serving batch with grouped heads and key channels that stand out
        dict(name="decode gqa B16 S8192", op="decode", B=16, s_lo=8192, s_hi=8192, H_q=32,
             H_kv=8, D=128, group=32, page=16, dtype="bf16", outliers=8),
        # long sequences of unequal lengths
        dict(name="decode ragged long", op="decode", B=4, s_lo=16384, s_hi=131072, H_q=32,
             H_kv=8, D=128, group=64, page=128, dtype="bf16", outliers=8),
        # drafts of four tokens checked for 16 sequences
        dict(name="chunk draft 16x4", op="chunk", B=16, n_lo=4, n_hi=4, s_lo=4096, s_hi=8192,
             H_q=32, H_kv=8, D=128, group=32, page=16, dtype="bf16"),
        # prompt chunks of 512 tokens at the end of long contexts
        dict(name="chunk 2x512 S32768", op="chunk", B=2, n_lo=512, n_hi=512, s_lo=33280,
             s_hi=33280, H_q=32, H_kv=8, D=128, group=64, page=64, dtype="bf16"),
        # whole prompts of unequal lengths, nothing before them
        dict(name="chunk prompts 4x4096", op="chunk", B=4, n_lo=1021, n_hi=4096, s_lo=0, s_hi=0,
             H_q=32, H_kv=8, D=64, group=32, page=32, dtype="fp16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "decode", "chunk"])
    H_kv = rng.choice([1, 2, 4, 8])
    H_q = H_kv * rng.choice([1, 2, 3, 4, 5, 8])
    D = rng.choice([64, 128])
    group = rng.choice([32, 64, 128] if D == 128 else [32, 64])
    page = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "norm_rope":
        D = rng.choice([64, 96, 128, 256])
        return dict(op=op, T=_log(rng, 1, 16384), H_q=H_q, H_kv=H_kv, D=D,
                    rot=rng.choice([D, D, D // 2]), axes=rng.choice([1, 3]),
                    interleaved=rng.choice([False, True]), norm=rng.choice([True, False]),
                    dtype=rng.choice(["bf16", "fp16", "fp32"]), far=_log(rng, 64, 1048576))
    if op == "append":
        n = _log(rng, 1, 4096)
        return dict(op=op, B=_log(rng, 1, max(1, min(128, 16384 // n))), n_lo=max(1, n // 2),
                    n_hi=n, s_lo=n, s_hi=n + _log(rng, 1, 16384), H_q=H_q, H_kv=H_kv, D=D,
                    group=group, page=page, axes=rng.choice([1, 3]),
                    norm=rng.choice([True, False]), dtype=dtype)
    if op == "decode":
        S = _log(rng, 1, 65536)
        return dict(op=op, B=_log(rng, 1, max(1, min(128, 262144 // S))), s_lo=S // 2, s_hi=S,
                    H_q=H_q, H_kv=H_kv, D=D, group=group, page=page, dtype=dtype,
                    outliers=rng.choice([0, 8]))
    n = _log(rng, 2, 1024)
    S = _log(rng, n, 16384)
    H_kv = min(H_kv, 4)
    H_q = H_kv * rng.choice([1, 2, 3, 4, 5, 8])
    return dict(op=op, B=_log(rng, 1, max(1, min(32, 2048 // n))), n_lo=max(1, n // 2), n_hi=n,
                s_lo=S, s_hi=S, H_q=H_q, H_kv=H_kv, D=D, group=group, page=page, dtype=dtype)


def _lengths(case):
    """New tokens and lengths (new tokens included) of each sequence: part of
    the case, so drawn from its own values.  s_hi = 0: nothing before the new
    tokens."""
    rng = random.Random("%(B)d %(s_lo)d %(s_hi)d %(H_q)d %(page)d" % case)
    n = [rng.randint(case["n_lo"], case["n_hi"]) if "n_lo" in case else 1
         for _ in range(case["B"])]
    S = [max(m if "n_lo" in case else 0, rng.randint(case["s_lo"], case["s_hi"])) for m in n]
    return n, S


# ---- work ----------------------------------------------------------------

def work(case):
    D, H_q, H_kv = case["D"], case["H_q"], case["H_kv"]
    e = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "norm_rope":
        rows = case["T"] * (H_q + H_kv)
        return dict(bytes=2 * rows * D * e + 8 * case["T"] * case["axes"], flops=10 * rows * D)
    n, S = _lengths(case)
    tok = H_kv * (D + 8 * (D // case["group"]))          # bytes of a stored token
    if case["op"] == "append":
        T = sum(n)
        heads = T * (2 * H_q + 2 * H_kv) * D * e          # q in and out, k and v in
        # written as codes, read back as codes, given out in 16 bits
        return dict(bytes=heads + 2 * T * tok + 2 * T * H_kv * D * 2 + 8 * T * case["axes"],
                    flops=T * D * (10 * H_q + 30 * H_kv))
    T = sum(n) if case["op"] == "chunk" else case["B"]
    pairs = sum(m * (s - m) + m * (m + 1) // 2 for m, s in zip(n, S)) \
        if case["op"] == "chunk" else sum(S)
    return dict(bytes=sum(S) * tok + 2 * T * H_q * D * e, flops=4 * pairs * H_q * D)


# ---- the pool's blocks -----------------------------------------------------

def _quantize(x, group):
    """codes, scale, zero of fp16 rows over groups of channels (32-bit IEEE
    arithmetic; a constant group has scale 0 and codes 0)."""
    g = x.float().unflatten(-1, (-1, group))
    lo, hi = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    # by a tensor: torch divides by a number as a product with its reciprocal
    scale = (hi - lo) / torch.full_like(hi, 15.0)
    code = torch.where(scale > 0, torch.round((g - lo) / scale), torch.zeros_like(g))
    return (code.clamp(0, 15).to(torch.uint8).flatten(-2), scale[..., 0].half(),
            (lo[..., 0] + 0.0).half())


def _pack_blocks(kc, ks, kz, vc, vs, vz):
    """[..., 16, D] codes and [..., 16, D/group] scales, zeros -> [..., block]
    bytes."""
    def meta(s, z):
        m = torch.stack((s, z), -2).unflatten(-3, (8, 2))       # [8, 2, {s, z}, groups]
        m = m.movedim(-4 + 1, -1)                               # [8, {s, z}, groups, 2]
        return m.transpose(-3, -2).contiguous().view(torch.uint8).flatten(-4)

    def nibbles(c):
        c = c.unflatten(-1, (-1, 2))
        return c[..., 0] | (c[..., 1] << 4)

    k = kc.unflatten(-1, (-1, 4, 8)).transpose(-3, -2).flatten(-4)
    v = vc.unflatten(-1, (-1, 8, 4)).unflatten(-4, (2, 4, 2))    # [h, t, s, i, g, r]
    d = v.dim() - 6
    v = v.permute(*range(d), d, d + 4, d + 1, d + 3, d + 2, d + 5).flatten(-6)
    return torch.cat((nibbles(k), meta(ks, kz), nibbles(v), meta(vs, vz)), -1)


def _unpack_blocks(blocks, D, group):
    """[..., block] bytes -> fp32 key and value rows [..., 16, D] that the
    blocks stand for (rounded to fp16 as the definition asks)."""
    nc, nm, ng = 8 * D, 64 * (D // group), D // group

    def codes(b):
        return torch.stack((b & 15, b >> 4), -1).flatten(-2)

    def meta(b):
        m = b.contiguous().view(torch.float16).unflatten(-1, (8, ng, 2, 2)).float()
        m = m.transpose(-4 + 1, -1)                              # [8, 2, {s, z}, groups]
        m = m.flatten(-4, -3)                                    # [16, {s, z}, groups]
        return (m[..., 0, :].repeat_interleave(group, -1),
                m[..., 1, :].repeat_interleave(group, -1))

    kc, km, vc, vm = torch.split(blocks, (nc, nm, nc, nm), -1)
    k = codes(kc).unflatten(-1, (16, 4, -1, 8)).transpose(-3, -2).flatten(-3)
    v = codes(vc).unflatten(-1, (2, 8, 4, D // 32, 2, 4))        # [h, g, t, i, s, r]
    d = v.dim() - 6
    v = v.permute(*range(d), d, d + 2, d + 4, d + 3, d + 1, d + 5)
    v = v.flatten(-6, -4).flatten(-3)
    out = []
    for c, m in ((k, km), (v, vm)):
        s, z = meta(m)
        # the product of a 4-bit code and an fp16 scale is exact in 32 bits
        out.append((c.float() * s + z).half().float())
    return out


# ---- inputs ----------------------------------------------------------------

def _gen(seed, stream):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000 + stream)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _frequencies(rot, axes):
    """Frequencies of the rotated pairs in 64 bits and the axis of each pair
    (a quarter of them time, the rest height and width)."""
    half = rot // 2
    inv = torch.tensor([10000.0 ** (-i / half) for i in range(half)], dtype=torch.float64)
    if axes == 1:
        return inv, [0] * half
    a, b = half // 4, half // 4 + (half - half // 4) // 2
    return inv, [0 if i < a else 1 if i < b else 2 for i in range(half)]


def prepare(case, seed):
    D, H_q, H_kv = case["D"], case["H_q"], case["H_kv"]
    dt = DTYPES[case["dtype"]]
    s = dict(case=case)
    if case["op"] in ("norm_rope", "append"):
        rot = case.get("rot", D)
        inv, axis = _frequencies(rot, case["axes"])
        s["inv_freq"], s["axis"] = inv.cuda(), torch.tensor(axis, device="cuda")
    if case["op"] == "norm_rope":
        T = case["T"]
        # q, k and v as one projection gives them: the heads are strided views
        x = _randn(_gen(seed, 0), T, (H_q + 2 * H_kv) * D).to(dt)
        x = x.view(T, H_q + 2 * H_kv, D)
        s["q"], s["k"] = x[:, :H_q], x[:, H_q:H_q + H_kv]
        g = _gen(seed, 1)
        s["positions"] = torch.randint(0, case["far"], (case["axes"], T), generator=g,
                                       device="cuda")
        if case["norm"]:
            s["q_weight"] = (1 + 0.1 * _randn(g, D)).to(dt)
            s["k_weight"] = (1 + 0.1 * _randn(g, D)).to(dt)
        if own:
            from bit_kv_cache_05_gb300.rope import Rope
            s["rope"] = Rope(inv, axis=axis, interleaved=case["interleaved"])
        return s

    B, page, group = case["B"], case["page"], case["group"]
    n, S = _lengths(case)
    need = [-(-max(m, 1) // page) for m in S]
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=_gen(seed, 2), device="cuda").int()
    table = torch.full((B, max(need)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b in range(B):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    s["table"] = table
    s["lens"] = torch.tensor(S, dtype=torch.int32, device="cuda")
    s["n_tokens"], s["max_new"], s["max_len"] = sum(n), max(n), max(max(S), 1)
    cu = [0]
    for m in n:
        cu.append(cu[-1] + m)
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    gain = torch.ones(H_kv, D, device="cuda")
    for h in range(H_kv):
        at = torch.randperm(D, generator=_gen(seed, 10 + h), device="cuda")
        gain[h, at[:case.get("outliers", 0)]] = 10.0
    parts = []
    for stream, f in ((3, gain), (4, None)):
        x = _randn(_gen(seed, stream), n_pages, H_kv, page // 16, 16, D)
        if f is not None:
            x *= f[None, :, None, None]
        parts += _quantize(x.half(), group)
        del x
    s["pool"] = _pack_blocks(*parts)
    del parts
    T = sum(n)
    if case["op"] == "append":
        x = _randn(_gen(seed, 5), T, (H_q + 2 * H_kv) * D).to(dt).view(T, -1, D)
        s["q"], s["k"], s["v"] = x[:, :H_q], x[:, H_q:H_q + H_kv], x[:, H_q + H_kv:]
        g = _gen(seed, 6)
        if case["norm"]:
            s["q_weight"] = (1 + 0.1 * _randn(g, D)).to(dt)
            s["k_weight"] = (1 + 0.1 * _randn(g, D)).to(dt)
        if case["axes"] > 1:
            s["positions"] = torch.randint(0, 4096, (case["axes"], T), generator=g,
                                           device="cuda")
    else:
        s["q"] = _randn(_gen(seed, 7), T, H_q, D).to(dt)
    if own:
        from bit_kv_cache_05_gb300.paged import PagedKiviCache
        s["cache"] = PagedKiviCache(n_pages, page=page, H_q=H_q, H_kv=H_kv, D=D, group=group,
                                    pool=s["pool"])
        if case["op"] == "append":
            from bit_kv_cache_05_gb300.rope import Rope
            s["rope"] = Rope(inv, axis=axis)
    return s


# ---- one pass ----------------------------------------------------------------

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    case = s["case"]
    op = case["op"]
    if op == "norm_rope":
        from bit_kv_cache_05_gb300.rope import norm_rope
        q, k = norm_rope(s["q"], s["k"], s["positions"], s["rope"], q_weight=s.get("q_weight"),
                         k_weight=s.get("k_weight"), eps=EPS)
        return dict(q=q, k=k)
    cache = s["cache"]
    if op == "append":
        # one new token each is the call without offsets
        cu = None if s["max_new"] == 1 else s["cu"]
        q = cache.append(s["k"], s["v"], s["table"], s["lens"], cu, q=s["q"], rope=s["rope"],
                         positions=s.get("positions"), q_weight=s.get("q_weight"),
                         k_weight=s.get("k_weight"), eps=EPS)
        k, v = cache.dequantize(s["table"], s["lens"], cu, n_tokens=s["n_tokens"])
        return dict(q=q, k=k, v=v)
    if op == "decode":
        return dict(out=cache.attend(s["q"], s["table"], s["lens"]))
    return dict(out=cache.attend(s["q"], s["table"], s["lens"], s["cu"], max_new=s["max_new"]))


def _norm_rotate(s, x, weight, positions, interleaved):
    """fp32 rows [T][H][D]: norm over each head, then the rotation."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
    inv, half = s["inv_freq"], s["inv_freq"].numel()
    # far positions need their angles in 64 bits
    angle = positions.double()[s["axis"]].T * inv                # [T][half]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    y, rest = x[..., :2 * half], x[..., 2 * half:]
    if interleaved:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = y[..., :half], y[..., half:]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, rest), -1)


def _token_places(s):
    """(sequence, position in the cache) of each new token."""
    n = s["cu"][1:] - s["cu"][:-1]
    T = s["n_tokens"]
    seq = torch.repeat_interleave(torch.arange(n.numel(), device="cuda"), n, output_size=T)
    pos = torch.arange(T, device="cuda") - s["cu"][seq] + (s["lens"] - n)[seq]
    return seq, pos.long()


def _run_plain(s):
    case = s["case"]
    op, D = case["op"], case["D"]
    if op == "norm_rope":
        dt = s["q"].dtype
        return {k: _norm_rotate(s, s[k], s.get(k + "_weight"), s["positions"],
                                case["interleaved"]).to(dt) for k in ("q", "k")}
    group, page, pool, table = case["group"], case["page"], s["pool"], s["table"]
    H_kv, dt = case["H_kv"], s["q"].dtype
    if op == "append":
        seq, pos = _token_places(s)
        positions = s.get("positions")
        if positions is None:
            positions = pos[None].expand(case["axes"], -1)
        q = _norm_rotate(s, s["q"], s.get("q_weight"), positions, False).to(dt)
        k = _norm_rotate(s, s["k"], s.get("k_weight"), positions, False).half()
        v = s["v"].half()
        # the blocks that the tokens fall into are unpacked to codes, changed
        # at the tokens' places and packed again: all as indexed bytes
        at = table[seq, pos // page].long()
        blk, tl = pos % page // 16, pos % 16
        bits = torch.arange(D, device="cuda")
        h = torch.arange(H_kv, device="cuda")[None, :, None]
        ng = D // group
        base = (at[:, None, None] * H_kv + h) * (page // 16) + blk[:, None, None]
        base = base * pool.shape[-1]
        flat = pool.view(-1)
        half = torch.arange(ng, device="cuda")
        tl3 = tl[:, None, None]
        for x, o, kind in ((k, 0, 0), (v, 8 * D + 64 * ng, 1)):
            c, sc, z = _quantize(x, group)
            b2 = torch.arange(D // 2, device="cuda") * 2          # even channels of a byte
            if kind == 0:
                byte = tl3 * (D // 2) + 4 * ((b2 % 32 // 8) * (D // 32) + b2 // 32) + b2 % 8 // 2
            else:
                word = ((8 * (tl3 // 8) + b2 % 32 // 4) * 4 + tl3 % 8 // 2) * (D // 32) + b2 // 32
                byte = 4 * word + 2 * (tl3 % 2) + b2 % 4 // 2
            flat[base + o + byte] = c[..., 0::2] | (c[..., 1::2] << 4)
            at16 = (base + o + 8 * D) // 2 + ((tl3 // 2) * ng + half) * 4 + tl3 % 2
            flat.view(torch.float16)[at16] = sc
            flat.view(torch.float16)[at16 + 2] = z
        kh, vh = _unpack_blocks(pool[at[:, None], h[0, :, 0], blk[:, None]], D, group)
        pick = tl[:, None, None, None].expand(-1, H_kv, 1, D)
        return dict(q=q, k=kh.gather(2, pick)[:, :, 0].half(),
                    v=vh.gather(2, pick)[:, :, 0].half())

    pages = table[:, :-(-s["max_len"] // page)].clamp(min=0).long()
    kh, vh = _unpack_blocks(pool[pages].transpose(1, 2).flatten(2, 3), D, group)
    kh, vh = kh.flatten(2, 3), vh.flatten(2, 3)                   # [B][H_kv][S][D]
    B, GQ = kh.shape[0], case["H_q"] // H_kv
    t = torch.arange(kh.shape[2], device="cuda")
    if op == "decode":
        q = s["q"].float().view(B, H_kv, GQ, D)
        last = (s["lens"] - 1)[:, None].expand(-1, GQ)            # newest token a row sees
    else:
        n = s["max_new"]
        seq, pos = _token_places(s)
        i = torch.arange(s["n_tokens"], device="cuda") - s["cu"][seq]
        q = torch.zeros(B, n, H_kv, GQ, D, device="cuda")
        q[seq, i] = s["q"].float().unflatten(1, (H_kv, GQ))
        q = q.permute(0, 2, 1, 3, 4).flatten(2, 3)                # [B][H_kv][n GQ][D]
        last = torch.full((B, n), -1, device="cuda")
        last[seq, i] = pos
        last = last.repeat_interleave(GQ, 1)
    score = torch.matmul(q, kh.transpose(-1, -2)) / math.sqrt(D)
    seen = t <= last[:, None, :, None]
    score = torch.where(seen, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.where(seen, torch.exp(score - torch.where(top > -math.inf, top, 0.0)), 0.0)
    den = p.sum(-1, keepdim=True)
    out = torch.matmul(p, vh) / torch.where(den > 0, den, 1.0)
    if op == "decode":
        return dict(out=out.flatten(1, 2).to(dt))
    out = out.unflatten(2, (n, GQ))[seq, :, i]                    # [T][H_kv][GQ][D]
    return dict(out=out.flatten(1, 2).to(dt))


# ---- the definition in 64 bits ---------------------------------------------

def _exact_rows(x, weight, inv, axis, positions, interleaved):
    """Norm and rotation of one tensor, pair by pair as complex numbers."""
    x = x.double()
    if weight is not None:
        x = x * weight.double() / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS)
    half = inv.numel()
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       positions.double()[axis].T * inv)[:, None]
    out = x.clone()
    re = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    im = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    z = torch.complex(x[..., re], x[..., im]) * turn
    out[..., re], out[..., im] = z.real, z.imag
    return out


def _exact_values(x, group):
    """What fp16 rows [..., D] become in 4 bits: the quantizer is defined in
    32-bit IEEE arithmetic, each step of which is a 64-bit one rounded."""
    out = torch.empty(x.shape, dtype=torch.float64, device="cuda")
    for a in range(0, x.shape[-1], group):
        g = x[..., a:a + group].double()
        lo, hi = g.min(-1, keepdim=True).values, g.max(-1, keepdim=True).values
        scale = ((hi - lo) / torch.full_like(hi, 15)).float().double()
        t = ((g - lo) / torch.where(scale > 0, scale, 1.0)).float().double()
        code = torch.round(t).clamp(0, 15) * (scale > 0)
        out[..., a:a + group] = (code * scale.half().double() + lo).float().half().double()
    return out


def _exact_cache(s, b, S):
    """Key and value rows [H_kv][S][D] of sequence b, element by element from
    the pool's bytes."""
    case, pool = s["case"], s["pool"]
    D, page, group, H_kv = case["D"], case["page"], case["group"], case["H_kv"]
    ng = D // group
    t = torch.arange(S, device="cuda")[:, None]
    c = torch.arange(D, device="cuda")
    at = s["table"][b].long()[t // page]
    tl = t % 16
    kb = tl * (D // 2) + 4 * ((c % 32) // 8 * (D // 32) + c // 32) + (c % 8) // 2
    vb = 4 * (((tl // 8 * 8 + c % 32 // 4) * 4 + tl % 8 // 2) * (D // 32) + c // 32) \
        + 2 * (tl % 2) + c % 4 // 2
    mb = ((tl // 2) * ng + c // group) * 4 + tl % 2
    flat, out = pool.view(-1), []
    flat16 = flat.view(torch.float16)
    for o, byte in ((0, kb), (8 * D + 64 * ng, vb)):
        rows = []
        for h in range(H_kv):
            base = ((at * H_kv + h) * (page // 16) + t % page // 16) * pool.shape[-1] + o
            code = flat[base + byte].to(torch.int32) >> (c % 2 * 4) & 15
            m = (base + 8 * D) // 2 + mb
            rows.append((code.double() * flat16[m].double() + flat16[m + 2].double())
                        .float().half().double())
        out.append(torch.stack(rows))
    return out


def exact(case, seed):
    s = prepare(case, seed)
    D, H_q, H_kv = case["D"], case["H_q"], case["H_kv"]
    if case["op"] == "norm_rope":
        return {k: _exact_rows(s[k], s.get(k + "_weight"), s["inv_freq"], s["axis"],
                               s["positions"], case["interleaved"]) for k in ("q", "k")}
    n, S = _lengths(case)
    GQ = H_q // H_kv
    if case["op"] == "append":
        pos = torch.cat([torch.arange(S[b] - n[b], S[b], device="cuda") for b in range(len(n))])
        positions = s["positions"] if "positions" in s else pos[None].repeat(case["axes"], 1)
        rows = [_exact_rows(s[k], s.get(k + "_weight"), s["inv_freq"], s["axis"], positions,
                            False) for k in ("q", "k")]
        return dict(q=rows[0], k=_exact_values(rows[1].half(), case["group"]),
                    v=_exact_values(s["v"].half(), case["group"]))
    outs, at = [], 0
    for b in range(len(n)):
        q = s["q"][at:at + n[b]].double()
        at += n[b]
        o = torch.zeros(n[b], H_q, D, dtype=torch.float64, device="cuda")
        if S[b] > 0:
            k, v = _exact_cache(s, b, S[b])
            hidden = torch.arange(S[b], device="cuda") > \
                torch.arange(S[b] - n[b], S[b], device="cuda")[:, None]
            for h in range(H_q):
                a = (q[:, h] @ k[h // GQ].T) * D ** -0.5
                o[:, h] = torch.softmax(a.masked_fill(hidden, -math.inf), -1) @ v[h // GQ]
        outs.append(o)
    return dict(out=torch.cat(outs))
