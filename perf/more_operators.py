"""Measured cases of the operators that speculative decoding over trees of drafts
and eviction need beside the paged 4-bit cache.

Five kinds of pass, each as a serving program makes it:

  tree     attention of a tree of drafted tokens over the paged cache: each node
           sees what was there before and the nodes that its bit mask names
  verify   which drafted tokens stay, and the token behind them, from the
           target's and the draft's probabilities and given random numbers
  keep     the tokens of the accepted path move together in the cache; the rows
           of the new tokens' places are read back
  weigh    attention of single tokens that also adds each stored token's softmax
           weight to an accumulator per kv head
  evict    per kv head the first, the newest and the heaviest tokens stay: their
           codes and accumulated weights move into the places of the others; the
           rows that stay are read back

`own` chooses between the plain form (elementary torch operations in 32 bits, sums
of probabilities in whole numbers of 2^-44) and the framework's kernels.  Both
work on the same state.

The pool is uint8 [n_pages][H_kv][page / 16][block]; a block holds 16 tokens of
one kv head: key codes, key (scale, zero), value codes, value (scale, zero), in
the orders that `_places` writes down.  A value stands for code * scale + zero,
rounded to fp16.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
UNIT = 2.0 ** 44           # sums of probabilities are whole numbers of 1 / UNIT


# ---- cases ---------------------------------------------------------------

def listed():
    return [
        # one conversation, a small tree behind a short context: latency counts
        dict(name="tree B1 x8 S700", op="tree", B=1, n_lo=8, n_hi=8, s_lo=700, s_hi=700, H_q=16,
             H_kv=8, D=128, group=32, page=64, dtype="fp16"),
        # a serving batch with trees of 16 nodes, grouped heads
        dict(name="tree B16 x16 S8192", op="tree", B=16, n_lo=16, n_hi=16, s_lo=4096, s_hi=8192,
             H_q=32, H_kv=8, D=128, group=32, page=16, dtype="bf16"),
        # large ragged trees behind long contexts
        dict(name="tree B2 x61 S65536", op="tree", B=2, n_lo=40, n_hi=61, s_lo=32768, s_hi=65536,
             H_q=32, H_kv=4, D=128, group=64, page=64, dtype="bf16"),
        # one chain of four drafts, a small vocabulary: latency counts
        dict(name="verify chain B1 V32000", op="verify", B=1, n_lo=5, n_hi=5, V=32000, tree=False,
             draft=True, dtype="fp32"),
        # chains of a serving batch, a large vocabulary
        dict(name="verify chain B64 V131072", op="verify", B=64, n_lo=5, n_hi=5, V=131072,
             tree=False, draft=True, dtype="fp32"),
        # trees with several candidates a node, an odd vocabulary: rows on odd addresses
        dict(name="verify tree B16 x32 V100003", op="verify", B=16, n_lo=24, n_hi=32, V=100003,
             tree=True, draft=True, dtype="fp32"),
        # the accepted path of each of 64 sequences' trees moves together
        dict(name="keep B64 x16", op="keep", B=64, n_lo=16, n_hi=16, s_lo=16, s_hi=2048, H_q=32,
             H_kv=8, D=128, group=32, page=16),
        # large trees, every head with its own keys
        dict(name="keep B128 x64 H32", op="keep", B=128, n_lo=33, n_hi=64, s_lo=64, s_hi=1024,
             H_q=32, H_kv=32, D=128, group=64, page=64),
        # a decode step of a serving batch that accumulates weights
        dict(name="weigh B16 S8192", op="weigh", B=16, s_lo=8192, s_hi=8192, H_q=32, H_kv=8,
             D=128, group=32, page=16, dtype="bf16"),
        # long sequences of unequal lengths, every head with its own keys
        dict(name="weigh ragged long", op="weigh", B=3, s_lo=16384, s_hi=65536, H_q=16, H_kv=16,
             D=128, group=64, page=128, dtype="fp16"),
        # a full cache, one token over its budget in each sequence
        dict(name="evict step B32 to 512", op="evict", B=32, s_lo=513, s_hi=513, budget=512,
             recent=64, first=4, H_q=32, H_kv=8, D=128, group=32, page=16),
        # after long prompts: a fraction of the tokens stays
        dict(name="evict prompts B4 to 4096", op="evict", B=4, s_lo=16384, s_hi=65536, budget=4096,
             recent=512, first=4, H_q=32, H_kv=8, D=128, group=64, page=64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tree", "verify", "keep", "weigh", "evict"])
    if op == "verify":
        V = _log(rng, 100, 131072)
        n = _log(rng, 1, 64)
        B = _log(rng, 1, max(1, min(128, 60000000 // (V * n))))
        return dict(op=op, B=B, n_lo=max(1, n // 2), n_hi=n, V=V, tree=rng.choice([True, False]),
                    draft=rng.choice([True, True, False]),
                    dtype=rng.choice(["fp32", "fp32", "bf16", "fp16"]))
    H_kv = rng.choice([1, 2, 4, 8])
    D = rng.choice([64, 128])
    c = dict(op=op, H_q=H_kv * rng.choice([1, 2, 3, 4, 5, 8]), H_kv=H_kv, D=D,
             group=rng.choice([32, 64, 128] if D == 128 else [32, 64]),
             page=rng.choice([16, 32, 64, 128]))
    if op in ("tree", "keep"):
        n = _log(rng, 1, 64)
        S = _log(rng, n, 16384 if op == "tree" else 2048)
        B = _log(rng, 1, max(1, min(64, 32768 // S)))
        c.update(B=B, n_lo=max(1, n // 2), n_hi=n, s_lo=max(n // 2, S // 2), s_hi=S)
    elif op == "weigh":
        S = _log(rng, 1, 65536)
        c.update(B=_log(rng, 1, max(1, min(128, 131072 // S))), s_lo=S // 2, s_hi=S)
    else:
        S = _log(rng, 1, 65536)
        budget = _log(rng, 1, max(1, min(S, 4096)))
        recent = rng.randint(0, budget)
        c.update(B=_log(rng, 1, max(1, min(64, 65536 // S))), s_lo=S // 2, s_hi=S, budget=budget,
                 recent=recent, first=rng.randint(0, min(4, budget - recent)))
    if op in ("tree", "weigh"):
        c["dtype"] = rng.choice(["bf16", "fp16"])
    return c


# Lengths, trees and paths are part of a case, so drawn from its own values.

def _rng(case):
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _lengths(case):
    """New tokens and lengths (new tokens included) of each sequence."""
    rng = _rng(case)
    n = [rng.randint(case["n_lo"], case["n_hi"]) if "n_lo" in case else 1
         for _ in range(case["B"])]
    S = [max(m if "n_lo" in case else 0, rng.randint(case["s_lo"], case["s_hi"])) for m in n] \
        if "s_lo" in case else n
    return n, S


def _parents(case):
    """Parent of each node within its sequence, node 0 the root (-1).  Trees
    widen near the root, as the best candidates of each level are followed."""
    rng, n = _rng(case), _lengths(case)[0]
    chain = case["op"] == "verify" and not case["tree"]
    out = []
    for m in n:
        p = [-1]
        for i in range(1, m):
            p.append(i - 1 if chain else min(int(rng.random() ** 1.5 * i), i - 1))
            if not chain and i > 1:
                p[i] = max(p[i], p[i - 1])          # nodes in the order of their parents
        out.append(p)
    return out


def _path(parents, rng):
    """An accepted path: from the root down, sometimes stopping early."""
    path, at = [0], 0
    while True:
        kids = [i for i, p in enumerate(parents) if p == at and i > 0]
        if not kids or rng.random() < 0.15:
            return path
        at = rng.choice(kids)
        path.append(at)


# ---- work ----------------------------------------------------------------

def work(case):
    n, S = _lengths(case)
    B = case["B"]
    if case["op"] == "verify":
        # a walk ends with the rows of one node: the target's, and the draft's
        # where a child was rejected
        e = 4 if case["dtype"] == "fp32" else 2
        rows = 2 if case["draft"] and case["n_hi"] > 1 else 1
        return dict(bytes=B * rows * case["V"] * e + sum(n) * 24, flops=4 * B * rows * case["V"])
    D, H_q, H_kv = case["D"], case["H_q"], case["H_kv"]
    tok = H_kv * (D + 8 * (D // case["group"]))          # bytes of a stored token
    if case["op"] == "tree":
        pairs = sum(m * (s - m) + m * (m + 1) // 2 for m, s in zip(n, S))
        return dict(bytes=sum(S) * tok + 4 * sum(n) * H_q * D, flops=4 * pairs * H_q * D)
    if case["op"] == "weigh":
        return dict(bytes=sum(S) * (tok + 8 * H_kv) + 4 * B * H_q * D,
                    flops=4 * sum(S) * H_q * D)
    if case["op"] == "keep":
        # the read-back: a token's codes in, two rows of 16 bits out
        moved = sum(len(_path(p, r)) - 1 for p, r in zip(_parents(case), _path_rngs(case)))
        return dict(bytes=2 * moved * tok + sum(n) * (tok + 4 * H_kv * D), flops=2 * sum(n) * H_kv * D)
    stay = [min(s, case["budget"]) for s in S]
    moved = sum(min(s - k, k) for s, k in zip(S, stay)) / 2
    return dict(bytes=sum(S) * 4 * H_kv + sum(stay) * 4 * H_kv + int(2 * moved * tok) +
                sum(stay) * (tok + 4 * H_kv * D), flops=2 * sum(stay) * H_kv * D)


def _path_rngs(case):
    return [random.Random("%d %d" % (b, case["s_hi"])) for b in range(case["B"])]


# ---- the pool ----------------------------------------------------------------

def _places(D, group):
    """16-bit places of a token's parts in its block: [16 tokens][what a token
    holds], the same order of parts for each token.  Key codes: 16 rows of D / 8
    words, word (D / 32) t + i with channels 32 i + 8 t ... + 7.  Value codes:
    word ((8 h + g) 4 + t) (D / 32) + i with channels 32 i + 4 g ... + 3 of token
    8 h + 2 t in its low half, of the next token in its high half.  (scale,
    zero): fp16, per token pair and group s, s', z, z'."""
    ng, I = D // group, D // 32
    rows = []
    for t in range(16):
        key = [t * (D // 4) + c for c in range(D // 4)]
        km = [4 * D + ((t // 2) * ng + j) * 4 + 2 * m + t % 2 for m in (0, 1) for j in range(ng)]
        o = 4 * D + 32 * ng
        val = [o + 2 * (((8 * (t // 8) + g) * 4 + t % 8 // 2) * I + i) + t % 2
               for g in range(8) for i in range(I)]
        vm = [o + 4 * D + ((t // 2) * ng + j) * 4 + 2 * m + t % 2
              for m in (0, 1) for j in range(ng)]
        rows.append(key + km + val + vm)
    return torch.tensor(rows, device="cuda")


def _channels(D):
    """Channel of each nibble of a token's key codes and value codes, in the
    order of `_places`, the lowest nibble of a place first."""
    key = [32 * i + 8 * t + r for t in range(4) for i in range(D // 32) for r in range(8)]
    val = [32 * i + 4 * g + r for g in range(8) for i in range(D // 32) for r in range(4)]
    return torch.tensor(key, device="cuda"), torch.tensor(val, device="cuda")


def _quantize(x, group):
    """codes, scale, zero of fp16 rows over groups of channels."""
    g = x.float().unflatten(-1, (-1, group))
    lo, hi = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    scale = (hi - lo) / torch.full_like(hi, 15.0)
    code = torch.where(scale > 0, torch.round((g - lo) / scale), torch.zeros_like(g))
    return code.clamp(0, 15).to(torch.int16).flatten(-2), scale[..., 0].half(), lo[..., 0].half()


def _store(x, group, channel):
    """What `_places` has of fp16 rows [..., D]: codes of four channels in 16
    bits, then scales, then zeros, all as int16."""
    code, s, z = _quantize(x, group)
    code = code[..., channel].unflatten(-1, (-1, 4))
    word = code[..., 0] | code[..., 1] << 4 | code[..., 2] << 8 | code[..., 3] << 12
    return torch.cat((word, s.view(torch.int16), z.view(torch.int16)), -1)


def _rows_of(part, D, group, inverse):
    """The fp32 values that int16 parts [..., D / 4 + 2 D / group] stand for."""
    nw, ng = D // 4, D // group
    w = part[..., :nw].to(torch.int32)
    code = torch.stack((w, w >> 4, w >> 8, w >> 12), -1).flatten(-2) & 15
    code = code[..., inverse].float().unflatten(-1, (ng, group))
    s = part[..., nw:nw + ng].contiguous().view(torch.float16).float()[..., None]
    z = part[..., nw + ng:].contiguous().view(torch.float16).float()[..., None]
    # the product of a 4-bit code and an fp16 scale is exact in 32 bits
    return (code * s + z).half().float().flatten(-2)


# ---- inputs ----------------------------------------------------------------

def _gen(seed, stream):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000 + stream)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _offsets(n):
    return torch.tensor([sum(n[:b]) for b in range(len(n) + 1)], dtype=torch.int32,
                        device="cuda")


def _prepare_verify(case, seed):
    n, V, T = _lengths(case)[0], case["V"], sum(_lengths(case)[0])
    dt, par = DTYPES[case["dtype"]], _parents(case)
    g = _gen(seed, 0)
    s = dict(case=case, cu=_offsets(n), n=n)
    s["parents"] = torch.tensor([x for p in par for x in p], dtype=torch.int32, device="cuda")
    logits = 2.5 * _randn(g, T, V)
    s["target"] = torch.softmax(logits, -1).to(dt)
    # the draft is near the target: most of its tokens are good ones
    q = torch.softmax(logits + 0.8 * _randn(g, T, V), -1).to(dt)
    del logits
    start = torch.repeat_interleave(s["cu"][:-1].long(), torch.tensor(n, device="cuda"))
    up = (start + s["parents"].clamp(min=0)).long()
    if case["draft"]:
        # a node's children are drawn from its row, one by one
        s["draft"] = q
        pick = [torch.multinomial(q[a:a + 256].float(), 64, replacement=True, generator=g)
                for a in range(0, T, 256)]
    else:
        # or are its best candidates
        pick = [torch.topk(q[a:a + 256].float(), min(64, V), -1).indices
                for a in range(0, T, 256)]
    pick = torch.cat(pick)
    nth = [sum(1 for j in range(1, i) if p[j] == p[i]) if i else 0
           for p in par for i in range(len(p))]
    nth = torch.tensor(nth, device="cuda") % pick.shape[1]
    s["tokens"] = pick[up, nth]
    s["uniforms"] = torch.rand(T, generator=g, device="cuda")
    return s


def prepare(case, seed):
    if case["op"] == "verify":
        return _prepare_verify(case, seed)
    D, H_q, H_kv, B, page, group = (case[k] for k in ("D", "H_q", "H_kv", "B", "page", "group"))
    n, S = _lengths(case)
    s = dict(case=case)
    need = [-(-max(m, 1) // page) for m in S]
    n_pages, width = sum(need) + 3, max(need)
    order = torch.randperm(n_pages, generator=_gen(seed, 2), device="cuda").int()
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b in range(B):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    s["table"] = table
    s["lens"] = torch.tensor(S, dtype=torch.int32, device="cuda")
    s["cu"], s["n_tokens"], s["max_new"], s["max_len"] = _offsets(n), sum(n), max(n), max(S)
    s["places"], channels = _places(D, group), _channels(D)
    s["inverse"] = [torch.argsort(c) for c in channels]
    parts = [_store(_randn(_gen(seed, 3 + k), n_pages, H_kv, page // 16, 16, D).half(), group,
                    channels[k]) for k in (0, 1)]
    pool = torch.empty(n_pages, H_kv, page // 16, 16 * D + 128 * (D // group), dtype=torch.uint8,
                       device="cuda")
    pool.view(torch.int16)[..., s["places"]] = torch.cat(parts, -1)
    s["pool"] = pool
    del parts
    if case["op"] in ("tree", "weigh"):
        s["q"] = _randn(_gen(seed, 5), sum(n), H_q, D).to(DTYPES[case["dtype"]])
    if case["op"] == "tree":
        masks = []
        for p in _parents(case):
            m = [1]
            for i in range(1, len(p)):
                m.append(m[p[i]] | 1 << i)
            masks += [x - (1 << 64) if x >> 63 else x for x in m]
        s["tree"] = torch.tensor(masks, dtype=torch.int64, device="cuda")
    if case["op"] == "keep":
        # each state its own path
        path, counts = [], []
        for p, b in zip(_parents(case), range(B)):
            one = _path(p, random.Random("%d %d" % (b, case["s_hi"])))
            path += one + [-1] * (len(p) - len(one))
            counts.append(len(one))
        s["path"] = torch.tensor(path, dtype=torch.int32, device="cuda")
        s["counts"] = torch.tensor(counts, dtype=torch.int32, device="cuda")
    if case["op"] in ("weigh", "evict"):
        # a few tokens have most of the weight, some none at all
        g = _gen(seed, 6)
        w = torch.exp(2 * _randn(g, B, H_kv, width * page))
        w *= torch.rand(w.shape, generator=g, device="cuda") > 0.05
        s["weights"] = w * (torch.arange(width * page, device="cuda") < s["lens"][:, None, None])
    if case["op"] == "evict":
        stay = [min(x, case["budget"]) for x in S]
        s["cu_stay"], s["n_stay"] = _offsets(stay), sum(stay)
    if own:
        from bit_kv_cache_05_gb300.paged import PagedKiviCache
        s["cache"] = PagedKiviCache(n_pages, page=page, H_q=H_q, H_kv=H_kv, D=D, group=group,
                                    pool=s["pool"])
    return s


# ---- one pass ----------------------------------------------------------------

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    op = s["case"]["op"]
    if op == "verify":
        from bit_kv_cache_05_gb300.drafts import verify_drafts
        path, counts, after = verify_drafts(s["target"], s["tokens"], s["uniforms"], s["cu"],
                                            parents=s["parents"], draft=s.get("draft"))
        return dict(path=path, counts=counts, after=after)
    cache = s["cache"]
    if op == "tree":
        return dict(out=cache.attend(s["q"], s["table"], s["lens"], s["cu"],
                                     max_new=s["max_new"], tree=s["tree"]))
    if op == "weigh":
        out = cache.attend(s["q"], s["table"], s["lens"], weights=s["weights"])
        return dict(out=out, weights=s["weights"])
    if op == "keep":
        lens = cache.keep(s["table"], s["lens"], s["cu"], s["path"], s["counts"])
        k, v = cache.dequantize(s["table"], s["lens"], s["cu"], n_tokens=s["n_tokens"])
        return dict(lens=lens, k=k, v=v)
    lens, weights = cache.evict(s["table"], s["lens"], s["weights"], s["case"]["budget"],
                                recent=s["case"]["recent"], first=s["case"]["first"])
    k, v = cache.dequantize(s["table"], lens, s["cu_stay"], n_tokens=s["n_stay"])
    return dict(lens=lens, weights=weights, k=k, v=v)


def _token_rows(s):
    """(sequence, place in the cache) of each new token."""
    n = s["cu"][1:] - s["cu"][:-1]
    T = s["n_tokens"]
    seq = torch.repeat_interleave(torch.arange(n.numel(), device="cuda"), n, output_size=T)
    return seq, (torch.arange(T, device="cuda") - s["cu"][seq] + (s["lens"] - n)[seq]).long()


def _halves(s, seq, pos):
    """Places in the pool's 16-bit view of all parts of tokens `pos` of sequences
    `seq` (one shape), for each kv head: [..., H_kv or as given, parts]."""
    case, pool = s["case"], s["pool"]
    blocks, size = case["page"] // 16, pool.shape[-1] // 2
    page = s["table"][seq, (pos // case["page"])].clamp(min=0).long()
    head = torch.arange(case["H_kv"], device="cuda")
    if pos.dim() == 1:                                   # every head the same token
        page, pos = page[:, None], pos[:, None]
    else:
        head = head[:, None]                             # [B][H_kv][tokens]
    block = (page * case["H_kv"] + head) * blocks + pos % case["page"] // 16
    return block[..., None] * size + s["places"][pos % 16]


def _read_back(s, seq, pos):
    """fp16 key and value rows [tokens][H_kv][D] as the cache stands for them."""
    D, group = s["case"]["D"], s["case"]["group"]
    part = s["pool"].view(torch.int16).view(-1)[_halves(s, seq, pos)]
    half = part.shape[-1] // 2
    return (_rows_of(part[..., :half], D, group, s["inverse"][0]).half(),
            _rows_of(part[..., half:], D, group, s["inverse"][1]).half())


def _whole(s):
    """fp32 key and value rows [B][H_kv][S][D] of whole sequences."""
    case = s["case"]
    pages = s["table"][:, :-(-s["max_len"] // case["page"])].clamp(min=0).long()
    part = s["pool"].view(torch.int16)[pages].transpose(1, 2).flatten(2, 3)[..., s["places"]]
    part = part.flatten(2, 3)
    half = part.shape[-1] // 2
    return (_rows_of(part[..., :half], case["D"], case["group"], s["inverse"][0]),
            _rows_of(part[..., half:], case["D"], case["group"], s["inverse"][1]))


def _softmax_rows(q, kh, seen):
    score = torch.matmul(q, kh.transpose(-1, -2)) / math.sqrt(q.shape[-1])
    score = torch.where(seen, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.where(seen, torch.exp(score - torch.where(top > -math.inf, top, 0.0)), 0.0)
    den = p.sum(-1, keepdim=True)
    return p / torch.where(den > 0, den, 1.0)


def _run_plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "verify":
        return _verify_plain(s)
    H_kv, GQ = case["H_kv"], case["H_q"] // case["H_kv"]
    if op == "tree":
        kh, vh = _whole(s)
        n, T = s["max_new"], s["n_tokens"]
        seq, pos = _token_rows(s)
        i = torch.arange(T, device="cuda") - s["cu"][seq]
        q = torch.zeros(len(kh), n, H_kv, GQ, case["D"], device="cuda")
        q[seq, i] = s["q"].float().unflatten(1, (H_kv, GQ))
        q = q.permute(0, 2, 1, 3, 4).flatten(2, 3)               # [B][H_kv][n GQ][D]
        mask = torch.zeros(len(kh), n, dtype=torch.int64, device="cuda")
        mask[seq, i] = s["tree"]
        t = torch.arange(kh.shape[2], device="cuda")
        j = t - (s["lens"] - (s["cu"][1:] - s["cu"][:-1]))[:, None]      # [B][S]
        bit = (mask[:, :, None] >> j.clamp(0, 63)[:, None]) & 1
        new = (j >= 0) & (t < s["lens"][:, None])
        seen = (j < 0)[:, None] | new[:, None] & (bit > 0)
        p = _softmax_rows(q, kh, seen.repeat_interleave(GQ, 1)[:, None])
        out = torch.matmul(p, vh).unflatten(2, (n, GQ))[seq, :, i]
        return dict(out=out.flatten(1, 2).to(s["q"].dtype))
    if op == "weigh":
        kh, vh = _whole(s)
        q = s["q"].float().unflatten(1, (H_kv, GQ))
        seen = torch.arange(kh.shape[2], device="cuda") < s["lens"][:, None, None, None]
        p = _softmax_rows(q, kh, seen)
        s["weights"][..., :kh.shape[2]] += p.sum(2)
        return dict(out=torch.matmul(p, vh).flatten(1, 2).to(s["q"].dtype), weights=s["weights"])
    flat = s["pool"].view(torch.int16).view(-1)
    if op == "keep":
        seq, pos = _token_rows(s)
        j = torch.arange(s["n_tokens"], device="cuda") - s["cu"][seq]
        stays = j < s["counts"][seq]
        source = torch.where(stays, s["path"], j)                # the others stay where they are
        moved = flat[_halves(s, seq, pos - j + source)]
        flat[_halves(s, seq, pos)] = moved
        lens = s["lens"] - (s["cu"][1:] - s["cu"][:-1]) + s["counts"]
        k, v = _read_back(s, seq, pos)
        return dict(lens=lens, k=k, v=v)
    return _evict_plain(s, flat)


def _evict_plain(s, flat):
    case = s["case"]
    w, lens = s["weights"], s["lens"].long()[:, None, None]
    first, recent, budget = case["first"], case["recent"], case["budget"]
    K = budget - recent
    t = torch.arange(w.shape[-1], device="cuda")
    full = lens > budget
    candidate = (t >= first) & (t < lens - recent)
    rank = torch.sort(torch.where(candidate, w, -math.inf), dim=-1, descending=True, stable=True)[1]
    rank = torch.empty_like(rank).scatter_(-1, rank, t.expand_as(rank))
    stays = candidate & (rank < K - first) | (t < first)
    hole = ~stays & (t < K)
    source = stays & (t >= K)
    order = torch.sort((~source).to(torch.uint8), dim=-1, stable=True)[1]    # sources first, in order
    nth = (hole.cumsum(-1) - 1).clamp(min=0)
    # the token that a place gets
    take = torch.where(hole, order.gather(-1, nth), t)
    take = torch.where(t < K, take, lens - budget + t)
    take = torch.where(full, take, t)[..., :budget].contiguous()
    lens_out = s["lens"].clamp(max=budget)
    here = t[:budget].expand_as(take)
    there = here < lens_out[:, None, None]
    seq = torch.arange(len(w), device="cuda")[:, None, None].expand_as(take)
    take, here = torch.where(there, take, 0), torch.where(there, here, 0)
    moved = flat[_halves(s, seq, take)]
    flat[_halves(s, seq, here)[there]] = moved[there]
    weights = torch.zeros_like(w)
    weights[..., :budget] = torch.where(there, w.gather(-1, take), 0.0)
    seq = torch.repeat_interleave(torch.arange(len(w), device="cuda"), lens_out.long(),
                                  output_size=s["n_stay"])
    k, v = _read_back(s, seq, torch.arange(s["n_stay"], device="cuda") - s["cu_stay"][seq])
    return dict(lens=lens_out, weights=weights, k=k, v=v)


def _verify_plain(s):
    """All sequences side by side, node by node: a node's children have higher
    numbers than it has."""
    cu, target, draft, u = s["cu"].long(), s["target"], s.get("draft"), s["uniforms"].double()
    B, V, T = s["case"]["B"], s["case"]["V"], len(u)
    tokens, parents = s["tokens"], s["parents"].long()
    n = cu[1:] - cu[:-1]
    every = torch.arange(B, device="cuda")
    at = torch.zeros(B, dtype=torch.int64, device="cuda")         # the node each walk is at
    c = torch.zeros(B, dtype=torch.float64, device="cuda")
    mass = torch.ones(B, dtype=torch.float64, device="cuda")
    gone = torch.zeros(B, V, dtype=torch.bool, device="cuda")     # without a draft: rejected tokens
    path = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    counts = torch.ones(B, dtype=torch.int64, device="cuda")
    path[cu[:-1]] = 0

    def residual():
        """Whole numbers of 1 / UNIT of what is left of the rows at `at`."""
        p = target[cu[:-1] + at].double()
        if draft is not None:
            # rows of nodes without a rejected child are not read: they may hold anything
            q = torch.where(c[:, None] > 0, draft[cu[:-1] + at].double(), 0.0)
            p = (p - c[:, None] * q).float().double()
        p = torch.where((p > 0) & ~gone, p, 0.0).clamp(max=1.0)
        return torch.round(p * UNIT).long()

    for i in range(1, int(s["case"]["n_hi"])):
        row = (cu[:-1] + i).clamp(max=T - 1)
        child = (i < n) & (parents[row] == at)
        x = tokens[row]
        p = target[cu[:-1] + at, x].double()
        if draft is not None:
            q = draft[cu[:-1] + at, x].double()
            w = (p - c * q).float().double()
            good = child & (mass > 0) & (u[row] * q * mass < w)
        else:
            w = torch.where(gone[every, x], 0.0, p)
            good = child & (mass > 0) & (u[row] * mass < w)
        bad = child & ~good
        if draft is not None:
            c = torch.where(good, 0.0, torch.where(bad, (c + mass).float().double(), c))
            left = residual().sum(-1).double() / UNIT
            mass = torch.where(good, 1.0, torch.where(bad, left, mass))
        else:
            less = torch.round(w.clamp(max=1.0) * UNIT) / UNIT
            mass = torch.where(good, 1.0, torch.where(bad, (mass - less).clamp(min=0), mass))
            gone &= ~good[:, None]
            gone[every, x] |= bad
        path[torch.where(good, cu[:-1] + counts, cu[:-1])] = torch.where(good, i, 0).int()
        counts += good
        at = torch.where(good, i, at)
    whole = residual()
    # nothing left after rounding: from the target's row itself
    empty = whole.sum(-1) == 0
    c, gone = torch.where(empty, 0.0, c), gone & ~empty[:, None]
    whole = torch.where(empty[:, None], residual(), whole)
    total = whole.sum(-1)
    U = torch.floor(u[cu[:-1]] * 2.0 ** 31).long()
    # floor(total U / 2^31) in 63 bits
    r = (total >> 31) * U + ((total & (2 ** 31 - 1)) * U >> 31)
    after = (whole.cumsum(-1) <= r[:, None]).sum(-1)
    after = torch.where(total > 0, after, -1)
    return dict(path=path, counts=counts.int(), after=after)


# ---- the definition in 64 bits ---------------------------------------------

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


def _exact_verify(case, s):
    """One walk after the other, each residual taken from the one before it."""
    paths, counts, after = [], [], []
    start = 0
    for b, m in enumerate(s["n"]):
        par = s["parents"][start:start + m].tolist()
        tok = s["tokens"][start:start + m].tolist()
        u = s["uniforms"][start:start + m].double().tolist()
        cur, path = 0, [0]
        p = s["target"][start].double()
        for i in range(1, m):
            if par[i] != cur:
                continue
            x = tok[i]
            if "draft" in s:
                q = s["draft"][start + cur].double()
                if u[i] * float(q[x]) < float(p[x]):
                    cur, p = i, s["target"][start + i].double()
                    path.append(i)
                    continue
                p = (p - q).clamp(min=0)
            else:
                if u[i] < float(p[x]):
                    cur, p = i, s["target"][start + i].double()
                    path.append(i)
                    continue
                p = p.clone()
                p[x] = 0
                p = p / (p.sum() if float(p.sum()) > 0 else 1.0)
                continue
            total = float(p.sum())
            p = p / total if total > 0 else s["target"][start + cur].double()
        at = torch.cumsum(p, 0)
        after.append(int((at <= u[0] * at[-1]).sum().clamp(max=case["V"] - 1)))
        paths += path + [-1] * (m - len(path))
        counts.append(len(path))
        start += m
    i32 = dict(dtype=torch.int32, device="cuda")
    return dict(path=torch.tensor(paths, **i32), counts=torch.tensor(counts, **i32),
                after=torch.tensor(after, device="cuda"))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "verify":
        return _exact_verify(case, s)
    D, H_q, H_kv, B = case["D"], case["H_q"], case["H_kv"], case["B"]
    n, S = _lengths(case)
    GQ = H_q // H_kv
    if case["op"] in ("tree", "weigh"):
        outs, at = [], 0
        weights = s["weights"].double() if case["op"] == "weigh" else None
        for b in range(B):
            q = s["q"][at:at + n[b]].double()
            o = torch.zeros(n[b], H_q, D, dtype=torch.float64, device="cuda")
            if S[b] > 0:
                k, v = _exact_cache(s, b, S[b])
                hidden = torch.zeros(n[b], S[b], dtype=torch.bool, device="cuda")
                if case["op"] == "tree":
                    for i, m in enumerate(s["tree"][at:at + n[b]].tolist()):
                        row = [not m >> j & 1 for j in range(n[b])]
                        hidden[i, S[b] - n[b]:] = torch.tensor(row, device="cuda")
                for h in range(H_q):
                    a = (q[:, h] @ k[h // GQ].T) * D ** -0.5
                    p = torch.softmax(a.masked_fill(hidden, -math.inf), -1)
                    o[:, h] = p @ v[h // GQ]
                    if weights is not None:
                        weights[b, h // GQ, :S[b]] += p.sum(0)
            at += n[b]
            outs.append(o)
        outs = dict(out=torch.cat(outs))
        return outs if weights is None else dict(outs, weights=weights)
    before = [_exact_cache(s, b, S[b]) if S[b] else None for b in range(B)]
    rows = ([], [])
    if case["op"] == "keep":
        at, lens = 0, []
        for b in range(B):
            m = int(s["counts"][b])
            base = S[b] - n[b]
            source = [base + x for x in s["path"][at:at + m].tolist()] + \
                list(range(base + m, S[b]))
            lens.append(base + m)
            for o, x in zip(rows, before[b]):
                o.append(x[:, source].transpose(0, 1))
            at += n[b]
        return dict(lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                    k=torch.cat(rows[0]), v=torch.cat(rows[1]))
    budget, recent, first = case["budget"], case["recent"], case["first"]
    K = budget - recent
    weights = torch.zeros_like(s["weights"], dtype=torch.float64)
    for b in range(B):
        if S[b] == 0:
            continue
        take = torch.arange(min(S[b], budget), device="cuda").repeat(H_kv, 1)
        for h in range(H_kv if S[b] > budget else 0):
            w = s["weights"][b, h, first:S[b] - recent].double()
            best = torch.sort(w, descending=True, stable=True).indices[:K - first] + first
            stays = torch.zeros(S[b], dtype=torch.bool, device="cuda")
            stays[best] = True
            stays[:first] = True
            take[h, :K][~stays[:K]] = torch.nonzero(stays[K:]).flatten() + K
            take[h, K:] = torch.arange(S[b] - recent, S[b], device="cuda")
        weights[b, :, :take.shape[1]] = s["weights"][b].double().gather(1, take)
        for o, x in zip(rows, before[b]):
            o.append(x.gather(1, take[..., None].expand(-1, -1, D)).transpose(0, 1))
    none = [torch.zeros(0, H_kv, D, dtype=torch.float64, device="cuda")]
    return dict(lens=s["lens"].clamp(max=budget), weights=weights, k=torch.cat(rows[0] + none),
                v=torch.cat(rows[1] + none))
