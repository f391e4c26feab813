"""Performance cases of the operators around the indexer: the rotation of queries and keys, the
writers of the two 8-bit pools (the indexer's keys and the layer's K and V) and the attention over
the K/V pool, at every visible position or at the positions that the select stored.

A case is a dict of plain values.  ``prepare`` makes what a serving program holds before the call,
``run`` makes one pass (the plain form in elementary torch operations, or the package's call where
``own`` is true), ``exact`` gives the same outputs in 64 bits, ``work`` the bytes and operations
that a pass cannot do without.
"""
from __future__ import annotations

import math

import torch

own = False

E4M3_MAX = 448.0
TINY = 2.0 ** -100  # the least largest-magnitude (index rows) and the least scale (K/V blocks)


# ---- the cases ---------------------------------------------------------------------------------

def listed():
    return [
        # One decode step of 64 requests: the queries of 64 heads, 64 of 128 elements rotated.
        dict(name="rotary decode", op="rotary", tokens=64, heads=64, dim=128, rot=64, offset=64,
             interleaved=True, dtype="bf16", max_pos=131072),
        # The queries of a long prompt, the whole head rotated in halves.
        dict(name="rotary prompt", op="rotary", tokens=8192, heads=64, dim=128, rot=128, offset=0,
             interleaved=False, dtype="bf16", max_pos=131072),
        # The indexer's inputs of one decode step: 64 query heads a token, one key into the pool.
        dict(name="index decode", op="index", batch=64, next_n=1, min_len=1024, max_len=32768,
             heads=64, dim=128, block=64, rot=64, offset=0, interleaved=False, dtype="bf16"),
        # The indexer's inputs of prompts of unequal length that arrive together.
        dict(name="index prompts", op="index", batch=13, next_n=0, min_len=300, max_len=2500,
             heads=64, dim=128, block=64, rot=64, offset=0, interleaved=False, dtype="bf16"),
        # One decode step's keys and values into the cache: one token a request, part-filled blocks.
        dict(name="append decode", op="append", batch=64, next_n=1, min_len=1024, max_len=8192,
             kv_heads=8, dim=128, block=64, rot=64, offset=0, interleaved=False, dtype="bf16"),
        # Whole prompts into the cache, unequal lengths, odd starts and ends of blocks.
        dict(name="append prompts", op="append", batch=11, next_n=0, min_len=1000, max_len=5000,
             kv_heads=8, dim=128, block=64, rot=128, offset=0, interleaved=False, dtype="bf16"),
        # Attention, the two short requests of the smallest workload: latency.
        dict(name="attention tiny", op="attention", batch=2, next_n=1, min_len=300, max_len=1000,
             zeros=0, spread="uniform", heads=64, kv_heads=8, dim=128, block=64, top_k=0,
             dtype="bf16"),
        # A decode batch over every position, eight query heads to a K/V head.
        dict(name="attention decode", op="attention", batch=64, next_n=1, min_len=1024,
             max_len=32768, zeros=0, spread="uniform", heads=64, kv_heads=8, dim=128, block=64,
             top_k=0, dtype="bf16"),
        # Draft verification: four tokens a request, each with its own extent.
        dict(name="attention draft", op="attention", batch=32, next_n=4, min_len=4096,
             max_len=65536, zeros=0, spread="uniform", heads=32, kv_heads=4, dim=64, block=32,
             top_k=0, dtype="bf16"),
        # One request over a very long cache, all heads on one K/V head: the axis is split.
        dict(name="attention one long", op="attention", batch=1, next_n=1, min_len=131071,
             max_len=131071, zeros=0, spread="uniform", heads=64, kv_heads=1, dim=128, block=64,
             top_k=0, dtype="fp16"),
        # Long contexts at the 2048 selected positions, two draft slots with selections of their own.
        dict(name="attention selected", op="attention", batch=8, next_n=2, min_len=131072,
             max_len=131072, zeros=0, spread="uniform", heads=64, kv_heads=1, dim=128, block=64,
             top_k=2048, dtype="bf16"),
        # The serving mix at its selected positions: short and long requests, some without tokens.
        dict(name="attention serving", op="attention", batch=128, next_n=1, min_len=64,
             max_len=65536, zeros=3, spread="log", heads=64, kv_heads=8, dim=128, block=64,
             top_k=2048, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "index", "append", "attention", "attention", "attention"])
    half = rng.random() < 0.5
    if op == "rotary":
        dim = rng.choice([64, 96, 128, 192])
        rot = rng.choice([dim, dim // 2, dim // 4])
        return dict(op=op, tokens=_log(rng, 1, 8192), heads=rng.randint(1, 64), dim=dim, rot=rot,
                    offset=rng.choice([0, dim - rot]), interleaved=half,
                    dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                    max_pos=_log(rng, 2048, 131072))
    if op in ("index", "append"):
        ragged = rng.random() < 0.5
        hi = _log(rng, 40, 2500 if ragged else 16384)
        case = dict(op=op, batch=_log(rng, 1, 12 if ragged else 128),
                    next_n=0 if ragged else rng.randint(1, 4), min_len=rng.randint(8, hi),
                    max_len=hi)
        if op == "index":
            case.update(heads=rng.choice([8, 16, 32, 64]), dim=rng.choice([64, 128, 192]))
        else:
            case.update(kv_heads=rng.choice([1, 2, 4, 8]), dim=rng.choice([64, 128]))
        rot = rng.choice([32, 64])
        case.update(block=rng.choice([32, 64, 128]), rot=rot,
                    offset=rng.choice([0, case["dim"] - rot]), interleaved=half,
                    dtype=rng.choice(["bf16", "fp16"]))
        return case
    kv_heads = rng.choice([1, 2, 4, 8])
    top_k = rng.choice([0, 0, rng.choice([64, 512, 2048])])
    hi = _log(rng, 64, 131072)
    batch = _log(rng, 1, max(1, min(64, (1 << 20) // hi)))
    return dict(op="attention", batch=batch, next_n=rng.randint(1, 4), min_len=rng.randint(8, hi),
                max_len=hi, zeros=rng.choice([0, 0, 1]) if batch > 2 else 0,
                spread=rng.choice(["uniform", "log"]), heads=kv_heads * rng.randint(1, 8),
                kv_heads=kv_heads, dim=rng.choice([64, 128]), block=rng.choice([32, 64, 128]),
                top_k=top_k, dtype=rng.choice(["bf16", "fp16"]))


# ---- sizes that follow from a case alone ---------------------------------------------------------

def _lens(case):
    """Request lengths: spread over [min_len, max_len] by the golden ratio, ends odd and even."""
    lo, hi = case["min_len"], case["max_len"]
    out = []
    for b in range(case["batch"]):
        u = (0.5 + b * 0.6180339887498949) % 1.0
        if case.get("spread") == "log":
            n = round(math.exp(math.log(lo) + u * (math.log(hi) - math.log(lo))))
        else:
            n = round(lo + u * (hi - lo))
        out.append(0 if b < case.get("zeros", 0) else int(n))
    return out


def _new(case):
    """New tokens of each request: next_n, or (next_n = 0) all but a few of its length: a prompt
    that continues what the cache already holds."""
    if case["next_n"]:
        return [case["next_n"]] * case["batch"]
    return [n - (b * 7 % min(n, 90)) for b, n in enumerate(_lens(case))]


def _extents(case):
    n = case["next_n"]
    return [max(0, l - n + t + 1) for l in _lens(case) for t in range(n)]


def _counts(case):
    """Selected positions of each row: at least its top_k, a few more as a threshold gives them."""
    return [min(e, min(e, case["top_k"]) + 5 * (r % 7)) for r, e in enumerate(_extents(case))]


def work(case):
    op, D = case["op"], case["dim"]
    size = 4 if case["dtype"] == "fp32" else 2
    if op == "rotary":
        x = case["tokens"] * case["heads"] * D
        rot = case["tokens"] * case["rot"]
        return {"bytes": 2 * size * x + 4 * rot + 4 * case["tokens"],
                "flops": 3 * rot * case["heads"]}
    if op == "index":
        T, H = sum(_new(case)), case["heads"]
        return {"bytes": T * (H + 1) * D * (size + 1) + T * (8 * H + 4) + 4 * T * case["rot"],
                "flops": T * (H + 1) * (3 * D + 3 * case["rot"])}
    if op == "append":
        T, H = sum(_new(case)), case["kv_heads"]
        return {"bytes": 2 * T * H * D * (size + 1) + 4 * T * case["rot"],
                "flops": T * H * (6 * D + 3 * case["rot"])}
    H, Hkv, n = case["heads"], case["kv_heads"], case["next_n"]
    if case["top_k"]:
        tokens, pairs = sum(_counts(case)), sum(_counts(case))
        extra = 4 * tokens  # the positions
    else:
        tokens, pairs = sum(_lens(case)), sum(_extents(case))
        extra = 0
    qo = 2 * size * case["batch"] * n * H * D
    return {"bytes": 2 * tokens * Hkv * D + 8 * Hkv * (tokens // case["block"] + 1) + qo + extra,
            "flops": 4 * pairs * H * D}


# ---- inputs ------------------------------------------------------------------------------------

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _table(max_pos, rot, dev):
    """cos and sin of every position, rounded once from 64 bits: float32 [max_pos, rot / 2, 2]."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
    a = torch.arange(max_pos, dtype=torch.float64, device=dev)[:, None] * inv
    return torch.stack((a.cos(), a.sin()), -1).float().contiguous()


def _randn8(shape, gen, dev, scale=1.0):
    """N(0, scale) in e4m3, drawn a part at a time."""
    out = torch.empty(shape, dtype=torch.uint8, device=dev)
    flat, step = out.view(-1), 1 << 28
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        x = torch.randn(n, generator=gen, device=dev, dtype=torch.float16)
        flat[i:i + n] = (x.float() * scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return out.view(torch.float8_e4m3fn)


def _paging(case, gen, dev):
    """Block tables over a shared pool whose pages are in random order; unused entries are 0."""
    bs, lens = case["block"], _lens(case)
    pages = [-(-n // bs) for n in lens]
    width, total = max(max(pages), 1), max(sum(pages), 1)
    perm = torch.randperm(total, generator=gen, device=dev).int()
    table = torch.zeros(case["batch"], width, dtype=torch.int32, device=dev)
    at = 0
    for b, p in enumerate(pages):
        table[b, :p] = perm[at:at + p]
        at += p
    return table, torch.tensor(lens, dtype=torch.int32, device=dev), total


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev)
    gen.manual_seed(seed)
    op, D = case["op"], case["dim"]
    dt = _DTYPES[case["dtype"]]
    s = dict(case=case)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev).to(dt)

    if op == "rotary":
        s["x"] = randn(case["tokens"], case["heads"], D)
        s["positions"] = torch.randint(case["max_pos"], (case["tokens"],), generator=gen,
                                       device=dev, dtype=torch.int32)
        s["table"] = _table(case["max_pos"], case["rot"], dev)
        return s
    s["bt"], s["seq_lens"], blocks = _paging(case, gen, dev)
    bs = case["block"]
    if op in ("index", "append"):
        new = _new(case)
        T = sum(new)
        s["starts"] = None
        if not case["next_n"]:
            at = [0]
            for n in new:
                at.append(at[-1] + n)
            s["starts"] = torch.tensor(at, dtype=torch.int32, device=dev)
        s["table"] = _table(max(_lens(case)), case["rot"], dev)
        # The most blocks that one request's new tokens touch (the plain form's padded width).
        s["touched"] = max((l - 1) // bs - max(l - n, 0) // bs + 1 for l, n in zip(_lens(case), new))
    if op == "index":
        s["k"] = randn(T, D)
        s["q"] = randn(T, case["heads"], D)
        s["weights"] = torch.rand(T, case["heads"], generator=gen, device=dev) * 2 - 1
        pool = torch.zeros(blocks, bs * (D + 4), dtype=torch.uint8, device=dev)
        pool[:, :bs * D] = _randn8((blocks, bs * D), gen, dev).view(torch.uint8)
        s["pool"] = pool
        return s
    Hkv = case["kv_heads"]
    shape = (blocks, Hkv, bs, D)
    if op == "append":
        # Tokens of a cache in use: what is there was written with the scale that fits it, and a
        # few channels of the new keys are large, so that some blocks have to grow.
        s["k_pool"], s["v_pool"] = (_randn8(shape, gen, dev, 60.0) for _ in range(2))
        s["k_scales"], s["v_scales"] = (
            torch.exp2(torch.randint(-8, -4, (blocks, Hkv), generator=gen, device=dev).float())
            for _ in range(2))
        s["k"], s["v"] = randn(T, Hkv, D), randn(T, Hkv, D)
        s["k"][:, :, D // 2] *= 8
        return s
    s["k_pool"], s["v_pool"] = (_randn8(shape, gen, dev, 100.0) for _ in range(2))
    s["k_scales"], s["v_scales"] = ((torch.rand(blocks, Hkv, generator=gen, device=dev) * 1.5 + 0.5)
                                    / 100 for _ in range(2))
    s["q"] = randn(case["batch"], case["next_n"], case["heads"], D)
    if case["top_k"]:
        rows, top_k = case["batch"] * case["next_n"], case["top_k"]
        counts = _counts(case)
        ties = torch.tensor([min(c, r % 3) for r, c in enumerate(counts)], device=dev)
        lo = (top_k - ties).int()
        s["ranges"] = torch.stack((lo, lo + torch.tensor(counts, device=dev).int()))
        cand = torch.zeros(rows, 2 * top_k + 64, 2, dtype=torch.int32, device=dev)
        for r, (e, c) in enumerate(zip(_extents(case), counts)):
            if c:
                at = int(top_k - min(c, r % 3))
                cand[r, at:at + c, 0] = torch.randperm(e, generator=gen, device=dev)[:c].int()
        s["candidates"] = cand
    return s


# ---- one pass ------------------------------------------------------------------------------------

def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _own_rotary(s):
    import paged_fp8_mqa_gb300 as idx
    c = s["case"]
    return idx.rotary(s["x"], s["positions"], s["table"], interleaved=c["interleaved"],
                      rot_offset=c["offset"])


def _own_index(s):
    import paged_fp8_mqa_gb300 as idx
    c = s["case"]
    q8, w = idx.index_prepare(s["k"], s["pool"], s["bt"], s["seq_lens"], token_starts=s["starts"],
                              q=s["q"], weights=s["weights"], table=s["table"],
                              interleaved=c["interleaved"], rot_offset=c["offset"])
    return (q8, w, *_pool_views(s))


def _own_append(s):
    import paged_fp8_mqa_gb300 as idx
    c = s["case"]
    idx.kv_append(s["k"], s["v"], s["k_pool"], s["v_pool"], s["k_scales"], s["v_scales"], s["bt"],
                  s["seq_lens"], token_starts=s["starts"], table=s["table"],
                  interleaved=c["interleaved"], rot_offset=c["offset"])
    return s["k_pool"], s["v_pool"], s["k_scales"], s["v_scales"]


def _own_attention(s):
    import paged_fp8_mqa_gb300 as idx
    return idx.attention_fp8(s["q"], s["k_pool"], s["v_pool"], s["k_scales"], s["v_scales"],
                             s["bt"], s["seq_lens"], candidates=s.get("candidates"),
                             ranges=s.get("ranges"))


_own = dict(rotary=_own_rotary, index=_own_index, append=_own_append, attention=_own_attention)


def _pool_views(s):
    """The indexer's pool as its values [blocks, block, dim] and its scales [blocks, block]."""
    bs, D = s["case"]["block"], s["case"]["dim"]
    p = s["pool"]
    v = p.as_strided((p.shape[0], bs, D), (p.stride(0), D, 1)).view(torch.float8_e4m3fn)
    f = p.view(torch.float32).as_strided((p.shape[0], bs), (p.stride(0) // 4, 1), bs * D // 4)
    return v, f


def _rotate(x, cs, c):
    """x float32 [T, H, D], cs [T, rot / 2, 2]: the pairs turned, the rest as it is."""
    off, rot = c["offset"], c["rot"]
    cos, sin = cs[:, None, :, 0], cs[:, None, :, 1]
    part = x[..., off:off + rot]
    if c["interleaved"]:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((x[..., :off], turned, x[..., off + rot:]), -1)


def _tokens(s, T):
    """Request and position of each new token: a request's are the last of its length."""
    n = s["seq_lens"].long()
    t = torch.arange(T, device=n.device)
    if s["starts"] is None:
        per = s["case"]["next_n"]
        b = t // per
        return b, n[b] - per + t % per
    st = s["starts"].long()
    b = torch.searchsorted(st, t, right=True) - 1
    return b, n[b] - (st[b + 1] - t)


def _plain_rotary(s):
    x = _rotate(s["x"].float(), s["table"][s["positions"].long()], s["case"])
    return x.to(s["x"].dtype)


def _rows8(x):
    """e4m3 rows and their float32 scales, largest magnitude over 448."""
    scale = x.abs().amax(-1).clamp_min(TINY) / E4M3_MAX
    return (x / scale[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn), scale


def _plain_index(s):
    c = s["case"]
    b, pos = _tokens(s, s["k"].shape[0])
    cs = s["table"][pos]
    k8, ks = _rows8(_rotate(s["k"].float()[:, None], cs, c)[:, 0])
    q8, qs = _rows8(_rotate(s["q"].float(), cs, c))
    page = s["bt"][b, pos // c["block"]].long()
    values, scales = _pool_views(s)
    values.view(torch.uint8)[page, pos % c["block"]] = k8.view(torch.uint8)
    scales[page, pos % c["block"]] = ks
    return q8, s["weights"] * qs, values, scales


def _pow2_scale(amax):
    """The least power of two, 2^-100 or more, that brings amax to at most 448."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8)
    return torch.exp2(torch.where(amax > 0, e, torch.full_like(e, -100)).clamp_min(-100).float())


def _plain_append(s):
    c = s["case"]
    bs, J = c["block"], s["touched"]
    dev = s["k"].device
    n = s["seq_lens"].long()
    T = s["k"].shape[0]
    if s["starts"] is None:
        first = torch.arange(c["batch"], device=dev) * c["next_n"]
        begin = n - c["next_n"]
    else:
        first = s["starts"].long()[:-1]
        begin = n - (s["starts"].long()[1:] - first)
    blk = begin[:, None] // bs + torch.arange(J, device=dev)              # [B, J]
    live = blk * bs < n[:, None]
    pos = blk[..., None] * bs + torch.arange(bs, device=dev)              # [B, J, bs]
    fresh = (pos >= begin[:, None, None]) & (pos < n[:, None, None])
    old = (pos < begin[:, None, None])
    page = s["bt"].gather(1, blk.clamp_max(s["bt"].shape[1] - 1)).long()
    t = (first[:, None, None] + pos - begin[:, None, None]).clamp(0, T - 1)
    _, at = _tokens(s, T)
    turned = _rotate(s["k"].float(), s["table"][at], c)
    for x, pool, scales in ((turned, s["k_pool"], s["k_scales"]),
                            (s["v"].float(), s["v_pool"], s["v_scales"])):
        new = x[t].permute(0, 1, 3, 2, 4)                                 # [B, J, H, bs, D]
        is_new, is_old = fresh[:, :, None, :, None], old[:, :, None, :, None]
        scale = _pow2_scale((new.abs() * is_new).amax((3, 4)))            # [B, J, H]
        had = old.any(-1)[..., None]
        was = scales[page]
        scale = torch.where(had, torch.maximum(scale, was), scale)
        held = pool.view(torch.uint8)[page].view(torch.float8_e4m3fn)
        again = (held.float() * (was / scale)[..., None, None]).clamp(-448, 448)
        fits = (new / scale[..., None, None]).clamp(-448, 448)
        value = torch.where(is_new, fits, again).to(torch.float8_e4m3fn).view(torch.uint8)
        value = torch.where(is_new | is_old, value, held.view(torch.uint8))
        pool.view(torch.uint8)[page[live]] = value[live]
        scales[page[live]] = scale[live]
    return s["k_pool"], s["v_pool"], s["k_scales"], s["v_scales"]


def _softmax_product(q, k, v, seen):
    """q [..., r, D] (scaled), k and v [..., L, D], seen [..., r, L]: rows that see nothing give 0."""
    z = (q @ k.transpose(-1, -2)).masked_fill(~seen, float("-inf"))
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - m.masked_fill(m == float("-inf"), 0.0))
    total = p.sum(-1, keepdim=True)
    return (p @ v) / total.masked_fill(total == 0, 1.0)


def _plain_attention(s):
    c = s["case"]
    B, n, H, D = s["q"].shape
    Hkv, bs = c["kv_heads"], c["block"]
    G = H // Hkv
    dev = s["q"].device
    lens = s["seq_lens"].long()
    q = s["q"].float() * (D ** -0.5)
    if c["top_k"]:
        lo, hi = s["ranges"].long()
        slot = torch.arange(s["candidates"].shape[1], device=dev)
        seen = (slot >= lo[:, None]) & (slot < hi[:, None])               # [R, S]
        pos = torch.where(seen, s["candidates"][..., 0].long(), 0)
        b = torch.arange(B, device=dev).repeat_interleave(n)
        page = s["bt"].long()[b[:, None], pos // bs]

        def rows(pool, scales):
            x = pool.view(torch.uint8)[page, :, pos % bs].view(torch.float8_e4m3fn)
            return (x.float() * scales[page][..., None]).transpose(1, 2)  # [R, Hkv, S, D]

        q = q.view(B * n, Hkv, G, D)
        o = _softmax_product(q, rows(s["k_pool"], s["k_scales"]), rows(s["v_pool"], s["v_scales"]),
                             seen[:, None, None, :])
        return o.reshape(B, n, H, D).to(s["q"].dtype)

    def whole(pool, scales):
        page = s["bt"].long()
        x = pool.view(torch.uint8)[page].view(torch.float8_e4m3fn)        # [B, W, Hkv, bs, D]
        x = x.float() * scales[page][..., None, None]
        return x.transpose(1, 2).reshape(B, Hkv, -1, D)

    pos = torch.arange(s["bt"].shape[1] * bs, device=dev)
    ext = lens[:, None] - n + 1 + torch.arange(n, device=dev)             # [B, n]
    seen = (pos < ext[..., None])[:, None, :, None, :].expand(B, 1, n, G, -1).reshape(B, 1, n * G, -1)
    q = q.view(B, n, Hkv, G, D).transpose(1, 2).reshape(B, Hkv, n * G, D)
    o = _softmax_product(q, whole(s["k_pool"], s["k_scales"]), whole(s["v_pool"], s["v_scales"]),
                         seen)
    return o.view(B, Hkv, n, G, D).transpose(1, 2).reshape(B, n, H, D).to(s["q"].dtype)


_plain = dict(rotary=_plain_rotary, index=_plain_index, append=_plain_append,
              attention=_plain_attention)


# ---- the same in 64 bits -------------------------------------------------------------------------

def _turn64(x, table, pos, c):
    """Each pair as a complex number times cos + i sin."""
    x = x.double().clone()
    w = torch.view_as_complex(table.double().contiguous())[pos][:, None]
    off, half = c["offset"], c["rot"] // 2
    i = torch.arange(half, device=x.device)
    a, b = (off + 2 * i, off + 2 * i + 1) if c["interleaved"] else (off + i, off + half + i)
    z = torch.complex(x[..., a], x[..., b]) * w
    x[..., a], x[..., b] = z.real, z.imag
    return x


def exact(case, seed):
    s = prepare(case, seed)
    op, D = case["op"], case["dim"]
    if op == "rotary":
        return _turn64(s["x"], s["table"], s["positions"].long(), case)
    lens, bs = _lens(case), case["block"]
    if op in ("index", "append"):
        new = _new(case)
        pos = torch.cat([torch.arange(l - n, l) for l, n in zip(lens, new)]).cuda()
        who = torch.cat([torch.full((n,), b) for b, n in enumerate(new)]).cuda()
        page, row = s["bt"].long()[who, pos // bs], pos % bs
    if op == "index":
        values, scales = (x.double() for x in _pool_views(s))
        k, q = _turn64(s["k"][:, None], s["table"], pos, case)[:, 0], _turn64(s["q"], s["table"], pos, case)
        ks, qs = (x.abs().amax(-1) / 448 for x in (k, q))
        values[page, row] = k / ks[:, None]
        scales[page, row] = ks
        return q / qs[..., None], s["weights"].double() * qs, values, scales
    if op == "append":
        outs = []
        for x, pool, was in ((_turn64(s["k"], s["table"], pos, case), s["k_pool"], s["k_scales"]),
                             (s["v"].double(), s["v_pool"], s["v_scales"])):
            pool, scale = pool.double(), was.double()
            at = 0
            for b, (l, n) in enumerate(zip(lens, new)):
                for j in range((l - n) // bs, (l - 1) // bs + 1):
                    p, t0, t1 = int(s["bt"][b, j]), max(l - n, j * bs), min(l, (j + 1) * bs)
                    part = x[at + t0 - (l - n):at + t1 - (l - n)]
                    need = torch.exp2(torch.ceil(torch.log2(part.abs().amax((0, 2)) / 448)))
                    if t0 > j * bs:
                        need = torch.maximum(need, scale[p])
                        pool[p, :, :t0 - j * bs] *= (scale[p] / need)[:, None, None]
                    pool[p, :, t0 - j * bs:t1 - j * bs] = (part / need[:, None]).transpose(0, 1)
                    scale[p] = need
                at += n
            outs.append((pool, scale))
        return outs[0][0], outs[1][0], outs[0][1], outs[1][1]
    B, n, H, _ = s["q"].shape
    Hkv = case["kv_heads"]
    out = torch.zeros(B, n, H, D, dtype=torch.float64, device="cuda")
    if sum(_extents(case)) * H * D * 4 > 1.2e13:
        return None  # over 20 seconds at this card's rate in 64 bits

    def rows(pool, scales, pages, at):
        x = pool.view(torch.uint8)[pages, :, at].view(torch.float8_e4m3fn).double()
        return x * scales[pages].double()[..., None]                      # [L, Hkv, D]

    for b, l in enumerate(lens):
        for t in range(n):
            r, e = b * n + t, max(0, l - n + t + 1)
            if not e:
                continue
            p = torch.arange(e, device="cuda")
            if case["top_k"]:
                p = s["candidates"][r, int(s["ranges"][0, r]):int(s["ranges"][1, r]), 0].long()
            pages, at = s["bt"].long()[b, p // bs], p % bs
            k, v = rows(s["k_pool"], s["k_scales"], pages, at), rows(s["v_pool"], s["v_scales"], pages, at)
            q = s["q"][b, t].double().view(Hkv, H // Hkv, D)
            z = torch.einsum("hgd,lhd->hgl", q, k) / math.sqrt(D)
            out[b, t] = torch.einsum("hgl,lhd->hgd", torch.softmax(z, -1), v).reshape(H, D)
    return out
