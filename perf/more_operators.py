"""Performance cases of what a layer with normalised heads, image and video positions and a 4-bit K/V
cache needs: the rotation by several axes, the norms of queries and keys with the rotation in the same
pass (forward, and forward with gradients), the writer and the reader of the 4-bit cache, and the
attention over it, at every visible position or at the positions that the select stored.

The cache: codes of four bits (E2M1: a sign and one of 0, 0.5, 1, 1.5, 2, 3, 4, 6), two a byte, the
even element in the low half.  A key has a power of two (UE8M0, one byte: 2^(byte - 127)) for each 32
elements, the least that brings them to at most 6; a value row has one float32 scale, its largest
magnitude over 6.

A case is a dict of plain values.  ``prepare`` makes what a program holds before the call, ``run``
makes one pass (the plain form in elementary torch operations, or the package's call where ``own`` is
true), ``exact`` gives the same outputs in 64 bits, ``work`` the bytes and operations that a pass
cannot do without.
"""
from __future__ import annotations

import math

import torch

own = False

TINY = 2.0 ** -96  # the least largest-magnitude of a value row
LEAST = -100       # the least exponent of a key group's scale
EPS = 1e-6


# ---- the cases ---------------------------------------------------------------------------------

def listed():
    return [
        # One decode step of 64 requests of a model with image positions: time, height and width.
        dict(name="axes decode", op="axes", tokens=64, heads=64, dim=128, rot=128, offset=0,
             interleaved=False, axes=3, spread=False, dtype="bf16", max_pos=32768),
        # The queries of a long video: an odd number of patches, the axes taken in turn.
        dict(name="axes video", op="axes", tokens=8191, heads=64, dim=128, rot=128, offset=0,
             interleaved=False, axes=3, spread=True, dtype="bf16", max_pos=32768),
        # Queries and keys of one decode step, views of one projection: norms and rotation at once.
        dict(name="norm decode", op="norm", tokens=64, heads=64, kv_heads=8, dim=128, rot=128,
             offset=0, interleaved=False, axes=1, spread=False, dtype="bf16", wdtype="bf16",
             max_pos=131072),
        # The same of a long prompt.
        dict(name="norm prompt", op="norm", tokens=8192, heads=64, kv_heads=8, dim=128, rot=128,
             offset=0, interleaved=False, axes=1, spread=False, dtype="bf16", wdtype="bf16",
             max_pos=131072),
        # A small model's training step over a few images: forward and all gradients, part of a head
        # of 64 rotated.
        dict(name="norm train small", op="train", tokens=301, heads=12, kv_heads=2, dim=64, rot=32,
             offset=0, interleaved=False, axes=3, spread=False, dtype="fp16", wdtype="fp32",
             max_pos=4096),
        # A layer's training step over 8192 tokens, forward and all gradients.
        dict(name="norm train", op="train", tokens=8192, heads=32, kv_heads=8, dim=128, rot=128,
             offset=0, interleaved=False, axes=1, spread=False, dtype="bf16", wdtype="fp32",
             max_pos=8192),
        # One token each of 64 short chats into the 4-bit cache, and what the requests hold read back.
        dict(name="append decode", op="append", batch=64, next_n=1, min_len=20, max_len=200,
             kv_heads=8, dim=128, block=64, rot=64, offset=0, interleaved=False, dtype="bf16"),
        # Prompts of unequal length that continue what the cache holds, and the whole contexts read
        # back for the attention among a prompt's tokens.
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
             max_len=65536, zeros=0, spread="uniform", heads=32, kv_heads=4, dim=128, block=32,
             top_k=0, dtype="bf16"),
        # The serving mix at its selected positions: short and long requests, some without tokens.
        dict(name="attention serving", op="attention", batch=128, next_n=1, min_len=64,
             max_len=65536, zeros=3, spread="log", heads=64, kv_heads=8, dim=128, block=64,
             top_k=2048, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["axes", "norm", "train", "append", "attention", "attention", "attention"])
    half = rng.random() < 0.5
    if op in ("axes", "norm", "train"):
        dim = rng.choice([64, 96, 128, 192])
        rot = rng.choice([dim, dim // 2, dim // 4])
        kv = rng.choice([1, 2, 4, 8])
        case = dict(op=op, tokens=_log(rng, 1, 8192), heads=kv * rng.randint(1, 64 // kv), dim=dim,
                    rot=rot, offset=rng.choice([0, dim - rot]), interleaved=half,
                    axes=rng.choice([2, 3, 4]) if op == "axes" else rng.choice([1, 1, 3]),
                    spread=rng.random() < 0.5, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                    max_pos=_log(rng, 2048, 131072))
        if op == "train":
            case.update(heads=min(case["heads"], 32), tokens=_log(rng, 1, 4096))
        if op != "axes":
            case.update(kv_heads=kv, wdtype=rng.choice([case["dtype"], "fp32"]))
        return case
    if op == "append":
        ragged = rng.random() < 0.5
        hi = _log(rng, 40, 2500)
        return dict(op=op, batch=_log(rng, 1, 12), next_n=0 if ragged else rng.randint(1, 4),
                    min_len=rng.randint(8, hi), max_len=hi, kv_heads=rng.choice([1, 2, 4, 8]),
                    dim=rng.choice([64, 128]), block=rng.choice([32, 64, 128]),
                    rot=rng.choice([32, 64]), offset=0, interleaved=half,
                    dtype=rng.choice(["bf16", "fp16"]))
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


def _sections(case):
    """Pairs of each axis: a quarter for the first, the rest shared out."""
    A, half = case["axes"], case["rot"] // 2
    first = half if A == 1 else max(1, half // 4)
    rest = [(half - first) // (A - 1) + (i < (half - first) % (A - 1)) for i in range(A - 1)]
    return [first, *rest]


def _pair_axes(case):
    """The axis of each pair: one section after the other, or in turn while an axis has some left."""
    left = _sections(case)
    if not case["spread"]:
        return [a for a, n in enumerate(left) for _ in range(n)]
    out = []
    while any(left):
        for a in range(len(left)):
            if left[a]:
                out.append(a)
                left[a] -= 1
    return out


def work(case):
    op, D = case["op"], case["dim"]
    size = 4 if case["dtype"] == "fp32" else 2
    if op in ("axes", "norm", "train"):
        T, heads = case["tokens"], case["heads"] + case.get("kv_heads", 0)
        x, rot = T * heads * D, T * case["rot"]
        angles = 4 * rot + 4 * T * case["axes"]
        if op == "axes":
            return {"bytes": 2 * size * x + angles, "flops": 3 * rot * heads}
        once = 4 * x + 3 * rot * heads
        if op == "norm":
            return {"bytes": 2 * size * x + angles, "flops": once}
        # Forward: x in, y out; the gradients: dy in, x again (what a forward leaves), dx out.
        return {"bytes": 5 * size * x + 2 * angles, "flops": 3 * once}
    if op == "append":
        H = case["kv_heads"]
        T, all_ = sum(_new(case)), sum(_lens(case))
        row = D + D // 32 + 4  # codes and scales of a token's key and value
        return {"bytes": 2 * size * (T + all_) * H * D + (T + all_) * H * row + 4 * T * case["rot"],
                "flops": T * H * (6 * D + 3 * case["rot"]) + 2 * all_ * H * D}
    H, Hkv, n = case["heads"], case["kv_heads"], case["next_n"]
    if case["top_k"]:
        tokens, pairs = sum(_counts(case)), sum(_counts(case))
        extra = 4 * tokens  # the positions
    else:
        tokens, pairs = sum(_lens(case)), sum(_extents(case))
        extra = 0
    qo = 2 * size * case["batch"] * n * H * D
    return {"bytes": tokens * Hkv * (D + D // 32 + 4) + qo + extra, "flops": 4 * pairs * H * D}


# ---- inputs ------------------------------------------------------------------------------------

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _table(max_pos, rot, dev):
    """cos and sin of every position, rounded once from 64 bits: float32 [max_pos, rot / 2, 2]."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
    a = torch.arange(max_pos, dtype=torch.float64, device=dev)[:, None] * inv
    return torch.stack((a.cos(), a.sin()), -1).float().contiguous()


def _positions(case, gen, dev):
    """int32 [axes, tokens]: text, whose axes agree, and in every second run of 32 tokens patches, which
    stand at a place of their own; with one axis [tokens]."""
    T, most = case["tokens"], case["max_pos"]
    text = torch.randint(most, (T,), generator=gen, device=dev, dtype=torch.int32)
    if case["axes"] == 1:
        return text
    patch = torch.randint(min(most, 96), (case["axes"], T), generator=gen, device=dev, dtype=torch.int32)
    image = torch.arange(T, device=dev) // 32 % 2 == 1
    return torch.where(image, patch, text).contiguous()


def _codes(shape, gen, dev):
    """Codes of a normal distribution, two a byte, drawn a part at a time."""
    z = torch.erfinv((torch.arange(256, device=dev) + 0.5) / 128 - 1) * 2 ** 0.5 * 2.2
    one = _code_of(z.float()).to(torch.int32)
    byte = (one[:, None] | one[None, :] << 4).to(torch.uint8).view(-1)  # by two random bytes
    out = torch.empty(shape, dtype=torch.uint8, device=dev)
    flat, step = out.view(-1), 1 << 27
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        flat[i:i + n] = byte[torch.randint(65536, (n,), generator=gen, device=dev, dtype=torch.int32)]
    return out


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

    if op in ("axes", "norm", "train"):
        T, H = case["tokens"], case["heads"]
        s["positions"] = _positions(case, gen, dev)
        s["table"] = _table(case["max_pos"], case["rot"], dev)
        s["axes"] = tuple(_pair_axes(case)) if case["axes"] > 1 else None
        s["pair_axis"] = torch.tensor(_pair_axes(case), device=dev)
        if op == "axes":
            s["x"] = randn(T, H, D)
            return s
        Hkv = case["kv_heads"]
        qkv = randn(T, H + 2 * Hkv, D)
        s["q"], s["k"] = qkv[:, :H], qkv[:, H:H + Hkv]
        for n in ("q_weight", "k_weight"):
            w = 1 + 0.2 * torch.randn(D, generator=gen, device=dev)
            s[n] = w.to(_DTYPES[case["wdtype"]])
        if op == "train":
            s["q_grad"], s["k_grad"] = randn(T, H, D), randn(T, Hkv, D)
        return s
    s["bt"], s["seq_lens"], blocks = _paging(case, gen, dev)
    bs, Hkv = case["block"], case["kv_heads"]
    s["k_pool"], s["v_pool"] = (_codes((blocks, Hkv, bs, D // 2), gen, dev) for _ in range(2))
    # Keys have channels that stand out: the second group's scales are a binade up.
    s["k_scales"] = torch.randint(124, 127, (blocks, Hkv, bs, D // 32), generator=gen, device=dev,
                                  dtype=torch.uint8)
    s["k_scales"][..., 1] += 1
    s["v_scales"] = torch.rand(blocks, Hkv, bs, generator=gen, device=dev) * 0.4 + 0.25
    if op == "append":
        new = _new(case)
        T = sum(new)
        s["starts"] = None
        at = [0]
        for n in new:
            at.append(at[-1] + n)
        if not case["next_n"]:
            s["starts"] = torch.tensor(at, dtype=torch.int32, device=dev)
        at = [0]
        for n in _lens(case):
            at.append(at[-1] + n)
        s["all_starts"] = torch.tensor(at, dtype=torch.int32, device=dev)
        s["total"] = at[-1]
        s["table"] = _table(max(_lens(case)), case["rot"], dev)
        s["k"], s["v"] = randn(T, Hkv, D), randn(T, Hkv, D)
        s["k"][:, :, D // 2] *= 8
        return s
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


def _own_axes(s):
    import paged_fp8_mqa_gb300 as idx
    c = s["case"]
    return idx.rotary(s["x"], s["positions"], s["table"], axes=s["axes"],
                      interleaved=c["interleaved"], rot_offset=c["offset"])


def _own_norm(s):
    import paged_fp8_mqa_gb300 as idx
    c = s["case"]
    return idx.norm_rotary(s["q"], s["k"], s["q_weight"], s["k_weight"], s["positions"], s["table"],
                           eps=EPS, axes=s["axes"], interleaved=c["interleaved"],
                           rot_offset=c["offset"])


def _own_train(s):
    import paged_fp8_mqa_gb300 as idx
    c = s["case"]
    leaves = [s[n].detach().requires_grad_() for n in ("q", "k", "q_weight", "k_weight")]
    out = idx.norm_rotary(*leaves, s["positions"], s["table"], eps=EPS, axes=s["axes"],
                          interleaved=c["interleaved"], rot_offset=c["offset"])
    return (*(x.detach() for x in out), *torch.autograd.grad(out, leaves, (s["q_grad"], s["k_grad"])))


def _own_append(s):
    import paged_fp8_mqa_gb300 as idx
    c = s["case"]
    cache = s["k_pool"], s["v_pool"], s["k_scales"], s["v_scales"]
    idx.kv_append_fp4(s["k"], s["v"], *cache, s["bt"], s["seq_lens"], token_starts=s["starts"],
                      table=s["table"], interleaved=c["interleaved"], rot_offset=c["offset"])
    k, v = idx.kv_read_fp4(*cache, s["bt"], s["seq_lens"], s["all_starts"], tokens=s["total"],
                           dtype=s["k"].dtype)
    return k, v


def _own_attention(s):
    import paged_fp8_mqa_gb300 as idx
    return idx.attention_fp4(s["q"], s["k_pool"], s["v_pool"], s["k_scales"], s["v_scales"],
                             s["bt"], s["seq_lens"], candidates=s.get("candidates"),
                             ranges=s.get("ranges"))


_own = dict(axes=_own_axes, norm=_own_norm, train=_own_train, append=_own_append,
            attention=_own_attention)


def _angles(s):
    """cos and sin of each token's pairs, [T, 1, rot / 2, 2], each pair's by its own axis."""
    p = s["positions"].long()
    if s["axes"] is None:
        return s["table"][p][:, None]
    pair = torch.arange(s["table"].shape[1], device=p.device)
    return s["table"][p[s["pair_axis"]].t(), pair][:, None]


def _rotate(x, cs, c, back=False):
    """x float32 [T, H, D]: the pairs turned (or turned back), the rest as it is."""
    off, rot = c["offset"], c["rot"]
    cos, sin = cs[..., 0], cs[..., 1]
    if back:
        sin = -sin
    part = x[..., off:off + rot]
    if c["interleaved"]:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((x[..., :off], turned, x[..., off + rot:]), -1)


def _plain_axes(s):
    return _rotate(s["x"].float(), _angles(s), s["case"]).to(s["x"].dtype)


def _inv_rms(x):
    return torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)


def _plain_norm(s):
    cs = _angles(s)
    out = []
    for n in "qk":
        x = s[n].float()
        y = x * _inv_rms(x) * s[n + "_weight"].float()
        out.append(_rotate(y, cs, s["case"]).to(s[n].dtype))
    return out


def _plain_train(s):
    cs = _angles(s)
    out, dx, dw = [], [], []
    for n in "qk":
        x, w = s[n].float(), s[n + "_weight"].float()
        r = _inv_rms(x)
        unit = x * r
        out.append(_rotate(unit * w, cs, s["case"]).to(s[n].dtype))
        g = _rotate(s[n + "_grad"].float(), cs, s["case"], back=True)
        gw = g * w
        dx.append(((gw - unit * (gw * unit).mean(-1, keepdim=True)) * r).to(s[n].dtype))
        # (a sum over every token and head: in 64 bits)
        dw.append((g * unit).sum((0, 1), dtype=torch.float64).to(s[n + "_weight"].dtype))
    return *out, *dx, *dw


_BORDERS = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]  # between the magnitudes
_UP = [False, True, False, True, False, True, False]  # ties to the even code: up at these


def _code_of(x):
    """The four-bit codes of x (magnitudes past 6: 6)."""
    a = x.abs()
    n = torch.zeros(x.shape, dtype=torch.uint8, device=x.device)
    for b, up in zip(_BORDERS, _UP):
        n += (a >= b) if up else (a > b)
    return n | (torch.signbit(x).to(torch.uint8) << 3)


def _pack(code):
    return code[..., 0::2] | code[..., 1::2] << 4


def _values(codes):
    """The numbers of packed codes, float32, twice as many in the last axis."""
    half = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    one = torch.cat((half, -half))
    two = torch.stack((one.repeat(16), one.repeat_interleave(16)), -1)
    return two[codes.int()].flatten(-2)


def _keys(codes, scales):
    v = _values(codes)
    return (v.unflatten(-1, (-1, 32)) * torch.exp2(scales.float() - 127)[..., None]).flatten(-2)


def _tokens(seq_lens, starts, per, T):
    """Request and position of each of T rows: a request's are the last of its length."""
    n = seq_lens.long()
    t = torch.arange(T, device=n.device)
    if starts is None:
        b = t // per
        return b, n[b] - per + t % per
    st = starts.long()
    b = torch.searchsorted(st, t, right=True) - 1
    return b, n[b] - (st[b + 1] - t)


def _plain_append(s):
    c = s["case"]
    bs = c["block"]
    b, pos = _tokens(s["seq_lens"], s["starts"], c["next_n"], s["k"].shape[0])
    page, row = s["bt"][b, pos // bs].long(), pos % bs
    k = _rotate(s["k"].float(), s["table"][pos][:, None], c).unflatten(-1, (-1, 32))
    m, e = torch.frexp(k.abs().amax(-1))
    e = torch.where(m <= 0.75, e - 3, e - 2).clamp_min(LEAST)       # the least with amax <= 6 * 2^e
    s["k_pool"][page, :, row] = _pack(_code_of((k * torch.exp2(-e.float())[..., None]).flatten(-2)))
    s["k_scales"][page, :, row] = (e + 127).to(torch.uint8)
    v = s["v"].float()
    most = v.abs().amax(-1).clamp_min(TINY)
    # (6 v over the largest, not v over the rounded scale: values halfway between two codes stay so)
    s["v_pool"][page, :, row] = _pack(_code_of(6 * v / most[..., None]))
    s["v_scales"][page, :, row] = most / 6
    b, pos = _tokens(s["seq_lens"], s["all_starts"], 0, s["total"])
    page, row = s["bt"][b, pos // bs].long(), pos % bs
    k = _keys(s["k_pool"][page, :, row], s["k_scales"][page, :, row])
    v = _values(s["v_pool"][page, :, row]) * s["v_scales"][page, :, row][..., None]
    return k.to(s["k"].dtype), v.to(s["k"].dtype)


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
        page, row = s["bt"].long()[b[:, None], pos // bs], pos % bs
        k = _keys(s["k_pool"][page, :, row], s["k_scales"][page, :, row]).transpose(1, 2)
        v = (_values(s["v_pool"][page, :, row]) * s["v_scales"][page, :, row][..., None]).transpose(1, 2)
        o = _softmax_product(q.view(B * n, Hkv, G, D), k, v, seen[:, None, None, :])
        return o.reshape(B, n, H, D).to(s["q"].dtype)

    def whole(x):
        return x.transpose(1, 2).reshape(B, Hkv, -1, D)                   # of [B, W, Hkv, bs, D]

    page = s["bt"].long()
    k = whole(_keys(s["k_pool"][page], s["k_scales"][page]))
    v = whole(_values(s["v_pool"][page]) * s["v_scales"][page][..., None])
    pos = torch.arange(s["bt"].shape[1] * bs, device=dev)
    ext = lens[:, None] - n + 1 + torch.arange(n, device=dev)             # [B, n]
    seen = (pos < ext[..., None])[:, None, :, None, :].expand(B, 1, n, G, -1).reshape(B, 1, n * G, -1)
    q = q.view(B, n, Hkv, G, D).transpose(1, 2).reshape(B, Hkv, n * G, D)
    o = _softmax_product(q, k, v, seen)
    return o.view(B, Hkv, n, G, D).transpose(1, 2).reshape(B, n, H, D).to(s["q"].dtype)


_plain = dict(axes=_plain_axes, norm=_plain_norm, train=_plain_train, append=_plain_append,
              attention=_plain_attention)


# ---- the same in 64 bits -------------------------------------------------------------------------

def _turn64(x, s, positions, case, back=False):
    """Each pair as a complex number times cos + i sin (or over it)."""
    x = x.double().clone()
    off, half = case["offset"], case["rot"] // 2
    table = torch.view_as_complex(s["table"].double().contiguous())
    axis = _pair_axes(case) if case.get("axes", 1) > 1 else [0] * half
    pos = positions.long().view(-1, x.shape[0])
    w = torch.stack([table[pos[a], i] for i, a in enumerate(axis)], -1)[:, None]
    i = torch.arange(half, device=x.device)
    a, b = (off + 2 * i, off + 2 * i + 1) if case["interleaved"] else (off + i, off + half + i)
    z = torch.complex(x[..., a], x[..., b]) * (w.conj() if back else w)
    x[..., a], x[..., b] = z.real, z.imag
    return x


def _decode64(codes):
    """Sign, two exponent bits, one mantissa bit."""
    n = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).double()
    sign, n = torch.where(n >= 8, -1.0, 1.0), n % 8
    e, m = torch.floor(n / 2), n % 2
    return sign * torch.where(e == 0, m / 2, (1 + m / 2) * 2.0 ** (e - 1))


def _round64(y):
    """The nearest number of four bits, ties to the even mantissa."""
    a = y.abs().clamp_max(6)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()
    return torch.copysign(torch.round(a / step) * step, y)


def exact(case, seed):
    s = prepare(case, seed)
    op, D = case["op"], case["dim"]
    if op == "axes":
        return _turn64(s["x"], s, s["positions"], case)
    if op in ("norm", "train"):
        out, dx, dw = [], [], []
        for n in "qk":
            x, w = s[n].double(), s[n + "_weight"].double()
            rms = torch.sqrt(x.square().sum(-1, keepdim=True) / D + EPS)
            out.append(_turn64(x / rms * w, s, s["positions"], case))
            if op == "train":
                g = _turn64(s[n + "_grad"], s, s["positions"], case, back=True)
                dw.append((g * x / rms).sum((0, 1)))
                dx.append(g * w / rms - x * (g * w * x).sum(-1, keepdim=True) / (D * rms ** 3))
        return *out, *dx, *dw
    lens, bs = _lens(case), case["block"]
    if op == "append":
        new = _new(case)
        dev = s["k"].device
        pos = torch.cat([torch.arange(l - n, l) for l, n in zip(lens, new)]).to(dev)
        turned = _turn64(s["k"], s, pos, case)
        ks, vs, at = [], [], 0
        for b, (l, n) in enumerate(zip(lens, new)):
            p = torch.arange(l - n, device=dev)
            page = s["bt"].long()[b, p // bs]
            k = _decode64(s["k_pool"][page, :, p % bs]).unflatten(-1, (-1, 32))
            k = k * torch.exp2(s["k_scales"][page, :, p % bs].double() - 127)[..., None]
            v = _decode64(s["v_pool"][page, :, p % bs]) * s["v_scales"][page, :, p % bs].double()[..., None]
            g = turned[at:at + n].unflatten(-1, (-1, 32))
            unit = torch.exp2(torch.ceil(torch.log2(g.abs().amax(-1, keepdim=True) / 6)))
            x = s["v"][at:at + n].double()
            most = x.abs().amax(-1, keepdim=True)
            ks += [k.flatten(-2), (_round64(g / unit) * unit).flatten(-2)]
            vs += [v, _round64(x * 6 / most) * (most / 6)]
            at += n
        return torch.cat(ks), torch.cat(vs)
    B, n, H, _ = s["q"].shape
    Hkv = case["kv_heads"]
    out = torch.zeros(B, n, H, D, dtype=torch.float64, device="cuda")
    if sum(_extents(case)) * H * D * 4 > 1.2e13:
        return None  # over 20 seconds at this card's rate in 64 bits
    for b, l in enumerate(lens):
        for t in range(n):
            r, e = b * n + t, max(0, l - n + t + 1)
            if not e:
                continue
            p = torch.arange(e, device="cuda")
            if case["top_k"]:
                p = s["candidates"][r, int(s["ranges"][0, r]):int(s["ranges"][1, r]), 0].long()
            page, at = s["bt"].long()[b, p // bs], p % bs
            k = _decode64(s["k_pool"][page, :, at]).unflatten(-1, (-1, 32))
            k = (k * torch.exp2(s["k_scales"][page, :, at].double() - 127)[..., None]).flatten(-2)
            v = _decode64(s["v_pool"][page, :, at]) * s["v_scales"][page, :, at].double()[..., None]
            q = s["q"][b, t].double().view(Hkv, H // Hkv, D)
            z = torch.einsum("hgd,lhd->hgl", q, k) / math.sqrt(D)
            out[b, t] = torch.einsum("hgl,lhd->hgd", torch.softmax(z, -1), v).reshape(H, D)
    return out
