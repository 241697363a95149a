"""Workloads of rotary positions, the 8-bit cache and its attention, and beam search, in plain torch and through the library.

``own`` selects what ``run`` computes: False, the operators written out in
elementary torch operations; True, the library's calls on the same state.
``exact`` gives the same outputs from the definitions in FP64.

The operators:

* ``rotary``: positions put into q and k (or taken out of their gradients):
  pairs of the first R dims of each head, halves apart or side by side, turn by
  position times a frequency, frequencies scaled for long contexts;
* ``cache8``: new tokens' K and V written into a cache of 8-bit codes with a
  scale for each block of tokens and head, and tokens read back from it;
* ``decode8``: attention of one new token per sequence over such a cache;
* ``beam``: the best continuations over beams and vocabulary, and the beams'
  token histories put in their new order.

Code pools are [pages, kv heads, tokens of a page, head size], scale pools
[pages, kv heads, blocks of a page]; a code c of a block with scale s stands
for c * s.  A block's scale is made when its first token is written: the
largest magnitude of what is written / 127 for integers, the least power of
two that brings it to 448 or below for floats.  A token too large for a block
that has been begun multiplies the scale by a power of two, and the codes that
are there are divided by it and rounded to nearest even.
"""
import math

import torch

own = False

DEV = "cuda"
FLOATS = {"f16": torch.float16, "f32": torch.float32}
CODES = {"i8": torch.int8, "e4m3": torch.float8_e4m3fn}
LARGEST = {"i8": 127.0, "e4m3": 448.0}
LEAST_SCALE = 2.0 ** -126


# -- cases ---------------------------------------------------------------------

def listed():
    return [
        # One step's new token of each of 64 sequences, far into a context eight times as long as trained: latency.
        {"name": "rotary_64_gqa128_f32", "op": "rotary", "tokens": 64, "heads": 32, "kv_heads": 8, "dim": 128,
         "turned": 128, "type": "f32", "layout": "half", "scaling": "parts", "factor": 8.0, "far": 131072,
         "transpose": False},
        # Gradients of packed prompts of 6001 tokens in all, half of each head turned.
        {"name": "rotary_6001_grad64_f16", "op": "rotary", "tokens": 6001, "heads": 14, "kv_heads": 2, "dim": 64,
         "turned": 32, "type": "f16", "layout": "interleaved", "scaling": "plain", "factor": 1.0, "far": 2048,
         "transpose": True},
        # One long prompt of the feed-forward workload's 8192 rows, positions interpolated.
        {"name": "rotary_8192_gqa128_f32", "op": "rotary", "tokens": 8192, "heads": 32, "kv_heads": 8, "dim": 128,
         "turned": 128, "type": "f32", "layout": "half", "scaling": "linear", "factor": 4.0, "far": 32768,
         "transpose": False},
        # One step's new token of 64 sequences written, and the last 16 tokens of each read: a short window.
        {"name": "cache8_64x1_i8", "op": "cache8", "seqs": 64, "tokens": 64, "page": 16, "block": 16, "pool": 512,
         "kv_heads": 8, "dim": 128, "codes": "i8", "window": 16, "out": "f32"},
        # Uneven prompts that go on from cached tokens, everything read back for their attention.
        {"name": "cache8_8x750_e4m3", "op": "cache8", "seqs": 8, "tokens": 6001, "page": 64, "block": 32, "pool": 300,
         "kv_heads": 12, "dim": 64, "codes": "e4m3", "window": 0, "out": "f16"},
        # Long prompts written into the cache and read back.
        {"name": "cache8_4x2048_i8", "op": "cache8", "seqs": 4, "tokens": 8190, "page": 64, "block": 64, "pool": 400,
         "kv_heads": 8, "dim": 128, "codes": "i8", "window": 0, "out": "f32"},
        # One sequence, a few pages: latency.
        {"name": "decode8_1x130_i8", "op": "decode8", "batch": 1, "longest": 130, "page": 16, "block": 16, "heads": 32,
         "kv_heads": 8, "dim": 128, "codes": "i8"},
        # A dozen samples, heads not grouped, two scales to a page.
        {"name": "decode8_12x2000_e4m3", "op": "decode8", "batch": 12, "longest": 2000, "page": 32, "block": 16,
         "heads": 12, "kv_heads": 12, "dim": 64, "codes": "e4m3"},
        # Two very long contexts.
        {"name": "decode8_2x65536_i8", "op": "decode8", "batch": 2, "longest": 65536, "page": 64, "block": 64,
         "heads": 32, "kv_heads": 8, "dim": 128, "codes": "i8"},
        # A serving batch of long contexts.
        {"name": "decode8_64x8000_i8", "op": "decode8", "batch": 64, "longest": 8000, "page": 64, "block": 64,
         "heads": 32, "kv_heads": 8, "dim": 128, "codes": "i8"},
        # One request with four beams over a vocabulary of odd size: latency.
        {"name": "beam_1x4_32003", "op": "beam", "seqs": 1, "beams": 4, "vocab": 32003, "history": 300},
        # A batch of requests with eight beams each over a large vocabulary.
        {"name": "beam_32x8_128000", "op": "beam", "seqs": 32, "beams": 8, "vocab": 128000, "history": 1000},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "rotary", "cache8", "cache8", "decode8", "decode8", "decode8", "beam", "beam"])
    heads, kv_heads, dim = rng.choice([(12, 12, 64), (32, 8, 128), (16, 2, 128), (8, 8, 80), (14, 2, 64), (9, 3, 40)])
    if op == "rotary":
        return {"op": op, "tokens": _log_uniform(rng, 1, 8000), "heads": heads, "kv_heads": kv_heads, "dim": dim,
                "turned": rng.choice([dim, dim // 2, dim // 4 * 2]), "type": rng.choice(["f16", "f32"]),
                "layout": rng.choice(["half", "interleaved"]),
                "scaling": rng.choice(["plain", "linear", "ntk", "parts"]), "factor": rng.choice([2.0, 4.0, 8.0, 32.0]),
                "far": _log_uniform(rng, 1, 1000000), "transpose": rng.random() < 0.4}
    codes = rng.choice(["i8", "e4m3"])
    page = rng.choice([16, 32, 64, 128])
    block = rng.choice([b for b in (16, 32, 64, 128) if b <= page])
    if op == "cache8":
        seqs = _log_uniform(rng, 1, 64)
        tokens = seqs if rng.random() < 0.4 else max(seqs, _log_uniform(rng, 1, 8000))
        return {"op": op, "seqs": seqs, "tokens": tokens, "page": page, "block": block,
                "pool": rng.randint(50, 150) + 2 * tokens // page + 8 * seqs, "kv_heads": kv_heads, "dim": dim,
                "codes": codes, "window": rng.choice([0, 0, rng.randint(1, 200)]), "out": rng.choice(["f16", "f32"])}
    if op == "decode8":
        batch = _log_uniform(rng, 1, 64)
        return {"op": op, "batch": batch, "longest": _log_uniform(rng, 1, min(65000, 500000 // batch)), "page": page,
                "block": block, "heads": heads, "kv_heads": kv_heads, "dim": dim, "codes": codes}
    seqs = _log_uniform(rng, 1, 32)
    return {"op": op, "seqs": seqs, "beams": rng.randint(1, 8), "vocab": _log_uniform(rng, 1000, 127000),
            "history": _log_uniform(rng, 1, 1000)}


# -- inputs ----------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _host_gen(seed):
    return torch.Generator().manual_seed(int(seed) * 2 + 1)


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _lengths(total, parts, seed):
    """`parts` lengths of at least one that add up to `total`, most within a factor of two of each other."""
    w = 0.7 + 0.6 * torch.rand(parts, generator=_host_gen(seed), dtype=torch.float64)
    n = (w / w.sum() * (total - parts)).floor().to(torch.int64) + 1
    n[-1] += total - int(n.sum())
    return n.tolist()


def _starts(lens):
    return torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32).to(DEV)


def _ceil(a, b):
    return -(-a // b)


def _ints(values):
    return torch.as_tensor(values).to(torch.int32).to(DEV)


def _frequencies(c):
    """Angle of a position for each pair, FP64, and the factor on the turned values."""
    n, far = c["turned"], 4096  # trained up to 4096 positions
    i = torch.arange(0, n, 2, dtype=torch.float64)
    base = 10000.0
    if c["scaling"] == "ntk" and n > 2:
        base = base * c["factor"] ** (n / (n - 2))
    f = base ** (-i / n)
    if c["scaling"] == "linear":
        f = f / c["factor"]
    if c["scaling"] != "parts":
        return f, 1.0
    # Pairs that turn often within the trained length keep their frequency, slow ones are interpolated.
    keep = ((far * f / (2 * math.pi) - 1.0) / (32.0 - 1.0)).clamp(0, 1)
    return keep * f + (1 - keep) * f / c["factor"], 1.0 + 0.1 * math.log(c["factor"])


def _codes(g, kind, *shape):
    """Codes of about normally distributed values, the largest of them near the largest code."""
    x = _randn(g, *shape) * (LARGEST[kind] / 4)
    x = x.clamp(-LARGEST[kind], LARGEST[kind])
    return x.round().to(torch.int8) if kind == "i8" else x.to(CODES[kind])


def _scales(g, kind, *shape):
    """Scales under which the codes are values of a size of 0.7 to 1.4."""
    s = (0.7 + 0.7 * torch.rand(*shape, generator=g, device=DEV)) * 4 / LARGEST[kind]
    return s if kind == "i8" else torch.exp2(torch.log2(s).floor())


def _pools(g, c):
    shape = (c["pool"], c["kv_heads"], c["page"], c["dim"])
    scales = (c["pool"], c["kv_heads"], c["page"] // c["block"])
    return {"k_codes": _codes(g, c["codes"], *shape), "v_codes": _codes(g, c["codes"], *shape),
            "k_scales": _scales(g, c["codes"], *scales), "v_scales": _scales(g, c["codes"], *scales)}


def _table(pool, seqs, width, pages, seed):
    """Sequence s's page ids, of which it has pages[s], in an order without system; -1 behind them."""
    ids = torch.randperm(pool, generator=_host_gen(seed + 3))[:seqs * width].reshape(seqs, width)
    return _ints(torch.where(torch.arange(width)[None, :] < pages[:, None], ids, torch.full_like(ids, -1)))


def _before(c):
    """Tokens that a sequence of a `cache8` case has already, on the average: its window and more."""
    return 3 * c["page"] // 2 + 2 * c["window"]


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    s = {"case": c}
    if c["op"] == "rotary":
        dt = FLOATS[c["type"]]
        s["q"] = _randn(g, c["tokens"], c["heads"], c["dim"], dtype=dt)
        s["k"] = _randn(g, c["tokens"], c["kv_heads"], c["dim"], dtype=dt)
        s["positions"] = torch.randint(0, c["far"], (c["tokens"],), generator=_host_gen(seed)).to(DEV)
        f, s["amplitude"] = _frequencies(c)
        s["frequencies"] = f.to(DEV)
        if own:
            import compensated_fp32_projection_amd as cf
            s["frequencies"], s["amplitude"] = cf.rotary_frequencies(
                c["turned"], scaling=c["scaling"], factor=c["factor"], trained=4096)
    elif c["op"] == "cache8":
        new = _lengths(c["tokens"], c["seqs"], seed)
        lens = torch.tensor(_lengths(c["seqs"] * _before(c), c["seqs"], seed + 5)) - 1
        after = lens + torch.tensor(new)
        width = int(_ceil(int(after.max()), c["page"]))
        c["pool"] = max(c["pool"], c["seqs"] * width)
        s.update(_pools(g, c))
        s["table"] = _table(c["pool"], c["seqs"], width, (after + c["page"] - 1) // c["page"], seed)
        first = (after - c["window"]).clamp(min=0) if c["window"] else torch.zeros_like(after)
        n_read = (after - first).tolist()
        s.update(k=_randn(g, c["tokens"], c["kv_heads"], c["dim"]), v=_randn(g, c["tokens"], c["kv_heads"], c["dim"]),
                 cu=_starts(new), lens=_ints(lens), most=max(new), first=_ints(first), cu_read=_starts(n_read),
                 n_read=sum(n_read))
    elif c["op"] == "decode8":
        b, page = c["batch"], c["page"]
        lens = torch.randint(_ceil(c["longest"], 2), c["longest"] + 1, (b,), generator=_host_gen(seed))
        width = _ceil(c["longest"], page)
        c["pool"] = b * width + 3
        s.update(_pools(g, c))
        s["table"] = _table(c["pool"], b, width, (lens + page - 1) // page, seed)
        s.update(q=_randn(g, b, c["heads"], c["dim"]), lens=_ints(lens))
    else:
        rows = c["seqs"] * c["beams"]
        s["logits"] = _randn(g, rows, c["vocab"]) * 3
        s["scores"] = -20 * torch.rand(c["seqs"], c["beams"], generator=g, device=DEV)
        s["done"] = torch.rand(c["seqs"], c["beams"], generator=g, device=DEV) < 0.1
        s["history"] = torch.randint(0, c["vocab"], (rows, c["history"]), generator=g, device=DEV, dtype=torch.int32)
    if own and c["op"] in ("cache8", "decode8"):
        import compensated_fp32_projection_amd as cf
        s["cache"] = cf.Cache8(s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"])
    return s


# -- plain forms -------------------------------------------------------------------

def _turn(x, cos, sin, c):
    n = c["turned"]
    y, rest = x.float()[..., :n], x[..., n:]
    a, b = (y[..., :n // 2], y[..., n // 2:]) if c["layout"] == "half" else (y[..., 0::2], y[..., 1::2])
    p, q = a * cos - b * sin, b * cos + a * sin
    y = torch.cat([p, q], dim=-1) if c["layout"] == "half" else torch.stack([p, q], dim=-1).flatten(-2)
    return torch.cat([y.to(x.dtype), rest], dim=-1)


def _plain_rotary(s):
    c = s["case"]
    angle = s["positions"].double()[:, None] * s["frequencies"]  # 64 bits: far positions
    if c["transpose"]:
        angle = -angle
    cos, sin = (s["amplitude"] * t for t in (torch.cos(angle), torch.sin(angle)))
    cos, sin = cos.float()[:, None, :], sin.float()[:, None, :]
    return _turn(s["q"], cos, sin, c), _turn(s["k"], cos, sin, c)


def _to_grid(y, kind):
    """y (64 bits: values next to a border) rounded to the nearest code, ties to even."""
    if kind == "i8":
        return y.round()
    e = torch.frexp(y)[1].clamp(min=-5)  # steps of 2^-9 below 2^-6
    step = torch.ldexp(torch.ones_like(y), e - 4)
    return (y / step).round() * step


def _write(codes, scales, x, s):
    """New tokens into a pool, block by block of each sequence."""
    c = s["case"]
    kind, page, block, h, d = c["codes"], c["page"], c["block"], c["kv_heads"], c["dim"]
    lens, new = s["lens"].long(), (s["cu"][1:] - s["cu"][:-1]).long()
    nb = _ceil(s["most"], block) + 1
    start = (lens // block * block)[:, None] + torch.arange(nb, device=DEV)[None, :] * block  # [sequences, blocks]
    pos = start[:, :, None] + torch.arange(block, device=DEV)
    row = pos - lens[:, None, None]
    is_new, is_old = (row >= 0) & (row < new[:, None, None]), row < 0
    touched = is_new.any(dim=2)
    at = torch.where(is_new, s["cu"][:-1].long()[:, None, None] + row, torch.zeros_like(row))
    y = torch.where(is_new[..., None, None], x[at], torch.zeros((), device=DEV))  # [sequences, blocks, tokens, h, d]
    most = y.abs().amax(dim=(2, 4))  # [sequences, blocks, h]
    entry = (start // page).clamp(max=s["table"].shape[1] - 1)
    to = torch.gather(s["table"].long(), 1, entry).clamp(min=0)
    part = start % page // block
    had = scales[to, :, part]
    ma, ea = torch.frexp(most)
    if kind == "i8":
        fresh = (most / 127.0).clamp(min=LEAST_SCALE)
    else:
        e = torch.where(most > 0, ea - 9 + (ma > 0.875).int(), torch.full_like(ea, -126)).clamp(min=-126)
        fresh = torch.ldexp(torch.ones_like(most), e)
    mc, ec = torch.frexp(had * LARGEST[kind])
    up = (ea - ec + (ma > mc).int()).clamp(min=0)
    up = torch.where(most > 0, up, torch.zeros_like(up))
    begun = (start < lens[:, None])[..., None]
    up = torch.where(begun, up, torch.zeros_like(up))
    scale = torch.where(begun, torch.ldexp(had, up), fresh)
    codes_new = _to_grid(y.double() / scale.double()[:, :, None, :, None], kind)
    off, bits = pos % page, codes.view(torch.uint8)
    old = bits[to[:, :, None].expand_as(off), :, off].view(codes.dtype).double()
    codes_old = _to_grid(old * torch.ldexp(torch.ones_like(most), -up).double()[:, :, None, :, None], kind)
    value = torch.where(is_new[..., None, None], codes_new, codes_old).float()
    put = (is_new | is_old) & touched[:, :, None]
    bits[to[:, :, None].expand_as(off)[put], :, off[put]] = value[put].to(codes.dtype).view(torch.uint8)
    scales[to[touched], :, part[touched]] = scale[touched]


def _read(codes, scales, s):
    c = s["case"]
    tok = torch.arange(s["n_read"], device=DEV)
    seq = torch.searchsorted(s["cu_read"][1:].contiguous(), tok.to(torch.int32), right=True)
    pos = (s["first"][seq] + tok - s["cu_read"][seq]).long()
    page, off = s["table"][seq, pos // c["page"]].long(), pos % c["page"]
    got = codes.view(torch.uint8)[page, :, off].view(codes.dtype).float()
    return (got * scales[page, :, off // c["block"]][..., None]).to(FLOATS[c["out"]])


def _plain_cache8(s):
    _write(s["k_codes"], s["k_scales"], s["k"], s)
    _write(s["v_codes"], s["v_scales"], s["v"], s)
    lens = s["lens"] + (s["cu"][1:] - s["cu"][:-1])
    return lens, _read(s["k_codes"], s["k_scales"], s), _read(s["v_codes"], s["v_scales"], s)


def _plain_decode8(s):
    c = s["case"]
    b, h, hk, d = c["batch"], c["heads"], c["kv_heads"], c["dim"]
    ids = s["table"].long().clamp(min=0)

    def rows(codes, scales):  # [sequences, kv heads, tokens, dim]
        x = codes.view(torch.uint8)[ids].view(codes.dtype).float().reshape(*ids.shape, hk, -1, c["block"], d)
        x = x * scales[ids][..., None, None]
        return x.transpose(1, 2).reshape(b, hk, -1, d)

    k = rows(s["k_codes"], s["k_scales"])
    scores = torch.matmul(s["q"].reshape(b, hk, h // hk, d), k.transpose(2, 3).contiguous()) * (1.0 / math.sqrt(d))
    del k
    at = torch.arange(scores.shape[3], device=DEV)
    scores = torch.where(at < s["lens"][:, None, None, None], scores, torch.full_like(scores, -math.inf))
    m = scores.amax(dim=3, keepdim=True)
    p = torch.exp(scores - torch.where(m == -math.inf, torch.zeros_like(m), m))
    total = p.sum(dim=3, keepdim=True)
    o = torch.matmul(p, rows(s["v_codes"], s["v_scales"]))
    return (o / torch.where(total == 0, torch.ones_like(total), total)).reshape(b, h, d)


def _plain_beam(s):
    c = s["case"]
    n, beams, vocab = c["seqs"], c["beams"], c["vocab"]
    x = s["logits"].double()  # 64 bits: long sums, and candidates next to each other
    m = x.amax(dim=1, keepdim=True)
    x = (x - (m + torch.log(torch.exp(x - m).sum(dim=1, keepdim=True)))).reshape(n, beams, vocab)
    x = x + s["scores"].double()[:, :, None]
    # A finished beam offers itself alone, as its last token (0) again.
    none = torch.full((), -math.inf, dtype=torch.float64, device=DEV)
    x = torch.where(s["done"][:, :, None], none, x)
    x[:, :, 0] = torch.where(s["done"], s["scores"].double(), x[:, :, 0])
    x = x.reshape(n, beams * vocab)
    at = torch.arange(beams * vocab, device=DEV)
    best, where = [], []
    for _ in range(beams):
        top = x.amax(dim=1, keepdim=True)
        i = torch.where(x == top, at, torch.full_like(at, beams * vocab)).amin(dim=1, keepdim=True)
        best.append(top)
        where.append(i)
        x.scatter_(1, i, -math.inf)
    where = torch.cat(where, dim=1)
    rows = where // vocab + torch.arange(n, device=DEV)[:, None] * beams
    tokens = where % vocab
    done = s["done"].flatten()[rows] | (tokens == 0)
    return (rows.to(torch.int32), tokens.to(torch.int32), torch.cat(best, dim=1).float(), done,
            s["history"][rows.flatten()])


# -- one pass --------------------------------------------------------------------

def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if own:
        import compensated_fp32_projection_amd as cf
        if op == "rotary":
            return cf.rotary(s["q"], s["k"], s["frequencies"], s["positions"], layout=c["layout"],
                             amplitude=s["amplitude"], transpose=c["transpose"])
        if op == "cache8":
            lens = cf.cache8_append(s["k"], s["v"], s["cu"], s["cache"], s["table"], s["lens"])
            k, v = cf.cache8_read(s["cache"], s["table"], s["cu_read"], s["n_read"], first=s["first"],
                                  dtype=FLOATS[c["out"]])
            return lens, k, v
        if op == "decode8":
            return cf.attention8_decode(s["q"], s["cache"], s["table"], s["lens"])
        parents, tokens, scores, done = cf.beam_select(s["logits"], s["scores"], done=s["done"], eos=0)
        return parents, tokens, scores, done, cf.beam_reorder(s["history"], parents)
    return {"rotary": _plain_rotary, "cache8": _plain_cache8, "decode8": _plain_decode8, "beam": _plain_beam}[op](s)


# -- the same from the definitions, in FP64 -------------------------------------------

def _exact_rotary(c, s):
    f, amplitude = _frequencies(c)
    angle = s["positions"].double()[:, None] * f.to(DEV)
    turn = torch.polar(torch.full_like(angle, amplitude), -angle if c["transpose"] else angle)[:, None, :]
    n, outs = c["turned"], []
    for x in (s["q"].double(), s["k"].double()):
        first = torch.arange(n // 2, device=DEV) * (1 if c["layout"] == "half" else 2)
        second = first + (n // 2 if c["layout"] == "half" else 1)
        z = torch.complex(x[..., first], x[..., second]) * turn
        x[..., first], x[..., second] = z.real, z.imag
        outs.append(x)
    return tuple(outs)


def _nearest(y, kind):
    if kind == "i8":
        return torch.round(y)
    size = y.abs().clamp(min=2.0 ** -6)
    step = torch.exp2(torch.floor(torch.log2(size)) - 3)
    return torch.round(y / step) * step


def _exact_pool(c, s, codes, scales, x):
    """Each block written in turn; returns the pool's codes and scales in FP64."""
    codes, scales, x = codes.double(), scales.double(), x.double()
    table, lens, cu = s["table"].tolist(), s["lens"].tolist(), s["cu"].tolist()
    page, block, top = c["page"], c["block"], LARGEST[c["codes"]]
    for i in range(c["seqs"]):
        n = cu[i + 1] - cu[i]
        for start in range(lens[i] // block * block, lens[i] + n, block):
            p, o = table[i][start // page], start % page
            a, b = max(start, lens[i]), min(start + block, lens[i] + n)
            new = x[cu[i] + a - lens[i]:cu[i] + b - lens[i]].transpose(0, 1)  # [heads, tokens, dim]
            most = new.abs().amax(dim=(1, 2))
            if start >= lens[i]:
                scale = (most / 127).float().double() if c["codes"] == "i8" else \
                    torch.exp2(torch.ceil(torch.log2((most / top).clamp(min=LEAST_SCALE))))
                scale = scale.clamp(min=LEAST_SCALE)
            else:
                scale = scales[p, :, o // block].clone()
                while bool((small := (scale * top).float().double() < most).any()):
                    scale = torch.where(small, scale * 2, scale)
                there = codes[p, :, o:o + a - start]
                ratio = (scales[p, :, o // block] / scale)[:, None, None]
                codes[p, :, o:o + a - start] = _nearest(there * ratio, c["codes"])
            codes[p, :, o + a - start:o + b - start] = _nearest(new / scale[:, None, None], c["codes"])
            scales[p, :, o // block] = scale
    return codes, scales


def _exact_cache8(c, s):
    outs = [None]
    first, cu = s["first"].tolist(), s["cu_read"].tolist()
    for name in ("k", "v"):
        codes, scales = _exact_pool(s["case"], s, s[name + "_codes"], s[name + "_scales"], s[name])
        values = codes * scales.repeat_interleave(c["block"], dim=2)[..., None]
        values = values.transpose(1, 2)  # [pages, tokens, heads, dim]
        rows = []
        for i in range(c["seqs"]):
            pages = values[s["table"][i].long().clamp(min=0)].flatten(0, 1)
            rows.append(pages[first[i]:first[i] + cu[i + 1] - cu[i]])
        outs.append(torch.cat(rows))
    return tuple(outs)


def _exact_decode8(c, s):
    g, d = c["heads"] // c["kv_heads"], c["dim"]
    out = torch.zeros(c["batch"], c["heads"], d, dtype=torch.float64, device=DEV)
    for b, n in enumerate(s["lens"].tolist()):
        ids = s["table"][b, :_ceil(n, c["page"])].long()
        k, v = ((s[x + "_codes"][ids].double() * s[x + "_scales"][ids].double().repeat_interleave(c["block"], dim=2)[..., None])
                .transpose(0, 1).reshape(c["kv_heads"], -1, d)[:, :n] for x in ("k", "v"))
        q = s["q"][b].double().reshape(c["kv_heads"], g, d)
        w = torch.softmax((q @ k.transpose(1, 2).contiguous()) / math.sqrt(d), dim=2)
        out[b] = (w @ v).reshape(c["heads"], d)
    return out


def _exact_beam(c, s):
    best = []
    logp = torch.log_softmax(s["logits"].double(), dim=1)
    for i in range(c["seqs"]):
        offers = []
        for j in range(c["beams"]):
            score = s["scores"][i, j].double()
            offers.append(score[None] if bool(s["done"][i, j]) else
                          score + logp[i * c["beams"] + j].sort(descending=True)[0][:c["beams"]])
        best.append(torch.cat(offers).sort(descending=True)[0][:c["beams"]])
    return None, None, torch.stack(best), None, None


def exact(case, seed):
    s = prepare(case, seed)
    return {"rotary": _exact_rotary, "cache8": _exact_cache8, "decode8": _exact_decode8,
            "beam": _exact_beam}[case["op"]](case, s)


# -- what one pass cannot do without ----------------------------------------------------

def work(case):
    c = case
    if c["op"] == "rotary":
        size = 2 if c["type"] == "f16" else 4
        values = c["tokens"] * (c["heads"] + c["kv_heads"])
        return {"bytes": 2 * size * values * c["dim"] + 8 * c["tokens"], "flops": 3 * values * c["turned"]}
    if c["op"] == "cache8":
        token = 2 * c["kv_heads"] * c["dim"]  # codes of K and V
        read = c["window"] * c["seqs"] if c["window"] else _before(c) * c["seqs"] + c["tokens"]
        # FP32 read and codes written; codes read and values written
        return {"bytes": 5 * token * c["tokens"] + (5 if c["out"] == "f32" else 3) * token * read, "flops": 0}
    if c["op"] == "decode8":
        tokens = 0.75 * c["longest"] * c["batch"]
        return {"bytes": tokens * 2 * c["kv_heads"] * (c["dim"] + 4 / c["block"]) + 8 * c["batch"] * c["heads"] * c["dim"],
                "flops": 4 * tokens * c["heads"] * c["dim"]}
    rows = c["seqs"] * c["beams"]
    return {"bytes": 4 * rows * c["vocab"] + 8 * rows * c["history"], "flops": 3 * rows * c["vocab"]}
