"""Workloads of the attention and cache operators, in plain torch and through the library.

``own`` selects what ``run`` computes: False, the operators written out in
elementary torch operations (FP32); True, the library's calls on the same
state.  ``exact`` gives the same outputs from the definitions in FP64.

The operators:

* ``prompt``: causal attention over packed prompts, grouped heads;
* ``decode``: one new token per sequence against a paged cache whose first
  pages all sequences of the batch share;
* ``append``: pages reserved for new tokens, and the tokens' K and V written
  into them;
* ``fork``: children of running sequences that share the whole pages and get
  a copy of the last, partly filled one;
* ``compact``: pages of ended sequences freed, the live pages moved to the
  front of the pool and the tables rewritten.

Cache pools are [pages, kv heads, tokens of a page, head size]; a table row
holds a sequence's page ids in order, -1 where it has none; ``refs`` counts
the tables' uses of each page, 0 for a free one.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f16": torch.float16, "f32": torch.float32}


# -- cases ---------------------------------------------------------------------

def listed():
    return [
        # A short question through a small encoder-sized layer: latency.
        {"name": "prompt_37_mha64_f32", "op": "prompt", "seqs": 1, "tokens": 37, "past": 0, "heads": 12,
         "kv_heads": 12, "dim": 64, "kv": "f32", "head_major": True},
        # The QKV projection workload's 512 tokens, heads as the rotary packing leaves them, as one prompt.
        {"name": "prompt_512_mha64_f32", "op": "prompt", "seqs": 1, "tokens": 512, "past": 0, "heads": 12,
         "kv_heads": 12, "dim": 64, "kv": "f32", "head_major": True},
        # Prompts of uneven lengths packed together, some of them going on from cached tokens.
        {"name": "prompt_8x750_gqa128_f16", "op": "prompt", "seqs": 8, "tokens": 6001, "past": 301, "heads": 32,
         "kv_heads": 8, "dim": 128, "kv": "f16", "head_major": False},
        # One long prompt of the feed-forward workload's 8192 rows.
        {"name": "prompt_8192_gqa128_f32", "op": "prompt", "seqs": 1, "tokens": 8192, "past": 0, "heads": 32,
         "kv_heads": 8, "dim": 128, "kv": "f32", "head_major": False},
        # One sequence, a few pages, nothing shared: latency.
        {"name": "decode_1_own130_f16", "op": "decode", "batch": 1, "shared": 0, "own": 130, "page": 16, "heads": 32,
         "kv_heads": 8, "dim": 128, "kv": "f16"},
        # Samples of one prompt on FP32 pages, heads not grouped.
        {"name": "decode_12_shared2000_f32", "op": "decode", "batch": 12, "shared": 2000, "own": 333, "page": 16,
         "heads": 12, "kv_heads": 12, "dim": 64, "kv": "f32"},
        # A serving batch behind one long system prompt.
        {"name": "decode_32_shared65536_f16", "op": "decode", "batch": 32, "shared": 65536, "own": 1000, "page": 64,
         "heads": 32, "kv_heads": 8, "dim": 128, "kv": "f16"},
        # One step's new token of each sequence.
        {"name": "append_64x1_f16", "op": "append", "seqs": 64, "tokens": 64, "page": 16, "pool": 2048,
         "kv_heads": 8, "dim": 128, "kv": "f16"},
        # Prompts written into the cache.
        {"name": "append_4x2048_f16", "op": "append", "seqs": 4, "tokens": 8190, "page": 64, "pool": 512,
         "kv_heads": 8, "dim": 128, "kv": "f16"},
        # A few samples of one sequence.
        {"name": "fork_4_f16", "op": "fork", "seqs": 1, "children": 4, "page": 16, "pool": 256, "kv_heads": 8,
         "dim": 128, "kv": "f16"},
        # Beams of many sequences.
        {"name": "fork_256_f16", "op": "fork", "seqs": 32, "children": 256, "page": 64, "pool": 1024, "kv_heads": 8,
         "dim": 128, "kv": "f16"},
        # A half-empty pool made dense.
        {"name": "compact_1024_f16", "op": "compact", "seqs": 40, "ended": 16, "page": 64, "pool": 1024,
         "kv_heads": 8, "dim": 128, "kv": "f16"},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "decode", "decode", "append", "fork", "compact"])
    heads, kv_heads, dim = rng.choice([(12, 12, 64), (32, 8, 128), (16, 2, 128), (8, 8, 80), (14, 2, 64), (9, 3, 40)])
    kv = rng.choice(["f16", "f32"])
    if op == "prompt":
        tokens = _log_uniform(rng, 1, 8000)
        return {"op": op, "seqs": rng.randint(1, min(8, tokens)), "tokens": tokens,
                "past": rng.choice([0, 0, rng.randint(1, 700)]), "heads": heads, "kv_heads": kv_heads, "dim": dim,
                "kv": kv, "head_major": rng.random() < 0.5}
    page = rng.choice([16, 32, 64, 128])
    if op == "decode":
        shared = rng.choice([0, _log_uniform(rng, 16, 60000)])
        return {"op": op, "batch": _log_uniform(rng, 1, 32), "shared": shared, "own": _log_uniform(rng, 1, 1000),
                "page": page, "heads": heads, "kv_heads": kv_heads, "dim": dim, "kv": kv}
    if op == "append":
        seqs = _log_uniform(rng, 1, 64)
        tokens = seqs if rng.random() < 0.4 else max(seqs, _log_uniform(rng, 1, 8000))
        return {"op": op, "seqs": seqs, "tokens": tokens, "page": page,
                "pool": rng.randint(300, 600) + 2 * tokens // page + 8 * seqs, "kv_heads": kv_heads, "dim": dim,
                "kv": kv}
    page = rng.choice([16, 32, 64])
    if op == "fork":
        children = _log_uniform(rng, 1, 200)
        return {"op": op, "seqs": rng.randint(1, 16), "children": children, "page": page,
                "pool": rng.randint(400, 900), "kv_heads": kv_heads, "dim": dim, "kv": kv}
    seqs = rng.randint(2, 40)
    return {"op": op, "seqs": seqs, "ended": rng.randint(1, seqs - 1), "page": page, "pool": rng.randint(200, 1000),
            "kv_heads": kv_heads, "dim": dim, "kv": kv}


# -- inputs ----------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _lengths(total, parts, seed):
    """`parts` lengths of at least one that add up to `total`, most within a factor of two of each other."""
    r = torch.Generator().manual_seed(int(seed) * 2 + 1)
    w = 0.7 + 0.6 * torch.rand(parts, generator=r, dtype=torch.float64)
    n = (w / w.sum() * (total - parts)).floor().to(torch.int64) + 1
    n[-1] += total - int(n.sum())
    return n.tolist()


def _starts(lens):
    return torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32).to(DEV)


def _pool(g, c):
    shape = (c["pool"], c["kv_heads"], c["page"], c["dim"])
    return _randn(g, *shape, dtype=TYPES[c["kv"]]), _randn(g, *shape, dtype=TYPES[c["kv"]])


def _ceil(a, b):
    return -(-a // b)


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    s = {"case": c}
    if c["op"] == "prompt":
        lq = _lengths(c["tokens"], c["seqs"], seed)
        past = _lengths(c["past"] + c["seqs"], c["seqs"], seed + 7)  # each sequence's cached tokens, plus one
        lk = [a + b - 1 for a, b in zip(lq, past)]
        tq, tk = sum(lq), sum(lk)
        dt = TYPES[c["kv"]]
        if c["head_major"]:
            q = _randn(g, c["heads"], tq, c["dim"]).transpose(0, 1)
            k = _randn(g, c["kv_heads"], tk, c["dim"], dtype=dt).transpose(0, 1)
            v = _randn(g, c["kv_heads"], tk, c["dim"], dtype=dt).transpose(0, 1)
        else:
            q = _randn(g, tq, c["heads"], c["dim"])
            k = _randn(g, tk, c["kv_heads"], c["dim"], dtype=dt)
            v = _randn(g, tk, c["kv_heads"], c["dim"], dtype=dt)
        s.update(q=q, k=k, v=v, cu_q=_starts(lq), cu_k=_starts(lk), max_q=max(lq), max_k=max(lk))
    elif c["op"] == "decode":
        n_shared = c["shared"] // c["page"]  # whole pages; the prefix's last tokens are each sequence's own
        tail = c["shared"] % c["page"]
        b = c["batch"]
        r = torch.Generator().manual_seed(int(seed) * 2 + 1)
        own_lens = tail + torch.randint(_ceil(c["own"], 2), c["own"] + 1, (b,), generator=r)
        width = _ceil(tail + c["own"], c["page"])
        pool = n_shared + b * width + 5
        c["pool"] = pool
        k_pages, v_pages = _pool(g, c)
        ids = torch.randperm(pool, generator=r).to(torch.int32)
        own_ids = ids[n_shared:n_shared + b * width].reshape(b, width)
        used = torch.arange(width)[None, :] * c["page"] < own_lens[:, None]
        own_ids = torch.where(used, own_ids, torch.full_like(own_ids, -1))
        table = torch.cat([ids[:n_shared][None, :].expand(b, -1), own_ids], dim=1)
        s.update(q=_randn(g, b, c["heads"], c["dim"]), k_pages=k_pages, v_pages=v_pages,
                 table=table.contiguous().to(DEV), shared_pages=n_shared,
                 lens=(own_lens + n_shared * c["page"]).to(torch.int32).to(DEV))
    elif c["op"] == "append":
        new = _lengths(c["tokens"], c["seqs"], seed)
        r = torch.Generator().manual_seed(int(seed) * 2 + 1)
        lens = torch.randint(0, 3 * c["page"], (c["seqs"],), generator=r)
        width = 3 + _ceil(2 * c["tokens"] // c["seqs"] + c["seqs"], c["page"])  # room for the longest
        k_pages, v_pages = _pool(g, c)
        ids = torch.randperm(c["pool"], generator=r).to(torch.int32)[:c["seqs"] * width].reshape(c["seqs"], width)
        held = torch.arange(width)[None, :] < (lens[:, None] + c["page"] - 1) // c["page"]
        table = torch.where(held, ids, torch.full_like(ids, -1))
        refs = torch.zeros(c["pool"], dtype=torch.int32)
        refs[table[table >= 0].long()] = 1
        s.update(k=_randn(g, c["tokens"], c["kv_heads"], c["dim"]), v=_randn(g, c["tokens"], c["kv_heads"], c["dim"]),
                 cu=_starts(new), lens=lens.to(torch.int32).to(DEV), table=table.contiguous().to(DEV),
                 refs=refs.to(DEV), k_pages=k_pages, v_pages=v_pages)
    else:
        r = torch.Generator().manual_seed(int(seed) * 2 + 1)
        n, pool = c["seqs"], c["pool"]
        spare = c["children"] if c["op"] == "fork" else pool // 4  # pages that stay free
        width = max(1, (pool - spare) // n)
        k_pages, v_pages = _pool(g, c)
        lens = torch.randint(1, width * c["page"] + 1, (n,), generator=r)
        ids = torch.randperm(pool, generator=r)[:n * width].to(torch.int32).reshape(n, width)
        used = torch.arange(width)[None, :] * c["page"] < lens[:, None]
        table = torch.where(used, ids, torch.full_like(ids, -1))
        refs = torch.zeros(pool, dtype=torch.int32)
        refs[table[table >= 0].long()] = 1
        s.update(k_pages=k_pages, v_pages=v_pages, lens=lens.to(torch.int32).to(DEV), refs=refs.to(DEV),
                 table=table.contiguous().to(DEV))
        if c["op"] == "fork":
            s["parents"] = torch.randint(0, n, (c["children"],), generator=r).to(torch.int32).to(DEV)
        else:
            gone = torch.randperm(n, generator=r)
            s["ended"] = s["table"][gone[:c["ended"]].to(DEV)].contiguous()
            s["running"] = s["table"][gone[c["ended"]:].to(DEV)].contiguous()
    return s


# -- plain forms -------------------------------------------------------------------

def _padded(cu, longest):
    """Indices [sequences, longest] of each sequence's tokens in the packed rows, and which of them exist."""
    at = torch.arange(longest, device=cu.device)
    start, n = cu[:-1].long(), (cu[1:] - cu[:-1]).long()
    valid = at[None, :] < n[:, None]
    return torch.where(valid, start[:, None] + at[None, :], torch.zeros_like(start)[:, None]), valid, n


def _softmax_product(scores, seen, v):
    """Rows of softmax(scores over the seen keys) @ v; zero where a row sees none."""
    scores = torch.where(seen, scores, torch.full_like(scores, -math.inf))
    m = scores.amax(dim=-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(scores - m)
    total = p.sum(dim=-1, keepdim=True)
    return torch.matmul(p, v) / torch.where(total == 0, torch.ones_like(total), total)


def _plain_prompt(s):
    c = s["case"]
    h, hk, d = c["heads"], c["kv_heads"], c["dim"]
    iq, vq, nq = _padded(s["cu_q"], s["max_q"])
    ik, vk, nk = _padded(s["cu_k"], s["max_k"])
    q = s["q"].float()[iq].permute(0, 2, 1, 3)  # [sequences, heads, rows, dim]
    k = s["k"].float()[ik].permute(0, 2, 1, 3)
    v = s["v"].float()[ik].permute(0, 2, 1, 3)
    b, lq, lk = q.shape[0], q.shape[2], k.shape[2]
    q = q.reshape(b, hk, h // hk * lq, d)
    scores = torch.matmul(q, k.transpose(2, 3).contiguous()) * (1.0 / math.sqrt(d))
    row = torch.arange(lq, device=DEV)[None, :, None] + (nk - nq)[:, None, None]
    seen = (torch.arange(lk, device=DEV)[None, None, :] <= row) & vk[:, None, :]
    scores = scores.reshape(b, h, lq, lk)
    o = _softmax_product(scores, seen[:, None], v.repeat_interleave(h // hk, dim=1).contiguous())
    out = torch.zeros(c["tokens"], h, d, dtype=torch.float32, device=DEV)
    out[iq[vq]] = o.permute(0, 2, 1, 3)[vq]
    return out


def _plain_decode(s):
    c = s["case"]
    b, h, hk, d, n = c["batch"], c["heads"], c["kv_heads"], c["dim"], s["shared_pages"]
    g = h // hk
    q = s["q"].reshape(b, hk, g, d)
    shared, mine = s["table"][0, :n].long(), s["table"][:, n:].long().clamp(min=0)

    def rows(pages, ids):  # pages of ids [..., w] as [..., kv heads, w * page, dim]
        x = pages[ids].float().transpose(-4, -3)
        return x.reshape(*x.shape[:-3], x.shape[-3] * x.shape[-2], d)

    scale = 1.0 / math.sqrt(d)
    ks, vs = rows(s["k_pages"], shared), rows(s["v_pages"], shared)
    ko, vo = rows(s["k_pages"], mine), rows(s["v_pages"], mine)
    first = torch.matmul(q.permute(1, 0, 2, 3).reshape(hk, b * g, d), ks.transpose(1, 2).contiguous())
    first = first.reshape(hk, b, g, -1).transpose(0, 1)
    scores = torch.cat([first, torch.matmul(q, ko.transpose(2, 3).contiguous())], dim=3) * scale
    at = torch.arange(scores.shape[3], device=DEV)
    scores = torch.where(at < s["lens"][:, None, None, None], scores, torch.full_like(scores, -math.inf))
    m = scores.amax(dim=3, keepdim=True)
    p = torch.exp(scores - torch.where(m == -math.inf, torch.zeros_like(m), m))
    total = p.sum(dim=3, keepdim=True)
    cut = n * c["page"]
    o = torch.matmul(p[..., :cut].transpose(0, 1).reshape(hk, b * g, cut).contiguous(), vs)
    o = o.reshape(hk, b, g, d).transpose(0, 1) + torch.matmul(p[..., cut:].contiguous(), vo)
    return (o / torch.where(total == 0, torch.ones_like(total), total)).reshape(b, h, d)


def _take_free(refs, wanted):
    """Page ids for the True places of `wanted` in order: the lowest free pages; -1 when there are no more."""
    free = torch.nonzero(refs <= 0).flatten()
    rank = wanted.flatten().long().cumsum(0) - 1
    got = torch.nn.functional.pad(free, (0, 1), value=-1)[rank.clamp(min=0, max=free.numel())]
    got = torch.where(wanted.flatten(), got, torch.full_like(got, -1))
    return got.reshape(wanted.shape).to(torch.int32)


def _plain_append(s):
    c = s["case"]
    page, table, refs = c["page"], s["table"], s["refs"]
    new = s["cu"][1:] - s["cu"][:-1]
    at = torch.arange(table.shape[1], device=DEV)[None, :]
    wanted = (at * page < (s["lens"] + new)[:, None]) & (table < 0)
    got = _take_free(refs, wanted)
    table = torch.where(wanted, got, table)
    refs = refs.clone()
    refs[got[got >= 0].long()] = 1
    tok = torch.arange(c["tokens"], device=DEV)
    seq = torch.searchsorted(s["cu"][1:].contiguous(), tok.to(torch.int32), right=True)
    pos = (s["lens"][seq] + tok - s["cu"][seq]).long()
    to = table[seq, pos // page].long()
    s["k_pages"][to, :, pos % page] = s["k"].to(s["k_pages"].dtype)
    s["v_pages"][to, :, pos % page] = s["v"].to(s["v_pages"].dtype)
    return table, refs, s["lens"] + new, s["k_pages"], s["v_pages"]


def _plain_fork(s):
    c = s["case"]
    page, refs = c["page"], s["refs"].clone()
    lens = s["lens"][s["parents"].long()]
    old = s["table"][s["parents"].long()]
    whole, part = (lens // page)[:, None], (lens % page != 0)[:, None]
    at = torch.arange(old.shape[1], device=DEV)[None, :]
    last = (at == whole) & part
    got = _take_free(refs, last)
    table = torch.where(at < whole, old, got)
    kept = old[(at < whole) & (old >= 0)].long()
    refs.index_put_((kept,), torch.ones_like(kept, dtype=torch.int32), accumulate=True)
    refs[got[got >= 0].long()] = 1
    src, dst = old[last & (got >= 0)].long(), got[last & (got >= 0)].long()
    s["k_pages"][dst] = s["k_pages"][src]
    s["v_pages"][dst] = s["v_pages"][src]
    return table, refs, lens, s["k_pages"], s["v_pages"]


def _plain_compact(s):
    refs = s["refs"].clone()
    gone = s["ended"][s["ended"] >= 0].long()
    refs.index_put_((gone,), torch.full_like(gone, -1, dtype=torch.int32), accumulate=True)
    live = refs > 0
    n = live.sum()
    at = torch.arange(refs.numel(), device=DEV)
    src = torch.nonzero(live & (at >= n)).flatten()
    dst = torch.nonzero(~live & (at < n)).flatten()
    s["k_pages"][dst] = s["k_pages"][src]
    s["v_pages"][dst] = s["v_pages"][src]
    to = at.clone()
    to[src] = dst
    refs[dst] = refs[src]
    refs = torch.where(at < n, refs, torch.zeros_like(refs))
    table = torch.where(s["running"] >= 0, to[s["running"].long().clamp(min=0)].to(torch.int32), s["running"])
    return table, refs, n.to(torch.int32).reshape(1), s["k_pages"], s["v_pages"]


# -- one pass --------------------------------------------------------------------

def run(state):
    s, op = state, state["case"]["op"]
    if own:
        import compensated_fp32_projection_amd as cf
        if op == "prompt":
            return cf.attention_prompt(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"])
        if op == "decode":
            return cf.attention_decode(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"],
                                       shared_pages=s["shared_pages"])
        if op == "append":
            table, refs = cf.cache_reserve(s["table"], s["lens"], s["refs"], s["cu"], page=s["case"]["page"])
            lens = cf.cache_append(s["k"], s["v"], s["cu"], s["k_pages"], s["v_pages"], table, s["lens"])
            return table, refs, lens, s["k_pages"], s["v_pages"]
        if op == "fork":
            table, refs, lens = cf.cache_fork(s["k_pages"], s["v_pages"], s["table"], s["lens"], s["refs"],
                                              s["parents"])
            return table, refs, lens, s["k_pages"], s["v_pages"]
        refs = cf.cache_free(s["ended"], s["refs"])
        table, refs, n = cf.cache_compact(s["k_pages"], s["v_pages"], s["running"], refs)
        return table, refs, n, s["k_pages"], s["v_pages"]
    return {"prompt": _plain_prompt, "decode": _plain_decode, "append": _plain_append, "fork": _plain_fork,
            "compact": _plain_compact}[op](s)


# -- the same from the definitions, in FP64 -------------------------------------------

def _exact_rows(q, k, v, limits):
    """Attention of rows q [rows, d] over keys k, v [n, d], row i seeing keys below limits[i]."""
    e = (q @ k.t()) / math.sqrt(q.shape[1])
    e.masked_fill_(torch.arange(k.shape[0], device=k.device)[None, :] >= limits[:, None], -math.inf)
    w = torch.softmax(e, dim=1)
    return torch.where(limits[:, None] > 0, w @ v, torch.zeros((), dtype=q.dtype, device=q.device))


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "prompt":
        cu_q, cu_k = s["cu_q"].tolist(), s["cu_k"].tolist()
        out = torch.zeros(c["tokens"], c["heads"], c["dim"], dtype=torch.float64, device=DEV)
        for i in range(c["seqs"]):
            a, b, a2, b2 = cu_q[i], cu_q[i + 1], cu_k[i], cu_k[i + 1]
            limits = (torch.arange(b - a, device=DEV) + (b2 - a2) - (b - a) + 1).clamp(0, b2 - a2)
            for h in range(c["heads"]):
                kh = h // (c["heads"] // c["kv_heads"])
                out[a:b, h] = _exact_rows(s["q"][a:b, h].double(), s["k"][a2:b2, kh].double(),
                                          s["v"][a2:b2, kh].double(), limits)
        return out
    if c["op"] == "decode":
        g, page = c["heads"] // c["kv_heads"], c["page"]
        out = torch.zeros(c["batch"], c["heads"], c["dim"], dtype=torch.float64, device=DEV)
        lens = s["lens"].tolist()
        for b in range(c["batch"]):
            n = lens[b]
            ids = s["table"][b, :_ceil(n, page)].long()
            for kh in range(c["kv_heads"]):
                k = s["k_pages"][ids, kh].reshape(-1, c["dim"])[:n].double()
                v = s["v_pages"][ids, kh].reshape(-1, c["dim"])[:n].double()
                rows = slice(kh * g, kh * g + g)
                out[b, rows] = _exact_rows(s["q"][b, rows].double(), k, v, torch.full((g,), n, device=DEV))
        return out
    table, refs = s["table"].tolist(), s["refs"].tolist()
    lens = s["lens"].tolist()
    page = c["page"]
    if c["op"] == "append":
        free = iter([i for i, r in enumerate(refs) if r <= 0])
        cu = s["cu"].tolist()
        to, off = [], []
        for i, row in enumerate(table):
            end = lens[i] + cu[i + 1] - cu[i]
            for j in range(_ceil(end, page)):
                if row[j] < 0:
                    row[j] = next(free)
                    refs[row[j]] = 1
            to += [row[p // page] for p in range(lens[i], end)]
            off += [p % page for p in range(lens[i], end)]
            lens[i] = end
        to, off = torch.tensor(to, device=DEV), torch.tensor(off, device=DEV)
        pages = []
        for x, into in ((s["k"], s["k_pages"]), (s["v"], s["v_pages"])):
            y = into.double()
            y[to, :, off] = x.double()
            pages.append(y)
        return None, None, None, pages[0], pages[1]
    moves = {}
    if c["op"] == "fork":
        free = iter([i for i, r in enumerate(refs) if r <= 0])
        for p in s["parents"].tolist():
            if lens[p] % page:
                moves[next(free)] = table[p][lens[p] // page]
    else:
        for row in s["ended"].tolist():
            for p in row:
                if p >= 0:
                    refs[p] -= 1
        n = sum(r > 0 for r in refs)
        high = [i for i, r in enumerate(refs) if r > 0 and i >= n]
        moves = dict(zip([i for i, r in enumerate(refs) if r <= 0 and i < n], high))
    pages = [x.double() for x in (s["k_pages"], s["v_pages"])]
    before = [x.clone() for x in pages]
    for dst, src in moves.items():
        for x, y in zip(pages, before):
            x[dst] = y[src]
    return None, None, None, pages[0], pages[1]


# -- what one pass cannot do without ----------------------------------------------------

def work(case):
    c = case
    size = 2 if c["kv"] == "f16" else 4
    kv_row = 2 * size * c["kv_heads"] * c["dim"]  # K and V of one token
    if c["op"] == "prompt":
        tq, tk = c["tokens"], c["tokens"] + c["past"]
        # sequences of about equal lengths, each row seeing its past and itself
        pairs = tq * (c["past"] / c["seqs"] + (tq / c["seqs"] + 1) / 2)
        return {"bytes": 8 * tq * c["heads"] * c["dim"] + tk * kv_row, "flops": 4 * c["dim"] * c["heads"] * pairs}
    if c["op"] == "decode":
        mine = c["shared"] % c["page"] + 0.75 * c["own"]
        shared = c["shared"] // c["page"] * c["page"]
        return {"bytes": (shared + c["batch"] * mine) * kv_row + 8 * c["batch"] * c["heads"] * c["dim"],
                "flops": 4 * c["dim"] * c["heads"] * c["batch"] * (shared + mine)}
    if c["op"] == "append":
        return {"bytes": c["tokens"] * (8 * c["kv_heads"] * c["dim"] + kv_row) + 8 * c["pool"], "flops": 0}
    page_bytes = kv_row * c["page"]
    if c["op"] == "fork":
        return {"bytes": 2 * c["children"] * page_bytes * (1 - 1 / c["page"]) + 8 * c["pool"], "flops": 0}
    # about half of the table's entries are in use; of n live pages, (pool - n) / pool lie at or above n
    held = c["seqs"] * max(1, (c["pool"] - c["pool"] // 4) // c["seqs"]) * 0.5
    live = held * (c["seqs"] - c["ended"]) / c["seqs"]
    return {"bytes": 2 * live * (c["pool"] - live) / c["pool"] * page_bytes + 12 * c["pool"], "flops": 0}
