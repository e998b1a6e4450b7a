"""Packed sequences and paged caches: the cases, the plain forms, and the calls a user makes.

A serving step holds the new tokens of all its requests packed one after another, and their
keys and values in pages of a pool that the requests share.  Four passes:

* pages:  finished requests give their pages back, the others take pages for their new
  tokens; block tables, positions and the slot of every token come out;
* rope:   a projection's output: queries and keys normalised for each head and rotated by
  their position, queries to packed rows, keys and values to their slots of the pool;
* prompt: causal attention of whole prompts over themselves, packed, grouped query heads;
* paged:  causal attention of each request's new tokens (one in decode, a chunk of a prompt)
  over its pages.

Shapes are those of the decode layers in dv_inputs.py (32/64/72/96 heads of 128, lengths 512
to 2048, the tiny binary32 layer with 8 heads of 32) and generic longer and grouped ones.
"""
import math
import random

import numpy as np
import torch

own = False

_TORCH = {"f32": torch.float32, "f16": torch.float16}
_ESIZE = {"f32": 4, "f16": 2}


# ------------------------------------------------------------------------------------------
# cases


def _case(name, op, B, H, Hkv, D, tok, ctx, dtype="f16", **kw):
    """B requests of up to tok new tokens after up to ctx cached ones."""
    c = {"name": name, "op": op, "B": B, "H": H, "Hkv": Hkv, "D": D, "tok": tok, "ctx": ctx,
         "dtype": dtype, "ragged": False, "singles": 0, "page": 0, "src": "f16", "norm": "",
         "rot": 0, "layout": "", "scaling": "", "factor": 1.0}
    c.update(kw)
    return c


def listed():
    return [
        # a decode step of a running batch, a sixth of its requests just finished: latency
        _case("pages_step", "pages", 48, 32, 32, 128, 1, 4095, ragged=True, page=16),
        # a large batch of prompt chunks
        _case("pages_chunks", "pages", 256, 64, 8, 128, 512, 8192, ragged=True, page=32),
        # one new token a request of the 6.7B-shaped layer, from a binary32 projection: latency
        _case("rope_token", "rope", 8, 32, 32, 128, 1, 575, page=16, src="f32", rot=128,
              layout="half", norm="rms"),
        # ragged chunks, part of the head rotated, interleaved, at far scaled positions
        _case("rope_far", "rope", 5, 72, 72, 128, 333, 120000, ragged=True, page=64, rot=64,
              layout="pairs", scaling="ramp", factor=8.0),
        # long prompts of grouped heads, normalised and rotated
        _case("rope_prompt", "rope", 8, 64, 8, 128, 2048, 0, page=16, src="f32", rot=128,
              layout="half", norm="rms", scaling="linear", factor=4.0),
        # a few short prompts of the tiny binary32 layer
        _case("prompt_tiny", "prompt", 3, 8, 8, 32, 300, 0, "f32", ragged=True),
        # a batch of prompts of different lengths, grouped heads
        _case("prompt_packed", "prompt", 12, 64, 8, 128, 2048, 0, ragged=True),
        # two long prompts
        _case("prompt_long", "prompt", 2, 32, 4, 128, 16384, 0),
        # one decode token at the 6.7B-shaped layer
        _case("paged_token", "paged", 1, 32, 32, 128, 1, 575, page=16),
        # a decode batch of grouped heads with ragged lengths
        _case("paged_decode", "paged", 64, 64, 8, 128, 1, 8191, ragged=True, page=16),
        # a mixed step at the 175B shape: most requests decode, some bring a chunk of a prompt
        _case("paged_mixed", "paged", 24, 96, 96, 128, 511, 2048, ragged=True, singles=16,
              page=32),
        # the next chunk of one long prompt
        _case("paged_chunk", "paged", 1, 64, 8, 128, 2048, 30000, page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(["pages", "rope", "prompt", "prompt", "paged", "paged", "paged"])
        dtype = "f16" if op == "pages" else rng.choice(["f16", "f16", "f16", "f32"])
        D = rng.choice([64, 128, 128])
        Hkv = _log(rng, 1, 96)
        G = rng.choice([1, 1, 2, 3, 4, 8])
        page = rng.choice([16, 32, 64, 128])
        c = _case("", op, _log(rng, 1, 64), Hkv * G, Hkv, D, 1, 0, dtype,
                  ragged=rng.random() < 0.7)
        if op == "pages":
            c.update(B=_log(rng, 1, 256), tok=_log(rng, 1, 512), ctx=_log(rng, 1, 8192))
        elif op == "rope":
            rot = rng.choice([D, D, D // 2, D // 4, 0])
            c.update(tok=_log(rng, 1, 2048), ctx=rng.choice([0, _log(rng, 1, 120000)]),
                     src=rng.choice(["f16", "f32"]), rot=rot,
                     layout=rng.choice(["half", "pairs"]), norm=rng.choice(["", "rms", "layer"]),
                     scaling=rng.choice(["", "linear", "base", "ramp"]))
            c["factor"] = rng.choice([2.0, 4.0, 8.0]) if c["scaling"] else 1.0
        elif op == "prompt":
            c.update(B=_log(rng, 1, 16), tok=_log(rng, 1, 16384))
        else:
            kind = rng.choice(["decode", "chunk", "mixed"])
            c.update(ctx=_log(rng, 1, 32768))
            if kind != "decode":
                c.update(tok=_log(rng, 2, 2048), B=_log(rng, 1, 24))
            if kind == "mixed":
                c.update(singles=c["B"] // 2)
        if dtype == "f32":
            # the tiny layer's kind: few narrow heads, short texts
            c.update(D=rng.choice([32, 32, 64]), B=min(c["B"], 8), ctx=min(c["ctx"], 2048),
                     tok=min(c["tok"], 512), H=min(Hkv, 8) * G, Hkv=min(Hkv, 8))
            c["rot"] = min(c["rot"], c["D"])
        if op != "prompt":
            c["page"] = page
        w = work(c)
        if (c["H"] <= 128 and _cost(c) <= most and w["flops"] <= 4e12
                and sum(_toks(c)) * c["H"] * c["D"] <= 3e8
                and (op == "rope" or sum(_ends(c)) * c["Hkv"] * c["D"] <= 8e8)):
            del c["name"]
            return c


def _spread(n, lo, hi, salt):
    """n whole numbers spread over lo..hi, the first of them hi: part of the case, not of its seed."""
    r = random.Random(1000003 * salt + 31 * n + hi)
    return [hi] + [r.randint(lo, hi) for _ in range(n - 1)]


def _lens(c):
    return _spread(c["B"], 0, c["ctx"], 1) if c["ragged"] else [c["ctx"]] * c["B"]


def _toks(c):
    t = _spread(c["B"], 1, c["tok"], 2) if c["ragged"] else [c["tok"]] * c["B"]
    return t[:c["B"] - c["singles"]] + [1] * c["singles"]


def _ends(c):
    return [a + b for a, b in zip(_lens(c), _toks(c))]


def _done(c):
    """The requests that have finished (they bring no new tokens)."""
    return [b % 6 == 5 for b in range(c["B"])]


def _pages(n, page):
    return -(-n // page)


def work(c):
    D, H, Hkv, e = c["D"], c["H"], c["Hkv"], _ESIZE[c["dtype"]]
    lens, toks, ends = _lens(c), _toks(c), _ends(c)
    if c["op"] == "pages":
        done, p = _done(c), c["page"]
        back = sum(_pages(n, p) for n, d in zip(lens, done) if d)
        new = sum(_pages(b, p) - _pages(a, p) for a, b, d in zip(lens, ends, done) if not d)
        live = sum(t for t, d in zip(toks, done) if not d)
        # lengths, counts, flags and offsets; pages given back and taken; positions and slots
        # (whose page is in the table already for the first tokens of a request)
        return {"bytes": 16 * c["B"] + 8 * back + 8 * new + 8 * live, "flops": 4 * live}
    if c["op"] == "rope":
        n, s = sum(toks), _ESIZE[c["src"]]
        b = n * ((H + 2 * Hkv) * D * (s + e) + 8) + (8 * D if c["norm"] else 0) + 4 * c["rot"]
        return {"bytes": b, "flops": n * (H + Hkv) * (3 * c["rot"] + (4 * D if c["norm"] else 0))}
    pairs = sum(t * a + t * (t + 1) // 2 for a, t in zip(lens, toks))
    b = 2 * sum(ends) * Hkv * D * e + 2 * sum(toks) * H * D * e
    if c["page"]:
        b += 4 * sum(_pages(n, c["page"]) for n in ends)
    return {"bytes": b, "flops": 4 * H * D * pairs}


def _cost(c):
    """Seconds, roughly, of the plain form and of the 64-bit one: what bounds a drawn case."""
    w = work(c)
    slow = 20 if c["op"] == "pages" else 1
    return w["bytes"] / 1e12 * slow + w["flops"] / 3e13


# ------------------------------------------------------------------------------------------
# inputs

_THETA = 500000.0
_ORIG = 8192.0  # trained length that "ramp" scales from
_RAMP = (1.0, 4.0)  # turns over that length: slower than 1 scaled by the factor, faster than 4 kept


def _held(c):
    """The first page and the number of pages that each request has in the pool before the pass:
    those of its cached tokens, of the new ones too where they are in the cache, or of the new ones
    alone where no others are used."""
    p = c["page"]
    first = [n // p if c["op"] == "rope" else 0 for n in _lens(c)]
    last = _lens(c) if c["op"] == "pages" else _ends(c)
    return first, [_pages(n, p) - f for n, f in zip(last, first)]


def prepare(c, seed):
    B, H, Hkv, D, page = c["B"], c["H"], c["Hkv"], c["D"], c["page"]
    dev, dt = "cuda", _TORCH[c["dtype"]]
    g = torch.Generator(dev).manual_seed(seed)
    host = np.random.default_rng(seed)
    lens, toks = _lens(c), _toks(c)
    n = sum(toks)

    def ints(x):
        return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)

    def normal(*shape, dtype=dt):
        return torch.randn(shape, generator=g, device=dev).to(dtype)

    s = {"case": c, "lens": ints(lens), "cu": ints(np.cumsum([0] + toks))}
    if page:
        first, count = _held(c)
        all_pages = [_pages(x, page) for x in _ends(c)]
        n_pages = sum(all_pages) - sum(first) + 3
        width = max(all_pages) + 1
        order = host.permutation(n_pages).astype(np.int32)
        tables = np.full((B, width), -1, dtype=np.int32)
        at = 0
        for b in range(B):
            tables[b, first[b]:first[b] + count[b]] = order[at:at + count[b]]
            at += count[b]
        s["tables"] = ints(tables)
    if c["op"] == "pages":
        free = np.full(n_pages, -1, dtype=np.int32)
        free[:n_pages - at] = order[at:]
        s["free"], s["n_free"] = ints(free), ints([n_pages - at])
        s["n_free_mid"], s["n_free_new"] = ints([0]), ints([0])
        s["done"] = ints(_done(c))
        s["n_tok"] = ints([0 if d else t for t, d in zip(toks, _done(c))])
        s["cu"], s["pos"], s["slots"] = ints([0] * (B + 1)), ints([0] * n), ints([0] * n)
    else:
        # queries, keys and values side by side, as a projection leaves them
        src = _TORCH[c["src"]] if c["op"] == "rope" else dt
        wide = H if c["op"] == "paged" else H + 2 * Hkv
        qkv = normal(n, wide, D, dtype=src)
        if c["op"] != "rope":
            qkv[:, :H] *= 2
        s["q"], s["k"], s["v"] = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
        s["out"] = torch.zeros(n, H, D, dtype=dt, device=dev)
    if c["op"] == "rope":
        pos = np.concatenate([np.arange(a, a + t) for a, t in zip(lens, toks)])
        row = np.repeat(np.arange(B), toks)
        s["pos"] = ints(pos)
        s["slots"] = ints(tables[row, pos // page] * page + pos % page)
        s["k_pool"], s["v_pool"] = (torch.zeros(n_pages, Hkv, page, D, dtype=dt, device=dev)
                                    for _ in range(2))
        if c["norm"]:
            s["q_gain"], s["k_gain"] = (1 + 0.1 * normal(D, dtype=torch.float32) for _ in range(2))
    if c["op"] == "paged":
        s["k_pool"], s["v_pool"] = (normal(n_pages, Hkv, page, D) for _ in range(2))
    if own:
        from attention_dv_predict_gb300 import dv

        dtype = {"f32": dv.DV_F32, "f16": dv.DV_F16}[c["dtype"]]
        desc = dv.make_seq_desc(H, Hkv, D, dtype, page, n_pages if page else 0)
        s["desc"], s["ws"] = desc, dv.SeqWorkspace(desc)
        if "k_pool" in s:
            s["cache"] = dv.PagedCache(desc, tensors={"k": s["k_pool"], "v": s["v_pool"]})
        if c["op"] == "pages":
            s["pt"] = dv.PageTables(desc, B, width, tensors={
                "tables": s["tables"], "free": s["free"], "n_free": s["n_free"]})
        if c["op"] == "rope":
            s["rope"] = dv.Rope(
                D, c["rot"], interleaved=c["layout"] == "pairs", theta=_THETA,
                scaling=c["scaling"] or "none", factor=c["factor"], orig_len=_ORIG, low=_RAMP[0],
                high=_RAMP[1], norm=dv.DV_LAYERNORM if c["norm"] == "layer" else dv.DV_RMSNORM,
                eps=1e-5, q_gain=s.get("q_gain"), k_gain=s.get("k_gain"))
    return s


# ------------------------------------------------------------------------------------------
# one pass


def _plain_pages(s):
    c = s["case"]
    page, B, n = c["page"], c["B"], s["slots"].numel()
    lens, tables = s["lens"].long(), s["tables"]
    # the finished requests' pages go on top of the stack, in the order of the requests
    held = torch.where(s["done"] != 0, (lens + page - 1) // page, 0)
    j = torch.arange(tables.shape[1], device="cuda")
    place = s["n_free"] + (held.cumsum(0) - held)[:, None] + j
    n_pages = s["free"].numel()
    stack = torch.cat([s["free"], s["n_free"]])  # (its last entry takes what is no page)
    stack[torch.where(j < held[:, None], place, n_pages)] = tables
    s["free"].copy_(stack[:n_pages])
    s["n_free_mid"].copy_(s["n_free"] + held.sum())
    # the others take theirs from the top
    end = lens + s["n_tok"]
    have = (lens + page - 1) // page
    need = (end + page - 1) // page - have
    upto = need.cumsum(0)
    fits = (need == 0) | (upto <= s["n_free_mid"])
    k = j - have[:, None]
    new = (k >= 0) & (k < need[:, None]) & fits[:, None]
    take = (s["n_free_mid"] - 1 - (upto - need)[:, None] - k).clamp(0, s["free"].numel() - 1)
    tables.copy_(torch.where(new, s["free"][take], tables))
    s["n_free_new"].copy_(s["n_free_mid"] - torch.where(fits, need, 0).sum())
    cu = s["cu"]
    cu[1:] = s["n_tok"].cumsum(0)
    t = torch.arange(n, device="cuda", dtype=torch.int32)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=B - 1)
    live = t < cu[-1]
    pos = lens[b] + t - cu[b]
    at = tables[b, (pos // page).clamp(0, tables.shape[1] - 1)].long() * page + pos % page
    s["pos"].copy_(torch.where(live, pos, -1))
    s["slots"].copy_(torch.where(live & fits[b], at, -1))


def _freqs(c):
    """Angle of each pair of dimensions per position (doubles)."""
    rot = c["rot"]
    theta = _THETA * c["factor"] ** (rot / (rot - 2)) if c["scaling"] == "base" else _THETA
    f = theta ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    if c["scaling"] == "linear":
        f = f / c["factor"]
    if c["scaling"] == "ramp":
        keep = np.clip((_ORIG * f / (2 * math.pi) - _RAMP[0]) / (_RAMP[1] - _RAMP[0]), 0, 1)
        f = f * (keep + (1 - keep) / c["factor"])
    return f


def _plain_rope(s):
    c = s["case"]
    rot, page, slots = c["rot"], c["page"], s["slots"].long()
    angle = s["pos"].double()[:, None] * torch.from_numpy(_freqs(c)).cuda() if rot else None
    for t, out in (("q", s["out"]), ("k", None)):
        x = s[t].float()
        if c["norm"]:
            if c["norm"] == "layer":
                x = x - x.mean(-1, keepdim=True)
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-5) * s[t + "_gain"]
        if rot:
            cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
            half = c["layout"] == "half"
            a = x[..., :rot // 2] if half else x[..., :rot:2]
            b = x[..., rot // 2:rot] if half else x[..., 1:rot:2]
            a, b = a * cos - b * sin, b * cos + a * sin
            turned = torch.cat([a, b], -1) if half else torch.stack([a, b], -1).flatten(-2)
            x = torch.cat([turned, x[..., rot:]], -1)
        if out is not None:
            out.copy_(x)
        else:
            s["k_pool"][slots // page, :, slots % page] = x.to(s["k_pool"].dtype)
    s["v_pool"][slots // page, :, slots % page] = s["v"].to(s["v_pool"].dtype)


def _rows_of(s, b, lo, end):
    """Keys and values of request b, [Hkv, end, D] as they lie; lo: its first packed row."""
    c = s["case"]
    if c["op"] == "prompt":
        return [s[t][lo:lo + end].transpose(0, 1) for t in ("k", "v")]
    pages = s["tables"][b, :_pages(end, c["page"])].long()
    return [s[t][pages].transpose(0, 1).flatten(1, 2)[:, :end] for t in ("k_pool", "v_pool")]


def _attend(s, out, dtype):
    """Causal attention in `dtype`, a piece of the queries at a time with the keys they see."""
    c = s["case"]
    H, Hkv, D = c["H"], c["Hkv"], c["D"]
    lo = 0
    for b, (past, n) in enumerate(zip(_lens(c), _toks(c))):
        kk, vv = _rows_of(s, b, lo, past + n)
        step = max(1, min(n, 2048, int(5e8) // (H * (past + n))))
        for i in range(0, n, step):
            m, end = min(step, n - i), past + min(i + step, n)
            for h in ([slice(0, Hkv)] if H * m * end <= 6e8 else
                      [slice(x, x + 1) for x in range(Hkv)]):
                k, v = kk[h, :end].to(dtype), vv[h, :end].to(dtype)
                q = s["q"][lo + i:lo + i + m].to(dtype).view(m, Hkv, H // Hkv, D)[:, h]
                q = q.permute(1, 2, 0, 3)  # [h, G, m, D]
                score = torch.matmul(q.flatten(1, 2), k.transpose(-1, -2)) / math.sqrt(D)
                score = score.view(k.shape[0], H // Hkv, m, end)
                p = torch.arange(past + i, past + i + m, device="cuda")[:, None]
                score.masked_fill_(torch.arange(end, device="cuda") > p, -math.inf)
                w = torch.exp(score - score.amax(-1, keepdim=True))
                o = torch.matmul(w.flatten(1, 2), v).view(q.shape)
                o = o / w.sum(-1, keepdim=True)
                out[lo + i:lo + i + m].view(m, Hkv, H // Hkv, D)[:, h] = \
                    o.permute(2, 0, 1, 3).to(out.dtype)
        lo += n


def run(s):
    c = s["case"]
    if own:
        from attention_dv_predict_gb300 import dv

        if c["op"] == "pages":
            dv.dv_page_release(s["pt"], s["lens"], s["done"], s["ws"], n_free_out=s["n_free_mid"])
            dv.dv_page_take(s["pt"], s["lens"], s["n_tok"], s["cu"], s["pos"], s["slots"],
                            s["ws"], n_free=s["n_free_mid"], n_free_out=s["n_free_new"])
        elif c["op"] == "rope":
            dv.dv_qk_rope(s["rope"], s["q"], s["k"], s["pos"], s["ws"], q_out=s["out"], v=s["v"],
                          cache=s["cache"], slots=s["slots"])
        elif c["op"] == "prompt":
            dv.dv_prompt_attn(s["desc"], s["q"], s["k"], s["v"], s["cu"], s["out"], s["ws"],
                              max_tok=c["tok"])
        else:
            dv.dv_paged_attn(s["cache"], s["q"], s["cu"], s["lens"], s["tables"], s["out"],
                             s["ws"], max_tok=max(_toks(c)))
    elif c["op"] == "pages":
        _plain_pages(s)
    elif c["op"] == "rope":
        _plain_rope(s)
    else:
        _attend(s, s["out"], torch.float32)
    if c["op"] == "pages":
        return [s[t] for t in ("tables", "free", "n_free_mid", "n_free_new", "cu", "pos", "slots")]
    if c["op"] == "rope":
        return [s["out"], s["k_pool"], s["v_pool"]]
    return [s["out"]]


# ------------------------------------------------------------------------------------------
# the definitions in 64 bits


def _exact_pages(c, s):
    page, lens = c["page"], _lens(c)
    tables, free = s["tables"].cpu().numpy(), s["free"].cpu().numpy()
    top, n = int(s["n_free"]), s["slots"].numel()
    for b in range(c["B"]):
        if _done(c)[b]:
            for j in range(_pages(lens[b], page)):
                free[top] = tables[b, j]
                top += 1
    mid, cu = top, [0]
    pos, slots = np.full(n, -1, np.int32), np.full(n, -1, np.int32)
    for b, t in enumerate(s["n_tok"].tolist()):
        for j in range(_pages(lens[b], page), _pages(lens[b] + t, page)):
            top -= 1
            tables[b, j] = free[top]
        for i in range(t):
            p = lens[b] + i
            pos[cu[-1] + i], slots[cu[-1] + i] = p, tables[b, p // page] * page + p % page
        cu.append(cu[-1] + t)
    return [torch.from_numpy(np.asarray(x, dtype=np.int32))
            for x in (tables, free, [mid], [top], cu, pos, slots)]


def _exact_rope(c, s):
    D, rot, page = c["D"], c["rot"], c["page"]
    slots = s["slots"].cpu().numpy()
    angle = np.outer(s["pos"].cpu().numpy().astype(np.float64), _freqs(c)) if rot else None
    outs = []
    for t in ("q", "k"):
        x = s[t].double().cpu().numpy()
        if c["norm"]:
            if c["norm"] == "layer":
                x = x - x.mean(-1, keepdims=True)
            x = x / np.sqrt(np.square(x).mean(-1, keepdims=True) + 1e-5)
            x = x * s[t + "_gain"].double().cpu().numpy()
        if rot:
            pair = np.arange(rot // 2)
            i, j = (pair, pair + rot // 2) if c["layout"] == "half" else (2 * pair, 2 * pair + 1)
            z = (x[..., i] + 1j * x[..., j]) * np.exp(1j * angle)[:, None]
            x[..., i], x[..., j] = z.real, z.imag
        outs.append(x)
    outs.append(s["v"].double().cpu().numpy())
    for a in (1, 2):
        pool = np.zeros(tuple(s["k_pool"].shape))
        pool[slots // page, :, slots % page] = outs[a]
        outs[a] = pool
    return [torch.from_numpy(x) for x in outs]


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "pages":
        return _exact_pages(c, s)
    if c["op"] == "rope":
        return _exact_rope(c, s) if sum(_toks(c)) * (c["H"] + c["Hkv"]) * c["D"] <= 2e8 else None
    if work(c)["flops"] > 5e12:
        return None
    H, Hkv, D = c["H"], c["Hkv"], c["D"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lo = 0
    for b, (past, n) in enumerate(zip(_lens(c), _toks(c))):
        kk, vv = _rows_of(s, b, lo, past + n)
        for h in range(H):
            k, v = kk[h * Hkv // H].double(), vv[h * Hkv // H].double()
            for i in range(0, n, 1024):
                m = min(1024, n - i)
                end = past + i + m
                x = (s["q"][lo + i:lo + i + m, h].double() @ k[:end].T) * D ** -0.5
                seen = torch.ones(m, end, dtype=torch.bool, device="cuda").tril(past + i)
                w = torch.softmax(torch.where(seen, x, -math.inf), -1)
                out[lo + i:lo + i + m, h] = w @ v[:end]
        lo += n
    return [out]
