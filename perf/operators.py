"""The KV-cache operators: their cases, their plain forms, and the calls a user makes of them.

Four passes over one cache [B, Hkv, cap, D] (binary32, binary16, or 8-bit codes with a
binary32 scale for each row of D values):

* append: new keys and values are written (quantised, for an 8-bit cache; block means of
  completed blocks kept) and read back as floating-point rows;
* keep:   drafted tokens are written, the accepted path's rows are moved together, and the
  span is read back;
* tree:   attention of up to 64 drafted tokens a row, each seeing the cached prefix and its
  own ancestors (one token a row is ordinary decode attention);
* block:  blocks of cached positions are scored against each query by their mean key, the
  best are taken, and attention runs over them alone.

Shapes are those of the decode layers in dv_inputs.py (32/72/96 heads of 128, lengths 512 to
2048, batches 1 to 32, the tiny binary32 layer with 8 heads of 32) and generic longer ones.
"""
import math
import random

import numpy as np
import torch

own = False

_ESIZE = {"f32": 4, "f16": 2, "i8": 1}
_TORCH = {"f32": torch.float32, "f16": torch.float16}


# ------------------------------------------------------------------------------------------
# cases


def _case(name, op, B, H, D, T, length, dtype, **kw):
    c = {"name": name, "op": op, "B": B, "H": H, "Hkv": H, "D": D, "T": T, "len": length,
         "ragged": False, "dtype": dtype, "block": 0, "src": "f32", "out": "f32", "pick": 0,
         "heads": 0}
    c.update(kw)
    return c


def listed():
    return [
        # one new token a row into an 8-bit cache, read back: latency
        _case("append_token", "append", 4, 32, 128, 1, 575, "i8"),
        # ragged chunks of a binary16 projection into an 8-bit cache with block means
        _case("append_ragged", "append", 5, 72, 128, 333, 1024, "i8", ragged=True, block=64,
              src="f16", out="f16"),
        # a batch of prompts filling an 8-bit cache with block means, read back as a
        # binary16 layer cache
        _case("append_prompt", "append", 8, 96, 128, 2048, 37, "i8", block=64, out="f16"),
        # a short draft on the tiny binary32 layer
        _case("keep_tiny", "keep", 3, 8, 32, 5, 64, "f32", ragged=True),
        # a whole batch's 48-token drafts on an 8-bit cache with block means
        _case("keep_batch", "keep", 32, 96, 128, 48, 1000, "i8", ragged=True, block=32),
        # a single token over the 6.7B-shaped layer's cache
        _case("tree_token", "tree", 1, 32, 128, 1, 512, "f16"),
        # 13-token trees, ragged rows, the heads a contextual predictor keeps (15 of 72)
        _case("tree_heads", "tree", 8, 72, 128, 13, 1024, "i8", ragged=True, heads=15),
        # grouped query heads (8 to a KV head), 7 drafted tokens, a longer cache
        _case("tree_grouped", "tree", 16, 64, 128, 7, 8191, "f16", Hkv=8),
        # 64-token trees for a whole batch at the 175B shape
        _case("tree_wide", "tree", 32, 96, 128, 64, 2048, "i8"),
        # 8 blocks of 64 for one row of the 6.7B-shaped layer
        _case("block_row", "block", 1, 32, 128, 1, 4095, "f16", block=64, pick=8),
        # 32 blocks of 64 from a long cache
        _case("block_long", "block", 2, 96, 128, 1, 32768, "i8", block=64, pick=32),
        # grouped heads, short blocks, a ragged batch
        _case("block_batch", "block", 32, 64, 128, 1, 8000, "i8", Hkv=16, block=32, pick=48,
              ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = max(work(c)["bytes"] + work(c)["flops"] / 100 for c in listed())
    while True:
        op = rng.choice(["append", "keep", "tree", "block"])
        dtype = rng.choice(["f16", "i8", "i8", "f32"])
        D = rng.choice([64, 128, 128, 32] if op != "block" else [64, 128, 128])
        Hkv = _log(rng, 1, 96)
        G = rng.choice([1, 1, 1, 2, 4, 8]) if op in ("tree", "block") else 1
        block = rng.choice([16, 32, 64, 128])
        c = _case("", op, _log(rng, 1, 32), Hkv * G, D, 1, _log(rng, 3, 4000), dtype, Hkv=Hkv,
                  ragged=rng.random() < 0.7, src=rng.choice(["f32", "f16"]),
                  out=rng.choice(["f32", "f16"]))
        if op == "append":
            c.update(T=_log(rng, 1, 2000), block=rng.choice([0, block]))
        elif op == "keep":
            c.update(T=rng.randint(2, 64), block=rng.choice([0, block]))
        elif op == "tree":
            c.update(T=_log(rng, 1, 64), src="f32", out="f32",
                     heads=rng.choice([0, 0, max(1, Hkv // 5)]))
        else:
            c.update(block=block, len=_log(rng, 200, 32768), src="f32", out="f32")
            c.update(pick=min(max(2, c["len"] // block), _log(rng, 2, 64)))
        if op != "block" and c["len"] + c["T"] < c["block"]:
            c["block"] = 0
        if c["Hkv"] * G > 128:
            continue
        w = work(c)
        if (w["bytes"] + w["flops"] / 100 <= most and
                c["B"] * Hkv * (c["len"] + c["T"]) * D <= 8e8):
            del c["name"]
            return c


def _spread(n, lo, hi, salt):
    """n whole numbers spread over lo..hi, the first of them hi: part of the case, not of its seed."""
    r = random.Random(1000003 * salt + 31 * n + hi)
    return [hi] + [r.randint(lo, hi) for _ in range(n - 1)]


def _lens(c):
    lo = 1 if c["op"] == "block" else 0
    return _spread(c["B"], lo, c["len"], 1) if c["ragged"] else [c["len"]] * c["B"]


def _toks(c):
    return _spread(c["B"], 1, c["T"], 2) if c["ragged"] else [c["T"]] * c["B"]


def _keeps(c):
    return [min(k, t) for k, t in zip(_spread(c["B"], 0, max(1, c["T"] // 2), 3), _toks(c))]


def work(c):
    D, Hkv, G = c["D"], c["Hkv"], c["H"] // c["Hkv"]
    row = D * _ESIZE[c["dtype"]] + (4 if c["dtype"] == "i8" else 0)  # one cached row
    lens, toks = _lens(c), _toks(c)
    out = D * (_ESIZE[c["out"]])
    if c["op"] == "append":
        # new rows in, cached rows out; the span's rows in, floating-point rows out; the key
        # rows of completed blocks that were cached before are read for the mean
        new, read = sum(toks) * Hkv, c["B"] * c["T"] * Hkv
        b = 2 * (new * (D * _ESIZE[c["src"]] + row) + read * (row + out))
        f = 2 * new * D * 4
        if c["block"]:
            n = c["block"]
            done = sum((l + t) // n - l // n for l, t in zip(lens, toks))
            old = sum(l % n for l, t in zip(lens, toks) if (l + t) // n > l // n)
            b += Hkv * (done * (D + 4) + old * row)
            f += Hkv * done * n * D * 2
        return {"bytes": b, "flops": f}
    if c["op"] == "keep":
        new, moved = sum(toks) * Hkv, sum(_keeps(c)) * Hkv
        b = 2 * (new * (D * _ESIZE[c["src"]] + row) + 2 * moved * row
                 + c["B"] * c["T"] * Hkv * (row + out))
        return {"bytes": b, "flops": 2 * new * D * 4}
    if c["op"] == "tree":
        hk = c["heads"] or Hkv
        b = hk * sum(l + t for l, t in zip(lens, toks)) * 2 * row + 2 * hk * G * sum(toks) * D * 4
        return {"bytes": b, "flops": 4 * hk * G * D * sum(t * (l + t) for l, t in zip(lens, toks))}
    n, b, f = c["block"], 0.0, 0.0
    for l in lens:
        nb = -(-l // n)
        k = min(nb, c["pick"])
        # the blocks of a group's query heads overlap as independent choices would
        union = nb * (1 - (1 - k / nb) ** G)
        b += Hkv * (nb * (D + 4) + union * n * 2 * row) + c["H"] * (2 * D * 4 + c["pick"] * 4)
        f += c["H"] * (2 * nb * D + 4 * k * n * D)
    return {"bytes": b, "flops": f}


# ------------------------------------------------------------------------------------------
# inputs


def _quantise(x):
    """Rows of codes (as binary32) and scales: scale = max(amax / 127, 2^-126), code = rint(x / scale)."""
    x = x.float()
    # (a tensor divisor: dividing by a Python number multiplies by its rounded reciprocal)
    s = (x.abs().amax(-1) / torch.full((), 127.0, device=x.device)).clamp_min(2.0 ** -126)
    return torch.round(x / s[..., None]).clamp(-127, 127), s


def _block_means(x, n):
    """Quantised means of x [..., blocks * n, D] over blocks of n positions: keys rounded to a grid
    of 2^(e-24) n (2^e above the block's largest magnitude) so that a binary32 sum is exact in any order."""
    x = x.unflatten(-2, (-1, n))
    e = torch.frexp(x.abs().amax((-1, -2))).exponent.clamp_min(-100)
    step = torch.ldexp(torch.ones_like(x[..., 0, 0]), e - 24)[..., None, None]
    total = torch.round(x / (step * n)).sum(-2)
    return _quantise(total * step[..., 0])


def _tree_masks(c, g):
    """Ancestors (and self) of each drafted token of random trees, as bits."""
    B, T = c["B"], c["T"]
    anc = np.zeros((B, T, T), dtype=bool)
    for i in range(T):
        anc[:, i, i] = True
        if i:
            parent = g.integers(-1, i, B)
            anc[:, i] |= np.where((parent >= 0)[:, None], anc[np.arange(B), parent], False)
    bits = (anc.astype(np.uint64) << np.arange(T, dtype=np.uint64)).sum(-1, dtype=np.uint64)
    return torch.from_numpy(bits.view(np.int64))


def prepare(c, seed):
    B, H, Hkv, D, T, n = c["B"], c["H"], c["Hkv"], c["D"], c["T"], c["block"]
    dev = "cuda"
    g = torch.Generator(dev).manual_seed(seed)
    host = np.random.default_rng(seed)
    cap = c["len"] + (0 if c["op"] == "block" else T)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev)

    s = {"case": c, "cap": cap}
    s["lens"] = torch.tensor(_lens(c), dtype=torch.int32, device=dev)
    if c["ragged"]:
        s["toks"] = torch.tensor(_toks(c), dtype=torch.int32, device=dev)
    for t in ("k", "v"):
        if c["dtype"] == "i8":
            s[t] = torch.empty(B, Hkv, cap, D, dtype=torch.int8, device=dev)
            s[t + "_scale"] = torch.empty(B, Hkv, cap, device=dev)
            for b in range(B):
                q, s[t + "_scale"][b] = _quantise(normal(Hkv, cap, D))
                s[t][b] = q.to(torch.int8)
        else:
            s[t] = normal(B, Hkv, cap, D).to(_TORCH[c["dtype"]])
    if n:
        nb = cap // n
        s["k_mean"] = torch.zeros(B, Hkv, nb, D, dtype=torch.int8, device=dev)
        s["k_mean_scale"] = torch.zeros(B, Hkv, nb, device=dev)
        for b in range(B if nb else 0):
            x = s["k"][b, :, :nb * n].float()
            if c["dtype"] == "i8":
                x = x * s["k_scale"][b, :, :nb * n, None]
            q, s["k_mean_scale"][b] = _block_means(x, n)
            s["k_mean"][b] = q.to(torch.int8)
    if c["op"] in ("append", "keep"):
        # keys and values side by side, as a projection leaves them
        kv = normal(B, T, 2, Hkv, D).to(_TORCH[c["src"]])
        s["new_k"], s["new_v"] = kv[:, :, 0], kv[:, :, 1]
        s["k_out"], s["v_out"] = (torch.zeros(B, Hkv, T, D, dtype=_TORCH[c["out"]], device=dev)
                                  for _ in range(2))
    if c["op"] == "keep":
        keep = _keeps(c)
        path = np.zeros((B, T), dtype=np.int32)
        for b in range(B):
            path[b, :keep[b]] = np.sort(host.choice(_toks(c)[b], keep[b], replace=False))
        s["path"] = torch.from_numpy(path).to(dev)
        s["keep"] = torch.tensor(keep, dtype=torch.int32, device=dev)
    if c["op"] in ("tree", "block"):
        s["q"] = 2 * normal(B, T, H, D)
        s["att"] = torch.zeros(B, T, H, D, device=dev)
    if c["op"] == "tree":
        s["mask"] = _tree_masks(c, host).to(dev)
        if c["heads"]:
            pick = np.sort(host.choice(Hkv, c["heads"], replace=False)).astype(np.int32)
            s["heads"] = torch.from_numpy(pick).to(dev)
            s["n_heads"] = torch.tensor([c["heads"]], dtype=torch.int32, device=dev)
    if c["op"] == "block":
        s["q"], s["att"] = s["q"][:, 0].contiguous(), s["att"][:, 0].contiguous()
        s["idx"] = torch.full((B, H, c["pick"]), -1, dtype=torch.int32, device=dev)
    if own:
        from attention_dv_predict_gb300 import dv

        desc = dv.make_kv_desc(H, Hkv, D, cap, {"f32": dv.DV_F32, "f16": dv.DV_F16,
                                                "i8": dv.DV_I8}[c["dtype"]], block=n)
        names = ("k", "v", "k_scale", "v_scale", "k_mean", "k_mean_scale")
        s["cache"] = dv.KvCache(desc, B, tensors={t: s[t] for t in names if t in s})
        s["ws"] = dv.KvWorkspace(desc, B, T)
    return s


# ------------------------------------------------------------------------------------------
# one pass


def _rows(s, t, pos):
    """The values of positions pos [B, P] of cache tensor t, [B, Hkv, P, D] in binary32."""
    b = torch.arange(pos.shape[0], device=pos.device)[:, None]
    x = s[t].transpose(1, 2)[b, pos].float()
    if t + "_scale" in s:
        x = x * s[t + "_scale"].transpose(1, 2)[b, pos][..., None]
    return x.transpose(1, 2)


def _plain_append(s):
    c = s["case"]
    B, T, n = c["B"], c["T"], c["block"]
    b = torch.arange(B, device="cuda")[:, None]
    i = torch.arange(T, device="cuda")
    pos = s["lens"].long()[:, None] + i
    toks = s.get("toks", torch.full_like(s["lens"], T)).long()
    live = i < toks[:, None]
    for t in ("k", "v"):
        x = s["new_" + t].float()
        if c["dtype"] == "i8":
            x, scale = _quantise(x)
            old = s[t + "_scale"].transpose(1, 2)
            old[b, pos] = torch.where(live[..., None], scale, old[b, pos])
        old = s[t].transpose(1, 2)
        old[b, pos] = torch.where(live[..., None, None], x.to(old.dtype), old[b, pos])
    if n:
        _plain_means(s, s["lens"], s["lens"] + toks)


def _plain_means(s, begin, end):
    """The means of the blocks whose last position lies in begin .. end - 1 of their row."""
    n, nb = s["case"]["block"], s["k_mean"].shape[2]
    if not nb:
        return
    x = s["k"][:, :, :nb * n].float()
    if "k_scale" in s:
        x = x * s["k_scale"][:, :, :nb * n, None]
    q, scale = _block_means(x, n)
    last = torch.arange(1, nb + 1, device="cuda") * n - 1
    hit = ((last >= begin[:, None]) & (last < end[:, None]))[:, None]
    s["k_mean"].copy_(torch.where(hit[..., None], q.to(torch.int8), s["k_mean"]))
    s["k_mean_scale"].copy_(torch.where(hit, scale, s["k_mean_scale"]))


def _plain_keep(s):
    c = s["case"]
    b = torch.arange(c["B"], device="cuda")[:, None]
    i = torch.arange(c["T"], device="cuda")
    live = i < s["keep"][:, None]
    to = s["lens"].long()[:, None] + i
    of = torch.where(live, s["lens"].long()[:, None] + s["path"], to)
    for t in ("k", "v", "k_scale", "v_scale"):
        if t in s:
            x = s[t].transpose(1, 2)
            x[b, to] = x[b, of]
    if c["block"]:
        _plain_means(s, s["lens"], s["lens"] + s["keep"])


def _plain_read(s):
    c = s["case"]
    pos = s["lens"].long()[:, None] + torch.arange(c["T"], device="cuda")
    return [_rows(s, t, pos).to(_TORCH[c["out"]]) for t in ("k", "v")]


def _softmax_rows(score, seen):
    """Weights of the seen scores; a row that sees nothing has none."""
    score = torch.where(seen, score, -math.inf)
    m = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total == 0, 1.0, total)


def _plain_tree(s):
    c = s["case"]
    B, T, D, H, Hkv = c["B"], c["T"], c["D"], c["H"], c["Hkv"]
    lens = s["lens"].long()
    toks = s.get("toks", torch.full_like(s["lens"], T)).long()
    P = c["len"] + T
    heads = s["heads"].long() if c["heads"] else torch.arange(Hkv, device="cuda")
    pos = torch.arange(P, device="cuda")
    j = pos - lens[:, None]  # the drafted token at a position
    drafted = (j >= 0) & (j < toks[:, None])
    anc = (s["mask"][:, :, None] >> j.clamp(0, 63)[:, None, :]) & 1
    seen = (j < 0)[:, None, :] | (drafted[:, None, :] & (anc == 1))  # [B, T, P]
    kv = []
    for t in ("k", "v"):
        x = s[t][:, heads, :P].float()
        if t + "_scale" in s:
            x = x * s[t + "_scale"][:, heads, :P, None]
        kv.append(torch.where((j < toks[:, None])[:, None, :, None], x, 0.0))
    q = s["q"].view(B, T, Hkv, H // Hkv, D)[:, :, heads].permute(0, 2, 3, 1, 4)  # [B, h, G, T, D]
    score = torch.matmul(q.flatten(2, 3), kv[0].transpose(-1, -2)) / math.sqrt(D)
    p = _softmax_rows(score.view(B, len(heads), -1, T, P), seen[:, None, None])
    o = torch.matmul(p.flatten(2, 3), kv[1]).view(B, len(heads), -1, T, D)
    o = o.permute(0, 3, 1, 2, 4)
    live = (torch.arange(T, device="cuda") < toks[:, None])[:, :, None, None, None]
    att = s["att"].view(B, T, Hkv, H // Hkv, D)
    att[:, :, heads] = torch.where(live, o, att[:, :, heads])
    return [s["att"]]


def _plain_block(s):
    c = s["case"]
    B, D, H, Hkv, n, k = c["B"], c["D"], c["H"], c["Hkv"], c["block"], c["pick"]
    G, lens = H // Hkv, s["lens"].long()
    nb = -(-c["len"] // n)
    qc, _ = _quantise(s["q"])
    # whole-number sums under 2^24: exact in binary32
    dots = torch.matmul(qc.view(B, Hkv, G, D), s["k_mean"].float().transpose(-1, -2))
    score = torch.full((B, H, nb), -math.inf, device="cuda")
    full = s["k_mean"].shape[2]
    score[:, :, :full] = (dots * s["k_mean_scale"][:, :, None]).view(B, H, full)
    blocks = torch.arange(nb, device="cuda")
    used = (lens + n - 1) // n
    held = (blocks < 1) | (blocks >= used[:, None] - 1)  # the first and the last block
    score = torch.where(held[:, None], math.inf, score)
    score = torch.where((blocks < used[:, None])[:, None], score, -math.inf)
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :k]
    if order.shape[-1] < k:
        order = torch.nn.functional.pad(order, (0, k - order.shape[-1]), value=nb)
    order = torch.where(order < used[:, None, None], order, nb + 1).sort(-1).values
    idx = torch.where(order < nb + 1, order, -1)
    s["idx"].copy_(idx)
    pos = (idx[..., None] * n + torch.arange(n, device="cuda")).flatten(-2)  # [B, H, k n]
    seen = (pos >= 0) & (pos < lens[:, None, None])
    pos = pos.clamp(0, s["cap"] - 1)
    row = (torch.arange(B, device="cuda")[:, None, None] * Hkv
           + (torch.arange(H, device="cuda") // G)[:, None]) * s["cap"] + pos
    x = s["k"].view(-1, D)[row].float()
    if c["dtype"] == "i8":
        x = x * s["k_scale"].view(-1)[row][..., None]
    score = torch.matmul(x, s["q"][..., None])[..., 0] / math.sqrt(D)
    p = _softmax_rows(score, seen)
    x = s["v"].view(-1, D)[row].float()
    if c["dtype"] == "i8":
        x = x * s["v_scale"].view(-1)[row][..., None]
    s["att"].copy_(torch.matmul(p[..., None, :], x)[..., 0, :])
    return [s["idx"], s["att"]]


def run(s):
    c = s["case"]
    if own:
        from attention_dv_predict_gb300 import dv

        cache, ws, lens, toks = s["cache"], s["ws"], s["lens"], s.get("toks")
        if c["op"] in ("append", "keep"):
            dv.dv_kv_append(cache, s["new_k"], s["new_v"], lens, ws, n_tok=toks)
            if c["op"] == "keep":
                dv.dv_kv_keep(cache, lens, s["path"], s["keep"], ws)
            dv.dv_kv_read(cache, lens, s["k_out"], s["v_out"], ws)
            out = [s["k_out"], s["v_out"]]
        elif c["op"] == "tree":
            dv.dv_tree_attn(cache, s["q"], lens, s["att"], ws, mask=s["mask"], n_tok=toks,
                            u_h=s.get("heads"), n_u_h=s.get("n_heads"))
            out = [s["att"]]
        else:
            dv.dv_block_topk(cache, s["q"], lens, s["idx"], ws)
            dv.dv_block_attn(cache, s["q"], lens, s["idx"], s["att"], ws)
            out = [s["idx"], s["att"]]
    elif c["op"] == "tree":
        out = _plain_tree(s)
    elif c["op"] == "block":
        out = _plain_block(s)
    else:
        _plain_append(s)
        if c["op"] == "keep":
            _plain_keep(s)
        out = _plain_read(s)
    if c["op"] in ("append", "keep") and c["block"]:
        # the 8-bit block means as the values they stand for
        out = out + [s["k_mean"] * s["k_mean_scale"][..., None]]
    return out


# ------------------------------------------------------------------------------------------
# the definitions in 64 bits


def _codes64(x):
    """Codes and scales of rows of doubles: the scale and the quotient are binary32 by definition."""
    s = np.maximum((np.abs(x).max(-1) / 127.0).astype(np.float32), np.float32(2.0 ** -126))
    return np.rint((x / s[..., None].astype(np.float64)).astype(np.float32)).astype(np.float64), s


def _means64(keys, n):
    """The value of the quantised mean of keys [h, n, D] (doubles)."""
    e = np.maximum(np.frexp(np.abs(keys).max((1, 2)))[1], -100)
    grid = np.ldexp(float(n), e - 24)[:, None, None]
    mean = np.rint(keys / grid).sum(1) * grid[:, 0] / n
    q, s = _codes64(mean)
    return (q.astype(np.float32) * s[..., None]).astype(np.float64)


def _host(s, t, b):
    """Cache tensor t of row b as binary32 values in doubles."""
    x = s[t][b].float()
    if t + "_scale" in s:
        x = x * s[t + "_scale"][b][..., None]
    return x.double()


def exact(c, seed):
    s = prepare(c, seed)
    B, T, D, H, Hkv, n = c["B"], c["T"], c["D"], c["H"], c["Hkv"], c["block"]
    G, lens, toks = H // Hkv, _lens(c), _toks(c)
    if c["op"] in ("append", "keep"):
        if B * Hkv * (c["len"] + T) * D > 3e8:
            return None
        outs, means = [[], []], []
        for b in range(B):
            both = []
            for t in ("k", "v"):
                x = _host(s, t, b).cpu().numpy()
                new = s["new_" + t][b].double().cpu().numpy().transpose(1, 0, 2)[:, :toks[b]]
                if c["dtype"] == "i8":
                    q, sc = _codes64(new)
                    new = (q.astype(np.float32) * sc[..., None]).astype(np.float64)
                elif c["dtype"] == "f16":
                    new = new.astype(np.float16).astype(np.float64)
                x[:, lens[b]:lens[b] + toks[b]] = new
                if c["op"] == "keep":
                    path = s["path"][b].tolist()
                    for i in range(_keeps(c)[b]):
                        x[:, lens[b] + i] = x[:, lens[b] + path[i]]
                both.append(x)
            if n:
                m = (s["k_mean"][b].double() * s["k_mean_scale"][b][..., None].double()).cpu().numpy()
                spans = [(both[0], lens[b], lens[b] + toks[b])]
                if c["op"] == "keep":
                    # a block that the draft filled has the draft's mean until its last row is kept
                    draft = _host(s, "k", b).cpu().numpy()
                    new = s["new_k"][b].double().cpu().numpy().transpose(1, 0, 2)[:, :toks[b]]
                    if c["dtype"] == "i8":
                        q, sc = _codes64(new)
                        new = (q.astype(np.float32) * sc[..., None]).astype(np.float64)
                    elif c["dtype"] == "f16":
                        new = new.astype(np.float16).astype(np.float64)
                    draft[:, lens[b]:lens[b] + toks[b]] = new
                    spans = [(draft, lens[b], lens[b] + toks[b]),
                             (both[0], lens[b], lens[b] + _keeps(c)[b])]
                for x, lo, hi in spans:
                    for j in range(m.shape[1]):
                        if lo <= j * n + n - 1 < hi:
                            m[:, j] = _means64(x[:, j * n:j * n + n], n)
                means.append(m)
            for o, x in zip(outs, both):
                o.append(x[:, lens[b]:lens[b] + T])
        out = [torch.from_numpy(np.stack(o)) for o in outs]
        return out + ([torch.from_numpy(np.stack(means))] if n else [])
    att = torch.zeros(B, T, H, D, dtype=torch.float64, device="cuda")
    if c["op"] == "tree":
        heads = s["heads"].tolist() if c["heads"] else list(range(Hkv))
        q = s["q"].double()
        for b in range(B):
            k, v = _host(s, "k", b), _host(s, "v", b)
            bits = s["mask"][b].cpu().numpy().view(np.uint64)
            sees = torch.ones(toks[b], lens[b] + toks[b], dtype=torch.bool)
            for i in range(toks[b]):
                for j in range(toks[b]):
                    sees[i, lens[b] + j] = bool((int(bits[i]) >> j) & 1)
            sees = sees.cuda()
            for h in heads:
                for a in range(h * G, h * G + G):
                    x = (q[b, :toks[b], a] @ k[h, :lens[b] + toks[b]].T) * D ** -0.5
                    w = torch.softmax(x.masked_fill(~sees, -math.inf), -1)
                    w = torch.where(sees.any(-1, keepdim=True), w, 0.0)
                    att[b, :toks[b], a] = w @ v[h, :lens[b] + toks[b]]
        return [att]
    idx = np.full((B, H, c["pick"]), -1, dtype=np.int32)
    for b in range(B):
        used = -(-lens[b] // n)
        k, v = _host(s, "k", b), _host(s, "v", b)
        qc = _codes64(s["q"][b].double().cpu().numpy())[0]
        mc = s["k_mean"][b].double().cpu().numpy()
        ms = s["k_mean_scale"][b].cpu().numpy()
        for h in range(H):
            dots = (mc[h // G] @ qc[h]).astype(np.float32) * ms[h // G]
            middle = sorted(range(1, used - 1), key=lambda j: (-dots[j], j))
            must = sorted({0, used - 1})
            got = sorted((must + middle)[:c["pick"]])
            idx[b, h, :len(got)] = got
            pos = torch.cat([torch.arange(j * n, min(j * n + n, lens[b])) for j in got]).cuda()
            w = torch.softmax(k[h // G, pos] @ s["q"][b, h].double() * D ** -0.5, -1)
            att[b, 0, h] = w @ v[h // G, pos]
    return [torch.from_numpy(idx), att[:, 0]]
