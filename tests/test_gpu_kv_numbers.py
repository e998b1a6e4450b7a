"""Attention over a KV cache where its numbers can go wrong, on the GPU: value rows of any size,
scores that rise, rows that must not depend on one another, NaN and infinities."""

import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import kv_ref
from test_gpu_kv import Case, close, dv, i32, mask_tensor, random_tree, skip_same, variant  # noqa: F401

pytestmark = pytest.mark.gpu


def half_ulp(x):
    return 2.0 ** (math.floor(math.log2(x)) - 24)


def sized_cache(c, pattern, e, rise, seed):
    """Fill an 8-bit Case: scores rise by `rise` (units of log2) over the first quarter of the
    positions for a query of 1 in dimension 0, value scales lie in [2^-e-1, 2^-e), zero rows as
    dv_kv_append stores them by `pattern`.  Returns keys' dimension 0 and values in 64 bits."""
    g = np.random.default_rng(seed)
    shape = (c.B, c.Hkv, c.cap)
    ramp = np.clip(np.arange(c.cap) / (c.cap / 4), 0, 1) * 200 - 100
    k0 = np.clip(np.rint(ramp + g.integers(-6, 7, shape)), -127, 127).astype(np.int8)
    codes = g.integers(64, 128, shape + (c.D,)).astype(np.int8)
    scale = (g.uniform(0.5, 1, shape) * 2.0 ** -e).astype(np.float32)
    zero = {"none": np.zeros(c.cap, bool), "first": np.arange(c.cap) < 100,
            "between": np.arange(c.cap) // 64 % 2 == 0}[pattern]
    codes[:, :, zero] = 0
    scale[:, :, zero] = 2.0 ** -126
    c.cache.k.zero_()
    c.cache.k[..., 0] = torch.from_numpy(k0).cuda()
    c.cache.k_scale.fill_(rise / 200)
    c.cache.v.copy_(torch.from_numpy(codes))
    c.cache.v_scale.copy_(torch.from_numpy(scale))
    return (k0 * float(np.float32(rise / 200)), codes * scale[..., None].astype(np.float64))


def sized_tolerance(e, rise, steps):
    """Relative to sum p |v|.  A score, one product, is off by at most 2^-21 of its size (its
    query's two parts 2^-22, the softmax scale, the product with it, the key's scale and the sum
    of the parts 2^-24 each).  Its weight's exponent, the score less a reference that takes the
    values' size too, is below |e| + 2 * rise + 16 and rounded once; ex2.approx, the weight's two
    parts and the value's scale add 2^-21.  That counts in the numerator and in the sum.  Every
    step of a tensor-core sum cuts off up to 2^-23."""
    w = math.log(2) * (rise / 2 * 2.0 ** -21 + half_ulp(abs(e) + 2 * rise + 16)) + 2.0 ** -21
    return 2 * w + steps * 2.0 ** -23


SIZES = [("none", e) for e in (0, 7, 14, 20, 30, 60)] + \
        [("first", e) for e in (-90, 0, 30)] + [("between", e) for e in (-90, -30, 8, 50)]


@pytest.mark.parametrize("pattern,e", SIZES)
@pytest.mark.parametrize("T,D,cap", [(3, 128, 1000), (3, 64, 6000), (12, 64, 1000),
                                     (40, 128, 1000), (12, 128, 9000)])
def test_tree_attn_values_of_any_size(dv, variant, T, D, cap, pattern, e):
    """Results are as exact for values of 2^-60 or 2^90 as for values of 1, also where scores rise
    from tile to tile and where the first rows, or every other tile's, are zeros."""
    skip_same(variant, "i8", D, T)
    rise = 12.0
    c = Case(dv, 2, 3, 1, D, 16, "i8", tokens=T)
    c = big(c, dv, cap, T)
    k0, v = sized_cache(c, pattern, e, rise, e + 1000)
    lens = [cap - T, cap // 2 + 5]
    q = torch.zeros(2, T, 3, D, device="cuda")
    q[..., 0] = 1.0
    out = torch.zeros_like(q)
    dv.dv_tree_attn(c.cache, q, i32(lens), out, c.ws, scale=math.log(2))
    c.ok()
    got = out.double().cpu().numpy()
    ln2 = float(np.float32(math.log(2)))
    tol = sized_tolerance(e, rise, 64 if cap <= 4096 else 224)
    for b in range(2):
        for t in (0, T - 1):
            n = lens[b] + t + 1
            s = ln2 * k0[b, :, :n]
            p = np.exp(s - s.max(-1, keepdims=True))
            want = np.einsum("hp,hpd->hd", p / p.sum(-1, keepdims=True), v[b, :, :n])
            err = np.abs(got[b, t] - want).max() / want.max()
            assert err <= tol, f"row {b} token {t}: off by {err:.3g} of its size, allowed {tol:.3g}"


def big(c, dv, cap, tokens, block=0):
    """c with a cache of `cap` positions that only the device holds."""
    c.cap = cap
    c.desc = dv.make_kv_desc(c.H, c.Hkv, c.D, cap, dv.DV_I8, block)
    c.cache = dv.KvCache(c.desc, c.B)
    c.ws = dv.KvWorkspace(c.desc, c.B, tokens)
    return c


@pytest.mark.parametrize("pattern,e", SIZES)
@pytest.mark.parametrize("D,cap", [(128, 1000), (64, 6000)])
def test_block_attn_values_of_any_size(dv, pattern, e, D, cap):
    rise = 12.0
    c = big(Case(dv, 2, 3, 1, D, 16, "i8"), dv, cap, 1, 16)
    k0, v = sized_cache(c, pattern, e, rise, e + 2000)
    lens = [cap, cap // 2 + 5]
    q = torch.zeros(2, 3, D, device="cuda")
    q[..., 0] = 1.0
    out = torch.zeros_like(q)
    idx = torch.arange(cap // 16, dtype=torch.int32, device="cuda").repeat(2, 3, 1)
    idx[1, :, (lens[1] + 15) // 16:] = -1
    dv.dv_block_attn(c.cache, q, i32(lens), idx, out, c.ws, scale=math.log(2))
    c.ok()
    got = out.double().cpu().numpy()
    tol = sized_tolerance(e, rise, 64 if cap <= 4096 else 224)
    for b in range(2):
        n = min(lens[b], cap // 16 * 16)
        s = float(np.float32(math.log(2))) * k0[b, :, :n]
        p = np.exp(s - s.max(-1, keepdims=True))
        want = np.einsum("hp,hpd->hd", p / p.sum(-1, keepdims=True), v[b, :, :n])
        err = np.abs(got[b] - want).max() / want.max()
        assert err <= tol, f"row {b}: off by {err:.3g} of its size, allowed {tol:.3g}"


@pytest.mark.parametrize("dtype", ["f16", "i8", "f32"])
@pytest.mark.parametrize("what", ["nan", "inf", "huge", "queries", "nan queries"])
@pytest.mark.parametrize("T,cap", [(6, 200), (6, 9000), (24, 200), (40, 9000)])
def test_rows_do_not_depend_on_one_another(dv, variant, dtype, what, T, cap):
    """To the bit: what a token does not see (behind the last token, and a drafted token that only
    itself sees), and other tokens' queries, do not show in its result."""
    if dtype == "f32" and cap > 200:
        pytest.skip("one form at any capacity")
    skip_same(variant, dtype, 64, T)
    B, Hkv, D = 2, 2, 64
    c = Case(dv, B, Hkv, 1, D, cap, dtype, tokens=T, seed=5)
    lens, n_tok, own = [cap - 70, 13], [T - 1, T], 2
    mask = [random_tree(c.rng, T) for _ in range(B)]
    for b in range(B):
        mask[b] = [m & ~(1 << own) for m in mask[b]]
        mask[b][own] = (1 << T) - 1
    q = torch.from_numpy(c.normal(B, T, Hkv, D)).cuda()

    def run():
        out = torch.zeros(B, T, Hkv, D, device="cuda")
        dv.dv_tree_attn(c.cache, q, i32(lens), out, c.ws, mask=mask_tensor(mask),
                        n_tok=i32(n_tok))
        c.ok()
        return out

    clean = run()
    if what == "queries":
        q[:, own] *= 300
    elif what == "nan queries":
        q[:, own, :, 7] = float("nan")
    else:
        x = {"nan": np.nan, "inf": np.inf, "huge": 3e4 if dtype == "f16" else 1e30}[what]
        for b in range(B):
            for p in [lens[b] + own] + list(range(lens[b] + n_tok[b], cap)):
                for t in ("k", "v"):
                    if dtype == "i8":
                        c.ref.scale[t][b, :, p] = x
                    else:
                        c.ref.raw[t][b, :, p] = x
        c.upload()
    got = run()
    for b in range(B):
        for t in range(n_tok[b]):
            if t != own:
                assert torch.equal(got[b, t], clean[b, t]), (b, t)
    assert not torch.equal(got[:, own], clean[:, own])


@pytest.mark.parametrize("dtype", ["f16", "i8"])
@pytest.mark.parametrize("T,D", [(3, 64), (12, 64), (12, 128)])
def test_long_rows_repeat_and_meet_poison(dv, variant, dtype, T, D):
    """So many long rows that a CTA attends several whole ones in chunks: the same bits from cold
    and warm calls, and with NaN or infinities where no token looks; one that is seen reaches its
    own head alone."""
    skip_same(variant, dtype, D, T)
    Hkv, cap = 160, 9000
    desc = dv.make_kv_desc(Hkv, Hkv, D, cap, 1 if dtype == "f16" else 2)
    cache, ws = dv.KvCache(desc, 1), dv.KvWorkspace(desc, 1, T)
    g = torch.Generator(device="cuda").manual_seed(T + D)
    for t in (cache.k, cache.v):
        t.random_(-100, 101, generator=g)
    if dtype == "i8":
        cache.k_scale.uniform_(0.01, 0.02, generator=g)
        cache.v_scale.uniform_(0.01, 0.02, generator=g)
    else:
        cache.k.mul_(2.0 ** -6)
        cache.v.mul_(2.0 ** -6)
    n = cap - T - 130
    mask = torch.full((1, T), (1 << T) - 1, dtype=torch.int64, device="cuda")
    mask &= ~2  # no token sees drafted token 1
    q = torch.randn(1, T, Hkv, D, generator=g, device="cuda")
    flush = torch.empty(1 << 28, dtype=torch.int8, device="cuda")

    def run():
        out = torch.zeros(1, T, Hkv, D, device="cuda")
        flush.fill_(1)
        dv.dv_tree_attn(cache, q, i32([n]), out, ws, mask=mask)
        assert dv.dv_check(ws) == 0
        return out

    def put(h, p, x):
        for t in (cache.k, cache.v) if dtype == "f16" else (cache.k_scale, cache.v_scale):
            t[0, h, p] = x

    clean = run()
    for _ in range(4):
        assert torch.equal(run(), clean)
    for x in (float("nan"), float("inf")):
        for p in (n + 1, slice(n + T, cap)):
            put(slice(None), p, x)
        assert torch.equal(run(), clean)
        put(77, 5000, x)
        out = run()
        assert not torch.isfinite(out[0, :, 77]).any()
        out[:, :, 77] = clean[:, :, 77]
        assert torch.equal(out, clean)
        put(77, 5000, 1.0)
        clean[:, :, 77] = run()[:, :, 77]
    assert torch.isfinite(clean).all()


@pytest.mark.parametrize("how", ["append", "keep"])
def test_mean_of_the_largest_keys(dv, how):
    """Keys at binary32's end: their mean rounds to an infinity, so the block comes first, like one
    that holds an infinity; below that it is a mean like others."""
    B, T, D, n = 1, 48, 32, 16
    c = Case(dv, B, 1, 1, D, 64, "f32", n)
    x = c.normal(B, T, 1, D)
    top = np.finfo(np.float32).max
    x[:, :n] = top
    x[:, n:2 * n] = np.float32(top * (1 - 2.0 ** -19))
    dev = torch.from_numpy(x).cuda()
    dv.dv_kv_append(c.cache, dev, dev, i32([0]), c.ws)
    if how == "keep":
        c.cache.k_mean.fill_(5)
        c.cache.k_mean_scale.fill_(7.0)
        path = torch.arange(T, dtype=torch.int32, device="cuda").reshape(1, T)
        dv.dv_kv_keep(c.cache, i32([0]), path, i32([T]), c.ws)
    c.ok()
    scale = c.cache.k_mean_scale[0, 0].cpu().numpy()
    codes = c.cache.k_mean[0, 0].cpu().numpy()
    assert np.isinf(scale[0]) and not codes[0].any()
    assert (codes[1] == 127).all() and abs(float(scale[1]) * 127 / top - 1) < 2.0 ** -18
    want, s = kv_ref.quantise(x[0, 2 * n:3 * n, 0].astype(np.float64).mean(0).astype(np.float32))
    assert np.abs(codes[2].astype(int) - want).max() <= 1 and abs(scale[2] / s - 1) < 2.0 ** -16
    idx = torch.zeros(B, 1, 2, dtype=torch.int32, device="cuda")
    dv.dv_block_topk(c.cache, -dev[:, 0, :, :] / top, i32([T]), idx, c.ws, n_first=0)
    c.ok()
    assert idx.flatten().tolist() == [0, 2]


@pytest.mark.parametrize("dtype,D", [("f32", 32), ("f16", 64), ("f16", 32)])
@pytest.mark.parametrize("T", [2, 12])
def test_infinite_keys(dv, variant, dtype, D, T):
    """A key with an infinity that a token sees: its score is an infinity or not a number.  The
    result is NaN, or as if the token did not see it (a score of -infinity); other heads and
    tokens that do not see it keep their bits."""
    skip_same(variant, dtype, D, T)
    B, H, cap = 1, 3, 300
    c = Case(dv, B, H, 1, D, cap, dtype, tokens=T, seed=1)
    n = 200
    q = torch.from_numpy(c.normal(B, T, H, D)).cuda()
    mask = [[((1 << T) - 1) & ~2] * T]  # drafted token 1 is not seen
    mask[0][T - 1] |= 2                 # but by the last one

    def run():
        out = torch.zeros(B, T, H, D, device="cuda")
        dv.dv_tree_attn(c.cache, q, i32([n]), out, c.ws, mask=mask_tensor(mask))
        c.ok()
        return out

    clean = run()
    c.cache.k[0, 0, n + 1, 3] = float("inf")
    out = run()
    assert torch.equal(out[:, :T - 1], clean[:, :T - 1])
    assert torch.equal(out[:, :, 1:], clean[:, :, 1:])
    mask[0][T - 1] &= ~2
    unseen = run()[0, T - 1, 0]
    got = out[0, T - 1, 0]
    assert torch.isnan(got).all() or torch.allclose(got, unseen, rtol=1e-5, atol=1e-6)


@pytest.mark.parametrize("dtype", ["f16", "i8", "f32"])
@pytest.mark.parametrize("D,cap", [(64, 700), (128, 9000)])
def test_block_attn_meets_poison(dv, dtype, D, cap):
    """NaN and infinities in blocks that are not listed, and behind the last position of a listed
    one, do not show; a listed one reaches its own head alone."""
    if dtype == "f32" and cap > 700:
        pytest.skip("one form at any capacity")
    H, n = 3, 32
    c = Case(dv, 1, H, 1, D, cap, dtype, n, seed=2)
    L = cap - 75
    nb = -(-L // n)
    listed = [j for j in range(nb) if j % 5 != 1]
    assert nb - 1 in listed
    idx = torch.full((1, H, nb), -1, dtype=torch.int32, device="cuda")
    idx[:, :, :len(listed)] = torch.tensor(listed, dtype=torch.int32, device="cuda")
    q = torch.from_numpy(c.normal(1, H, D)).cuda()

    def run():
        out = torch.zeros(1, H, D, device="cuda")
        dv.dv_block_attn(c.cache, q, i32([L]), idx, out, c.ws)
        c.ok()
        return out

    clean = run()
    sides = (c.cache.k_scale, c.cache.v_scale) if dtype == "i8" else (c.cache.k, c.cache.v)
    for x in (float("nan"), float("inf")):
        for t in sides:
            for j in range(1, nb, 5):
                t[:, :, j * n:(j + 1) * n] = x
            t[:, :, L:] = x
        assert torch.equal(run(), clean)
    sides[1][0, 1, 2 * n + 5] = float("nan")
    out = run()
    assert not torch.isfinite(out[0, 1]).any()
    assert torch.equal(out[0, [0, 2]], clean[0, [0, 2]])


@pytest.mark.parametrize("dtype,B,Hkv,T", [("f16", 6, 4, 12), ("f16", 6, 8, 20), ("i8", 6, 4, 12),
                                           ("i8", 8, 8, 40)])
def test_short_rows_in_a_large_cache(dv, dtype, B, Hkv, T):
    """Capacity of more than 4096 positions, rows of a hundred: the rules choose the kernel."""
    c = Case(dv, B, Hkv, 1, 64, 6000, dtype, tokens=T, seed=T)
    lens = [0, 1, 63, 64, 100, 17, 129, 5][:B]
    q = c.normal(B, T, Hkv, 64)
    out = torch.zeros(q.shape, device="cuda")
    dv.dv_tree_attn(c.cache, torch.from_numpy(q).cuda(), i32(lens), out, c.ws)
    c.ok()
    close(out, *kv_ref.tree(c.ref, q, lens, [T] * B, None, 0.125))


def test_wrappers_refuse_tensors_of_other_ranks(dv):
    """Too few dimensions are a ValueError too."""
    c = Case(dv, 2, 2, 1, 32, 50, "i8", 16)
    lens, x, o = i32([0, 0]), torch.zeros(2, 2, device="cuda"), torch.zeros(2, device="cuda")
    for call in (lambda: dv.dv_kv_append(c.cache, o, o, lens, c.ws),
                 lambda: dv.dv_kv_read(c.cache, lens, x, x, c.ws),
                 lambda: dv.dv_kv_keep(c.cache, lens, lens, lens, c.ws),
                 lambda: dv.dv_tree_attn(c.cache, o, lens, o, c.ws),
                 lambda: dv.dv_block_topk(c.cache, x, lens, lens, c.ws),
                 lambda: dv.dv_block_attn(c.cache, x, lens, lens, x, c.ws)):
        with pytest.raises(ValueError):
            call()
    c.same_cache()


def test_two_calls_at_once(dv, variant):
    """Calls on two streams, a workspace each, on one cache."""
    c = Case(dv, 4, 4, 1, 128, 3000, "i8", 64, tokens=20)
    lens = i32([2900, 2100, 50, 1500])
    s = [torch.cuda.Stream() for _ in range(2)]
    ws = [dv.KvWorkspace(c.desc, 4, 20) for _ in range(2)]
    q = [torch.from_numpy(c.normal(4, 20, 4, 128)).cuda() for _ in range(2)]
    want = [torch.zeros_like(q[0]) for _ in range(2)]
    for i in range(2):
        dv.dv_tree_attn(c.cache, q[i], lens, want[i], ws[i])
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(s[i]):
                out = torch.zeros_like(q[i])
                dv.dv_tree_attn(c.cache, q[i], lens, out, ws[i])
                outs.append((i, out))
    torch.cuda.synchronize()
    assert all(dv.dv_check(w) == 0 for w in ws)
    assert all(torch.equal(o, want[i]) for i, o in outs)


FIRST_CALLS = """
import torch
from attention_dv_predict_gb300 import dv
def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")
for dt, D in ((0, 32), (1, 64), (2, 128)):
    desc = dv.make_kv_desc(4, 4, D, 200, dt, 16)
    c, ws = dv.KvCache(desc, 2), dv.KvWorkspace(desc, 2, 16)
    x = torch.randn(2, 12, 4, D, device="cuda")
    lens, n = i32([60, 5]), i32([12, 12])
    path = torch.arange(12, dtype=torch.int32, device="cuda").repeat(2, 1)
    k, v = (torch.zeros(2, 4, 12, D, device="cuda") for _ in range(2))
    out, one = torch.zeros_like(x), torch.zeros(2, 4, D, device="cuda")
    idx = torch.zeros(2, 4, 2, dtype=torch.int32, device="cuda")
    def step():
        dv.dv_kv_append(c, x, x, lens, ws)
        dv.dv_tree_attn(c, x, lens, out, ws)
        dv.dv_kv_keep(c, lens, path, n, ws)
        dv.dv_kv_read(c, lens, k, v, ws)
        dv.dv_block_topk(c, x[:, 0], lens, idx, ws)
        dv.dv_block_attn(c, x[:, 0], lens, idx, one, ws)
    for kernel in (1, 2):
        dv.dv_set_tree_kernel(kernel)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        g.replay()
        got = [t.clone() for t in (out, one, k, v, idx)]
        step()
        assert all(torch.equal(a, b) for a, b in zip(got, (out, one, k, v, idx)))
        assert dv.dv_check(ws) == 0 and bool(out.any())
print("captured")
"""


def test_first_calls_are_captured():
    """A process whose first call of every operator is recorded into a graph."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "captured", r.stderr[-2000:]
