"""The KV-cache operators on the GPU against plain 64-bit implementations.

Codes, scales, block means and selected blocks are defined to the bit and must be equal.
Attention tolerances come from kv_ref.attend, which derives them from each case's values.
"""

import numpy as np
import pytest
import torch

import kv_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dv():
    from attention_dv_predict_gb300 import build

    build.build()
    from attention_dv_predict_gb300 import dv as mod

    return mod


DT = {"f32": 0, "f16": 1, "i8": 2}


@pytest.fixture(params=[1, 2], ids=["mma", "tcgen05"])
def variant(dv, request):
    """Both tree kernels (they are the same one where only one serves)."""
    dv.dv_set_tree_kernel(request.param)
    yield request.param
    dv.dv_set_tree_kernel(0)


def skip_same(variant, dtype, D, rows):
    if variant == 2 and (dtype == "f32" or D not in (64, 128) or rows <= 8):
        pytest.skip("one kernel serves this shape")


class Case:
    """A random cache on the device and its host twin."""

    def __init__(self, dv, B, Hkv, G, D, cap, dtype, block=0, tokens=64, seed=0):
        self.dv, self.B, self.Hkv, self.H, self.D, self.cap = dv, B, Hkv, Hkv * G, D, cap
        self.rng = np.random.default_rng(seed)
        self.ref = kv_ref.RefCache(B, Hkv, cap, D, dtype, block, self.rng)
        self.desc = dv.make_kv_desc(self.H, Hkv, D, cap, DT[dtype], block)
        self.cache = dv.KvCache(self.desc, B)
        self.ws = dv.KvWorkspace(self.desc, B, min(tokens, cap))
        self.upload()

    def upload(self):
        for t in ("k", "v"):
            getattr(self.cache, t).copy_(torch.from_numpy(self.ref.raw[t]))
            if self.ref.scale:
                getattr(self.cache, t + "_scale").copy_(torch.from_numpy(self.ref.scale[t]))
        if self.ref.block:
            self.cache.k_mean.copy_(torch.from_numpy(self.ref.mean))
            self.cache.k_mean_scale.copy_(torch.from_numpy(self.ref.mean_scale))

    def normal(self, *shape, dtype=np.float32):
        return self.rng.standard_normal(shape).astype(dtype)

    def ok(self, status=0):
        assert self.dv.dv_check(self.ws) == status

    def same_cache(self):
        for t in ("k", "v"):
            np.testing.assert_array_equal(getattr(self.cache, t).cpu().numpy(), self.ref.raw[t])
            if self.ref.scale:
                np.testing.assert_array_equal(getattr(self.cache, t + "_scale").cpu().numpy(),
                                              self.ref.scale[t])
        if self.ref.block:
            np.testing.assert_array_equal(self.cache.k_mean.cpu().numpy(), self.ref.mean)
            np.testing.assert_array_equal(self.cache.k_mean_scale.cpu().numpy(),
                                          self.ref.mean_scale)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def close(got, want, tol):
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all()
    bad = np.abs(got - want) - tol[..., None]
    assert (bad <= 0).all(), f"off by {np.abs(got - want).max():.3g}, allowed {tol.max():.3g}"


# ------------------------------------------------------------------ append, read, keep


@pytest.mark.parametrize("dtype", ["f32", "f16", "i8"])
@pytest.mark.parametrize("D,block,T", [(128, 64, 1), (128, 16, 70), (32, 32, 65), (64, 0, 3),
                                       (16, 128, 200)])
@pytest.mark.parametrize("src", ["f32", "f16"])
def test_append_and_read(dv, dtype, D, block, T, src):
    B, Hkv, cap = 5, 3, 300
    c = Case(dv, B, Hkv, 1, D, cap, dtype, block)
    lens = [0, 63, cap - T, 17, 95]
    n_tok = [T, T, T, 0, (T + 1) // 2]
    k, v = (c.normal(B, T, Hkv, D, dtype=np.float16 if src == "f16" else np.float32)
            for _ in range(2))
    if dtype == "i8":  # halves of a step, zeros, one huge value
        k[0, 0, 0] = 0
        k[0, 0, 1] = np.linspace(-127, 127, D).round() / 2
        v[0, 0, 0, 3] = 6e4
    dv.dv_kv_append(c.cache, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), i32(lens),
                    c.ws, n_tok=i32(n_tok))
    c.ok()
    c.ref.append(k, v, lens, n_tok)
    c.same_cache()
    for out in (torch.float32, torch.float16):
        ko, vo = (torch.zeros(B, Hkv, T, D, dtype=out, device="cuda") for _ in range(2))
        dv.dv_kv_read(c.cache, i32(lens), ko, vo, c.ws)
        c.ok()
        for o, t in ((ko, "k"), (vo, "v")):
            x = c.ref.values(t)
            want = np.stack([x[b, :, lens[b]:lens[b] + T] for b in range(B)])
            want = want.astype(np.float32)
            want = want.astype(np.float16) if out == torch.float16 else want
            np.testing.assert_array_equal(o.cpu().numpy(), want)


@pytest.mark.parametrize("dtype", ["f32", "f16", "i8"])
def test_append_strided_rows(dv, dtype):
    """Slices of a fused projection [B, T, 3, H, D], and a layer cache [B, H, cap, D] read as rows."""
    B, Hkv, T, D = 2, 4, 9, 64
    c = Case(dv, B, Hkv, 1, D, 40, dtype, 16)
    qkv = c.normal(B, T, 3, Hkv, D)
    dev = torch.from_numpy(qkv).cuda()
    dv.dv_kv_append(c.cache, dev[:, :, 1], dev[:, :, 2], i32([3, 11]), c.ws)
    c.ok()
    c.ref.append(qkv[:, :, 1], qkv[:, :, 2], [3, 11], [T, T])
    c.same_cache()
    layer = c.normal(B, Hkv, 50, D, dtype=np.float16)
    dev = torch.from_numpy(layer).cuda()[:, :, 5:25].transpose(1, 2)
    dv.dv_kv_append(c.cache, dev, dev, i32([0, 20]), c.ws)
    c.ok()
    rows = layer[:, :, 5:25].transpose(0, 2, 1, 3)
    c.ref.append(rows, rows, [0, 20], [20, 20])
    c.same_cache()


def test_append_non_finite(dv):
    """A row with a NaN or an infinity reads back as NaN (8 bits); its block comes first."""
    c = Case(dv, 1, 1, 1, 32, 64, "i8", 16)
    x = c.normal(1, 20, 1, 32)
    x[0, 3, 0, 5], x[0, 18, 0, 0] = np.nan, -np.inf
    dev = torch.from_numpy(x).cuda()
    dv.dv_kv_append(c.cache, dev, dev, i32([0]), c.ws)
    c.ok()
    c.ref.append(x, x, [0], [20])
    c.same_cache()
    assert np.isinf(c.ref.mean_scale[0, 0, 0]) and np.isfinite(c.ref.mean_scale[0, 0, 1])
    out = torch.zeros(1, 1, 20, 32, device="cuda")
    dv.dv_kv_read(c.cache, i32([0]), out, out.clone(), c.ws)
    bad = torch.isnan(out).all(-1)[0, 0].nonzero().flatten().tolist()
    assert bad == [3, 18] and torch.isfinite(out[0, 0, :3]).all()


def test_append_tiny_and_huge(dv):
    c = Case(dv, 1, 2, 1, 64, 8, "i8")
    x = c.normal(1, 8, 2, 64)
    x[0, 0] *= 1e-42 / 4
    x[0, 1] *= 1e-36
    x[0, 2] *= 5e37
    x[0, 3] = 0
    x[0, 4, :, :] = 3.4e38
    dev = torch.from_numpy(x).cuda()
    dv.dv_kv_append(c.cache, dev, dev, i32([0]), c.ws)
    c.ok()
    c.ref.append(x, x, [0], [8])
    c.same_cache()


@pytest.mark.parametrize("exp", [0, -30, -90, -118, 60])
def test_append_near_halves(dv, exp):
    """Values within a few last places of half a code: the rounded quotient decides."""
    B, T, H, D = 1, 400, 2, 128
    c = Case(dv, B, H, 1, D, T, "i8")
    s = (c.rng.uniform(1, 2, (B, T, H, 1)) * 2.0 ** exp).astype(np.float32)
    k = c.rng.integers(-126, 126, (B, T, H, D)) + 0.5
    x = (k * s).astype(np.float32)
    x = (x.view(np.int32) + c.rng.integers(-2, 3, x.shape).astype(np.int32)).view(np.float32)
    x[..., 0] = 127 * s[..., 0]
    dev = torch.from_numpy(x).cuda()
    dv.dv_kv_append(c.cache, dev, dev, i32([0]), c.ws)
    c.ok()
    c.ref.append(x, x, [0], [T])
    c.same_cache()


@pytest.mark.parametrize("dtype,D", [("f32", 32), ("f16", 128), ("i8", 128), ("i8", 16)])
def test_keep(dv, dtype, D):
    B, Hkv, T, cap = 6, 2, 37, 150
    c = Case(dv, B, Hkv, 1, D, cap, dtype, 16)
    lens = [0, 5, 15, 100, cap - T, 60]
    paths = [list(range(T)), [0, 2, 3, 11, 36], [36], [], [1, 2, 3, 4, 5, 6, 30, 31, 32, 33, 34],
             list(range(1, T))]
    x = c.normal(B, T, Hkv, D)
    dev = torch.from_numpy(x).cuda()
    dv.dv_kv_append(c.cache, dev, dev.flip(1), i32(lens), c.ws)
    c.ref.append(x, x[:, ::-1], lens, [T] * B)
    path = np.zeros((B, T), np.int32)
    for b, p in enumerate(paths):
        path[b, :len(p)] = p
    dv.dv_kv_keep(c.cache, i32(lens), torch.from_numpy(path).cuda(), i32([len(p) for p in paths]),
                  c.ws)
    c.ok()
    c.ref.keep(lens, path, [len(p) for p in paths])
    c.same_cache()


def test_bad_rows_are_skipped(dv):
    """Out-of-range lengths, counts and paths: that row alone is left as it was, and reported."""
    B, T, cap = 4, 8, 40
    c = Case(dv, B, 2, 1, 32, cap, "i8", 16)
    x = c.normal(B, T, 2, 32)
    dev = torch.from_numpy(x).cuda()
    for lens, n_tok in (([-1, 0, cap - T + 1, 5], [T] * 4), ([3, 0, cap, 5], [-1, T, 1, T + 1])):
        dv.dv_kv_append(c.cache, dev, dev, i32(lens), c.ws, n_tok=i32(n_tok))
        c.ok(dv.DV_ERR_DEVICE_INDEX)
        c.ok()
        good = [1, 3] if lens[0] == -1 else [1]
        c.ref.append(x, x, [lens[b] if b in good else 0 for b in range(B)],
                     [n_tok[b] if b in good else 0 for b in range(B)])
        c.same_cache()
    out = torch.full((B, 2, T, 32), 7.0, device="cuda")
    dv.dv_kv_read(c.cache, i32([-1, 0, cap - T + 1, 2 ** 31 - 1]), out, out.clone(), c.ws)
    c.ok(dv.DV_ERR_DEVICE_INDEX)
    assert (out[[0, 2, 3]] == 7).all() and (out[1] != 7).any()
    path = np.tile(np.arange(T, dtype=np.int32), (B, 1))
    path[0, 3] = 2                      # not ascending
    path[1, :3] = [1, 2, T]             # beyond the draft
    path[2, :2] = [-1, 3]
    dv.dv_kv_keep(c.cache, i32([0, 0, 0, cap - 3]), torch.from_numpy(path).cuda(),
                  i32([5, 3, 2, 4]), c.ws)
    c.ok(dv.DV_ERR_DEVICE_INDEX)
    c.same_cache()
    # tree: rows 0 and 2 are out of range; block selection likewise
    q = torch.from_numpy(c.normal(B, 2, 2, 32)).cuda()
    o = torch.full((B, 2, 2, 32), 7.0, device="cuda")
    dv.dv_tree_attn(c.cache, q, i32([-5, 3, cap - 1, 6]), o, c.ws)
    c.ok(dv.DV_ERR_DEVICE_INDEX)
    assert (o[[0, 2]] == 7).all() and (o[[1, 3]] != 7).all()
    idx = torch.full((B, 2, 2), 9, dtype=torch.int32, device="cuda")
    dv.dv_block_topk(c.cache, q[:, 0], i32([-5, 3, cap + 1, cap]), idx, c.ws)
    c.ok(dv.DV_ERR_DEVICE_INDEX)
    assert (idx[[0, 2]] == 9).all() and idx[1, 0].tolist() == [0, -1]


# ------------------------------------------------------------------ attention over a tree


def random_tree(rng, T):
    bits = []
    for i in range(T):
        p = rng.integers(-1, i) if i else -1
        bits.append((bits[p] if p >= 0 else 0) | 1 << i)
    return bits


def mask_tensor(mask):
    return torch.from_numpy(np.array(mask, dtype=np.uint64).view(np.int64)).cuda()


TREES = [
    # Hkv, G, D, T, cap
    (2, 1, 128, 1, 700), (3, 1, 128, 5, 200), (2, 1, 128, 8, 300), (2, 2, 128, 7, 300),
    (2, 1, 128, 13, 260), (1, 4, 128, 7, 200), (2, 1, 128, 33, 260), (2, 1, 128, 64, 400),
    (1, 8, 128, 17, 200), (2, 3, 64, 9, 333), (2, 1, 64, 50, 200), (3, 2, 32, 11, 150),
    (2, 1, 16, 6, 100), (1, 1, 256, 9, 150), (1, 16, 64, 64, 129),
]


@pytest.mark.parametrize("dtype", ["f32", "f16", "i8"])
@pytest.mark.parametrize("Hkv,G,D,T,cap", TREES)
def test_tree_attn(dv, variant, dtype, Hkv, G, D, T, cap):
    skip_same(variant, dtype, D, T * G)
    if dtype == "f32" and D == 256:
        pytest.skip("head_dim * 4 above 512 bytes is not supported")
    B = 5
    c = Case(dv, B, Hkv, G, D, cap, dtype, tokens=T, seed=T + D)
    lens = [0, 1, cap - T, 63, 64 if cap >= 64 + T else 0]
    n_tok = [T, T, T, max(1, T // 2), min(T, 3)]
    lens[3] = min(63, cap - T)
    q = 2 * c.normal(B, T, c.H, D)
    mask = [random_tree(c.rng, T) for _ in range(B)]
    mask[1][0] = 0
    mask[0][T - 1] = 0  # sees nothing: no prefix, no token
    if T == 64:
        mask[2][T - 1] = 2 ** 64 - 1
    out = torch.full((B, T, c.H, D), -9.0, device="cuda")
    dv.dv_tree_attn(c.cache, torch.from_numpy(q).cuda(), i32(lens), out, c.ws,
                    mask=mask_tensor(mask), n_tok=i32(n_tok))
    c.ok()
    want, tol = kv_ref.tree(c.ref, q, lens, n_tok, mask, D ** -0.5,
                            out=np.full((B, T, c.H, D), -9.0))
    close(out, want, tol)
    assert (out[0, T - 1] == 0).all()
    # causal without a mask; strided queries; another scale
    big = torch.zeros(B, T, c.H, 2, D, device="cuda")
    big[:, :, :, 1] = torch.from_numpy(q).cuda()
    dv.dv_tree_attn(c.cache, big[:, :, :, 1], i32(lens), out, c.ws, scale=-0.05)
    c.ok()
    close(out, *kv_ref.tree(c.ref, q, lens, [T] * B, None, -0.05))


@pytest.mark.parametrize("dtype", ["f16", "i8", "f32"])
@pytest.mark.parametrize("T", [1, 12, 40])
def test_tree_attn_listed_heads(dv, variant, dtype, T):
    """Only the listed KV heads are computed; repeated and bad entries do no harm."""
    skip_same(variant, dtype, 64, 2 * T)
    B, Hkv, G, D, cap = 2, 9, 2, 64 if dtype != "f32" else 32, 190
    c = Case(dv, B, Hkv, G, D, cap, dtype, tokens=T)
    lens, q = [120, 77], c.normal(B, T, Hkv * G, D)
    qd = torch.from_numpy(q).cuda()
    base = np.full((B, T, Hkv * G, D), 5.0)
    out = torch.full(base.shape, 5.0, device="cuda")
    dv.dv_tree_attn(c.cache, qd, i32(lens), out, c.ws, u_h=i32([7, 2, 2, 0, 4]), n_u_h=i32([4]))
    c.ok()
    want, tol = kv_ref.tree(c.ref, q, lens, [T] * B, None, D ** -0.5, heads=[0, 2, 7], out=base)
    close(out, want, tol)
    out.fill_(5.0)
    dv.dv_tree_attn(c.cache, qd, i32(lens), out, c.ws, u_h=i32([0, 9, -1, 8]), n_u_h=i32([4]))
    c.ok(dv.DV_ERR_DEVICE_INDEX)
    want, tol = kv_ref.tree(c.ref, q, lens, [T] * B, None, D ** -0.5, heads=[0, 8], out=base)
    close(out, want, tol)
    out.fill_(5.0)
    dv.dv_tree_attn(c.cache, qd, i32(lens), out, c.ws, u_h=i32([0, 1]), n_u_h=i32([0]))
    c.ok()
    assert (out == 5).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "i8"])
@pytest.mark.parametrize("bad", ["nan", "inf", "huge"])
@pytest.mark.parametrize("T", [6, 24])
def test_unseen_positions_cannot_change_a_result(dv, variant, dtype, bad, T):
    """NaN, infinities and huge values behind the last token and in drafted tokens others see."""
    skip_same(variant, dtype, 64, T)
    B, Hkv, D, cap = 2, 2, 64, 140
    c = Case(dv, B, Hkv, 1, D, cap, dtype, tokens=T, seed=3)
    lens, n_tok = [70, 13], [T - 1, T]
    x = {"nan": np.nan, "inf": np.inf, "huge": 3e4 if dtype == "f16" else 1e30}[bad]
    mask = [random_tree(c.rng, T) for _ in range(B)]
    poisoned = 2
    for b in range(B):
        for t in range(T):
            mask[b][t] &= ~(1 << poisoned) if t != poisoned else ~0
    q = c.normal(B, T, Hkv, D)
    clean, tol = kv_ref.tree(c.ref, q, lens, n_tok, mask, D ** -0.5)
    for b in range(B):
        for p in [lens[b] + poisoned] + list(range(lens[b] + n_tok[b], cap)):
            for t in ("k", "v"):
                if dtype == "i8":
                    c.ref.scale[t][b, :, p] = x
                else:
                    c.ref.raw[t][b, :, p] = x
    c.upload()
    out = torch.zeros(B, T, Hkv, D, device="cuda")
    dv.dv_tree_attn(c.cache, torch.from_numpy(q).cuda(), i32(lens), out, c.ws,
                    mask=mask_tensor(mask), n_tok=i32(n_tok))
    c.ok()
    got = out.double().cpu().numpy()
    for b in range(B):
        for t in range(n_tok[b]):
            if t != poisoned:
                assert (np.abs(got[b, t] - clean[b, t]) <= tol[b, t][:, None]).all(), (b, t)
            elif bad != "huge":
                assert not np.isfinite(got[b, t]).all(-1).any()


@pytest.mark.parametrize("T", [3, 20])
def test_tree_attn_wide_range(dv, variant, T):
    """Scores far apart, weights that underflow, values of very different size."""
    for dtype in ("f32", "f16", "i8"):
        c = Case(dv, 1, 1, 1, 64, 500, dtype)
        q = 40 * c.normal(1, T, 1, 64)
        size = 10.0 ** c.rng.uniform(-3, 3, (1, 1, 500, 1))
        v = (c.ref.values("v") * size).astype(np.float32)
        if dtype == "i8":
            c.ref.raw["v"], c.ref.scale["v"] = kv_ref.quantise(v)
        else:
            c.ref.raw["v"] = v.astype(c.ref.raw["v"].dtype)
        c.upload()
        out = torch.zeros(1, T, 1, 64, device="cuda")
        dv.dv_tree_attn(c.cache, torch.from_numpy(q).cuda(), i32([500 - T]), out, c.ws)
        c.ok()
        close(out, *kv_ref.tree(c.ref, q, [500 - T], [T], None, 0.125))


@pytest.mark.parametrize("T,dtype", [(3, "i8"), (11, "i8"), (11, "f16")])
def test_tree_attn_one_long_row_among_short_ones(dv, variant, T, dtype):
    """Units cut over many CTAs, and many units in one, in one call; twice on one workspace."""
    skip_same(variant, dtype, 128, T)
    B = 40
    c = Case(dv, B, 2, 1, 128, 5000, dtype, tokens=T)
    lens = [4980] + [b % 7 for b in range(1, B)]
    q = c.normal(B, T, 2, 128)
    out = torch.zeros(B, T, 2, 128, device="cuda")
    for _ in range(2):
        out.fill_(1.0)
        dv.dv_tree_attn(c.cache, torch.from_numpy(q).cuda(), i32(lens), out, c.ws)
        c.ok()
        close(out, *kv_ref.tree(c.ref, q, lens, [T] * B, None, 128 ** -0.5))


def test_tree_attn_rules_choose_both_kernels(dv):
    """Sizes on both sides of the launch rule, without a forced variant."""
    for dtype, T, Hkv, cap in (("f16", 30, 8, 1500), ("i8", 64, 12, 1100), ("i8", 12, 2, 300)):
        c = Case(dv, 6, Hkv, 1, 128, cap, dtype, tokens=T)
        lens = [cap - T - 97 * b if cap > 1000 else 40 * b for b in range(6)]
        q = c.normal(6, T, Hkv, 128)
        out = torch.zeros(q.shape, device="cuda")
        dv.dv_tree_attn(c.cache, torch.from_numpy(q).cuda(), i32(lens), out, c.ws)
        c.ok()
        close(out, *kv_ref.tree(c.ref, q, lens, [T] * 6, None, 128 ** -0.5))


# ------------------------------------------------------------------ selected blocks


@pytest.mark.parametrize("dtype", ["f32", "f16", "i8"])
@pytest.mark.parametrize("Hkv,G,D,block,k,first,last,cap", [
    (3, 1, 128, 64, 4, 1, 1, 1000), (2, 4, 128, 32, 9, 0, 2, 777), (2, 1, 64, 16, 20, 2, 1, 2000),
    (1, 2, 64, 128, 3, 1, 1, 900), (2, 1, 32, 16, 2, 1, 1, 400), (1, 1, 128, 16, 30, 0, 1, 9000),
    (1, 1, 128, 64, 1, 0, 1, 300), (1, 1, 32, 16, 40, 1, 1, 20000),
])
def test_block_topk_and_attn(dv, dtype, Hkv, G, D, block, k, first, last, cap):
    B = 5
    c = Case(dv, B, Hkv, G, D, cap, dtype, block)
    lens = [cap, 1, 0, cap // 2 // block * block, cap // 3]
    q = 2 * c.normal(B, c.H, D)
    qd = torch.from_numpy(q).cuda()
    idx = torch.full((B, c.H, k), 77, dtype=torch.int32, device="cuda")
    dv.dv_block_topk(c.cache, qd, i32(lens), idx, c.ws, n_first=first, n_last=last)
    c.ok()
    want = kv_ref.topk(c.ref, q, lens, k, first, last)
    np.testing.assert_array_equal(idx.cpu().numpy(), want)
    out = torch.full((B, c.H, D), -9.0, device="cuda")
    dv.dv_block_attn(c.cache, qd, i32(lens), idx, out, c.ws)
    c.ok()
    close(out, *kv_ref.block_attend(c.ref, q, lens, want, D ** -0.5))
    assert (out[2] == 0).all()


@pytest.mark.parametrize("dtype", ["f16", "i8", "f32"])
def test_block_attn_any_list(dv, dtype):
    """Blocks in any order, holes, entries out of range (reported, skipped)."""
    c = Case(dv, 2, 1, 2, 64, 400, dtype, 32)
    lens, q = [333, 64], c.normal(2, 2, 64)
    idx = np.array([[[10, 0, -1, 4], [-1, -1, -1, -1]], [[1, 0, 7, 7], [0, -1, 1, 1]]], np.int32)
    out = torch.full((2, 2, 64), 3.0, device="cuda")
    dv.dv_block_attn(c.cache, torch.from_numpy(q).cuda(), i32(lens), torch.from_numpy(idx).cuda(),
                     out, c.ws)
    c.ok()
    close(out, *kv_ref.block_attend(c.ref, q, lens, idx, 0.125))
    assert (out[0, 1] == 0).all()
    idx[0, 0] = [10, 11, 0, -2]
    dv.dv_block_attn(c.cache, torch.from_numpy(q).cuda(), i32(lens), torch.from_numpy(idx).cuda(),
                     out, c.ws)
    c.ok(dv.DV_ERR_DEVICE_INDEX)
    close(out, *kv_ref.block_attend(c.ref, q, lens, idx, 0.125))


def test_block_topk_ties_and_extremes(dv):
    """Equal scores go to the lower block; infinite scales first; zero and non-finite queries."""
    c = Case(dv, 1, 1, 1, 32, 16 * 300, "f32", 16)
    c.ref.mean[:] = 1
    c.ref.mean_scale[:] = 0.5
    c.ref.mean_scale[0, 0, 200] = np.inf
    c.ref.mean_scale[0, 0, 100:110] = 0.75
    c.upload()
    for q in (np.ones((1, 1, 32)), -np.ones((1, 1, 32)), np.zeros((1, 1, 32))):
        q = q.astype(np.float32)
        idx = torch.zeros(1, 1, 20, dtype=torch.int32, device="cuda")
        dv.dv_block_topk(c.cache, torch.from_numpy(q).cuda(), i32([4800]), idx, c.ws)
        c.ok()
        np.testing.assert_array_equal(idx.cpu().numpy(), kv_ref.topk(c.ref, q, [4800], 20))
        assert 200 in idx.flatten().tolist()
    q[0, 0, 3] = np.nan
    dv.dv_block_topk(c.cache, torch.from_numpy(q).cuda(), i32([4800]), idx, c.ws)
    c.ok()
    assert idx.flatten().tolist() == [0] + list(range(1, 18)) + [200, 299]


# ------------------------------------------------------------------ together, streams, graphs


@pytest.mark.parametrize("dtype,D", [("i8", 128), ("f16", 64), ("f32", 32)])
def test_a_speculative_decode(dv, variant, dtype, D):
    """Prompt, then rounds of draft, tree attention, keep, and block-sparse decode of one token."""
    B, Hkv, G, T, block, cap = 3, 2, 2, 9, 16, 300
    c = Case(dv, B, Hkv, G, D, cap, dtype, block, tokens=T, seed=9)
    lens = np.array([0, 0, 0])
    n = [150, 37, 16]
    x = c.normal(B, 150, Hkv, D)
    dev = torch.from_numpy(x).cuda()
    dv.dv_kv_append(c.cache, dev, 0.5 * dev, i32(lens), c.ws, n_tok=i32(n))
    c.ref.append(x, 0.5 * x, lens, n)
    lens = lens + n
    for step in range(4):
        k, v, q = c.normal(B, T, Hkv, D), c.normal(B, T, Hkv, D), c.normal(B, T, Hkv * G, D)
        mask = [random_tree(c.rng, T) for _ in range(B)]
        dl = i32(lens)
        dv.dv_kv_append(c.cache, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), dl, c.ws)
        out = torch.zeros(B, T, Hkv * G, D, device="cuda")
        dv.dv_tree_attn(c.cache, torch.from_numpy(q).cuda(), dl, out, c.ws,
                        mask=mask_tensor(mask))
        c.ref.append(k, v, lens, [T] * B)
        close(out, *kv_ref.tree(c.ref, q, lens, [T] * B, mask, D ** -0.5))
        n_keep = c.rng.integers(0, T + 1, B)
        path = np.zeros((B, T), np.int32)
        for b in range(B):
            path[b, :n_keep[b]] = np.sort(c.rng.choice(T, n_keep[b], replace=False))
        dv.dv_kv_keep(c.cache, dl, torch.from_numpy(path).cuda(), i32(n_keep), c.ws)
        c.ref.keep(lens, path, n_keep)
        lens = lens + n_keep
        idx = torch.zeros(B, Hkv * G, 3, dtype=torch.int32, device="cuda")
        o1 = torch.zeros(B, Hkv * G, D, device="cuda")
        q1 = torch.from_numpy(q).cuda()[:, 0]
        dv.dv_block_topk(c.cache, q1, i32(lens), idx, c.ws)
        dv.dv_block_attn(c.cache, q1, i32(lens), idx, o1, c.ws)
        want = kv_ref.topk(c.ref, q[:, 0], lens, 3)
        np.testing.assert_array_equal(idx.cpu().numpy(), want)
        close(o1, *kv_ref.block_attend(c.ref, q[:, 0], lens, want, D ** -0.5))
        c.same_cache()
    c.ok()


def test_one_workspace_for_several_shapes(dv, variant):
    """Calls of different shapes, one after another, leave the workspace ready for each other."""
    big = Case(dv, 4, 4, 1, 128, 700, "i8", tokens=64)
    small = Case(dv, 2, 8, 4, 64, 900, "f16", 32, seed=1)
    for _ in range(2):
        for c, T in ((big, 64), (small, 3), (big, 2)):
            q = c.normal(c.B, T, c.H, c.D)
            out = torch.zeros(q.shape, device="cuda")
            lens = [600 - 90 * b for b in range(c.B)]
            dv.dv_tree_attn(c.cache, torch.from_numpy(q).cuda(), i32(lens), out, big.ws)
            big.ok()
            close(out, *kv_ref.tree(c.ref, q, lens, [T] * c.B, None, c.D ** -0.5))
    short = dv.KvWorkspace(big.desc, 4, 64)
    short.nbytes -= 256
    q = torch.zeros(4, 64, 4, 128, device="cuda")
    with pytest.raises(dv.DvError) as e:
        dv.dv_tree_attn(big.cache, q, i32([0] * 4), torch.zeros_like(q), short)
    assert e.value.status == dv.DV_ERR_WORKSPACE


def test_graph_replay_and_side_stream(dv):
    """One step captured and replayed on new inputs, lengths advancing on the device."""
    B, Hkv, D, T = 3, 4, 128, 1
    c = Case(dv, B, Hkv, 1, D, 600, "i8", 64)
    lens0 = np.array([510, 63, 200])
    lens = i32(lens0)
    kv = torch.zeros(B, T, 2, Hkv, D, device="cuda")
    q = torch.zeros(B, T, Hkv, D, device="cuda")
    out, o2 = torch.zeros_like(q), torch.zeros(B, Hkv, D, device="cuda")
    idx = torch.zeros(B, Hkv, 3, dtype=torch.int32, device="cuda")
    one = torch.ones_like(lens)
    s = torch.cuda.Stream()

    def step():
        dv.dv_kv_append(c.cache, kv[:, :, 0], kv[:, :, 1], lens, c.ws, stream=s)
        dv.dv_tree_attn(c.cache, q, lens, out, c.ws, stream=s)
        with torch.cuda.stream(s):
            lens.add_(one)
        dv.dv_block_topk(c.cache, q[:, 0], lens, idx, c.ws, stream=s)
        dv.dv_block_attn(c.cache, q[:, 0], lens, idx, o2, c.ws, stream=s)

    s.wait_stream(torch.cuda.current_stream())
    saved = {n: getattr(c.cache, n).clone() for n in ("k", "v", "k_scale", "v_scale", "k_mean",
                                                      "k_mean_scale")}
    step()  # (set-up of the kernels before the capture)
    s.synchronize()
    for n, t in saved.items():
        getattr(c.cache, n).copy_(t)
    lens.copy_(i32(lens0))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step()
    for i in range(5):
        k, v, qq = c.normal(B, T, Hkv, D), c.normal(B, T, Hkv, D), c.normal(B, T, Hkv, D)
        kv[:, :, 0].copy_(torch.from_numpy(k))
        kv[:, :, 1].copy_(torch.from_numpy(v))
        q.copy_(torch.from_numpy(qq))
        g.replay()
        torch.cuda.synchronize()
        c.ref.append(k, v, lens0 + i, [1] * B)
        close(out, *kv_ref.tree(c.ref, qq, lens0 + i, [1] * B, None, D ** -0.5))
        want = kv_ref.topk(c.ref, qq[:, 0], lens0 + i + 1, 3)
        np.testing.assert_array_equal(idx.cpu().numpy(), want)
        close(o2, *kv_ref.block_attend(c.ref, qq[:, 0], lens0 + i + 1, want, D ** -0.5))
    c.same_cache()
    c.ok()


def test_results_repeat(dv, variant):
    """The same call twice gives the same bits (units cut over CTAs merge in a fixed order)."""
    c = Case(dv, 2, 3, 2, 128, 3000, "f16", 64, tokens=20)
    q = torch.from_numpy(c.normal(2, 20, 6, 128)).cuda()
    out = [torch.zeros(2, 20, 6, 128, device="cuda") for _ in range(6)]
    for o in out:
        dv.dv_tree_attn(c.cache, q, i32([2900, 1234]), o, c.ws)
    c.ok()
    assert all(torch.equal(out[0], o) for o in out[1:])


@pytest.mark.parametrize("dtype", ["f16", "i8"])
def test_cold_calls_equal_warm_ones(dv, variant, dtype):
    """The first call on a cache whose lines are in no cache, bit for bit as later ones: hand-overs
    inside the kernels must not depend on how long a load takes."""
    T = 11 if variant == 2 else 5
    flush = torch.empty(1 << 28, dtype=torch.int8, device="cuda")
    for seed in range(4):
        c = Case(dv, 40, 2, 1, 128, 3000, dtype, tokens=T, seed=seed)
        lens = i32([2900] + [(b * 37) % 200 for b in range(1, 40)])
        q = torch.from_numpy(c.normal(40, T, 2, 128)).cuda()
        out = [torch.zeros(40, T, 2, 128, device="cuda") for _ in range(4)]
        for i, o in enumerate(out):
            if i < 3:
                flush.fill_(i)
            dv.dv_tree_attn(c.cache, q, lens, o, c.ws)
        c.ok()
        assert all(torch.equal(out[3], o) for o in out)


@pytest.mark.parametrize("dtype", ["f16", "i8"])
@pytest.mark.parametrize("T", [2, 9, 64])
@pytest.mark.parametrize("rise", [0.0, 200.0], ids=["flat", "rising"])
def test_tree_attn_very_long_rows(dv, variant, dtype, T, rise):
    """100000 positions, so many heads that a CTA attends whole rows: sums of thousands of steps.

    Values lie in [1, 2), so a sum cut off at every step shows as a bias.  At most 64 tiles of 64
    (two streams of 32 tiles of 4 steps, or 64 steps) are summed by tensor cores, each step off by
    less than 2^-23 of the sum: 128 of them; sums of up to 64 further roundings; the quotient.
    (3000 steps of a row summed without a limit would lose 3000 x 2^-23 / 6.)  Scores that rise by
    200 move the reference point from chunk to chunk; a score has the rounding of its 64 products'
    sum, 2^-21 of its size, and a weight that times log2(e)."""
    Hkv, D, cap = 160, 64, 100100
    desc = dv.make_kv_desc(Hkv, Hkv, D, cap, DT[dtype])
    g = torch.Generator(device="cuda").manual_seed(T)
    cache = dv.KvCache(desc, 1)
    n = cap - T - 3
    pos = torch.arange(cap, device="cuda") / n
    if dtype == "f16":
        cache.k.normal_(generator=g).mul_(0.25)
        cache.k[..., 0] = pos
        cache.v.uniform_(1, 2, generator=g)
    else:
        cache.k.random_(-100, 101, generator=g)
        cache.k[..., 0] = (100 * pos).round().clamp(max=100).to(torch.int8)
        cache.v.random_(64, 128, generator=g)
        cache.k_scale.fill_(2.0 ** -8)
        cache.v_scale.fill_(2.0 ** -6)
    ws = dv.KvWorkspace(desc, 1, T)
    q = torch.randn(1, T, Hkv, D, generator=g, device="cuda")
    top = cache.k[0, 0, n - 1, 0].double() * (1 if dtype == "f16" else 2.0 ** -8)
    q[..., 0] = rise * D ** 0.5 / top.item()
    out = torch.zeros(1, T, Hkv, D, device="cuda")
    dv.dv_tree_attn(cache, q, i32([n]), out, ws)
    assert dv.dv_check(ws) == 0
    j = torch.arange(n + T, device="cuda")
    seen = j[None] <= n + torch.arange(T, device="cuda")[:, None]
    for h in (0, 77, Hkv - 1):
        k, v = cache.k[0, h, :n + T].double(), cache.v[0, h, :n + T].double()
        if dtype == "i8":
            k, v = k * 2.0 ** -8, v * 2.0 ** -6
        s = (q[0, :, h].double() @ k.T * D ** -0.5).masked_fill(~seen, -torch.inf)
        want = s.softmax(-1) @ v
        size = (q[0, :, h].double().abs() @ k.abs().T * D ** -0.5).max().item()
        tol = 2 * (192 * 2.0 ** -23 + 2 * size * 2.0 ** -21)
        err = (out[0, :, h].double() - want).abs().max().item()
        assert err <= tol, f"off by {err:.3g}, allowed {tol:.3g}"


@pytest.mark.parametrize("dtype", ["f16", "i8"])
@pytest.mark.parametrize("D", [64, 128])
def test_tree_attn_many_long_rows(dv, variant, dtype, D):
    """Several whole rows of more than 64 tiles in every CTA's run, cut ones between them; rows of
    other batch entries end in other tiles, one is empty.  Tolerance as above."""
    B, Hkv, T, cap = 5, 128, 9, 5200
    desc = dv.make_kv_desc(Hkv, Hkv, D, cap, DT[dtype])
    g = torch.Generator(device="cuda").manual_seed(D)
    cache = dv.KvCache(desc, B)
    for t in (cache.k, cache.v):
        t.random_(-100, 101, generator=g)
    if dtype == "i8":
        cache.k_scale.fill_(2.0 ** -6)
        cache.v_scale.fill_(2.0 ** -6)
    else:
        cache.k.mul_(2.0 ** -6)
        cache.v.mul_(2.0 ** -6)
    lens = [cap - T, 4999, 4096, 0, 4160 - T]
    ws = dv.KvWorkspace(desc, B, T)
    q = torch.randn(B, T, Hkv, D, generator=g, device="cuda")
    out = torch.full((B, T, Hkv, D), 7.0, device="cuda")
    dv.dv_tree_attn(cache, q, i32(lens), out, ws)
    assert dv.dv_check(ws) == 0
    unit = 2.0 ** -6 if dtype == "i8" else 1.0
    for b, n in enumerate(lens):
        k, v = (t[b, :, :n + T].double() * unit for t in (cache.k, cache.v))
        s = torch.einsum("thd,hpd->htp", q[b].double(), k) * D ** -0.5
        size = torch.einsum("thd,hpd->htp", q[b].double().abs(), k.abs()).max().item() * D ** -0.5
        j, t = torch.arange(n + T, device="cuda"), torch.arange(T, device="cuda")
        want = s.masked_fill(j > n + t[:, None], -torch.inf).softmax(-1) @ v
        tol = 2 * (192 * 2.0 ** -23 + 2 * size * 2.0 ** -21)
        err = (out[b].double().transpose(0, 1) - want).abs().max().item()
        assert err <= tol, f"row {b} off by {err:.3g}, allowed {tol:.3g}"


def test_offsets_beyond_32_bits(dv):
    """A cache of more than 2^32 values a side: its last row and head."""
    B, Hkv, D, cap, T = 3, 8, 128, (1 << 21) - 77, 4
    desc = dv.make_kv_desc(Hkv, Hkv, D, cap, dv.DV_I8, 128)
    assert B * Hkv * cap * D > 1 << 32
    cache = dv.KvCache(desc, B)
    ws = dv.KvWorkspace(desc, B, T)
    rng = np.random.default_rng(0)
    x = rng.standard_normal((B, 300, Hkv, D)).astype(np.float32)
    lens = i32([0, cap - 300 - T, cap - 300])
    dv.dv_kv_append(cache, torch.from_numpy(x).cuda(), torch.from_numpy(x).cuda(), lens, ws,
                    n_tok=i32([300, 300, 300]))
    codes, scale = kv_ref.quantise(x)
    for b, at in enumerate((0, cap - 300 - T, cap - 300)):
        np.testing.assert_array_equal(cache.k[b, :, at:at + 300].cpu().numpy(),
                                      codes[b].transpose(1, 0, 2))
    out = torch.zeros(B, Hkv, 5, D, device="cuda")
    dv.dv_kv_read(cache, i32([295, cap - 5 - T, cap - 5]), out, out.clone(), ws)
    want = (codes.astype(np.float32) * scale[..., None])[:, 295:].transpose(0, 2, 1, 3)
    np.testing.assert_array_equal(out.cpu().numpy(), want)
    idx = torch.full((B, Hkv, 2), -1, dtype=torch.int32, device="cuda")
    idx[:, :, 0] = (cap - 1) // 128
    idx[:, :, 1] = (cap - 1) // 128 - 1
    q = torch.from_numpy(rng.standard_normal((B, Hkv, D)).astype(np.float32)).cuda()
    o = torch.zeros(B, Hkv, D, device="cuda")
    dv.dv_block_attn(cache, q, i32([cap] * B), idx, o, ws)
    assert dv.dv_check(ws) == 0
    first = ((cap - 1) // 128 - 1) * 128
    for b in range(B):
        kk = (cache.k[b, :, first:].double() * cache.k_scale[b, :, first:, None].double()).cpu()
        vv = (cache.v[b, :, first:].double() * cache.v_scale[b, :, first:, None].double()).cpu()
        for h in range(Hkv):
            w, tol = kv_ref.attend(q[b, h].double().cpu().numpy(), kk[h].numpy(), vv[h].numpy(),
                                   D ** -0.5)
            assert np.abs(o[b, h].double().cpu().numpy() - w).max() <= tol
    del cache
    torch.cuda.empty_cache()


def test_wrappers_check_their_tensors(dv):
    c = Case(dv, 2, 2, 1, 32, 50, "i8", 16)
    q = torch.zeros(2, 3, 2, 32, device="cuda")
    out, lens = torch.zeros_like(q), i32([0, 0])
    for kw in (dict(q=q.bfloat16()), dict(q=q[:1]), dict(q=q.transpose(2, 3)), dict(q=q.cpu()),
               dict(out=out.half()), dict(out=out[:, :2]), dict(lens=lens.long()),
               dict(lens=lens.cpu()), dict(mask=torch.zeros(2, 3, dtype=torch.int32,
                                                            device="cuda")),
               dict(n_tok=lens[:1]), dict(u_h=lens)):
        a = dict(q=q, lens=lens, out=out)
        a.update(kw)
        with pytest.raises(ValueError):
            dv.dv_tree_attn(c.cache, a.pop("q"), a.pop("lens"), a.pop("out"), c.ws, **a)
    with pytest.raises(ValueError):
        dv.KvCache(c.desc, 2, tensors={n: getattr(c.cache, n) for n in ("k", "v")})
    with pytest.raises(dv.DvError):  # rows not on 16-byte steps
        x = torch.zeros(2, 3, 2, 33, device="cuda")[..., :32]
        dv.dv_kv_append(c.cache, x, x, lens, c.ws)
    c.same_cache()
