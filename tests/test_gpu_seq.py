"""The operators over packed sequences and paged caches on the GPU against plain 64-bit ones.

Tables, positions, slots and counts must be equal.  Tolerances of numbers come from seq_ref, which
derives them from each case's values."""

import math

import numpy as np
import pytest
import torch

import seq_ref

pytestmark = pytest.mark.gpu

NP = {"f32": np.float32, "f16": np.float16}
TT = {"f32": torch.float32, "f16": torch.float16}


@pytest.fixture(scope="module")
def dv():
    from attention_dv_predict_gb300 import build

    build.build()
    from attention_dv_predict_gb300 import dv as mod

    return mod


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def close(got, want, tol):
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all()
    bad = np.abs(got - want) > tol
    assert not bad.any(), (f"{bad.sum()} of {bad.size} off, worst {np.abs(got - want).max():.3g}, "
                           f"first at {np.argwhere(bad)[0]}, allowed {tol[bad].max():.3g}")


# ------------------------------------------------------------------ pages


def page_case(rng, B, page, width, spare, tok):
    lens = rng.integers(0, width * page - tok + 1, B)
    n_tok = rng.integers(0, tok + 1, B)
    held = [seq_ref.pages(int(n), page) for n in lens]
    N = sum(held) + spare
    order = rng.permutation(N).astype(np.int32)
    tables = np.full((B, width), -1, np.int32)
    at = 0
    for b in range(B):
        tables[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    free = np.full(N, -1, np.int32)
    free[:N - at] = order[at:]
    return lens, n_tok, tables, free, N - at


@pytest.mark.parametrize("B,page,width,spare,tok", [
    (1, 16, 3, 2, 1), (1, 128, 1, 1, 128), (33, 16, 40, 40, 1), (64, 32, 9, 700, 200),
    (256, 64, 20, 256, 70), (1024, 16, 6, 4000, 33), (5, 32, 4, 3, 64), (40, 16, 30, 25, 90)])
def test_release_and_take(dv, B, page, width, spare, tok):
    """Few spare pages: some requests are not served."""
    rng = np.random.default_rng(B + page)
    lens, n_tok, tables, free, n_free = page_case(rng, B, page, width, spare, tok)
    done = rng.random(B) < 0.3
    n_tok[done] = 0
    T = int(n_tok.sum()) + int(rng.integers(1, 40))
    desc = dv.make_seq_desc(4, 4, 64, dv.DV_F16, page, len(free))
    ws = dv.SeqWorkspace(desc)
    pt = dv.PageTables(desc, B, width, tensors={"tables": i32(tables), "free": i32(free),
                                                "n_free": i32([n_free])})
    dv.dv_page_release(pt, i32(lens), i32(done), ws)
    want_free, mid, st = seq_ref.release(tables, free, n_free, lens, done, page)
    assert dv.dv_check(ws) == st == 0
    assert pt.n_free.item() == mid
    np.testing.assert_array_equal(pt.free.cpu().numpy(), want_free)
    np.testing.assert_array_equal(pt.tables.cpu().numpy(), tables)
    cu, pos, slots = i32([-7] * (B + 1)), i32([-7] * T), i32([-7] * T)
    after = i32([-7])
    want = seq_ref.take(tables, want_free, mid, lens, n_tok, page, T)
    for out in (after, None):  # a count of its own, then in place: the same answers
        dv.dv_page_take(pt, i32(lens), i32(n_tok), cu, pos, slots, ws, n_free_out=out)
        assert dv.dv_check(ws) in (want[5] or {0})
        assert (pt.n_free if out is None else out).item() == want[1]
        for got, w in zip((pt.tables, cu, pos, slots), (want[0], *want[2:5])):
            np.testing.assert_array_equal(got.cpu().numpy(), w)


def test_take_skips_and_reports(dv):
    page, width, B, T = 16, 4, 7, 40
    desc = dv.make_seq_desc(2, 2, 32, dv.DV_F32, page, 20)
    ws = dv.SeqWorkspace(desc)
    free = np.arange(20, dtype=np.int32)[::-1].copy()
    tables = np.full((B, width), 5, np.int32)

    def run(lens, n_tok, n_free, tables=tables, free=free, T=T):
        pt = dv.PageTables(desc, B, width, tensors={"tables": i32(tables), "free": i32(free),
                                                    "n_free": i32([n_free])})
        cu, pos, slots = i32([0] * (B + 1)), i32([0] * T), i32([0] * T)
        dv.dv_page_take(pt, i32(lens), i32(n_tok), cu, pos, slots, ws)
        want = seq_ref.take(tables, free, n_free, lens, n_tok, page, T)
        assert dv.dv_check(ws) in (want[5] or {0})
        assert pt.n_free.item() == want[1]
        for got, w in zip((pt.tables, cu, pos, slots), (want[0], *want[2:5])):
            np.testing.assert_array_equal(got.cpu().numpy(), w)

    run([-1, 3, 60, 5, 65, 0, 2 ** 31 - 1], [2, 2, 9, -1, 0, 3, 2 ** 31 - 1], 20)
    run([0] * B, [17, 33, 1, 16, 0, 0, 9], 4)     # the second and the last are not served
    run([0] * B, [5] * B, 20, T=31)               # more tokens than places
    run([0] * B, [0] * B, 0)
    bad = tables.copy()
    bad[:, 0] = [-1, 20, 3, 4, 5, 6, 7]           # page numbers out of range
    run([3] * B, [2] * B, 20, tables=bad)
    worse = free.copy()
    worse[18:] = [99, -3]
    run([0] * B, [1] * B, 20, free=worse)
    for n in (-1, 21):                            # a count out of range: nothing is taken
        pt = dv.PageTables(desc, B, width, tensors={"tables": i32(tables), "free": i32(free),
                                                    "n_free": i32([n])})
        cu, pos, slots = i32([0] * (B + 1)), i32([0] * T), i32([0] * T)
        dv.dv_page_take(pt, i32([0] * B), i32([1] * B), cu, pos, slots, ws)
        assert dv.dv_check(ws) in (dv.DV_ERR_DEVICE_INDEX, dv.DV_ERR_PAGES)
        assert pt.n_free.item() == n and (slots == -1).all()
        np.testing.assert_array_equal(pt.tables.cpu().numpy(), tables)


def test_release_skips_and_reports(dv):
    page, width, B, N = 16, 4, 5, 12
    desc = dv.make_seq_desc(2, 2, 32, dv.DV_F32, page, N)
    ws = dv.SeqWorkspace(desc)
    tables = np.arange(B * width, dtype=np.int32).reshape(B, width) % N
    free = np.full(N, -1, np.int32)
    for lens, n_free, tab in (([20, -1, 40, 65, 16], 0, tables), ([64] * B, 0, tables),
                              ([64] * B, 9, tables), ([10] * B, -1, tables),
                              ([10] * B, N + 1, tables), ([33] * B, 1, np.where(tables == 5, N, tables)),
                              ([33] * B, 1, np.where(tables == 9, -1, tables))):
        pt = dv.PageTables(desc, B, width, tensors={"tables": i32(tab), "free": i32(free),
                                                    "n_free": i32([n_free])})
        dv.dv_page_release(pt, i32(lens), i32([1] * B), ws)
        assert dv.dv_check(ws) == dv.DV_ERR_DEVICE_INDEX
        if 0 <= n_free <= N:
            want, n, _ = seq_ref.release(tab, free, n_free, lens, [1] * B, page)
        else:
            want, n = free, n_free
        assert pt.n_free.item() == n
        np.testing.assert_array_equal(pt.free.cpu().numpy(), want)


# ------------------------------------------------------------------ norms and rotation


def rope_case(dv, T, H, Hkv, D, rot, src, dst, interleaved=False, norm=None, scaling="none",
              far=5000, page=16, mscale=1.0, seed=0):
    rng = np.random.default_rng(seed)
    qkv = rng.standard_normal((T, H + 2 * Hkv, D)).astype(NP[src])
    pos = rng.integers(0, far, T).astype(np.int32)
    n_pages = seq_ref.pages(T, page) + 2
    slots = rng.permutation(n_pages * page)[:T].astype(np.int32)
    gains = [(1 + 0.2 * rng.standard_normal(D)).astype(np.float32) if norm else None
             for _ in range(2)]
    kw = dict(scaling=scaling, factor=4.0, orig_len=2048.0, low=1.0, high=16.0)
    desc = dv.make_seq_desc(H, Hkv, D, dv.DV_F32 if dst == "f32" else dv.DV_F16, page, n_pages)
    cache, ws = dv.PagedCache(desc), dv.SeqWorkspace(desc)
    cache.k.fill_(7)
    cache.v.fill_(7)
    r = dv.Rope(D, rot, interleaved=interleaved, theta=10000.0, mscale=mscale,
                norm=dv.DV_LAYERNORM if norm == "layer" else dv.DV_RMSNORM, eps=1e-5,
                q_gain=None if gains[0] is None else dev(gains[0]),
                k_gain=None if gains[1] is None else dev(gains[1]), **kw)
    f = seq_ref.freqs(rot, 10000.0, **kw) if rot else None
    want = [seq_ref.rope(qkv[:, lo:hi], pos, f, rot, interleaved, mscale, g, norm == "layer", 1e-5)
            for lo, hi, g in ((0, H, gains[0]), (H, H + Hkv, gains[1]))]
    return qkv, pos, slots, cache, ws, r, want, page


def rounded(want, dst):
    """The tolerance with the result's rounding."""
    x, tol = want
    step = 2.0 ** -24 if dst == "f32" else 2.0 ** -11
    return x, tol + (np.abs(x) + tol) * step + (0 if dst == "f32" else 2.0 ** -25)


def pool_rows(t, slots, page):
    return t.cpu()[slots // page, :, slots % page]


@pytest.mark.parametrize("src,dst", [("f32", "f16"), ("f16", "f16"), ("f32", "f32"),
                                     ("f16", "f32")])
@pytest.mark.parametrize("T,H,Hkv,D,rot,interleaved,norm,scaling", [
    (1, 1, 1, 128, 128, False, "rms", "none"), (37, 32, 8, 128, 128, False, "rms", "linear"),
    (9, 8, 8, 32, 32, True, None, "none"), (70, 72, 72, 128, 64, True, None, "ramp"),
    (5, 6, 2, 64, 48, False, "layer", "base"), (11, 5, 5, 64, 20, False, "rms", "ramp_index"),
    (3, 3, 1, 8, 4, False, "rms", "none"), (4, 4, 2, 16, 10, True, "layer", "none"),
    (300, 16, 1, 128, 0, False, "rms", "none"), (2, 200, 100, 64, 64, False, None, "none")])
def test_rope(dv, src, dst, T, H, Hkv, D, rot, interleaved, norm, scaling):
    qkv, pos, slots, cache, ws, r, want, page = rope_case(
        dv, T, H, Hkv, D, rot, src, dst, interleaved, norm, scaling)
    x = dev(qkv)
    for out in ("f32", "f16"):
        q_out = torch.zeros(T, H, D, dtype=TT[out], device="cuda")
        k_out = torch.zeros(T, Hkv, D, dtype=TT[out], device="cuda")
        dv.dv_qk_rope(r, x[:, :H], x[:, H:H + Hkv], i32(pos), ws, q_out=q_out, k_out=k_out,
                      v=x[:, H + Hkv:], cache=cache, slots=i32(slots))
        assert dv.dv_check(ws) == 0
        close(q_out, *rounded(want[0], out))
        close(k_out, *rounded(want[1], out))
    close(pool_rows(cache.k, slots, page), *rounded(want[1], dst))
    np.testing.assert_array_equal(pool_rows(cache.v, slots, page).numpy(),
                                  qkv[:, H + Hkv:].astype(NP[dst]))
    rest = np.setdiff1d(np.arange(cache.k.shape[0] * page), slots)
    assert (pool_rows(cache.k, rest, page) == 7).all() and (pool_rows(cache.v, rest, page) == 7).all()


def test_rope_wide_heads(dv):
    for src, dst in (("f16", "f16"), ("f32", "f16")):
        qkv, pos, slots, cache, ws, r, want, page = rope_case(dv, 19, 4, 2, 256, 256, src, dst,
                                                              norm="rms")
        x = dev(qkv)
        q_out = torch.zeros(19, 4, 256, dtype=torch.float16, device="cuda")
        dv.dv_qk_rope(r, x[:, :4], x[:, 4:6], i32(pos), ws, q_out=q_out, v=x[:, 6:], cache=cache,
                      slots=i32(slots))
        assert dv.dv_check(ws) == 0
        close(q_out, *rounded(want[0], "f16"))
        close(pool_rows(cache.k, slots, page), *rounded(want[1], "f16"))


@pytest.mark.parametrize("far", [1 << 20, (1 << 31) - 1])
def test_rope_far_positions(dv, far):
    """Angles of far positions: 2^-33 of a turn there is more than the step's own rounding moves."""
    D, T = 128, 64
    rng = np.random.default_rng(3)
    x = rng.standard_normal((T, 2, D)).astype(np.float32)
    pos = rng.integers(far // 2, far, T)
    desc = dv.make_seq_desc(1, 1, D, dv.DV_F32)
    ws = dv.SeqWorkspace(desc)
    r = dv.Rope(D, D, theta=500000.0)
    q, k = dev(x[:, :1]), dev(x[:, 1:])
    dv.dv_qk_rope(r, q, k, i32(pos), ws)
    assert dv.dv_check(ws) == 0
    # the angle in whole 2^-64 turns, as defined, reduced in integers
    steps = [int(v) % (1 << 64) for v in r.steps.cpu().tolist()]
    ang = np.array([[(s * int(p)) % (1 << 64) / 2.0 ** 64 * 2 * math.pi for s in steps] for p in pos])
    for got, row in ((q, x[:, 0]), (k, x[:, 1])):
        a, b = row[:, :D // 2].astype(np.float64), row[:, D // 2:].astype(np.float64)
        want = np.concatenate([a * np.cos(ang) - b * np.sin(ang), b * np.cos(ang) + a * np.sin(ang)], 1)
        tol = np.tile((np.abs(a) + np.abs(b)) * 2.0 ** -21, 2)
        close(got[:, 0], want, tol)
    f = seq_ref.freqs(D, 500000.0)
    np.testing.assert_allclose(np.array(steps) / 2.0 ** 64 * 2 * math.pi, f, rtol=1e-13,
                               atol=1.01 * 2 * math.pi * 2.0 ** -65)  # (half a step)


def test_rope_skips_and_reports(dv):
    T, H, Hkv, D = 6, 3, 3, 64
    qkv, pos, slots, cache, ws, r, want, page = rope_case(dv, T, H, Hkv, D, D, "f32", "f16")
    pos[2] = -1
    slots[3] = -1
    n = cache.k.shape[0] * page
    slots[4] = n
    x = dev(qkv)
    q_out = torch.full((T, H, D), 3.0, dtype=torch.float16, device="cuda")
    dv.dv_qk_rope(r, x[:, :H], x[:, H:2 * H], i32(pos), ws, q_out=q_out, v=x[:, 2 * H:], cache=cache,
                  slots=i32(slots))
    assert dv.dv_check(ws) == dv.DV_ERR_DEVICE_INDEX
    assert dv.dv_check(ws) == 0
    assert (q_out[2] == 3).all()
    on = [0, 1, 3, 4, 5]
    close(q_out[on], *(y[on] for y in rounded(want[0], "f16")))
    on = [0, 1, 5]
    close(pool_rows(cache.k, slots[on], page), *(y[on] for y in rounded(want[1], "f16")))
    rest = np.setdiff1d(np.arange(n), slots[on])
    assert (pool_rows(cache.k, rest, page) == 7).all() and (pool_rows(cache.v, rest, page) == 7).all()


def test_rope_strides_and_in_place(dv):
    """Head-major rows, a slice of a wider projection, and the rows themselves as the result."""
    T, H, D = 21, 4, 64
    rng = np.random.default_rng(1)
    desc = dv.make_seq_desc(H, H, D, dv.DV_F32)
    ws, r = dv.SeqWorkspace(desc), dv.Rope(D, D)
    x = rng.standard_normal((2, H, T, D)).astype(np.float32)
    pos = np.arange(T, dtype=np.int32)
    t = dev(x)
    q, k = t[0].transpose(0, 1), t[1].transpose(0, 1)
    dv.dv_qk_rope(r, q, k, i32(pos), ws)
    f = seq_ref.freqs(D, 10000.0)
    for got, w in ((q, x[0]), (k, x[1])):
        close(got, *rounded(seq_ref.rope(w.transpose(1, 0, 2), pos, f, D), "f32"))
    wide = dev(rng.standard_normal((T, 3 * H, 2 * D)).astype(np.float32))
    before = wide.clone()
    q, k = wide[:, :H, D:], wide[:, 2 * H:, :D]
    qn, kn = q.cpu().numpy().copy(), k.cpu().numpy().copy()
    dv.dv_qk_rope(r, q, k, i32(pos), ws)
    for got, w in ((q, qn), (k, kn)):
        close(got, *rounded(seq_ref.rope(w, pos, f, D), "f32"))
    before[:, :H, D:], before[:, 2 * H:, :D] = q, k
    assert torch.equal(wide, before)  # nothing else has moved


# ------------------------------------------------------------------ attention


class Seqs:
    """Random requests: packed new tokens, pages in a random order, and their host twins."""

    def __init__(self, dv, toks, lens, Hkv, G, D, dtype, page=0, spare=2, seed=0, behind=0,
                 q_scale=2.0):
        self.dv, self.toks, self.lens, self.dtype, self.page = dv, toks, lens, dtype, page
        self.Hkv, self.H, self.D = Hkv, Hkv * G, D
        rng = self.rng = np.random.default_rng(seed)
        self.cu = np.cumsum([0] + list(toks)).astype(np.int32)
        self.T = int(self.cu[-1]) + behind
        B, t = len(toks), NP[dtype]
        wide = self.H + 2 * Hkv
        qkv = rng.standard_normal((self.T, wide, D)).astype(t)
        qkv[:, :self.H] *= t(q_scale)
        self.qkv = qkv
        self.q = qkv[:, :self.H]
        ends = [a + n for a, n in zip(lens, toks)]
        self.K, self.V = [], []
        if page:
            held = [seq_ref.pages(n, page) for n in ends]
            self.width = max(held + [1]) + 1
            self.n_pages = sum(held) + spare
            order = rng.permutation(self.n_pages).astype(np.int32)
            self.tables = np.full((B, self.width), -1, np.int32)
            at = 0
            for b in range(B):
                self.tables[b, :held[b]] = order[at:at + held[b]]
                at += held[b]
            shape = (self.n_pages, Hkv, page, D)
            self.pk, self.pv = (rng.standard_normal(shape).astype(t) for _ in range(2))
            for b in range(B):
                pg = self.tables[b, :held[b]]
                for dst, pool in ((self.K, self.pk), (self.V, self.pv)):
                    dst.append(pool[pg].transpose(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :ends[b]])
        else:
            self.n_pages = 0
            for b in range(B):
                rows = qkv[self.cu[b]:self.cu[b + 1]].transpose(1, 0, 2)
                self.K.append(rows[self.H:self.H + Hkv])
                self.V.append(rows[self.H + Hkv:])
        self.desc = dv.make_seq_desc(self.H, Hkv, D, dv.DV_F32 if dtype == "f32" else dv.DV_F16,
                                     page, self.n_pages)
        self.ws = dv.SeqWorkspace(self.desc)
        self.out = torch.full((self.T, self.H, D), 9.0, dtype=TT[dtype], device="cuda")
        self.upload()

    def upload(self):
        self.x = dev(self.qkv)
        if self.page:
            self.cache = self.dv.PagedCache(self.desc, tensors={"k": dev(self.pk), "v": dev(self.pv)})
            self.d_lens, self.d_tables = i32(self.lens), i32(self.tables)
        self.d_cu = i32(self.cu)

    def run(self, max_tok=None, scale=None, out=None):
        out = self.out if out is None else out
        q = self.x[:, :self.H]
        if self.page:
            self.dv.dv_paged_attn(self.cache, q, self.d_cu, self.d_lens, self.d_tables, out, self.ws,
                                  max_tok=max_tok, scale=scale)
        else:
            self.dv.dv_prompt_attn(self.desc, q, self.x[:, self.H:self.H + self.Hkv],
                                   self.x[:, self.H + self.Hkv:], self.d_cu, out, self.ws,
                                   max_tok=max_tok, scale=scale)
        return out

    def want(self, scale=None):
        scale = self.D ** -0.5 if scale is None else scale
        return seq_ref.packed(self.q, self.K, self.V, self.cu,
                              self.lens if self.page else [0] * len(self.toks), scale,
                              self.dtype == "f16", out=np.full(self.q.shape, 9.0))

    def check(self, max_tok=None, scale=None, status=0):
        out = self.run(max_tok, scale)
        assert self.dv.dv_check(self.ws) == status
        close(out, *self.want(scale))


KINDS = [("f32", 32), ("f32", 8), ("f32", 128), ("f16", 128), ("f16", 64), ("f16", 32),
         ("f16", 256), ("f16", 16)]


@pytest.mark.parametrize("dtype,D", KINDS)
@pytest.mark.parametrize("Hkv,G", [(1, 1), (2, 4), (3, 3), (1, 5)])
@pytest.mark.parametrize("toks", [[1], [127], [128], [129], [0, 5, 0, 33, 64, 1, 0], [257, 300],
                                  [7] * 20, [640]])
def test_prompt(dv, dtype, D, Hkv, G, toks):
    Seqs(dv, toks, [0] * len(toks), Hkv, G, D, dtype, behind=3).check()


@pytest.mark.parametrize("dtype,D", [("f32", 32), ("f32", 64), ("f16", 128), ("f16", 64), ("f16", 32)])
@pytest.mark.parametrize("Hkv,G", [(2, 1), (1, 8), (2, 7)])
@pytest.mark.parametrize("toks,lens,page", [
    ([1], [0], 16), ([1], [575], 16), ([1] * 9, [0, 1, 15, 16, 127, 128, 129, 300, 4000], 16),
    ([1, 130, 0, 17, 2], [1000, 5, 77, 0, 127], 32), ([200], [1300], 64), ([256, 257], [128, 0], 128),
    ([33] * 5, [64, 63, 65, 0, 900], 64)])
def test_paged(dv, dtype, D, Hkv, G, toks, lens, page):
    Seqs(dv, toks, lens, Hkv, G, D, dtype, page, behind=2).check(max_tok=max(toks))


@pytest.mark.parametrize("dtype,D", [("f32", 32), ("f16", 128), ("f16", 64)])
def test_longer(dv, dtype, D):
    """Many tiles: units cut over CTAs, in pairs and alone, and a token after a long past."""
    Seqs(dv, [1500, 1, 700], [0] * 3, 1, 2, D, dtype).check()
    Seqs(dv, [1, 1, 1], [20000, 3, 9000], 1, 4, D, dtype, 16).check(max_tok=1)
    Seqs(dv, [300, 1], [9000, 12000], 1, 1, D, dtype, 64).check()


def test_many_requests(dv):
    """More requests than threads scan at once, most of them empty."""
    rng = np.random.default_rng(0)
    toks = [int(x) for x in rng.integers(0, 4, 1024) * (rng.random(1024) < 0.5)]
    for dtype, D in (("f32", 32), ("f16", 64)):
        Seqs(dv, toks, [0] * 1024, 2, 2, D, dtype).check()
        lens = [int(x) for x in rng.integers(0, 40, 1024)]
        Seqs(dv, toks, lens, 1, 2, D, dtype, 16).check()


@pytest.mark.parametrize("dtype,D", [("f32", 32), ("f16", 128), ("f16", 64), ("f16", 32)])
def test_all_empty(dv, dtype, D):
    c = Seqs(dv, [0, 0, 0], [5, 0, 3], 2, 2, D, dtype, 16, behind=4)
    c.check()
    c = Seqs(dv, [0, 0, 0], [0, 0, 0], 2, 2, D, dtype, behind=4)
    c.check()


@pytest.mark.parametrize("dtype,D", [("f32", 32), ("f16", 128), ("f16", 64), ("f16", 256)])
@pytest.mark.parametrize("page", [0, 32])
def test_unseen_rows_may_hold_anything(dv, dtype, D, page):
    """NaN and infinities behind a row's own position, in other requests and in unused page rows
    change no bit."""
    toks, lens = [200, 90, 1, 131], [60, 0, 40, 7] if page else [0] * 4
    c = Seqs(dv, toks, lens, 2, 2, D, dtype, page, behind=5)
    c.check()
    clean = c.out.clone()
    for bad in (np.nan, np.inf, -np.inf):
        d = Seqs(dv, toks, lens, 2, 2, D, dtype, page, behind=5)
        cut = 150  # of the first request: its rows from there on are poisoned
        H, Hkv = d.H, d.Hkv
        if page:
            end = lens[0] + cut
            used = np.zeros((d.n_pages, page), bool)
            for b in range(4):
                for p in range(end if b == 0 else lens[b] + toks[b]):
                    used[d.tables[b, p // page], p % page] = True
            d.pk.transpose(0, 2, 1, 3)[~used] = bad
            d.pv.transpose(0, 2, 1, 3)[~used] = bad
        else:
            d.qkv[cut:200, H:] = bad
        d.qkv[cut:200, :H] = bad
        d.qkv[-5:] = bad
        d.upload()
        d.run()
        assert torch.equal(d.out[:cut], clean[:cut]) and torch.equal(d.out[200:], clean[200:])
        assert not torch.isfinite(d.out[cut:200].float()).any()


@pytest.mark.parametrize("dtype,D", [("f32", 32), ("f16", 128), ("f16", 64)])
def test_seen_nan_shows(dv, dtype, D):
    for n in (100, 400):
        for at in (0, 37, n - 1):
            for what in ("k", "v"):
                c = Seqs(dv, [n], [0], 1, 1, D, dtype)
                c.qkv[at, 1 if what == "k" else 2, 3] = np.nan
                c.upload()
                c.run()
                fine = torch.isfinite(c.out[:, 0].float())
                assert fine[:at].all()
                assert not fine[at:, 3].any()


@pytest.mark.parametrize("dtype,D", [("f32", 32), ("f16", 128), ("f16", 64)])
def test_scores_that_rise_and_fall(dv, dtype, D):
    """Scores along the positions that outgrow any fixed range of weights, and one far outlier."""
    n = 700
    for seed, ramp in enumerate((np.linspace(-60, 60, n), np.linspace(60, -60, n),
                                 np.where(np.arange(n) == 333, 100, 0), np.full(n, -90.0))):
        c = Seqs(dv, [n], [0], 1, 1, D, dtype, seed=seed)
        c.qkv[:, 0] = 0
        c.qkv[:, 0, 0] = 4
        c.qkv[:, 1, 0] = ramp / 4 * math.sqrt(D)
        c.upload()
        c.K = [c.qkv[:, 1:2].transpose(1, 0, 2)]
        c.V = [c.qkv[:, 2:3].transpose(1, 0, 2)]
        c.q = c.qkv[:, :1]
        c.check()


@pytest.mark.parametrize("dtype,D", [("f32", 32), ("f16", 128)])
def test_scale(dv, dtype, D):
    for scale in (1e-6, 0.02, 1.0):
        Seqs(dv, [150, 3], [0, 0], 2, 1, D, dtype, q_scale=0.5).check(scale=scale)


@pytest.mark.parametrize("dtype,D", [("f32", 32), ("f16", 128), ("f16", 64)])
def test_bad_requests_are_skipped(dv, dtype, D):
    c = Seqs(dv, [40, 9, 70, 3], [10, 20, 0, 5], 2, 2, D, dtype, 16)
    want, tol = c.want()
    for cu, lens in ((None, [10, -1, 0, 5]), (None, [10, 2 ** 31 - 1, 0, 5]),
                     ([0, 40, 39, 119, 122], None), ([0, 40, 49, 119, 123], None),
                     ([-1, 40, 49, 119, 122], None)):
        if cu is not None:
            c.d_cu = i32(cu)
        if lens is not None:
            c.d_lens = i32(lens)
        c.out.fill_(9)
        c.run()
        assert dv.dv_check(c.ws) == dv.DV_ERR_DEVICE_INDEX
        rows = np.ones(c.T, bool)
        if lens is not None:
            rows[40:49] = False
            assert (c.out[40:49] == 9).all()
        elif cu[2] == 39:  # (the second runs backwards; the third is another request)
            rows[39:119] = False
        elif cu[4] == 123:
            rows[119:] = False
            assert (c.out[119:] == 9).all()
        else:
            rows[:40] = False
            assert (c.out[:40] == 9).all()
        close(c.out[rows], want[rows], tol[rows])
        c.upload()
    # more tokens than max_tok says
    c.out.fill_(9)
    c.run(max_tok=69)
    assert dv.dv_check(c.ws) == dv.DV_ERR_DEVICE_INDEX
    assert (c.out[49:119] == 9).all()
    close(c.out[:49], want[:49], tol[:49])


@pytest.mark.parametrize("dtype,D", [("f32", 32), ("f16", 128), ("f16", 64)])
def test_bad_pages_read_as_zeros(dv, dtype, D):
    for bad in (-1, 2 ** 30, None):
        c = Seqs(dv, [40, 9], [100, 20], 2, 2, D, dtype, 16)
        c.d_tables[0, 3] = c.n_pages if bad is None else bad
        for t in (c.K, c.V):
            t[0] = t[0].copy()
            t[0][:, 48:64] = 0
        c.check(status=dv.DV_ERR_DEVICE_INDEX)


@pytest.mark.parametrize("dtype,D", [("f32", 32), ("f16", 128), ("f16", 64)])
def test_strides(dv, dtype, D):
    """Head-major rows and slices of wider ones."""
    T, H, Hkv = 150, 4, 2
    rng = np.random.default_rng(2)
    q, k, v = (rng.standard_normal((h, T, D)).astype(NP[dtype]) for h in (H, Hkv, Hkv))
    desc = dv.make_seq_desc(H, Hkv, D, dv.DV_F32 if dtype == "f32" else dv.DV_F16)
    ws = dv.SeqWorkspace(desc)
    out = torch.zeros(T, H, D, dtype=TT[dtype], device="cuda")
    want, tol = seq_ref.packed(q.transpose(1, 0, 2), [k], [v], [0, T], [0], D ** -0.5,
                               dtype == "f16")
    dv.dv_prompt_attn(desc, dev(q).transpose(0, 1), dev(k).transpose(0, 1), dev(v).transpose(0, 1),
                      i32([0, T]), out, ws)
    assert dv.dv_check(ws) == 0
    close(out, want, tol)
    wide = torch.zeros(T, 2 * H, 2 * D, dtype=TT[dtype], device="cuda")
    wide[:, H:, D:] = dev(q).transpose(0, 1)
    dv.dv_prompt_attn(desc, wide[:, H:, D:], dev(k).transpose(0, 1), dev(v).transpose(0, 1),
                      i32([0, T]), out, ws)
    close(out, want, tol)
    with pytest.raises(dv.DvError):  # one row for all heads
        dv.dv_prompt_attn(desc, dev(q).transpose(0, 1), dev(k[:1]).transpose(0, 1).expand(T, Hkv, D),
                          dev(v).transpose(0, 1), i32([0, T]), out, ws)


def test_results_repeat(dv):
    for args in (([300, 1, 129], [4000, 9000, 0], 2, 4, 128, "f16", 16),
                 ([1] * 30, list(range(0, 6000, 200)), 2, 2, 64, "f16", 32),
                 ([100, 7], [900, 0], 2, 2, 32, "f32", 16)):
        c = Seqs(dv, *args)
        first = c.run().clone()
        for _ in range(20):
            c.out.fill_(0)
            assert torch.equal(c.run(), first)
        # its rows alone in a call: the same to rounding, and another workspace's contents no matter
        c.ws = dv.SeqWorkspace(c.desc)
        assert torch.equal(c.run(), first)


# ------------------------------------------------------------------ together


def step(dv, s, x, n_tok, out):
    """One serving step over the new tokens' projection x [T, H + 2 Hkv, D]."""
    H, Hkv = s["desc"].n_heads, s["desc"].n_kv_heads
    dv.dv_page_take(s["pt"], s["lens"], n_tok, s["cu"], s["pos"], s["slots"], s["ws"])
    dv.dv_qk_rope(s["rope"], x[:, :H], x[:, H:H + Hkv], s["pos"], s["ws"], q_out=s["q"],
                  v=x[:, H + Hkv:], cache=s["cache"], slots=s["slots"])
    dv.dv_paged_attn(s["cache"], s["q"], s["cu"], s["lens"], s["pt"].tables, out, s["ws"])


def serving(dv, B, H, Hkv, D, page, n_pages, width, T, dtype):
    desc = dv.make_seq_desc(H, Hkv, D, dv.DV_F32 if dtype == "f32" else dv.DV_F16, page, n_pages)
    gain = torch.ones(D, device="cuda")
    return {"desc": desc, "ws": dv.SeqWorkspace(desc), "cache": dv.PagedCache(desc),
            "pt": dv.PageTables(desc, B, width), "lens": i32([0] * B),
            "cu": i32([0] * (B + 1)), "pos": i32([0] * T), "slots": i32([0] * T),
            "q": torch.zeros(T, H, D, dtype=TT[dtype], device="cuda"),
            "rope": dv.Rope(D, D, theta=10000.0, q_gain=gain, k_gain=gain, eps=1e-6)}


@pytest.mark.parametrize("dtype,D", [("f16", 128), ("f32", 32)])
def test_a_serving_run(dv, dtype, D):
    """Prompts in chunks, then single tokens, some requests finished and others begun in their
    pages: every step equals attention over the whole history."""
    B, H, Hkv, page, T = 6, 8, 2, 16, 256
    rng = np.random.default_rng(5)
    s = serving(dv, B, H, Hkv, D, page, 60, 20, T, dtype)
    hist = [[] for _ in range(B)]  # each request's projections so far
    f = seq_ref.freqs(D, 10000.0)
    plan = [[40, 0, 17, 100, 1, 33], [60, 30, 1, 1, 1, 1], [1, 1, 1, 1, 1, 1], None,
            [1, 90, 1, 64, 1, 1], [1] * B]
    lens = np.zeros(B, np.int64)
    for n_tok in plan:
        if n_tok is None:  # the fourth and the second have finished
            done = [0, 1, 0, 1, 0, 0]
            dv.dv_page_release(s["pt"], s["lens"], i32(done), s["ws"])
            for b in range(B):
                if done[b]:
                    hist[b], lens[b] = [], 0
            s["lens"].copy_(i32(lens))
            continue
        n = sum(n_tok)
        x = rng.standard_normal((T, H + 2 * Hkv, D)).astype(NP[dtype])
        out = torch.full((T, H, D), 9.0, dtype=TT[dtype], device="cuda")
        step(dv, s, dev(x), i32(n_tok), out)
        assert dv.dv_check(s["ws"]) == 0
        assert (out[n:] == 9).all()
        cu = np.cumsum([0] + n_tok)
        for b in range(B):
            hist[b] += list(x[cu[b]:cu[b + 1]])
            if not n_tok[b]:
                continue
            rows = np.stack(hist[b])
            pos = np.arange(len(rows))
            k = seq_ref.rope(rows[:, H:H + Hkv], pos, f, D, gain=np.ones(D))[0].astype(NP[dtype])
            q = seq_ref.rope(x[cu[b]:cu[b + 1], :H], pos[lens[b]:], f, D, gain=np.ones(D))[0]
            q = q.astype(NP[dtype])
            for h in range(H):
                K, V = k[:, h // 4], rows[:, H + Hkv + h // 4]
                want, tol = seq_ref.attend(q[:, h].astype(np.float64), K.astype(np.float64),
                                           V.astype(np.float64), pos[lens[b]:], D ** -0.5,
                                           dtype == "f16")
                # q and k may round the other way: a step of 2^-10 (2^-22) of each of D products,
                # independent of the others; their sum is below the largest times sqrt(D) steps,
                # and rows normalised to length sqrt(D) bound it by 2 sqrt(D) steps a score
                eps = (2.0 ** -10 if dtype == "f16" else 2.0 ** -20) * 2 * math.sqrt(D) * D ** -0.5
                tol = tol + 4 * eps * np.abs(V.astype(np.float64)).max()
                close(out[cu[b]:cu[b + 1], h], want, tol)
        lens += n_tok
        s["lens"].copy_(i32(lens))
    held = sum(seq_ref.pages(int(n), page) for n in lens)
    assert s["pt"].n_free.item() == 60 - held
    own = [s["pt"].tables[b, :seq_ref.pages(int(lens[b]), page)].tolist() for b in range(B)]
    flat = sum(own, []) + s["pt"].free[:60 - held].tolist()
    assert sorted(flat) == list(range(60))  # no page lost, none held twice


def test_prompt_paged_and_tree_agree(dv):
    """The same tokens as one packed prompt, in pages, and (their last 64) as drafted tokens over a
    contiguous cache."""
    n, H, Hkv, D, page = 500, 8, 2, 128, 16
    c = Seqs(dv, [n], [0], Hkv, H // Hkv, D, "f16")
    c.check()
    want, tol = c.want()
    n_pages = seq_ref.pages(n, page)
    s = serving(dv, 1, H, Hkv, D, page, n_pages, n_pages, n, "f16")
    s["rope"] = dv.Rope(D, 0)  # (no norm, no rotation: rows as they are)
    out = torch.zeros(n, H, D, dtype=torch.float16, device="cuda")
    step(dv, s, c.x, i32([n]), out)
    assert dv.dv_check(s["ws"]) == 0
    close(out, want, tol)
    kd = dv.make_kv_desc(H, Hkv, D, n, dv.DV_F16)
    cache, ws = dv.KvCache(kd, 1), dv.KvWorkspace(kd, 1, 64)
    x = c.x[None]
    dv.dv_kv_append(cache, x[:, :, H:H + Hkv], x[:, :, H + Hkv:], i32([0]), ws)
    tree = torch.zeros(1, 64, H, D, device="cuda")
    dv.dv_tree_attn(cache, x[:, n - 64:, :H], i32([n - 64]), tree, ws)
    assert dv.dv_check(ws) == 0
    close(tree[0], want[n - 64:], tol[n - 64:])


def test_captured_step(dv):
    """A step captured once and replayed with other lengths, counts and data."""
    B, H, Hkv, D, page, T, width = 4, 8, 2, 128, 16, 96, 30
    s = serving(dv, B, H, Hkv, D, page, 80, width, T, "f16")
    x = torch.zeros(T, H + 2 * Hkv, D, dtype=torch.float16, device="cuda")
    out = torch.zeros(T, H, D, dtype=torch.float16, device="cuda")
    n_tok = i32([1] * B)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        step(dv, s, x, n_tok, out)
    free0 = s["pt"].n_free.item()
    assert free0 == 80  # nothing has run yet
    twin = serving(dv, B, H, Hkv, D, page, 80, width, T, "f16")
    rng = np.random.default_rng(9)
    lens = np.zeros(B, np.int64)
    for toks in ([20, 1, 40, 3], [1, 0, 1, 60], [1, 1, 1, 1], [30, 30, 0, 30]):
        data = dev(rng.standard_normal(tuple(x.shape)).astype(np.float16))
        for d in (s, twin):
            d["lens"].copy_(i32(lens))
        x.copy_(data)
        n_tok.copy_(i32(toks))
        out.fill_(5)
        graph.replay()
        ref = torch.full_like(out, 5)
        step(dv, twin, data, i32(toks), ref)
        assert dv.dv_check(s["ws"]) == 0 and dv.dv_check(twin["ws"]) == 0
        assert torch.equal(out, ref)
        assert torch.equal(s["pt"].tables, twin["pt"].tables)
        lens += toks


def test_two_streams_at_once(dv):
    """Calls on two streams, a workspace each."""
    cs = [Seqs(dv, [300, 1, 64], [2000, 5000, 0], 2, 4, 128, "f16", 16, seed=i) for i in range(2)]
    alone = [c.run().clone() for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, st in zip(cs, streams):
            with torch.cuda.stream(st):
                c.run()
        torch.cuda.synchronize()
        for c, want in zip(cs, alone):
            assert torch.equal(c.out, want)
            assert dv.dv_check(c.ws) == 0
            c.out.fill_(0)
        torch.cuda.synchronize()


# ------------------------------------------------------------------ edges of the ranges


@pytest.mark.parametrize("Hkv,G", [(1, 256), (1, 160), (1, 131), (2, 48), (1, 12)])
def test_wide_groups(dv, Hkv, G):
    """Query heads that fill a unit's rows alone, do not divide them, or are a prime number."""
    for D, dtype in ((64, "f16"), (32, "f32")):
        Seqs(dv, [5, 70], [0, 0], Hkv, G, D, dtype).check()
        Seqs(dv, [1, 1, 3], [200, 0, 77], Hkv, G, D, dtype, 16).check(max_tok=3)


def test_pool_beyond_32_bits(dv):
    """Pages behind the first 2^31 elements of a pool, written by dv_qk_rope and attended."""
    H, Hkv, D, page = 8, 8, 128, 128
    n_pages = (1 << 31) // (Hkv * page * D) + 40
    desc = dv.make_seq_desc(H, Hkv, D, dv.DV_F16, page, n_pages)
    shape = (n_pages, Hkv, page, D)
    cache = dv.PagedCache(desc, tensors={n: torch.empty(shape, dtype=torch.float16, device="cuda")
                                         for n in ("k", "v")})
    ws = dv.SeqWorkspace(desc)
    T = 300
    rng = np.random.default_rng(0)
    qkv = rng.standard_normal((T, 3 * H, D)).astype(np.float16)
    x = dev(qkv)
    table = np.array([[n_pages - 1, n_pages - 30, n_pages - 7]], np.int32)
    pos = np.arange(T, dtype=np.int32)
    slots = table[0, pos // page] * page + pos % page
    q = torch.zeros(T, H, D, dtype=torch.float16, device="cuda")
    dv.dv_qk_rope(dv.Rope(D, 0), x[:, :H], x[:, H:2 * H], i32(pos), ws, q_out=q, v=x[:, 2 * H:],
                  cache=cache, slots=i32(slots))
    out = torch.zeros(T, H, D, dtype=torch.float16, device="cuda")
    dv.dv_paged_attn(cache, q, i32([0, T]), i32([0]), i32(table), out, ws)
    assert dv.dv_check(ws) == 0
    K = qkv[:, H:2 * H].transpose(1, 0, 2)
    V = qkv[:, 2 * H:].transpose(1, 0, 2)
    close(out, *seq_ref.packed(qkv[:, :H], [K], [V], [0, T], [0], D ** -0.5, True))
    one = torch.zeros(1, H, D, dtype=torch.float16, device="cuda")
    dv.dv_paged_attn(cache, q[-1:], i32([0, 1]), i32([T - 1]), i32(table), one, ws, max_tok=1)
    want, tol = seq_ref.packed(qkv[-1:, :H], [K], [V], [0, 1], [T - 1], D ** -0.5, True)
    close(one, want, tol)


def test_first_call_inside_a_capture(dv):
    """Each operator's first call of a process may be a captured one, on a stream of its own."""
    import subprocess
    import sys

    code = """
import sys; sys.path.insert(0, %r); sys.path.insert(0, %r)
import torch
from attention_dv_predict_gb300 import dv
from test_gpu_seq import serving, step, i32
s = serving(dv, 2, 4, 2, 64, 16, 20, 8, 40, "f16")
x = torch.randn(40, 8, 64, device="cuda").half()
out = torch.zeros(40, 4, 64, dtype=torch.float16, device="cuda")
n_tok, done = i32([30, 10]), i32([1, 0])
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    dv.dv_page_release(s["pt"], s["lens"], done, s["ws"])
    step(dv, s, x, n_tok, out)
    dv.dv_prompt_attn(s["desc"], x[:, :4], x[:, 4:6], x[:, 6:], s["cu"], out, s["ws"])
g.replay()
assert dv.dv_check(s["ws"]) == 0 and torch.isfinite(out).all() and out.abs().sum() > 0
st = torch.cuda.Stream()
st.wait_stream(torch.cuda.current_stream())
want = out.clone()
out.zero_()
torch.cuda.synchronize()
dv.dv_prompt_attn(s["desc"], x[:, :4], x[:, 4:6], x[:, 6:], s["cu"], out, s["ws"], stream=st)
st.synchronize()
assert torch.equal(out, want)
"""
    import os

    here = os.path.dirname(os.path.abspath(__file__))
    subprocess.run([sys.executable, "-c", code % (os.path.dirname(here), here)], check=True,
                   timeout=300)


def test_wrappers_refuse(dv):
    T, H, Hkv, D, page = 8, 4, 2, 64, 16
    desc = dv.make_seq_desc(H, Hkv, D, dv.DV_F16, page, 10)
    cache, ws, pt = dv.PagedCache(desc), dv.SeqWorkspace(desc), dv.PageTables(desc, 2, 3)
    x = torch.zeros(T, H + 2 * Hkv, D, dtype=torch.float16, device="cuda")
    q, k, v = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
    out = torch.zeros(T, H, D, dtype=torch.float16, device="cuda")
    cu, lens, pos, slots = i32([0, 4, 8]), i32([0, 0]), i32(range(T)), i32(range(T))
    r = dv.Rope(D, D)

    def prompt(**kw):
        a = dict(desc=desc, q=q, k=k, v=v, cu=cu, out=out, ws=ws)
        a.update(kw)
        dv.dv_prompt_attn(**a)

    def paged(**kw):
        a = dict(cache=cache, q=q, cu=cu, lens=lens, tables=pt.tables, out=out, ws=ws)
        a.update(kw)
        dv.dv_paged_attn(**a)

    def rope(**kw):
        a = dict(rope=r, q=q, k=k, pos=pos, ws=ws, q_out=out, v=v, cache=cache, slots=slots)
        a.update(kw)
        dv.dv_qk_rope(**a)

    def take(**kw):
        a = dict(pt=pt, lens=lens, n_tok=lens, cu=cu, pos=pos, slots=slots, ws=ws)
        a.update(kw)
        dv.dv_page_take(**a)

    prompt(), rope(), take()
    assert dv.dv_check(ws) == 0
    bad = [(prompt, dict(q=q.float())), (prompt, dict(q=q[:, :3])), (prompt, dict(q=q[0])),
           (prompt, dict(k=q)), (prompt, dict(v=v.cpu())), (prompt, dict(cu=cu.long())),
           (prompt, dict(out=out.float())), (prompt, dict(out=x[:, :H])),
           (prompt, dict(q=x.transpose(1, 2)[:, :H, :H])), (prompt, dict(scale=0.0)),
           (prompt, dict(max_tok=0)), (paged, dict(lens=cu)), (paged, dict(tables=pt.tables[0])),
           (paged, dict(lens=lens.cpu())), (paged, dict(q=q[:, :, :32])),
           (rope, dict(k=q)), (rope, dict(slots=None)), (rope, dict(cache=None)),
           (rope, dict(pos=pos[:4])), (rope, dict(rope=dv.Rope(32, 32))),
           (rope, dict(q_out=out[:4])), (rope, dict(k=k.float())),
           (take, dict(cu=cu[:2])), (take, dict(slots=slots[:4])), (take, dict(lens=lens.long()))]
    for f, kw in bad:
        with pytest.raises((ValueError, dv.DvError)):
            f(**kw)
    for f in (lambda: dv.PagedCache(dv.make_seq_desc(H, Hkv, D, dv.DV_F16)),
              lambda: dv.PageTables(dv.make_seq_desc(H, Hkv, D, dv.DV_F16), 2, 3),
              lambda: dv.SeqWorkspace(dv.make_seq_desc(H, 3, D, dv.DV_F16)),
              lambda: dv.PagedCache(desc, tensors={"k": cache.k}),
              lambda: dv.PagedCache(desc, tensors={"k": cache.k, "v": cache.v.float()}),
              lambda: dv.Rope(D, 7), lambda: dv.Rope(D, D, theta=0.5),
              lambda: dv.Rope(D, D, q_gain=torch.ones(3, device="cuda"))):
        with pytest.raises((ValueError, dv.DvError)):
            f()
    assert dv.dv_check(ws) == 0


@pytest.mark.parametrize("dtype,D", [("f32", 32), ("f16", 128), ("f16", 64)])
def test_one_position_is_its_value(dv, dtype, D):
    """A first token sees itself alone: its result is its value row, to the bit."""
    c = Seqs(dv, [1, 3, 1, 200], [0] * 4, 2, 3, D, dtype)
    c.run()
    first = c.cu[:4]
    np.testing.assert_array_equal(c.out.cpu().numpy()[first],
                                  np.repeat(c.qkv[first, c.H + c.Hkv:], 3, 1))


@pytest.mark.parametrize("dtype,D", [("f32", 32), ("f16", 128), ("f16", 64)])
@pytest.mark.parametrize("page", [0, 16])
def test_scores_of_any_size(dv, dtype, D, page):
    """Equal scores near the end of the type's squares: the plain mean of the values.

    Every position's score is the same sum of the same products, so the weights are
    equal; n of them are summed with their values in binary32 (n 2^-24 of the sum of
    |v|, twice for the sum and the quotient), and the result is rounded once.
    """
    n, big = 200, 6e4 if dtype == "f16" else 1e15
    for sign in (1, -1):
        c = Seqs(dv, [n, 1], [0, n if page else 0], 1, 2, D, dtype, page=page)
        c.qkv[:, :2] = big
        c.qkv[:, 2] = sign * big
        if page:
            c.pk[:] = sign * big
        c.upload()
        got = c.run().double().cpu().numpy()
        assert dv.dv_check(c.ws) == 0
        half = torch.finfo(TT[dtype]).eps / 2
        for b in range(2):
            V = c.V[b][0].astype(np.float64)
            for i in range(c.toks[b]):
                m = (c.lens[b] + i if page else i) + 1
                want, size = V[:m].mean(0), np.abs(V[:m]).mean(0)
                tol = half * np.abs(want) + 3 * m * 2.0 ** -24 * size
                assert (np.abs(got[c.cu[b] + i] - want) <= tol).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("tok", [1, 100, 200])
def test_long_sums_are_not_cut_off(dv, tok, D):
    """Outputs of one sign over many tiles of one stream: no bias.

    A sum of the tensor cores may be short by a step of binary32 (2^-23) for each of its
    products of 16 positions, 4 a tile of 64, and sums 256 tiles: 2^-13 of itself at
    most.  All else rounds, so its mean over 8 heads x D outputs and the last tokens is
    far smaller (a rounded weight and result: 2^-11 / sqrt(outputs)).
    """
    H, page, n = 8192 // D, 128, 1 << 17
    desc = dv.make_seq_desc(H, H, D, dv.DV_F16, page, n // page)
    ws, cache = dv.SeqWorkspace(desc), dv.PagedCache(desc)
    g = torch.Generator("cuda").manual_seed(3)
    cache.k.normal_(generator=g)
    cache.v.uniform_(0.5, 1, generator=g)
    q = torch.randn(tok, H, D, device="cuda", generator=g).half()
    out = torch.empty_like(q)
    tables = torch.arange(n // page, device="cuda").int().view(1, -1)
    dv.dv_paged_attn(cache, q, i32([0, tok]), i32([n - tok]), tables, out, ws)
    assert dv.dv_check(ws) == 0
    means = []
    for h in range(0, H, H // 8):
        K, V = (t[:, h].reshape(n, D).double() for t in (cache.k, cache.v))
        want = torch.softmax(K @ q[-1, h].double() * D ** -0.5, 0) @ V
        rel = out[-1, h].double() / want - 1
        assert rel.abs().max() <= 2 * 2.0 ** -11 + 2.0 ** -13
        means.append(rel.mean().item())
    assert abs(sum(means) / 8) <= 2.0 ** -13 + 4 * 2.0 ** -11 / math.sqrt(8 * D)


@pytest.mark.parametrize("dtype,D", [("f32", 32), ("f16", 128), ("f16", 64)])
def test_infinite_keys(dv, dtype, D):
    """Keys of -infinity have no weight; a row that sees nothing else gives 0."""
    n, dead = 300, 150
    c = Seqs(dv, [n], [0], 1, 1, D, dtype)
    c.qkv[:, 0] = np.abs(c.qkv[:, 0]) + NP[dtype](0.01)
    c.qkv[:dead, 1] = -np.inf
    c.upload()
    got = c.run().double().cpu().numpy()
    assert dv.dv_check(c.ws) == 0
    assert (got[:dead] == 0).all()
    q, K, V = (c.qkv[dead:, i].astype(np.float64) for i in range(3))
    s = q @ K.T * D ** -0.5
    w = np.tril(np.exp(s - s.max(1, keepdims=True)))
    w /= w.sum(1, keepdims=True)
    half = torch.finfo(TT[dtype]).eps / 2
    # a weight and the result rounded once each, scores of at most max|s| in binary32
    tol = (2 * half + 2.0 ** -20 * (1 + np.abs(s).max())) * (w @ np.abs(V))
    assert (np.abs(got[dead:, 0] - w @ V) <= tol).all()


@pytest.mark.parametrize("tok", [1, 100, 200])
@pytest.mark.parametrize("rise", [25.0, -25.0, 3.0])
def test_long_sums_with_moving_references(dv, tok, rise):
    """Scores that rise or fall over 2^17 positions: early parts keep their weight.

    Values are in 0.5 to 1, so a weight's rounding (2^-11), the result's (2^-11), the tensor
    cores' sums (2^-13) and scores of at most 32 in binary32 (8 D steps of 2^-24 of them, of
    which a weight's relative error is that) bound the relative error.
    """
    D, H, page, n = 64, 128, 128, 1 << 17
    desc = dv.make_seq_desc(H, H, D, dv.DV_F16, page, n // page)
    ws, cache = dv.SeqWorkspace(desc), dv.PagedCache(desc)
    g = torch.Generator("cuda").manual_seed(4)
    cache.k.normal_(generator=g)
    ramp = torch.linspace(0, rise, n, device="cuda").view(n // page, 1, page)
    cache.k[..., 0] = (ramp * D ** 0.5 / 4).half()
    cache.v.uniform_(0.5, 1, generator=g)
    q = torch.randn(tok, H, D, device="cuda", generator=g).half() * 0.25
    q[..., 0] = 4
    out = torch.empty_like(q)
    tables = torch.arange(n // page, device="cuda").int().view(1, -1)
    dv.dv_paged_attn(cache, q, i32([0, tok]), i32([n - tok]), tables, out, ws)
    assert dv.dv_check(ws) == 0
    for h in range(0, H, H // 8):
        K, V = (t[:, h].reshape(n, D).double() for t in (cache.k, cache.v))
        want = torch.softmax(K @ q[-1, h].double() * D ** -0.5, 0) @ V
        rel = out[-1, h].double() / want - 1
        assert rel.abs().max() <= 2 * 2.0 ** -11 + 2.0 ** -13 + 8 * D * 2.0 ** -24 * 32


@pytest.mark.parametrize("src", ["f32", "f16"])
@pytest.mark.parametrize("D,rot,interleaved", [
    (128, 64, False), (128, 64, True), (128, 96, False), (128, 8, False), (64, 48, False),
    (64, 20, False), (64, 2, True), (32, 12, True), (16, 10, True), (8, 4, False), (8, 2, True),
    (256, 128, False), (256, 64, True), (128, 0, False)])
def test_values_that_do_not_turn_are_kept(dv, src, D, rot, interleaved):
    """Infinities, NaN and -0 behind the turned part stay where and what they are, to the bit (a
    NaN: some NaN), and the turned part does not see them."""
    T, H, Hkv = 13, 6, 2
    dst = "f16" if D == 256 else src
    qkv, pos, slots, cache, ws, r, want, page = rope_case(dv, T, H, Hkv, D, rot, src, dst,
                                                          interleaved)
    rng = np.random.default_rng(D + rot)
    odd = rng.choice(np.array([np.inf, -np.inf, np.nan, -0.0, 0.0, 1.5]), qkv[..., rot:].shape)
    qkv[..., rot:] = odd
    x = dev(qkv)

    def kept(got, rows, out):
        got, rows = got.cpu().numpy(), rows.astype(NP[out])
        nan = np.isnan(rows)
        assert (np.isnan(got) == nan).all()
        whole = np.uint32 if out == "f32" else np.uint16
        np.testing.assert_array_equal(np.where(nan, 0, np.ascontiguousarray(got).view(whole)),
                                      np.where(nan, 0, np.ascontiguousarray(rows).view(whole)))

    for out in ("f32", "f16"):
        q_out = torch.zeros(T, H, D, dtype=TT[out], device="cuda")
        k_out = torch.zeros(T, Hkv, D, dtype=TT[out], device="cuda")
        dv.dv_qk_rope(r, x[:, :H], x[:, H:H + Hkv], i32(pos), ws, q_out=q_out, k_out=k_out,
                      v=x[:, H + Hkv:], cache=cache, slots=i32(slots))
        assert dv.dv_check(ws) == 0
        for got, lo, w in ((q_out, 0, want[0]), (k_out, H, want[1])):
            kept(got[..., rot:], qkv[:, lo:lo + got.shape[1], rot:], out)
            if rot:
                close(got[..., :rot], *(y[..., :rot] for y in rounded(w, out)))
    stored = pool_rows(cache.k, slots, page)
    kept(stored[..., rot:], qkv[:, H:H + Hkv, rot:], dst)
    if rot:
        close(stored[..., :rot], *(y[..., :rot] for y in rounded(want[1], dst)))
    kept(pool_rows(cache.v, slots, page), qkv[:, H + Hkv:], dst)


# What tensor cores may cut off of a sum, of the sum of its terms' sizes: 64 tiles of 64 positions
# between additions in binary32 are 256 products of 16 terms; each cuts its terms and the sum before
# them (17) off below 2^-25 of the largest, and the new sum below 2^-23 of itself.
CUT = 256 * (17 * 2.0 ** -25 + 2.0 ** -23)


def shared_cache(dv, B, tok, N, D, seed):
    """B requests of one query head over the same N cached positions (whole units of attention,
    at least one for every CTA), their descriptor and what the calls take beside queries."""
    page = 128
    desc = dv.make_seq_desc(1, 1, D, dv.DV_F16, page, N // page)
    cache = dv.PagedCache(desc)
    tables = i32(range(N // page))[None].expand(B, -1).contiguous()
    args = i32(range(0, B * tok + 1, tok)), i32([N - tok] * B), tables
    out = torch.zeros(B * tok, 1, D, dtype=torch.float16, device="cuda")
    return cache, args, out, torch.Generator("cuda").manual_seed(seed)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("tok,B", [(1, 304), (40, 304), (200, 152)])
def test_small_terms_beside_large_ones(dv, tok, B, D):
    """A term that outweighs 16384 others 2^25 times, and its opposite behind them: what is left is
    the others' sum.

    Weights are powers of two (exact in binary16); the sum loses CUT of the terms' sizes; binary32
    adds the tiles' sums of weights (2^-24 each, at most 512) and forms the quotient; the result
    is rounded once (2^-11, or 2^-25)."""
    pair = tok > 128
    nt = 256 if pair else 512  # 256 tiles a stream
    N = nt * 64
    cache, args, out, gen = shared_cache(dv, B, tok, N, D, D + tok)
    K, V = torch.zeros(N, D, device="cuda"), torch.zeros(N, D, device="cuda")
    K[:, 0] = -25.0
    for d, v in enumerate((1 - 2.0 ** -10, 1.0, 0.75, 0.5)):
        V[:, d::4] = v
    # (the two streams of a unit of up to 128 rows have every other tile each)
    for p, sign in ((0, 1.0), ((nt - 6) * 64 + 5, -1.0)):
        for at in ([p] if pair else [p, p + 64]):
            K[at, 0], V[at] = 0.0, sign
    cache.k.copy_(K.view(cache.k.shape))
    cache.v.copy_(V.view(cache.v.shape))
    q = torch.zeros(B * tok, 1, D, dtype=torch.float16, device="cuda")
    q[:, 0, 0] = 1
    ws = dv.SeqWorkspace(cache.desc)
    dv.dv_paged_attn(cache, q, *args, out, ws, max_tok=tok, scale=math.log(2))
    assert dv.dv_check(ws) == 0
    w = torch.exp2(K[:, 0].double())
    seen = torch.arange(N, device="cuda") <= torch.arange(N - tok, N, device="cuda")[:, None]
    p = w * seen
    p /= p.sum(1, keepdim=True)
    want, size = p @ V.double(), p @ V.double().abs()
    tol = CUT * size + want.abs() * (2.0 ** -11 + 514 * 2.0 ** -24) + 2.0 ** -25
    for b in range(B):
        close(out[b * tok:(b + 1) * tok, 0], want.cpu().numpy(), tol.cpu().numpy())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("tok,B", [(1, 304), (200, 152)])
def test_long_sums_of_whole_units(dv, tok, B, D):
    """Positive values over 262144 positions, no unit cut: 2048 tiles (a pair: 4096) of a stream.

    Each output: CUT, 2^-11 for the weights' rounding and 2^-11 for the result's, and binary32: a
    score's error, at most (D + 16) 2^-23 of its products' sizes (as in seq_ref, twice in a weight),
    and at most 4096 + 64 additions of 2^-24.  The mean: roundings are of either sign, so the mean of
    them over 4096 outputs and more is under 4 x 2^-11 / 64, and what is left is within CUT.  Sums
    that are never set aside lose 6e-4 in the mean, three times what is allowed."""
    N = 1 << 18
    cache, args, out, gen = shared_cache(dv, B, tok, N, D, 7 * D + tok)
    cache.k.normal_(generator=gen)
    cache.v.uniform_(0.5, 1, generator=gen)
    q = torch.randn(B * tok, 1, D, generator=gen, device="cuda").half()
    ws = dv.SeqWorkspace(cache.desc)
    dv.dv_paged_attn(cache, q, *args, out, ws, max_tok=tok)
    assert dv.dv_check(ws) == 0
    K, V = cache.k.view(N, D).double(), cache.v.view(N, D).double()
    rows = torch.arange(0, B * tok, max(1, B * tok // 64), device="cuda")[:64]
    s = q[rows, 0].double() @ K.T * D ** -0.5
    big = (q[rows, 0].double().abs() @ K.abs().T).amax(1, keepdim=True) * D ** -0.5
    s.masked_fill_(torch.arange(N, device="cuda") > (N - tok + rows % tok)[:, None], -math.inf)
    want = torch.softmax(s, 1) @ V
    r = out[rows, 0].double() / want - 1
    tol = CUT + 2 * 2.0 ** -11 + 2 * (D + 16) * 2.0 ** -23 * big + 4160 * 2.0 ** -24
    assert (r.abs() <= tol).all(), (r.abs().max().item(), tol.min().item())
    assert r.mean().abs() <= CUT + 4 * 2.0 ** -11 / 64, r.mean().item()


@pytest.mark.parametrize("args", [([300, 1, 129], [4000, 9000, 0], 2, 4, 128, "f16", 16),
                                  ([1] * 12, list(range(0, 6000, 500)), 2, 2, 64, "f16", 32),
                                  ([100, 7], [900, 0], 2, 2, 32, "f32", 16),
                                  ([700, 1, 90], [0] * 3, 1, 5, 128, "f16")])
def test_a_request_alone(dv, args):
    """A request's rows alone in a call and in a batch: each within the bound of seq_ref, so at most
    twice that apart (other requests move cuts between CTAs, and with max_tok the grouping)."""
    c = Seqs(dv, *args)
    got = c.run().double().cpu().numpy()
    assert dv.dv_check(c.ws) == 0
    want, tol = c.want()
    cu, lens, tables = c.cu, c.lens, getattr(c, "tables", None)
    x = c.x
    for b in range(len(cu) - 1):
        n = int(cu[b + 1] - cu[b])
        rows = slice(cu[b], cu[b + 1])
        c.x = x[cu[b]:cu[b + 1]].contiguous()
        c.d_cu = i32([0, n])
        if c.page:
            c.d_lens, c.d_tables = i32(lens[b:b + 1]), i32(tables[b:b + 1])
        for max_tok in (None, n):
            out = torch.zeros(n, c.H, c.D, dtype=c.out.dtype, device="cuda")
            c.run(max_tok=max_tok, out=out)
            assert dv.dv_check(c.ws) == 0
            close(out, want[rows], tol[rows])
            close(out, got[rows], 2 * tol[rows])


@pytest.mark.parametrize("dtype,D", [("f16", 128), ("f16", 64), ("f32", 32)])
@pytest.mark.parametrize("G", [5, 10, 11])
def test_groups_that_fill_no_unit(dv, G, D, dtype):
    """Mixed steps whose query heads a KV head leave much of a unit's rows empty: tight, loose and
    default bounds on the tokens, which choose other groups."""
    toks, lens = [1, 40, 1, 0, 1, 150, 1], [700, 30, 0, 9, 65, 128, 2000]
    c = Seqs(dv, toks, lens, 2, G, D, dtype, 16)
    for max_tok in (150, None):
        c.check(max_tok=max_tok)
    Seqs(dv, [1] * 20, list(range(0, 1000, 50)), 1, G, D, dtype, 16).check()


@pytest.mark.parametrize("dtype,D,tok,N", [
    ("f16", 64, 1, (1 << 30) - 77), ("f16", 128, 200, (1 << 30) - 77), ("f16", 128, 40, 1 << 30),
    ("f32", 32, 1, (1 << 26) - 9)])
def test_longest_requests(dv, dtype, D, tok, N):
    """A block table of up to 2^30 positions (61 pages over and over): a position's weight times
    how often it is seen.

    Bounds: scores as in seq_ref; binary16: CUT, and 2^-11 each for the weights and the result;
    additions in binary32 of 2^-24 each: of a CTA's tiles (152 CTAs; 64 more within a tile and where
    pieces meet) or, on CUDA cores, of its positions (608 CTAs), in numerator and denominator."""
    page, P = 128, 61
    desc = dv.make_seq_desc(1, 1, D, dv.DV_F16 if dtype == "f16" else dv.DV_F32, page, P)
    cache, ws = dv.PagedCache(desc), dv.SeqWorkspace(desc)
    g = torch.Generator("cuda").manual_seed(D + tok)
    cache.k.normal_(generator=g)
    cache.v.uniform_(0.5, 1, generator=g)
    tables = (torch.arange(seq_ref.pages(N, page), device="cuda") % P).int()[None].contiguous()
    q = torch.randn(tok, 1, D, generator=g, device="cuda").to(TT[dtype])
    out = torch.zeros_like(q)
    dv.dv_paged_attn(cache, q, i32([0, tok]), i32([N - tok]), tables, out, ws, max_tok=tok)
    assert dv.dv_check(ws) == 0
    K, V = (t.view(-1, D).double() for t in (cache.k, cache.v))
    s = q[:, 0].double() @ K.T * D ** -0.5
    big = (q[:, 0].double().abs() @ K.abs().T).amax(1, keepdim=True) * D ** -0.5
    n = torch.arange(N - tok + 1, N + 1, device="cuda")[:, None]
    times = n // (P * page) + (torch.arange(P * page, device="cuda") < n % (P * page))
    w = torch.exp(s - s.amax(1, keepdim=True)) * times
    want = w @ V / w.sum(1, keepdim=True)
    tol = 2 * (D + 16) * 2.0 ** -23 * big
    if dtype == "f16":
        tol = tol + CUT + 2 * 2.0 ** -11 + (N / 64 / 152 + 64) * 2.0 ** -24
    else:
        tol = tol + 2 * (N / 608 + 1024) * 2.0 ** -24
    r = (out[:, 0].double() / want - 1).abs()
    assert (r <= tol).all(), (r.max().item(), tol.min().item())
