"""The KV-cache operators' argument checks and their plain host forms (no GPU)."""

import ctypes as C
import math
import os
import subprocess

import numpy as np
import pytest
import torch

import kv_ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def dv():
    from attention_dv_predict_gb300 import build

    build.build()
    from attention_dv_predict_gb300 import dv as mod

    return mod


def test_struct_layouts_match_header(dv, tmp_path):
    src = tmp_path / "sizes.c"
    src.write_text(
        '#include <stdio.h>\n#include <stddef.h>\n#include "dv.h"\n'
        'int main(void){printf("%zu %zu %zu %zu %zu %d %d %d\\n", sizeof(dv_kv_desc),'
        " offsetof(dv_kv_desc, block), sizeof(dv_kv_cache), sizeof(dv_kv_rows),"
        " offsetof(dv_kv_rows, stride_h), DV_I8, DV_KV_MAX_BATCH, DV_TREE_MAX_TOKENS);"
        "return 0;}\n")
    exe = tmp_path / "sizes"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True,
                                          check=True).stdout.split()]
    assert got == [C.sizeof(dv.KvDesc), dv.KvDesc.block.offset, C.sizeof(dv.KvCachePointers),
                   C.sizeof(dv.KvRows), dv.KvRows.stride_h.offset, dv.DV_I8, dv.DV_KV_MAX_BATCH,
                   dv.DV_TREE_MAX_TOKENS]


def test_workspace_size_validates(dv):
    good = dv.make_kv_desc(64, 8, 128, 8192, dv.DV_I8, 64)
    n = dv.kv_workspace_size(good, 4, 1)
    assert 0 < n <= dv.kv_workspace_size(good, 4, 64) < 1 << 27
    # the size does not depend on the batch: one workspace serves any
    assert dv.kv_workspace_size(good, 256, 1) == n
    for B, T in ((0, 1), (257, 1), (1, 0), (1, 8193)):
        assert dv.kv_workspace_size(good, B, T) == 0
    bad = [(64, 7, 128, 8192, dv.DV_I8, 0), (0, 1, 128, 8, dv.DV_F16, 0),
           (512, 512, 128, 8, dv.DV_F16, 0), (8, 8, 96, 64, dv.DV_F16, 0),
           (8, 8, 512, 64, dv.DV_I8, 0), (8, 8, 256, 64, dv.DV_F32, 0),
           (8, 8, 8, 64, dv.DV_I8, 0), (8, 8, 128, 0, dv.DV_I8, 0),
           (8, 8, 128, 64, 3, 0), (8, 8, 128, 64, dv.DV_I8, 24), (8, 8, 128, 63, dv.DV_I8, 64),
           (8, 8, 128, 64, dv.DV_I8, -1), (8, 8, 128, 16384 * 16, dv.DV_I8, 16),
           (8, 8, 8, 64, dv.DV_F32, 16), (8, 8, 128, (1 << 28) + 1, dv.DV_I8, 0)]
    for b in bad:
        assert dv.kv_workspace_size(dv.make_kv_desc(*b), 1, 1) == 0, b
    # DV_I8 is no layer type
    assert dv.workspace_size(dv.make_desc(256, 8, 32, 1024, 32, dv.DV_I8, 65), 1) == 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake-pointer checks run only without a GPU")
def test_argument_checks_fail_before_any_launch(dv):
    lib, INV, UNS, WS = dv._lib, dv.DV_ERR_INVALID_ARG, dv.DV_ERR_UNSUPPORTED, dv.DV_ERR_WORKSPACE
    desc = dv.make_kv_desc(16, 8, 128, 512, dv.DV_I8, 64)
    P = [0x100000 + 4096 * i for i in range(12)]
    cache = dv.KvCachePointers(*P[:6])
    row = (P[6], dv.DV_F32, 1 << 16, 1 << 12, 128)
    ws, nws = 0x2000000, 1 << 30
    odd = 0x100002

    def call(fn, **kw):
        a = dict(desc=desc, cache=cache, rows=dv.KvRows(*row), B=2, T=4, lens=P[7], n_tok=None,
                 mask=None, scale=0.1, u_h=None, n_u_h=None, max_u_h=0, out=P[8], out2=P[9],
                 path=P[10], n_keep=P[11], idx=P[10], k=4, first=1, last=1, dt=dv.DV_F32, ws=ws,
                 nws=nws)
        a.update(kw)
        d = C.byref(a["desc"]) if a["desc"] is not None else None
        c = C.byref(a["cache"]) if a["cache"] is not None else None
        r = C.byref(a["rows"]) if a["rows"] is not None else None
        tail = (a["ws"], a["nws"], None)
        if fn == "append":
            return lib.dv_kv_append(d, c, r, r, a["B"], a["T"], a["lens"], a["n_tok"], *tail)
        if fn == "read":
            return lib.dv_kv_read(d, c, a["B"], a["T"], a["lens"], a["dt"], a["out"], a["out2"],
                                  *tail)
        if fn == "keep":
            return lib.dv_kv_keep(d, c, a["B"], a["T"], a["lens"], a["path"], a["n_keep"], *tail)
        if fn == "tree":
            return lib.dv_tree_attn(d, c, r, a["B"], a["T"], a["lens"], a["n_tok"], a["mask"],
                                    a["scale"], a["u_h"], a["n_u_h"], a["max_u_h"], a["out"],
                                    *tail)
        if fn == "topk":
            return lib.dv_block_topk(d, c, r, a["B"], a["lens"], a["k"], a["first"], a["last"],
                                     a["idx"], *tail)
        return lib.dv_block_attn(d, c, r, a["B"], a["lens"], a["idx"], a["k"], a["scale"],
                                 a["out"], *tail)

    no_block = dv.make_kv_desc(16, 8, 128, 512, dv.DV_I8, 0)
    rows_bad = [dv.KvRows(None, *row[1:]), dv.KvRows(P[6] + 8, *row[1:]),
                dv.KvRows(P[6], dv.DV_I8, *row[2:]), dv.KvRows(P[6], dv.DV_F32, 2, 4, 4),
                dv.KvRows(P[6], dv.DV_F16, 8, 8, 4), dv.KvRows(P[6], dv.DV_F32, 0, -128, 4)]
    cache_bad = [dv.KvCachePointers(None, *P[1:6]), dv.KvCachePointers(P[0], P[1] + 8, *P[2:6]),
                 dv.KvCachePointers(P[0], P[1], None, *P[3:6]),
                 dv.KvCachePointers(*P[:4], None, P[5]), dv.KvCachePointers(*P[:5], None)]
    for fn in ("append", "read", "keep", "tree", "topk", "battn"):
        common = [dict(desc=None), dict(cache=None), dict(B=0), dict(B=257), dict(lens=None),
                  dict(lens=odd)] + [dict(cache=c) for c in cache_bad]
        if fn in ("append", "tree", "topk", "battn"):
            common += [dict(rows=None)] + [dict(rows=r) for r in rows_bad]
        if fn in ("append", "read", "keep", "tree"):
            common += [dict(T=0), dict(T=513)]
        if fn in ("append", "tree"):
            common += [dict(n_tok=odd)]
        if fn in ("read", "tree", "battn"):
            common += [dict(out=None), dict(out=P[8] + 4)]
        if fn == "read":
            common += [dict(dt=dv.DV_I8), dict(out2=None)]
        if fn in ("keep", "tree"):
            common += [dict(T=65)]
        if fn == "keep":
            common += [dict(path=None), dict(n_keep=odd)]
        if fn == "tree":
            common += [dict(mask=0x100004), dict(u_h=P[10]), dict(u_h=P[10], n_u_h=P[11]),
                       dict(u_h=P[10], n_u_h=P[11], max_u_h=9), dict(max_u_h=1),
                       dict(n_u_h=P[11])]
        if fn in ("tree", "battn"):
            common += [dict(scale=math.inf), dict(scale=math.nan)]
        if fn in ("topk", "battn"):
            common += [dict(desc=no_block), dict(k=0), dict(k=16385), dict(idx=None)]
        if fn == "topk":
            common += [dict(last=0), dict(first=-1), dict(first=4), dict(first=2, last=3)]
        for kw in common:
            assert call(fn, **kw) == INV, (fn, kw)
        assert call(fn, desc=dv.make_kv_desc(16, 8, 96, 512, dv.DV_I8, 64)) == UNS, fn
        for kw in (dict(ws=None), dict(ws=ws + 16), dict(nws=1024)):
            assert call(fn, **kw) == WS, (fn, kw)


def test_wrappers_refuse_host_tensors(dv):
    desc = dv.make_kv_desc(8, 8, 32, 64, dv.DV_F32)
    with pytest.raises(ValueError):
        dv.KvCache(desc, 1, tensors={"k": torch.zeros(1, 8, 64, 32),
                                     "v": torch.zeros(1, 8, 64, 32)})
    with pytest.raises(ValueError):
        dv.KvCache(desc, 1, tensors={"k": torch.zeros(1, 8, 64, 32)})
    with pytest.raises(dv.DvError):
        dv.KvCache(dv.make_kv_desc(8, 3, 32, 64, dv.DV_F32), 1, tensors={})


def test_tree_kernel_variant_switch(dv):
    """Host-only: the variant switch accepts 0, 1 and 2 and refuses the rest."""
    for bad in (-1, 3):
        with pytest.raises(dv.DvError) as e:
            dv.dv_set_tree_kernel(bad)
        assert e.value.status == dv.DV_ERR_INVALID_ARG
    for ok in (1, 2, 0):
        dv.dv_set_tree_kernel(ok)


# ------------------------------------------------------------------ the host forms themselves


def test_quantise_is_nearest_code():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((50, 64)) * 10.0 ** rng.integers(-30, 30, (50, 1))).astype(np.float32)
    x[3] = 0
    q, s = kv_ref.quantise(x)
    assert np.abs(q).max() == 127 and (s >= 2.0 ** -126).all() and not q[3].any()
    # within half a step (and the quotient's rounding) of the value
    err = np.abs(q * s[:, None].astype(np.float64) - x)
    assert (err <= s[:, None] * (0.5 + 2.0 ** -17)).all()
    q, s = kv_ref.quantise(np.float32([[1, np.nan], [np.inf, 0]]))
    assert np.isnan(s).all() and not q.any()


@pytest.mark.parametrize("n", [16, 128])
def test_block_mean_is_the_mean(n):
    rng = np.random.default_rng(1)
    c = kv_ref.RefCache(1, 2, 2 * n, 32, "f32", n, rng)
    x = c.values("k").reshape(1, 2, 2, n, 32)
    got = c.mean * c.mean_scale[..., None].astype(np.float64)
    # half a code step, and the keys' rounding to the grid
    tol = 0.5 * c.mean_scale[..., None] + np.abs(x).max((3, 4))[..., None] * n * 2.0 ** -24
    assert (np.abs(got - x.mean(3)) <= tol * 1.001).all()


def test_tree_of_a_causal_mask_is_step_by_step():
    """Drafted tokens with their ancestors' bits equal one token after another."""
    rng = np.random.default_rng(2)
    c = kv_ref.RefCache(1, 1, 12, 16, "f32", 0, rng)
    q = rng.standard_normal((1, 4, 2, 16)).astype(np.float32)
    a, _ = kv_ref.tree(c, q, [7], [4], None, 0.25)
    b, _ = kv_ref.tree(c, q, [7], [4], [[1, 3, 7, 15]], 0.25)
    assert np.array_equal(a, b)
    for t in range(4):
        one, _ = kv_ref.tree(c, q[:, t:t + 1], [7 + t], [1], [[1]], 0.25)
        np.testing.assert_allclose(one[0, 0], a[0, t], rtol=1e-12)


def test_all_blocks_is_dense():
    rng = np.random.default_rng(3)
    c = kv_ref.RefCache(1, 2, 100, 16, "f32", 16, rng)
    q = rng.standard_normal((1, 2, 16)).astype(np.float32)
    idx = kv_ref.topk(c, q, [99], 9)
    assert (idx[0, 0] == [0, 1, 2, 3, 4, 5, 6, -1, -1]).all()
    a, _ = kv_ref.block_attend(c, q, [99], idx, 0.25)
    b, _ = kv_ref.tree(c, q[:, None], [99], [1], [[0]], 0.25)
    np.testing.assert_allclose(a, b[:, 0], rtol=1e-12)


def test_division_by_127_correction():
    """q + (a - 127 q) / 127 rounds to a / 127 for every significand (the scale's arithmetic)."""
    y = np.float32(1) / np.float32(127)
    m = np.arange(1 << 23, 1 << 24, dtype=np.int64).astype(np.float32)
    q = m * y
    r = m.astype(np.float64) - 127.0 * q.astype(np.float64)
    assert (r == r.astype(np.float32)).all()  # the remainder is exact
    got = (q.astype(np.float64) + r * np.float64(y)).astype(np.float32)
    assert (got == m / np.float32(127)).all()
