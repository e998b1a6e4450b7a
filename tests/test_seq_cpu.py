"""Argument checks of the operators over packed sequences, and their host function (no GPU)."""

import ctypes as C
import math
import os
import subprocess

import numpy as np
import pytest
import torch

import seq_ref

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
        'int main(void){printf("%zu %zu %zu %zu %zu %zu %zu %zu %d %d\\n", sizeof(dv_seq_desc),'
        " offsetof(dv_seq_desc, page), sizeof(dv_page_pool), sizeof(dv_rope),"
        " offsetof(dv_rope, mscale), offsetof(dv_rope, norm), offsetof(dv_rope, eps),"
        " offsetof(dv_rope, k_gain), DV_SEQ_MAX_BATCH, DV_ERR_PAGES);return 0;}\n")
    exe = tmp_path / "sizes"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True,
                                          check=True).stdout.split()]
    R = dv.RopeParams
    assert got == [C.sizeof(dv.SeqDesc), dv.SeqDesc.page.offset, C.sizeof(dv.PagePoolPointers),
                   C.sizeof(R), R.mscale.offset, R.norm.offset, R.eps.offset, R.k_gain.offset,
                   dv.DV_SEQ_MAX_BATCH, dv.DV_ERR_PAGES]
    assert dv.status_string(dv.DV_ERR_PAGES) != dv.status_string(99)


def test_workspace_size_validates(dv):
    assert 0 < dv.seq_workspace_size(dv.make_seq_desc(64, 8, 128, dv.DV_F16, 16, 1000)) < 1 << 27
    assert dv.seq_workspace_size(dv.make_seq_desc(64, 8, 128, dv.DV_F16)) > 0
    bad = [(64, 7, 128, 1, 0, 0), (0, 1, 128, 1, 0, 0), (8, 0, 128, 1, 0, 0), (257, 1, 128, 1, 0, 0),
           (8, 8, 96, 1, 0, 0), (8, 8, 4, 1, 0, 0), (8, 8, 512, 1, 0, 0), (8, 8, 256, 0, 0, 0),
           (8, 8, 128, 2, 0, 0), (8, 8, 128, 1, 16, 0), (8, 8, 128, 1, 0, 9), (8, 8, 128, 1, 24, 9),
           (8, 8, 128, 1, -16, 9), (8, 8, 128, 1, 128, (1 << 23) + 1), (8, 8, 128, 1, 16, -1)]
    for b in bad:
        assert dv.seq_workspace_size(dv.make_seq_desc(*b)) == 0, b


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake-pointer checks run only without a GPU")
def test_argument_checks_fail_before_any_launch(dv):
    lib, INV, UNS, WS = dv._lib, dv.DV_ERR_INVALID_ARG, dv.DV_ERR_UNSUPPORTED, dv.DV_ERR_WORKSPACE
    desc = dv.make_seq_desc(16, 8, 128, dv.DV_F16, 16, 100)
    bare = dv.make_seq_desc(16, 8, 128, dv.DV_F16)
    P = [0x100000 + 4096 * i for i in range(12)]
    odd = 0x100002
    f16, f32 = dv.DV_F16, dv.DV_F32

    def rows(p=P[0], dt=f16, st=1 << 14, sh=128):
        return C.byref(dv.KvRows(p, dt, 0, st, sh))

    def rope(**kw):
        r = dict(steps=P[1], rot_dim=128, interleaved=0, mscale=1.0, norm=dv.DV_RMSNORM, eps=1e-6,
                 q_gain=P[2], k_gain=P[3])
        r.update(kw)
        return C.byref(dv.RopeParams(*[r[n] for n, _ in dv.RopeParams._fields_]))

    def call(fn, **kw):
        a = dict(desc=desc, B=2, T=64, max_tok=40, lens=P[4], done=P[5], n_tok=P[5], width=6,
                 tables=P[6], free=P[7], n_free=P[8], n_out=P[8], cu=P[9], pos=P[10], slots=P[11],
                 q=rows(), k=rows(), v=rows(), q_out=rows(), k_out=rows(), rope=rope(),
                 pool=C.byref(dv.PagePoolPointers(P[1], P[2])), scale=0.1, out=P[3], ws=0x2000000,
                 nws=1 << 30)
        a.update(kw)
        d = C.byref(a["desc"]) if a["desc"] is not None else None
        tail = (a["ws"], a["nws"], None)
        if fn == "release":
            return lib.dv_page_release(d, a["B"], a["lens"], a["done"], a["width"], a["tables"],
                                       a["free"], a["n_free"], a["n_out"], *tail)
        if fn == "take":
            return lib.dv_page_take(d, a["B"], a["lens"], a["n_tok"], a["width"], a["tables"],
                                    a["free"], a["n_free"], a["n_out"], a["cu"], a["pos"],
                                    a["slots"], a["T"], *tail)
        if fn == "rope":
            return lib.dv_qk_rope(d, a["rope"], a["T"], a["pos"], a["q"], a["k"], a["v"],
                                  a["q_out"], a["k_out"], a["pool"], a["slots"], *tail)
        if fn == "prompt":
            return lib.dv_prompt_attn(d, a["B"], a["T"], a["max_tok"], a["q"], a["k"], a["v"],
                                      a["cu"], a["scale"], a["out"], *tail)
        return lib.dv_paged_attn(d, a["pool"], a["B"], a["T"], a["max_tok"], a["q"], a["cu"],
                                 a["lens"], a["tables"], a["width"], a["scale"], a["out"], *tail)

    everywhere = [(dict(desc=None), INV), (dict(desc=dv.make_seq_desc(16, 8, 96, f16, 16, 9)), UNS),
                  (dict(desc=dv.make_seq_desc(16, 5, 128, f16, 16, 9)), INV), (dict(nws=4096), WS),
                  (dict(ws=0x2000010), WS), (dict(ws=None), WS)]
    batched = [(dict(B=0), INV), (dict(B=1025), INV)]
    tabled = [(dict(desc=bare), INV), (dict(width=0), INV), (dict(width=(1 << 26) + 1), INV),
              (dict(lens=None), INV), (dict(tables=None), INV)]
    stack = [(dict(free=None), INV), (dict(n_free=odd), INV), (dict(n_out=None), INV)]
    sized = [(dict(T=0), INV), (dict(T=(1 << 28) + 1), INV)]
    misrow = [(n, dict([(n, x)])) for n in ("q", "k", "v") for x in (
        rows(p=odd), rows(p=None), rows(dt=2), rows(st=-8), rows(sh=4), rows(st=1 << 40))]
    attn = [(dict(max_tok=0), INV), (dict(cu=None), INV), (dict(out=odd), INV),
            (dict(scale=0.0), INV), (dict(scale=-1.0), INV), (dict(scale=math.nan), INV),
            (dict(scale=math.inf), INV), (dict(scale=3e38), INV), (dict(scale=1e-39), INV),
            (dict(q=rows(dt=f32)), INV), (dict(q=rows(sh=64)), INV), (dict(q=rows(st=0)), INV)]
    checks = {
        "release": everywhere + batched + tabled + stack + [(dict(done=None), INV)],
        "take": everywhere + batched + tabled + stack + sized + [
            (dict(n_tok=None), INV), (dict(cu=None), INV), (dict(pos=odd), INV),
            (dict(slots=None), INV)],
        "rope": everywhere + sized + [(x, INV) for _, x in misrow] + [
            (dict(pos=None), INV), (dict(rope=None), INV), (dict(q_out=rows(sh=0)), INV),
            (dict(k_out=rows(st=64)), INV), (dict(k=rows(dt=f32)), INV), (dict(v=rows(dt=f32)), INV),
            (dict(pool=None), INV), (dict(pool=None, slots=None), INV), (dict(slots=None), INV),
            (dict(desc=bare), INV), (dict(k_out=None, pool=None, slots=None, v=None), INV),
            (dict(rope=rope(rot_dim=130)), INV), (dict(rope=rope(rot_dim=-2)), INV),
            (dict(rope=rope(rot_dim=7)), INV), (dict(rope=rope(steps=None)), INV),
            (dict(rope=rope(mscale=math.nan)), INV), (dict(rope=rope(interleaved=2)), INV),
            (dict(rope=rope(norm=2)), INV), (dict(rope=rope(eps=0.0)), INV),
            (dict(rope=rope(q_gain=P[2] + 4)), INV), (dict(rope=rope(k_gain=P[2] + 4)), INV),
            (dict(pool=C.byref(dv.PagePoolPointers(odd, P[2]))), INV)],
        "prompt": everywhere + batched + sized + attn + [(x, INV) for _, x in misrow] + [
            (dict(k=rows(dt=f32)), INV), (dict(v=rows(sh=0)), INV)],
        "paged": everywhere + batched + tabled + sized + attn
        + [(x, INV) for n, x in misrow if n == "q"] + [
            (dict(pool=None), INV), (dict(pool=C.byref(dv.PagePoolPointers(P[1], odd))), INV)],
    }
    for fn, cases in checks.items():
        for kw, status in cases:
            assert call(fn, **kw) == status, (fn, kw)


@pytest.mark.parametrize("rot", [2, 4, 64, 96, 128, 256])
@pytest.mark.parametrize("scaling", ["none", "linear", "base", "ramp", "ramp_index"])
@pytest.mark.parametrize("theta", [10000.0, 500000.0, 1.5])
def test_rope_steps(dv, rot, scaling, theta):
    if scaling == "base" and rot == 2:
        pytest.skip("refused: no other pair to stretch")
    kw = dict(factor=8.0, orig_len=4096.0, low=1.0, high=32.0)
    host = (C.c_uint64 * (rot // 2))()
    assert dv._lib.dv_rope_steps(rot, theta, dv.DV_ROPE_SCALING[scaling], *kw.values(), host) == 0
    got = np.array([v / 2.0 ** 64 * 2 * math.pi for v in host])
    # a handful of roundings of binary64, and the rounding to whole steps: half a step is 2^-65
    # turns, 2 pi 2^-65 = 1.71e-19
    np.testing.assert_allclose(got, seq_ref.freqs(rot, theta, scaling, **kw), rtol=1e-13,
                               atol=1.01 * 2 * math.pi * 2.0 ** -65)


def test_rope_steps_refuses(dv):
    host = (C.c_uint64 * 128)()
    good = [64, 1e4, 3, 8.0, 4096.0, 1.0, 32.0]
    assert dv._lib.dv_rope_steps(*good, host) == 0
    for i, v in ((0, 0), (0, 3), (0, 258), (1, 1.0), (1, math.nan), (1, math.inf), (2, 5), (2, -1),
                 (3, 0.5), (3, math.inf), (3, math.nan), (4, 0.0), (4, math.nan), (5, 32.0),
                 (5, 0.0), (6, math.inf)):
        bad = list(good)
        bad[i] = v
        assert dv._lib.dv_rope_steps(*bad, host) == dv.DV_ERR_INVALID_ARG, (i, v)
    assert dv._lib.dv_rope_steps(2, 1e4, 2, 8.0, 0.0, 1.0, 32.0, host) == dv.DV_ERR_INVALID_ARG
    assert dv._lib.dv_rope_steps(*good, None) == dv.DV_ERR_INVALID_ARG


def test_the_plain_forms_on_small_cases():
    """seq_ref by hand: pages, slots, a quarter turn, a mean."""
    t, n, cu, pos, slots, seen = seq_ref.take(np.full((2, 3), -1, np.int32),
                                              np.arange(4, dtype=np.int32), 4, [0, 0], [17, 1], 16, 20)
    assert t[0, :2].tolist() == [3, 2] and t[1, 0] == 1 and n == 1 and not seen
    assert cu.tolist() == [0, 17, 18] and slots[[0, 15, 16, 17, 18]].tolist() == [48, 63, 32, 16, -1]
    free, n, st = seq_ref.release(t, np.full(4, 9, np.int32), 1, [17, 1], [1, 0], 16)
    assert free.tolist() == [9, 3, 2, 9] and n == 3 and st == 0
    x = np.array([[[1.0, 0, 2, 0]]])
    got, _ = seq_ref.rope(x, [1], np.array([math.pi / 2]), 2, False)
    np.testing.assert_allclose(got[0, 0], [0, 1, 2, 0], atol=1e-15)
    got, _ = seq_ref.attend(np.zeros((2, 2)), np.ones((3, 2)), np.arange(6.0).reshape(3, 2), [0, 1],
                            1.0, False)
    np.testing.assert_allclose(got, [[0, 1], [1, 2]])


@pytest.mark.parametrize("rot", [2, 4, 6, 64, 96, 128, 256])
@pytest.mark.parametrize("scaling", ["none", "linear", "base", "ramp", "ramp_index"])
@pytest.mark.parametrize("theta,factor,orig,low,high", [
    (10000.0, 8.0, 4096.0, 1.0, 32.0), (500000.0, 3.7, 8192.0, 1.0, 4.0),
    (1000003.7, 1.0, 131072.0, 0.3, 1.1), (1.7e308, 1e300, 1e6, 1e-3, 64.0),
    (1.0000001, 40.0, 10000.0, 1.0, 32.0)])
def test_rope_steps_are_rounded_from_the_exact_angle(dv, rot, scaling, theta, factor, orig, low,
                                                     high):
    """Half a unit of 2^-64 turns (and 2^-20 of one for binary128's own roundings: 113 bits of a
    number below 2^62 are 2^-51 of a unit, some hundred times): 80 digits decide."""
    import decimal

    if scaling == "base" and rot == 2:
        pytest.skip("refused: no other pair to stretch")
    host = (C.c_uint64 * (rot // 2))()
    assert dv._lib.dv_rope_steps(rot, theta, dv.DV_ROPE_SCALING[scaling], factor, orig, low, high,
                                 host) == 0
    with decimal.localcontext() as ctx:
        ctx.prec = 80
        X = decimal.Decimal

        def arctan_inverse(n):
            total = term = X(1) / n
            k = 1
            while abs(term) > X(10) ** -85:
                term = -term / (n * n)
                k += 2
                total += term / k
            return total

        pi = 4 * (4 * arctan_inverse(5) - arctan_inverse(239))  # (Machin)
        th, fa, og, lo, hi = (X(v) for v in (theta, factor, orig, low, high))
        log = th.ln()
        if scaling == "base":
            log += fa.ln() * rot / (rot - 2)
        for i in range(rot // 2):
            f = (-2 * i * log / rot).exp()
            w = X(1)
            if scaling == "ramp":
                w = (og * f / (2 * pi) - lo) / (hi - lo)
            if scaling == "ramp_index":
                a, b = (rot * (og / (2 * pi * r)).ln() / (2 * log) for r in (hi, lo))
                a = max(a.to_integral_value(decimal.ROUND_FLOOR), X(0))
                b = min(b.to_integral_value(decimal.ROUND_CEILING), X(rot - 1))
                b += X(0.001) if a == b else 0
                w = 1 - (i - a) / (b - a)
            w = min(max(w, X(0)), X(1))
            if scaling == "linear":
                f /= fa
            elif scaling.startswith("ramp"):
                f *= w + (1 - w) / fa
            off = abs(X(host[i]) - f / (2 * pi) * 2 ** 64)
            assert off <= X(0.5) + X(2) ** -20, (i, off)
