"""Arguments at the edges of the KV-cache operators' ranges (no GPU)."""

import ctypes as C

import pytest
import torch

from test_kv_cpu import dv  # noqa: F401


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake-pointer checks run only without a GPU")
@pytest.mark.parametrize("scale", [2.4e38, -3e38])
def test_scales_that_overflow_in_base_two_are_refused(dv, scale):
    """scale x log2(e) must be finite: an infinite one turns every zero query into NaN."""
    desc = dv.make_kv_desc(16, 8, 128, 512, dv.DV_F16, 64)
    P = [0x100000 + 4096 * i for i in range(10)]
    d, c = C.byref(desc), C.byref(dv.KvCachePointers(P[0], P[1], None, None, P[2], P[3]))
    rows = C.byref(dv.KvRows(P[4], dv.DV_F32, 1 << 16, 1 << 12, 128))
    tail = (0x2000000, 1 << 30, None)
    assert dv._lib.dv_tree_attn(d, c, rows, 2, 4, P[5], None, None, scale, None, None, 0, P[6],
                                *tail) == dv.DV_ERR_INVALID_ARG
    assert dv._lib.dv_block_attn(d, c, rows, 2, P[5], P[7], 4, scale, P[6],
                                 *tail) == dv.DV_ERR_INVALID_ARG
