"""Coefficients of the update's polynomial that its number format cannot hold (no GPU needed)."""
import ctypes
import math

import numpy as np
import pytest

F = 0x10000             # 32-byte aligned, never dereferenced: the calls fail validation first


@pytest.mark.parametrize("a", [15.99, 16.0, -16.0, 1e9, math.inf, math.nan])
def test_a_that_overflows_is_refused(a):
    """B = a I + b A + c A A is held in fp16 times 2^12: its diagonal overflows from 65520 / 4096 = 15.996 on."""
    from mxfp8_grouped_gemm_gb300 import build
    build.build()
    import mxfp8_grouped_gemm_gb300 as m
    with np.errstate(over="ignore"):
        assert np.isfinite(np.float16(15.989 * 4096)) and not np.isfinite(np.float16(15.997 * 4096))
    L = m.lib()
    ws = L.mxg_muon_workspace_bytes(2, 64, 128)
    args = m.MuonArgs(batch=2, rows=64, cols=128, grad=F, steps=5, a=a, b=0.0, c=0.0, scale=1.0, update=F, workspace=F,
                      workspace_bytes=ws - 1, dev_status=F)
    assert L.mxg_muon_update(ctypes.byref(args), None) == 1
    args.a = 15.9
    assert L.mxg_muon_update(ctypes.byref(args), None) == 5          # what is left to refuse is the workspace
