"""The query of the update's form (no GPU needed; without one the rules see a single SM)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def m():
    from mxfp8_grouped_gemm_gb300 import build
    build.build()
    import mxfp8_grouped_gemm_gb300 as m
    return m


def test_arguments(m):
    L, form = m.lib(), (ctypes.c_int * 4)()
    assert L.mxg_muon_form(1, 4, 4, None) == 1 and L.mxg_muon_form(0, 4, 4, form) == 1
    assert L.mxg_muon_form(65536, 4, 4, form) == 2
    with pytest.raises(m.MxgError):
        m.mxg_muon_form(1, 0, 4)


@pytest.mark.parametrize("short,parts", [(1, 2), (64, 2), (65, 1), (300, 1)])
def test_wide_and_tall_take_the_same_form(m, short, parts):
    f = m.mxg_muon_form(3, short, 9000)
    assert f["parts"] == parts and f["cluster"] == 0 and f["tile"] in (64, 128, 256)
    assert m.mxg_muon_form(3, 9000, short)["parts"] == parts


@pytest.mark.parametrize("batch", [1, 200])
@pytest.mark.parametrize("m_,n,most", [(4, 1 << 21, 16384), (64, 16385, 16384), (100, 300000, 16384), (128, 1 << 21, 16384),
                                       (129, 65537, 65536), (200, 1 << 20, 65536), (1000, 1 << 18, 65536)])
def test_no_accumulator_takes_a_longer_contraction(m, m_, n, most, batch):
    """Whether SMs are idle or not: the tensor cores cut their sums, which long ones must not show."""
    for rows, cols in ((m_, n), (n, m_)):
        shares = m.mxg_muon_form(batch, rows, cols)["shares"]
        # the shares are cut at whole stages of 64 (one tile: 128) columns
        assert -(-n // shares) <= most and shares <= 16 * -(-n // most)
        ws = m.mxg_muon_workspace_bytes(batch, rows, cols)
        assert ws >= batch * shares * 64 * 64 * 4
