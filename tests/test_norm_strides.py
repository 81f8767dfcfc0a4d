"""Row and stream strides of the norms whose last row lies past what an address can hold: refused
before anything is launched (on the CPU)."""
import ctypes

import pytest

from bidirectional_mamba_state_amd import bdssm

BASE, GB = 1 << 40, 1 << 30
FAR = [(1 << 63) - 1, 1 << 62, (1 << 63) // 7 + 1, (1 << 63) // 14 + 1]


@pytest.mark.parametrize("stride", FAR)
def test_gated_norm(stride):
    nd = bdssm.norm_dims(8, 100, bdssm.BF16)
    got = bdssm.load().bdssm_gated_norm(ctypes.byref(nd), BASE, BASE + GB, stride, None, 0, BASE + 2 * GB, None)
    assert got == bdssm.ERR_UNSUPPORTED


@pytest.mark.parametrize("stride", FAR)
def test_residual_norm(stride):
    nd = bdssm.norm_dims(8, 100, bdssm.BF16, rows_per_stream=1)
    r = bdssm.Residual(BASE, BASE + GB, None, None, BASE + 2 * GB, None, None, stride, 1.0)
    got = bdssm.load().bdssm_residual_norm(ctypes.byref(nd), ctypes.byref(r), BASE + 4 * GB, None, None)
    assert got == bdssm.ERR_UNSUPPORTED
