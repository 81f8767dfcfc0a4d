"""The norms where mean square and eps are below float32's smallest normal number (2^-126): rows
of zeros and of tiny values, against the formula in float64."""
import numpy as np
import pytest

from bidirectional_mamba_state_amd import bdssm

pytestmark = pytest.mark.gpu

ULP = 2.0**-149  # between float32 numbers below 2^-126


def _rows(width):
    """A row of zeros, and rows whose squares are below 2^-126 (2^-64 and 2^-66: not rounded)."""
    x = np.zeros((4, width), np.float32)
    x[1], x[2] = 2.0**-64, -(2.0**-66)
    x[3, ::2] = 2.0**-65
    return x


def _norm(x, eps):
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)


@pytest.mark.parametrize("eps", [2.0**-130, 2.0**-140, 2.0**-126])
@pytest.mark.parametrize("width", [64, 520, 2048, 4104])
def test_tiny_rows(width, eps):
    """The mean (width a power of two times a small number, so that 1 / width errs by 2^-24 at most)
    and its sum with eps are rounded below 2^-126 to multiples of 2^-149, by 2^-19 of eps at most;
    the root halves that."""
    import torch
    x = _rows(width)
    want = _norm(x.astype(np.float64), eps)
    xd = torch.from_numpy(x).cuda()
    nd = bdssm.norm_dims(4, width, bdssm.F32, eps=eps)
    u = torch.full_like(xd, float("nan"))
    bdssm.residual_norm(nd, xd, None, None, None, u)
    tol = 2.0**-20 + (2 * ULP / eps)
    assert np.all(np.abs(u.double().cpu().numpy() - want) <= tol * np.abs(want))
    out = torch.full_like(xd, float("nan"))
    z = torch.full_like(xd, 30.0)  # silu(30) = 30 to float32's precision (exp(-30) < 2^-43)
    bdssm.gated_norm(nd, xd, z, None, out, norm_first=True)
    assert np.all(np.abs(out.double().cpu().numpy() / 30 - want) <= (tol + 2.0**-20) * np.abs(want))
