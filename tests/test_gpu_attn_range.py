"""bdssm_attn_step with values near the end of float32's range: a row's weighted sum overflows
only where sum_j |v_j| does, however its scores rise from tile to tile."""
import pytest

from bidirectional_mamba_state_amd import bdssm
from test_gpu_attn import Case, _case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [bdssm.BF16, bdssm.F32])
@pytest.mark.parametrize("lens,tokens", [([120], 8), ([120], 40), ([120, 40], 3)])
def test_large_values_under_rising_scores(dtype, D, lens, tokens):
    """Every value is 2^119, so that 128 of them add to 2^126 and a row's result is 2^119; scores
    rise by 7.9 powers of two after the first 64 keys (to be seen past any reference kept there)."""
    import torch
    _case(f"large values {dtype} {D} {lens} {tokens}")
    c = Case(lens, [tokens] * len(lens), H=2, KV=1, D=D, dtype=dtype, own_keys=False)
    c.q.zero_()
    c.q[:, :, 0] = 1.0
    c.kp.zero_()
    c.vp.fill_(2.0**119)
    late = 7.9 / 1.4426950408889634 / c.scale
    for b, n in enumerate(lens):
        for j in range(64, n):
            c.kp[int(c.table[b, j // c.page]), :, j % c.page, 0] = late
    got = c.run().float()
    assert torch.isfinite(got).all()
    assert ((got / 2.0**119 - 1).abs() <= 2.0**-7).all()
