"""Rows that share a workgroup with a row that attends to an infinity or a NaN: bdssm_attn_step
computes them again apart, by the same rules."""
import pytest

from bidirectional_mamba_state_amd import bdssm
from test_gpu_attn import Case, _case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [bdssm.BF16, bdssm.F32])
def test_rows_beside_a_nan_keep_their_results(dtype, D):
    """Queries and keys of whole quarters and small whole values, one tile of keys: scores, sums of
    (rounded) weights and weighted sums are exact in float32 in any order with bf16 (weights of 8
    bits above 2^-12, 40 of them: 24 bits), so a row's result is the same to the last bit whether a
    neighbour's key holds a NaN or not. With float32 weights the sums round: 40 terms by 2^-24 each,
    twice, and so does the division."""
    import torch
    _case(f"neighbours {dtype} {D}")
    c = Case([0], [40], H=4, KV=2, D=D, dtype=dtype, block=8)
    g = torch.Generator(device="cuda")
    g.manual_seed(D)
    pick = lambda t: torch.randint(-2, 3, t.shape, generator=g, device="cuda").to(t.dtype)  # noqa: E731
    c.q.copy_(pick(c.q) / 4)
    c.k.copy_(pick(c.k) / 2)
    c.v.copy_(pick(c.v))
    before = c.run()
    c.v[33, :, 5] = float("nan")  # seen by tokens 32 to 39
    after = c.run()
    assert torch.isnan(after[32:, :, 5]).all() and torch.isfinite(after[:32]).all()
    if dtype == bdssm.BF16:
        assert torch.equal(after[:32], before[:32])
    else:
        w = c.v[:32].abs().amax().float()
        assert (after[:32] - before[:32]).abs().max() <= 2 * 82 * 2.0**-24 * w
