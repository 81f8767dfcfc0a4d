"""The example stack's fork (examples/hybrid_stack.py) where streams end: a parent outside the batch
leaves a row empty in both caches, the attention layers' pages and the Mamba layers' states."""
import pytest

from test_gpu_attn import _case
from test_gpu_hybrid import _module, _rel, _stack

pytestmark = pytest.mark.gpu

OPTIONS = dict(batch=3, rotary=True, cap=20.0, bias=True, managed=True)


@pytest.mark.parametrize("parents", [[-1, 0, 2], [1, -7, -1], [3, 1, 2**31 - 1]], ids=["ended", "two", "past the batch"])
def test_a_row_without_a_parent_is_empty_in_both_caches(parents):
    """Its states are zero; the other rows have their parents' states and operand forms to the last bit; and
    the next step is that of streams that hold the same tokens and no more (bf16 roundings of the
    activations aside, as in test_gpu_hybrid.py)."""
    import torch
    _case(f"ended streams {parents}")
    m = _module()
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    prompt = torch.randn((3, 96, 256), generator=g, device="cuda")
    noisy, t = torch.randn((3, 32, 256), generator=g, device="cuda"), torch.full((3,), 0.5, device="cuda")
    s, before = _stack(m, **OPTIONS), _stack(m, **OPTIONS)
    for x in (s, before):
        x.prefill(prompt.reshape(-1, 256).clone(), 96)
    s.fork(torch.tensor(parents, dtype=torch.int32, device="cuda"))
    goes_on = [0 <= p < 3 for p in parents]
    assert s.lens[0].tolist() == [96 if x else 0 for x in goes_on]
    for a, b in zip(s.layers, before.layers):
        if isinstance(a, m.MambaLayer):
            for row, p in enumerate(parents):
                assert torch.equal(a.state[row], b.state[p]) if goes_on[row] else not a.state[row].any()
            ops = torch.empty_like(a.ops)
            m.bdssm.state_ops(a.dims, a.state, ops)
            assert torch.equal(a.ops, ops)
    got = s.denoise(noisy.reshape(-1, 256).clone(), t).view(3, 32, 256)
    empty = _stack(m, **OPTIONS)
    for row, p in enumerate(parents):
        again = noisy[row].repeat(3, 1, 1).reshape(-1, 256)
        want = (before if goes_on[row] else empty).denoise(again.clone(), t).view(3, 32, 256)[p if goes_on[row] else 0]
        assert torch.isfinite(got[row]).all() and _rel(got[row], want) < 0.05
