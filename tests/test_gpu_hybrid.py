"""The example stack (examples/hybrid_stack.py) run through the library: a prompt built at once
and the same prompt built block by block by commits leave the same caches and the same next
step; a denoising step writes no cache; a step in a HIP graph replays."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _module():
    spec = importlib.util.spec_from_file_location("hybrid_stack", os.path.join(ROOT, "examples", "hybrid_stack.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _stack(m, **kw):
    d = dict(batch=2, width=256, mamba_heads=8, attn_heads=6, kv_heads=2, layers=4, attn_every=3, max_tokens=256)
    d.update(kw)
    return m.HybridStack(**d)


def _rel(a, b):
    return ((a - b).float().norm() / b.float().norm()).item()


@pytest.mark.parametrize("window", [0, 40])
def test_prompt_at_once_equals_commits(window):
    """The same tokens through prefix scans with block-ordered attention, or block by block: the
    caches differ by bf16 roundings of intermediate activations only (each layer rounds its
    input, output and scan result to bf16, 2^-8 each; four layers: below 5 %)."""
    import torch
    m = _module()
    one, many = (_stack(m, window=window, sinks=4 if window else 0) for _ in range(2))
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    x = torch.randn((2, 96, 256), generator=g, device="cuda")
    one.prefill(x.reshape(-1, 256).clone(), 96)
    for i in range(0, 96, 32):
        many.commit(x[:, i:i + 32].reshape(-1, 256).clone())
    torch.cuda.synchronize()
    assert one.lens[0].tolist() == many.lens[0].tolist() == [96, 96]
    for a, b in zip(one.layers, many.layers):
        if isinstance(a, m.MambaLayer):
            assert _rel(a.state, b.state) < 0.05
        else:
            used = a.model.table[:, :2].flatten().long()
            assert _rel(a.cache.k[used], b.cache.k[used]) < 0.05 and _rel(a.cache.v[used], b.cache.v[used]) < 0.05
    noisy = torch.randn((64, 256), generator=g, device="cuda")
    t = torch.full((2,), 0.5, device="cuda")
    ya, yb = one.denoise(noisy.clone(), t), many.denoise(noisy.clone(), t)
    assert torch.isfinite(ya).all() and _rel(ya, yb) < 0.05


def test_denoising_writes_no_cache_and_replays_in_a_graph():
    import torch
    m = _module()
    s = _stack(m)
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    s.prefill(torch.randn((2 * 64, 256), generator=g, device="cuda"), 64)
    noisy, t = torch.randn((64, 256), generator=g, device="cuda"), torch.full((2,), 0.3, device="cuda")
    attn = [l for l in s.layers if isinstance(l, m.AttentionLayer)][0]
    before = [attn.cache.k.clone(), attn.cache.v.clone(), s.layers[0].state.clone(), s.lens[0].clone()]
    want = s.denoise(noisy.clone(), t)
    torch.cuda.synchronize()
    for a, b in zip(before, (attn.cache.k, attn.cache.v, s.layers[0].state, s.lens[0])):
        assert torch.equal(a, b)
    x = noisy.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.denoise(x, t)  # warm
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.denoise(x, t)
    for _ in range(3):
        x.copy_(noisy)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(x, want)
        assert torch.equal(s.denoise(noisy.clone(), t), want)  # eager work between replays
