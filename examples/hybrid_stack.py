"""A block-diffusion Mamba hybrid's stack of layers on one MI355X, decoding block by block: Mamba
layers over their cached states and attention layers over a paged cache, joined by the fused
norms. Random weights, hidden vectors instead of tokens (no embedding and no output head).

    python examples/hybrid_stack.py            the 350M shape, 4 streams, prefix 4,096
    python examples/hybrid_stack.py --tiny     a few small layers

The stack alternates groups of Mamba layers with one attention layer. Between layers the
residual stream is updated by bdssm.residual_norm (the layer's output norm, the timestep's gate
and the residual add, then the next layer's input norm with the timestep's gain and shift); a
Mamba layer's scan output meets its gate in bdssm.gated_norm. Matrix products with the weights
are torch's.

  prefill   whole blocks of a prompt at once: prefix scans and block-ordered attention fill the
            states and the pages (no timestep: the cache must not depend on it)
  denoise   one step of the active block: block steps and attention read the caches, write none
  commit    the clean pass over the finished block: states advance, keys and values are appended
"""
import argparse
import math
import os
import sys
import time

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from bidirectional_mamba_state_amd import bdssm  # noqa: E402

N, P = 128, 64  # d_state and head size of the scan
BLOCK = 32


class MambaLayer:
    """One layer's weights and its cached state, in both forms: float32 (the master copy) and the
    block step's operand form."""

    def __init__(self, model, heads, g):
        d, inner = model.width, heads * P
        self.heads, self.inner = heads, inner
        self.w_in = model.weight(g, d, 2 * inner + 2 * N + heads)
        self.w_out = model.weight(g, inner, d)
        self.norm_w = torch.ones(inner, device="cuda")
        self.A = -torch.exp(torch.rand(heads, generator=g, device="cuda") * math.log(16.0))
        self.D = torch.randn(heads, generator=g, device="cuda")
        self.dims = bdssm.dims(model.batch, heads, P, N, 1, bdssm.BF16, bdssm.BF16)
        self.state = torch.zeros((model.batch, heads, N, P), device="cuda")
        self.ops = torch.zeros(bdssm.state_ops_bytes(self.dims), dtype=torch.uint8, device="cuda")

    def inputs(self, u, tokens):
        """(z, (x, dt, B, C)) of the layer's input rows u."""
        b, i = u.shape[0] // tokens, self.inner
        h = u @ self.w_in
        x, B, C = (h[:, s : s + n].contiguous().view(b, tokens, -1) for s, n in ((i, i), (2 * i, N), (2 * i + N, N)))
        dt = torch.nn.functional.softplus(h[:, 2 * i + 2 * N :].float() - 4.0).clamp(1e-3, 0.1).to(h.dtype)
        return h[:, :i], (x.view(b, tokens, self.heads, P), dt.view(b, tokens, self.heads).contiguous(),
                          B.view(b, tokens, 1, N), C.view(b, tokens, 1, N))

    def output(self, y, z):
        rows = z.shape[0]
        out = torch.empty((rows, self.inner), dtype=z.dtype, device="cuda")
        bdssm.gated_norm(bdssm.norm_dims(rows, self.inner, bdssm.BF16), y, z, self.norm_w, out)
        return out @ self.w_out

    def __call__(self, u, tokens, mode):
        z, seq = self.inputs(u, tokens)
        y = torch.empty_like(seq[0])
        if mode == "denoise":
            bdssm.block_step_ops(self.dims, tokens, self.ops, seq, seq, self.A, self.D, y)
        elif mode == "commit":
            bdssm.commit_refresh(self.dims, tokens, seq, self.A, self.D, self.state, self.ops, y=y)
        else:
            need = bdssm.prefix_scan_workspace(self.dims, tokens, 64, True, False)
            ws = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
            bdssm.prefix_scan(self.dims, tokens, 64, seq, self.A, self.D, None, y, None, self.state, ws, need)
            bdssm.state_ops(self.dims, self.state, self.ops)
        return self.output(y, z)


class AttentionLayer:
    """One layer's weights and its paged cache. Pages of all streams come from one pool; the table
    is shared by the stack's attention layers, which cache the same tokens."""

    def __init__(self, model, g):
        d, H, KV = model.width, model.attn_heads, model.kv_heads
        self.model, self.H, self.KV = model, H, KV
        self.w_qkv = model.weight(g, d, (H + 2 * KV) * 64)
        self.w_out = model.weight(g, H * 64, d)
        shape = (model.pages, KV, model.page, 64)
        self.cache = bdssm.KvCache(model.attn, torch.zeros(shape, dtype=torch.bfloat16, device="cuda"),
                                   torch.zeros(shape, dtype=torch.bfloat16, device="cuda"), model.table, model.lens[0], 0)

    def __call__(self, u, tokens, mode):
        m, n, H, KV = self.model, u.shape[0], self.H, self.KV
        qkv = u @ self.w_qkv
        q, k, v = (qkv[:, s * 64 : (s + h) * 64].view(n, h, 64) for s, h in ((0, H), (H, KV), (H + KV, KV)))
        mask = m.mask if mode == "denoise" else m.block_mask
        out = torch.empty((n, H, 64), dtype=u.dtype, device="cuda")
        ws = m.ws if tokens == BLOCK else m.workspace(tokens, self.cache.max_len, mask)
        bdssm.attn_step(m.attn, tokens, q, k, v, self.cache, mask, out, ws)
        if mode != "denoise":
            bdssm.kv_append(m.attn, tokens, k, v, self.cache, m.lens[1])
        return out.view(n, -1) @ self.w_out


class HybridStack:
    def __init__(self, batch, width, mamba_heads, attn_heads, kv_heads, layers, attn_every, max_tokens, window=0, sinks=0,
                 seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.batch, self.width, self.attn_heads, self.kv_heads = batch, width, attn_heads, kv_heads
        self.page, per = 64, -(-max_tokens // 64)
        self.pages = batch * per
        self.table = torch.randperm(self.pages, generator=g, device="cuda").to(torch.int32).view(batch, per)
        self.lens = [torch.zeros(batch, dtype=torch.int32, device="cuda") for _ in range(2)]
        self.length = 0  # the same for every stream here
        self.attn = bdssm.attn_dims(batch, attn_heads, kv_heads, 64, bdssm.BF16, self.page)
        self.mask = bdssm.attn_mask(0.125, 0, window, sinks)          # inside the active block: no order
        self.block_mask = bdssm.attn_mask(0.125, BLOCK, window, sinks)  # clean tokens: by blocks
        self.layers = [AttentionLayer(self, g) if (i + 1) % (attn_every + 1) == 0 else MambaLayer(self, mamba_heads, g)
                       for i in range(layers)]
        # a block's workspace: the longest cache's serves every length, the layers take turns
        self.ws = max((self.workspace(BLOCK, per * self.page, m) for m in (self.mask, self.block_mask)), key=torch.numel)
        self.norm_w = torch.ones(width, device="cuda")
        self.w_time = self.weight(g, 64, 3 * width * layers)

    def workspace(self, tokens, max_len, mask):
        return torch.empty(bdssm.attn_step_workspace(self.attn, tokens, max_len, mask), dtype=torch.uint8, device="cuda")

    def weight(self, g, rows, cols):
        return (torch.randn((rows, cols), generator=g, device="cuda") / math.sqrt(rows)).bfloat16()

    def modulation(self, t):
        """Per layer (gate, gain, shift) of every stream's timestep: slices of one projection."""
        f = torch.cat([torch.sin(t[:, None] * torch.arange(1, 33, device="cuda")),
                       torch.cos(t[:, None] * torch.arange(1, 33, device="cuda"))], 1).bfloat16()
        mod = 0.1 * (f @ self.w_time).view(self.batch, len(self.layers), 3, self.width)
        mod[:, :, :2] += 1.0
        return mod

    def forward(self, x, tokens, mode, t=None):
        """x [batch * tokens, width] float32, the residual stream, is updated in place and
        returned. t: the streams' timesteps (denoise only)."""
        rows, w = x.shape
        nd = bdssm.norm_dims(rows, w, bdssm.BF16, rows_per_stream=tokens, x_dtype=bdssm.F32)
        mod = None if t is None else self.modulation(t)
        part = lambda i, k: None if mod is None or i >= len(self.layers) else mod[:, i, k]  # noqa: E731
        u = torch.empty((rows, w), dtype=torch.bfloat16, device="cuda")
        bdssm.residual_norm(nd, x, None, self.norm_w, None, u, gain=part(0, 1), shift=part(0, 2))
        for i, layer in enumerate(self.layers):
            o = layer(u, tokens, mode)
            last = i + 1 == len(self.layers)
            bdssm.residual_norm(nd, x, o, self.norm_w, x, None if last else u, post_w=self.norm_w, gate=part(i, 0),
                                gain=part(i + 1, 1), shift=part(i + 1, 2), res_scale=1.0 / math.sqrt(2.0 * len(self.layers)))
        if mode != "denoise":  # the caches hold `tokens` more
            self.lens.reverse()
            self.length += tokens
            for layer in self.layers:
                if isinstance(layer, AttentionLayer):
                    layer.cache.set_lens(self.lens[0])
                    layer.cache.max_len = self.length
        return x

    def prefill(self, x, tokens):
        return self.forward(x, tokens, "prefill")

    def denoise(self, x, t):
        return self.forward(x, x.shape[0] // self.batch, "denoise", t)

    def commit(self, x):
        return self.forward(x, x.shape[0] // self.batch, "commit")


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tiny", action="store_true")
    ap.add_argument("--blocks", type=int, default=2)
    ap.add_argument("--steps", type=int, default=8, help="denoising steps of a block")
    ap.add_argument("--window", type=int, default=0, help="sliding window of the attention layers (with 4 sinks)")
    a = ap.parse_args()
    batch, prefix = (2, 256) if a.tiny else (4, 4096)
    shape = dict(width=256, mamba_heads=8, attn_heads=4, kv_heads=2, layers=4, attn_every=3) if a.tiny else \
        dict(width=1024, mamba_heads=32, attn_heads=16, kv_heads=4, layers=24, attn_every=5)
    model = HybridStack(batch, max_tokens=prefix + a.blocks * BLOCK, window=a.window, sinks=4 if a.window else 0, **shape)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    rows = lambda n: torch.randn((batch * n, model.width), generator=g, device="cuda")  # noqa: E731
    model.prefill(rows(prefix), prefix)
    for block in range(a.blocks):
        noisy = rows(BLOCK)
        torch.cuda.synchronize()
        began = time.perf_counter()
        for step in range(a.steps):
            out = model.denoise(noisy.clone(), torch.full((batch,), 1.0 - step / a.steps, device="cuda"))
            noisy = noisy + (out - noisy) / (a.steps - step)
        model.commit(noisy.clone())
        torch.cuda.synchronize()
        ms = (time.perf_counter() - began) * 1e3
        print(f"block {block}: {a.steps} steps and commit of {batch} x {BLOCK} in {ms:.1f} ms, "
              f"{model.length} tokens cached, rms {out.square().mean().sqrt().item():.3f}", flush=True)


if __name__ == "__main__":
    main()
