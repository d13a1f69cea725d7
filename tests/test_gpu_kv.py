"""Attention and experts together, as a decoder runs them: prompts in chunks,
then verify windows with rejected drafts, over paged caches of two layers
(sparse_moe_expert_gemv_b200/kv.py), each layer's attention checked in 64
bits and followed by its MoE layer in place."""
from types import SimpleNamespace

import numpy as np
import pytest
import torch

from sparse_moe_expert_gemv_b200 import inputs as I
from tests import _attn as A

pytestmark = pytest.mark.gpu
LAYERS, D, F, E, K = 2, 256, 128, 16, 2
N_Q, N_KV, DIM, PAGE = 4, 2, 64, 16


@pytest.fixture(scope="module")
def B():
    from sparse_moe_expert_gemv_b200 import binding
    return binding


class Decoder:
    """Two layers: norm, fused projection, attention, output projection, MoE."""

    def __init__(self, B, *, window=0, n_sink=0, e4m3=False, max_seqs=3):
        from sparse_moe_expert_gemv_b200.kv import PagedKV
        self.B = B
        self.ctx = ctx = B.moe_create(D, F, E, K, I.Q4)
        B.moe_configure(ctx, LAYERS, 1, 0, 256)
        g = torch.Generator(device="cuda").manual_seed(5)
        self.w_qkv, self.w_out = [], []
        for layer in range(LAYERS):
            codes, scales, _ = I.experts_torch(0, I.Q4, D, F, layer, 0, E, "cuda")
            B.moe_load_experts(ctx, layer, 0, E, codes, scales)
            sc, ss, _ = I.shared_np(0, I.Q4, D, F, layer)
            B.moe_load_shared(ctx, layer, sc, ss)
            B.moe_set_router(ctx, layer, I.router_np(0, E, D, layer))
            B.moe_set_norm(ctx, layer, None, 1e-6)
            self.w_qkv.append((torch.randn((D, (N_Q + 2 * N_KV) * DIM), generator=g, device="cuda") / 16).bfloat16())
            self.w_out.append((torch.randn((N_Q * DIM, D), generator=g, device="cuda") / 16).bfloat16())
        one = torch.ones(N_KV, device="cuda") / 32 if e4m3 else None
        self.kv = PagedKV(B, ctx, n_layers=LAYERS, n_q=N_Q, n_kv=N_KV, head_dim=DIM, page_size=PAGE, n_pages=64,
                          max_seqs=max_seqs, max_len=300, e4m3=e4m3, k_scale=one, v_scale=one, window=window,
                          n_sink=n_sink)
        self.norm = B.QkNorm(1 + 0.1 * torch.randn(DIM, generator=g, device="cuda"), None, 1e-6)
        self.rope = B.Rope(10000.0 ** (-torch.arange(0, DIM, 2, dtype=torch.float64, device="cuda") / DIM), DIM)

    def layers(self, x, qkv, h, out, check=None):
        n = x.shape[0]
        for layer in range(LAYERS):
            self.B.moe_rmsnorm(self.ctx, layer, x, n, h)
            torch.matmul(h, self.w_qkv[layer], out=qkv[layer].view(n, -1))
            self.kv.attend(layer, qkv[layer], out, self.norm, self.rope)
            if check:
                check(layer, qkv[layer], out)
            x += torch.matmul(out.view(n, -1), self.w_out[layer])
            self.B.moe_prefill(self.ctx, layer, x, n)

    def buffers(self, n):
        return (torch.empty((LAYERS, n, N_Q + 2 * N_KV, DIM), dtype=torch.bfloat16, device="cuda"),
                torch.empty((n, D), dtype=torch.bfloat16, device="cuda"),
                torch.empty((n, N_Q, DIM), dtype=torch.bfloat16, device="cuda"))

    def attention_ok(self, layer, qkv, out):
        """The attention of the open step against the cache in 64 bits."""
        kv = self.kv

        def rows64(b, which):
            t, s = (kv.k[layer], kv.scales[0]) if which == "k" else (kv.v[layer], kv.scales[1])
            if not kv.pages[b]:
                return torch.zeros((0, N_KV, DIM), dtype=torch.float64, device="cuda")
            # (a page that was given back: no row sees it, any will do)
            x = A.as_bytes(t)[torch.tensor([max(p, 0) for p in kv.pages[b]], device="cuda")]
            x = (x.view(t.dtype) if t.dtype == A.E4M3 else x).double()
            if s is not None:
                x = x * s.double()[:, None, None]
            return x.permute(0, 2, 1, 3).reshape(-1, N_KV, DIM)[:kv.length[b]]

        view = SimpleNamespace(n_kv=N_KV, e4m3=kv.k[0].dtype == A.E4M3, kv=kv.length, rows64=rows64)
        n = sum(kv.rows)
        want, tol = A.attention64(qkv[:n, :N_Q].contiguous(), view, kv.rows, DIM ** -0.5, kv.window, kv.n_sink,
                                  chunk=kv.most_rows * (N_Q // N_KV) > 64)
        over = (out[:n].double() - want).abs() - tol
        assert torch.isfinite(out[:n]).all() and over.max() <= 0, float(over.max())


def tokens(n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((n, D), generator=g, device="cuda").bfloat16()


@pytest.mark.parametrize("window,n_sink,e4m3", [(0, 0, False), (40, 3, False), (0, 0, True)])
def test_prompts_then_verify_windows(B, window, n_sink, e4m3):
    dec = Decoder(B, window=window, n_sink=n_sink, e4m3=e4m3)
    try:
        steps = [[70, 0, 33], [0, 120, 0], [3, 3, 3], [1, 0, 4], [2, 5, 1], [50, 1, 1], [1, 1, 1]]
        for i, rows in enumerate(steps):
            n = dec.kv.step(rows)
            x = tokens(n, i)
            dec.layers(x, *dec.buffers(n), check=dec.attention_ok)
            B.moe_sync(dec.ctx, 60000)
            assert torch.isfinite(x).all()
            for s, r in enumerate(rows):
                if r in (3, 4, 5):
                    dec.kv.trim(s, r - 1)  # all but one draft token rejected
    finally:
        B.moe_destroy(dec.ctx)


def test_captured_windows_replay(B):
    """A captured decode step of both layers, replayed for later windows,
    gives what eager calls give."""
    rows, outs = [2, 2, 2], []
    for captured in (False, True):
        dec = Decoder(B)
        try:
            n = dec.kv.step([40, 9, 17])
            dec.layers(tokens(n, 1), *dec.buffers(n))
            n = sum(rows)
            x, buffers, got, graph = tokens(n, 2), dec.buffers(n), [], None
            for i in range(4):
                dec.kv.step(rows)
                x.copy_(tokens(n, 10 + i))
                if captured and i == 1:
                    torch.cuda.synchronize()
                    graph = torch.cuda.CUDAGraph()
                    with torch.cuda.graph(graph):
                        dec.layers(x, *buffers)
                if graph is not None:
                    graph.replay()
                else:
                    dec.layers(x, *buffers)
                got.append(x.clone())
            B.moe_sync(dec.ctx, 60000)
            torch.cuda.synchronize()
            outs.append(torch.stack(got))
            del graph
        finally:
            B.moe_destroy(dec.ctx)
    assert torch.equal(outs[0], outs[1])


def test_contexts_without_moe_configure(B):
    """Attention needs no weights: a context that was only created."""
    from sparse_moe_expert_gemv_b200.kv import PagedKV
    ctx = B.moe_create(D, F, E, K, I.Q4)
    try:
        kv = PagedKV(B, ctx, n_layers=1, n_q=N_Q, n_kv=N_KV, head_dim=DIM, page_size=PAGE, n_pages=4, max_seqs=1,
                     max_len=64)
        n = kv.step([5])
        qkv = torch.randn((n, N_Q + 2 * N_KV, DIM), device="cuda").bfloat16()
        out = torch.full((n, N_Q, DIM), np.nan, dtype=torch.bfloat16, device="cuda")
        kv.attend(0, qkv, out)
        B.moe_sync(ctx, 60000)
        # the first token sees itself alone
        assert torch.equal(out[0], qkv[0, N_Q + N_KV:].repeat_interleave(N_Q // N_KV, 0))
    finally:
        B.moe_destroy(ctx)
