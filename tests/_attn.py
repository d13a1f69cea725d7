"""Inputs and 64-bit reference of the attention tests (tests/test_gpu_attn.py)."""
import math

import torch

E4M3 = torch.float8_e4m3fn


def as_bytes(t):
    return t.view(torch.uint8) if t.dtype == E4M3 else t


class Cache:
    """A paged cache of shuffled pages.  Rows that no sequence holds -- unused
    pages and the ends of last pages -- are NaN."""

    def __init__(self, kv, n_kv, dim, page, e4m3, seed, device="cuda", spare=2):
        g = torch.Generator(device=device).manual_seed(seed)
        self.kv, self.page, self.n_kv, self.dim, self.e4m3 = list(kv), page, n_kv, dim, e4m3
        need = [-(-n // page) for n in kv]
        n_pages = sum(need) + spare
        order = torch.randperm(n_pages, generator=g, device=device).tolist()
        self.table = torch.full((len(kv), max(need + [1])), -1, dtype=torch.int32)
        self.pages = []
        for b, n in enumerate(need):
            mine, order = order[:n], order[n:]
            self.pages.append(mine)
            self.table[b, :n] = torch.tensor(mine, dtype=torch.int32)
        self.table = self.table.to(device)
        shape = (n_pages, n_kv, page, dim)
        kind = E4M3 if e4m3 else torch.bfloat16
        spread = 64.0 if e4m3 else 1.0
        self.k = torch.full(shape, float("nan"), device=device).to(kind)
        self.v = torch.full(shape, float("nan"), device=device).to(kind)
        self.k_scale = self.v_scale = None
        if e4m3:
            self.k_scale = (0.75 + 0.5 * torch.rand(n_kv, generator=g, device=device)) / spread
            self.v_scale = (0.75 + 0.5 * torch.rand(n_kv, generator=g, device=device)) / spread
        for b, n in enumerate(kv):
            for i, p in enumerate(self.pages[b]):
                m = min(page, n - i * page)
                for t in (self.k, self.v):
                    x = torch.randn((n_kv, m, dim), generator=g, device=device) * spread
                    as_bytes(t)[p, :, :m] = as_bytes(x.to(kind))

    def rows64(self, b, which):
        """[kv, n_kv, dim] fp64 values of sequence b."""
        t, s = (self.k, self.k_scale) if which == "k" else (self.v, self.v_scale)
        if not self.pages[b]:
            return torch.zeros((0, self.n_kv, self.dim), dtype=torch.float64, device=t.device)
        x = as_bytes(t)[torch.tensor(self.pages[b], device=t.device)]
        x = (x.view(E4M3) if self.e4m3 else x).double()
        if s is not None:
            x = x * s.double()[:, None, None]
        return x.permute(0, 2, 1, 3).reshape(-1, self.n_kv, self.dim)[:self.kv[b]]

    def batch(self, B, rows, extra_rows=0):
        dev = self.k.device
        off = [0]
        for r in rows:
            off.append(off[-1] + r)
        return B.KvBatch(self.k, self.v, self.table, torch.tensor(off, dtype=torch.int32, device=dev),
                         torch.tensor(self.kv, dtype=torch.int32, device=dev), off[-1] + extra_rows,
                         k_scale=self.k_scale, v_scale=self.v_scale)


def attention64(q, cache, rows, scale, window, sinks, chunk=False):
    """(o, tol) in fp64 for q [n, n_q, dim].

    tol bounds the kernels' rounding, derived term by term.  With
    A = sum p |v| / sum p:
      scores    fp32 sums of exact products: |ds| <= D 2^-23 scale sum |q||k|,
                so each probability is off by a factor within 1 +- 2 ds (a
                probability and the sum it is divided by), and by 2^-20 for
                ex2 and the maximum's multiple;
      p         rounded to bf16, 2^-8 of itself (chunks, and windows over a
                bf16 cache); in windows over an e4m3 cache to fp16, 2^-11 of
                itself and 2^-25 where it is subnormal (the sum is at least 1):
                n 2^-25 max |v|;
      q         (e4m3 caches) fp16 after division by a power of two: exact but
                for elements below 2^-14 of the row's largest, 2^-25 of it:
                |ds| <= scale 2^-24 max|q| sum |k|;
      output    rounded to bf16, 2^-8 of itself.
    """
    n_q, dim, group = q.shape[1], q.shape[2], q.shape[1] // cache.n_kv
    o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(o)
    at = 0
    for b, r in enumerate(rows):
        if r == 0:
            continue
        n = cache.kv[b]
        k, v = cache.rows64(b, "k"), cache.rows64(b, "v")
        i = torch.arange(n - r, n, device=q.device)[:, None]
        j = torch.arange(n, device=q.device)[None]
        seen = j <= i
        if window:
            seen = seen & ((i - j < window) | (j < sinks))
        any_row = seen.any(0)
        k = torch.where(any_row[:, None, None], k, 0.0)
        v = torch.where(any_row[:, None, None], v, 0.0)
        for h in range(n_q):
            qh, kh, vh = q[at:at + r, h].double(), k[:, h // group], v[:, h // group]
            p = torch.softmax(torch.where(seen, qh @ kh.T * scale, -math.inf), -1)
            big = (qh.abs() @ kh.abs().T).amax(-1, keepdim=True)
            ds = dim * 2.0 ** -23 * scale * big
            if cache.e4m3:
                ds = ds + scale * 2.0 ** -24 * qh.abs().amax(-1, keepdim=True) * kh.abs().sum(-1).max()
            a = p @ vh.abs()
            oh = p @ vh
            t = (2.0 ** -11 if cache.e4m3 and not chunk else 2.0 ** -8) * a + (2 * ds + 2.0 ** -20) * a + 2.0 ** -8 * oh.abs()
            if cache.e4m3:
                t = t + n * 2.0 ** -25 * vh.abs().max()
            o[at:at + r, h], tol[at:at + r, h] = oh, t * (1 + 2.0 ** -6)
        at += r
    return o, tol


def norm_rope64(x, gamma, eps, pos, inv_freq, rot, interleaved):
    """fp64 norm and rotation of x [n, heads, dim]; also a bound on the error
    before the last rounding: fp32 products, sums and angles (2^-23 each)."""
    x = x.double()
    if eps is not None:
        x = x * (x.square().mean(-1, keepdim=True) + eps).rsqrt()
        if gamma is not None:
            x = x * gamma.double()
    mag = x.abs().clone()
    if inv_freq is not None:
        a = pos.double()[:, None, None] * inv_freq.double()
        if interleaved:
            i0 = torch.arange(0, rot, 2, device=x.device)
            i1 = i0 + 1
        else:
            i0 = torch.arange(rot // 2, device=x.device)
            i1 = i0 + rot // 2
        u, w = x[..., i0].clone(), x[..., i1].clone()
        x[..., i0] = u * a.cos() - w * a.sin()
        x[..., i1] = w * a.cos() + u * a.sin()
        mag[..., i0] = mag[..., i1] = u.abs() + w.abs()
    # norm: mean and rsqrt about 16 roundings; rotation: sin, cos, two products, a sum
    return x, mag * 2.0 ** -19
