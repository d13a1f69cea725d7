"""The attention half of a decoder's layers over a paged key/value cache.

``PagedKV`` owns the caches of all layers, gives their pages to sequences and
keeps the device tables that the attention calls read; ``attend`` is one
layer's step: the call's keys and values appended (norms and rotation on the
way), then attention of its queries over the cache.  With ``moe_forward`` /
``moe_prefill`` behind it this is the engine article's per-layer flow ("93
token/s on one 8 GB card", section "Doorbell handshake": attention, then the
router and the experts).  Windows of draft tokens that are not accepted are
taken back with ``trim`` (section "Speculative decoding").

The bookkeeping is plain host code; every step on the GPU is a library call.
The tables are updated in place, so a CUDA graph that captured ``attend``
replays for the next step of the same shape.
``step`` writes them on torch's current stream and waits for that: run
``attend`` on the same stream, or open a step only when the one before is done.
"""
from __future__ import annotations

import torch


class PagedKV:
    """Paged caches for up to ``max_seqs`` sequences of at most ``max_len``
    tokens in ``n_layers`` layers, on a context of its own geometry
    (``moe_attn_configure`` is called here).

    window > 0: attention sees that many last tokens and the first ``n_sink``;
    pages that no later token can see are given back."""

    def __init__(self, B, ctx, *, n_layers, n_q, n_kv, head_dim, page_size, n_pages, max_seqs, max_len,
                 e4m3=False, k_scale=None, v_scale=None, window=0, n_sink=0, device="cuda"):
        self.B, self.ctx = B, ctx
        self.n_q, self.n_kv, self.dim, self.page = n_q, n_kv, head_dim, page_size
        self.window, self.n_sink = window, n_sink
        self.max_seqs, self.max_len = max_seqs, max_len
        kind = torch.float8_e4m3fn if e4m3 else torch.bfloat16
        shape = (n_pages, n_kv, page_size, head_dim)
        if B is not None:
            B.moe_attn_configure(ctx, n_q, n_kv, head_dim, page_size, B.MOE_KV_E4M3 if e4m3 else B.MOE_KV_BF16)
        self.k = [torch.zeros(shape, dtype=kind, device=device) for _ in range(n_layers)]
        self.v = [torch.zeros(shape, dtype=kind, device=device) for _ in range(n_layers)]
        self.scales = (k_scale, v_scale)
        most = -(-max_len // page_size)
        self.table = torch.full((max_seqs, most), -1, dtype=torch.int32, device=device)
        self.row_off = torch.zeros(max_seqs + 1, dtype=torch.int32, device=device)
        self.kv_len = torch.zeros(max_seqs, dtype=torch.int32, device=device)
        self._table = torch.full((max_seqs, most), -1, dtype=torch.int32)
        self._free = list(range(n_pages - 1, -1, -1))
        self.pages = [[] for _ in range(max_seqs)]   # a sequence's pages in order; -1: given back
        self.length = [0] * max_seqs                 # cached tokens
        self.rows = [0] * max_seqs                   # rows of the present step
        self.most_rows = 0
        self._batches = {}

    # ------------------------------------------------------- bookkeeping
    def free_pages(self):
        return len(self._free)

    def _unseen(self, s):
        """Places of the pages that no token from position ``length[s]`` on sees."""
        if not self.window:
            return []
        whole = min(max(0, self.length[s] - self.window + 1) // self.page, len(self.pages[s]))
        return [i for i in range(-(-self.n_sink // self.page), whole) if self.pages[s][i] >= 0]

    def step(self, rows):
        """Opens a step: rows[s] new tokens of sequence slot s (the batch's
        rows in slot order).  Gives them pages and brings the device tables up
        to date.  Raises MemoryError, changing nothing, when there are not enough
        pages."""
        if len(rows) != self.max_seqs or any(r < 0 for r in rows):
            raise ValueError(f"rows: one count for each of {self.max_seqs} slots")
        if any(n + r > self.max_len for n, r in zip(self.length, rows)):
            raise ValueError(f"a sequence would grow past {self.max_len} tokens")
        # what can be given back is counted before anything changes: a refused
        # step leaves the one before it open, and a trim of that one brings
        # tokens back into the window
        unseen = [self._unseen(s) if rows[s] else [] for s in range(self.max_seqs)]
        need = [max(0, -(-(n + r) // self.page) - len(p)) for n, r, p in zip(self.length, rows, self.pages)]
        free = len(self._free) + sum(map(len, unseen))
        if sum(need) > free:
            raise MemoryError(f"{sum(need)} pages needed, {free} free")
        for s, places in enumerate(unseen):
            for i in places:
                self._free.append(self.pages[s][i])
                self.pages[s][i] = -1
                self._table[s, i] = -1
        off = [0]
        for s, r in enumerate(rows):
            for _ in range(need[s]):
                p = self._free.pop()
                self._table[s, len(self.pages[s])] = p
                self.pages[s].append(p)
            self.length[s] += r
            off.append(off[-1] + r)
        self.rows = list(rows)
        self.most_rows = max(rows, default=0)
        self.table.copy_(self._table)
        self.row_off.copy_(torch.tensor(off, dtype=torch.int32))
        self.kv_len.copy_(torch.tensor(self.length, dtype=torch.int32))
        return off[-1]

    def trim(self, s, n):
        """Takes back the last n tokens of slot s (of its present step only);
        their pages stay with the sequence."""
        if n < 0 or n > self.rows[s]:
            raise ValueError(f"slot {s}: {n} of the {self.rows[s]} tokens of its last step")
        self.length[s] -= n
        self.rows[s] -= n

    def release(self, s):
        """Ends slot s: all its pages are free again."""
        self._free.extend(p for p in self.pages[s] if p >= 0)
        self.pages[s] = []
        self._table[s] = -1
        self.length[s] = self.rows[s] = 0

    # ------------------------------------------------------ a layer's step
    def batch(self, layer, n_rows):
        """The library's view of this layer's cache for calls of n_rows rows."""
        key = (layer, n_rows)
        if key not in self._batches:
            if len(self._batches) >= 16 * len(self.k):  # prompts come in any number of rows
                self._batches.clear()
            ks, vs = self.scales
            self._batches[key] = self.B.KvBatch(self.k[layer], self.v[layer], self.table, self.row_off, self.kv_len,
                                                n_rows, k_scale=ks, v_scale=vs)
        return self._batches[key]

    def attend(self, layer, qkv, out, norm=None, rope=None, scale=None, stream=None):
        """qkv [n, n_q + 2 n_kv, head_dim] bf16, a fused projection's rows of
        the open step (n at least its rows): keys and values go to the cache,
        out [n, n_q, head_dim] receives the attention.  qkv's query part is
        overwritten with the normalised, rotated queries."""
        B, n = self.B, qkv.shape[0]
        q, k, v = qkv[:, :self.n_q], qkv[:, self.n_q:self.n_q + self.n_kv], qkv[:, self.n_q + self.n_kv:]
        batch = self.batch(layer, n)
        scale = self.dim ** -0.5 if scale is None else scale
        B.moe_kv_append(self.ctx, batch, q, k, v, norm, rope, q, stream=stream)
        call = B.moe_attn_forward if self.most_rows <= 32 else B.moe_attn_prefill
        call(self.ctx, batch, q, max(1, self.most_rows), scale, self.window, self.n_sink, out, stream=stream)
