"""The attention half of a layer, as this library serves it beside the experts:
query/key norms with the rotary positions, the paged key/value cache and the
attention that reads it.  Cases, inputs, plain forms and 64-bit values.

A sequence's cache is a list of pages; a page of a KV head holds `page` keys
(values) of `dim` elements.  A call brings `rows` new tokens of every
sequence; `kv` counts a sequence's cached tokens, the call's own included, so
row t of a sequence sits at position kv - rows + t.  Row i sees key j when
j <= i and (no window, or i - j < window, or j < sinks).
"""
import math

import torch

own = False

_ctx = {}  # the library's contexts by model geometry: one per served model


# ------------------------------------------------------------------- cases
def _case(name, op, **kw):
    c = dict(name=name, op=op, n_q=16, n_kv=4, dim=128, page=64, cache="bf16", seqs=1, rows=1, kv=1,
             ragged=False, window=0, sinks=0, rot=128, interleaved=False, norm=True, far=0)
    c.update(kw)
    return c


def listed():
    return [
        # one verify window of four draft tokens: the smallest call, all latency
        _case("rope_window", "rope", rows=4),
        # a prompt's chunk of 8192 tokens
        _case("rope_chunk", "rope", rows=8192),
        # odd rows far into a long context, half of each head rotated in adjacent pairs, no norm
        _case("rope_odd_far", "rope", rows=1001, n_q=32, n_kv=8, dim=64, rot=32, interleaved=True, norm=False,
              far=1000000),
        # eight sequences' verify windows appended to a bf16 cache
        _case("append_window", "append", seqs=8, rows=4, kv=4096, ragged=True),
        # 64 sequences' windows of five, 8-bit cache, small pages
        _case("append_batch_e4m3", "append", seqs=64, rows=5, kv=999, ragged=True, cache="e4m3", page=16),
        # a chunk of a long prompt
        _case("append_chunk", "append", rows=8192, kv=16384),
        # one user, one token, 32768 tokens resident
        _case("decode_one", "forward", kv=32768),
        # 64 sequences' verify windows of five over ragged caches
        _case("decode_batch", "forward", seqs=64, rows=5, kv=4096, ragged=True),
        # a sliding window with its first tokens kept, 8-bit cache, odd lengths
        _case("decode_sinks_e4m3", "forward", seqs=32, rows=3, kv=30011, ragged=True, cache="e4m3", window=1024,
              sinks=4, n_q=32, n_kv=4, dim=64, rot=64),
        # many users at full length: the largest cache that is read
        _case("decode_long", "forward", seqs=64, kv=32768, n_kv=2, page=128),
        # the second 8192-token chunk of a prompt
        _case("prefill_chunk", "prefill", rows=8192, kv=16384),
        # ragged prompts with a sliding window and sinks behind cached prefixes
        _case("prefill_ragged_sinks", "prefill", seqs=5, rows=1501, kv=5003, ragged=True, window=1024, sinks=4,
              n_q=24, n_kv=4, page=32),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))




def draw(rng):
    op = rng.choice(("rope", "append", "forward", "forward", "prefill", "prefill"))
    n_q, n_kv = rng.choice(((16, 2), (16, 4), (32, 8), (8, 1), (12, 4), (16, 16), (10, 2), (24, 4)))
    dim = rng.choice((64, 128, 128))
    c = dict(op=op, n_q=n_q, n_kv=n_kv, dim=dim, page=rng.choice((16, 32, 64, 128)),
             cache=rng.choice(("bf16", "bf16", "e4m3")), seqs=1, rows=1, kv=1, ragged=rng.random() < 0.7,
             window=0, sinks=0, rot=rng.choice((dim, dim // 2)), interleaved=rng.random() < 0.3,
             norm=rng.random() < 0.7, far=0)
    if op == "rope":
        c.update(rows=_log_int(rng, 1, 8192), far=rng.choice((0, 30000, 1000000)), cache="bf16")
    elif op == "append":
        seqs = _log_int(rng, 1, 64)
        rows = _log_int(rng, 1, 8192 // seqs)
        c.update(seqs=seqs, rows=rows, kv=rows + _log_int(rng, 1, 16384 // seqs))
    elif op == "forward":
        seqs, rows = _log_int(rng, 1, 64), rng.randint(1, 8)
        most = min(32768, 64 * 32768 * 2 * 128 // (seqs * n_kv * dim))
        kv = max(rows, _log_int(rng, 1, most))
        c.update(seqs=seqs, rows=rows, kv=kv)
    else:
        seqs = rng.choice((1, 1, 2, 3, 5))
        rows = _log_int(rng, 33, 8192 // seqs)
        most = min(16384, (16 * 8192 * 16384) // (seqs * rows * n_q))
        c.update(seqs=seqs, rows=rows, kv=rows + rng.choice((0, _log_int(rng, 1, max(1, most - rows)))))
    if op in ("forward", "prefill") and rng.random() < 0.4:
        c.update(window=_log_int(rng, 1, 4096), sinks=rng.choice((0, 1, 4, 70)))
    return c


def _spread(n, most, least):
    """n whole numbers in [least, most], the first `most`, the others spread unevenly."""
    return [most] + [least + int((most - least) * ((i * 0.6180339887) % 1.0)) for i in range(1, n)]


def _plan(c):
    """(rows, kv) of each sequence."""
    if not c["ragged"] or c["seqs"] == 1:
        return [c["rows"]] * c["seqs"], [c["kv"]] * c["seqs"]
    rows = _spread(c["seqs"], c["rows"], 0 if c["rows"] > 1 else 1)
    kv = [max(a, b) for a, b in zip(rows, reversed(_spread(c["seqs"], c["kv"], c["kv"] // 8)))]
    return rows, kv


# ------------------------------------------------------------------ inputs
def _page_list(c, kv, device, g):
    """A page table [seqs, most] over shuffled pages, and the number of pages."""
    need = [-(-n // c["page"]) for n in kv]
    most = max(need)
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=g, device=device).to(torch.int32)
    start = torch.tensor([sum(need[:i]) for i in range(len(need))], device=device)
    at = start[:, None] + torch.arange(most, device=device)[None]
    used = torch.arange(most, device=device)[None] < torch.tensor(need, device=device)[:, None]
    table = torch.where(used, order[at.clamp(max=n_pages - 1)], torch.zeros((), dtype=torch.int32, device=device))
    return table.contiguous(), n_pages


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev).manual_seed(int(seed))
    bf = torch.bfloat16

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device=dev) * scale).to(bf)

    rows, kv = _plan(c)
    n, n_q, n_kv, dim = sum(rows), c["n_q"], c["n_kv"], c["dim"]
    s = dict(case=c, n=n, scale=1.0 / math.sqrt(dim))
    if c["op"] in ("rope", "append"):
        # q, k and v are parts of one projection's rows, as a fused projection leaves them
        qkv = normal(n, n_q + 2 * n_kv, dim)
        s.update(q=qkv[:, :n_q], k=qkv[:, n_q:n_q + n_kv], v=qkv[:, n_q + n_kv:])
        s["inv_freq"] = 10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64) / c["rot"])
        s["inv_freq_dev"] = s["inv_freq"].to(dev)
        gamma = lambda: (1.0 + 0.1 * torch.randn(dim, generator=g, device=dev)) if c["norm"] else None  # noqa: E731
        s["q_gamma"], s["k_gamma"], s["eps"] = gamma(), gamma(), 1e-6
        s["q_out"] = torch.empty(n, n_q, dim, dtype=bf, device=dev)
    if c["op"] == "rope":
        s["pos"] = (c["far"] + torch.arange(n, device=dev)).to(torch.int32)
        s["k_out"] = torch.empty(n, n_kv, dim, dtype=bf, device=dev)
        return s
    s["most_rows"] = max(rows)
    s["row_off"] = torch.tensor([sum(rows[:i]) for i in range(len(rows) + 1)], dtype=torch.int32, device=dev)
    s["kv_len"] = torch.tensor(kv, dtype=torch.int32, device=dev)
    s["table"], n_pages = _page_list(c, kv, dev, g)
    shape = (n_pages, n_kv, c["page"], dim)
    if c["cache"] == "e4m3":
        s["k_cache"] = normal(*shape, scale=64.0).to(torch.float8_e4m3fn)
        s["v_cache"] = normal(*shape, scale=64.0).to(torch.float8_e4m3fn)
        s["k_scale"] = (0.75 + 0.5 * torch.rand(n_kv, generator=g, device=dev)) / 64.0
        s["v_scale"] = (0.75 + 0.5 * torch.rand(n_kv, generator=g, device=dev)) / 64.0
    else:
        s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"] = normal(*shape), normal(*shape), None, None
    if c["op"] != "append":
        s["q"] = normal(n, n_q, dim, scale=2.0)  # logits of a standard deviation of two
        s["out"] = torch.empty(n, n_q, dim, dtype=bf, device=dev)
    return s


# ------------------------------------------------------------- plain forms
def _norm_rope(x, gamma, eps, pos, s):
    """RMS norm of each head (where gamma is given), then the rotation; 32 bits, angles in 64."""
    c = s["case"]
    x = x.float()
    if gamma is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * gamma
    angle = pos.double()[:, None] * s["inv_freq_dev"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    rot = c["rot"]
    if c["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _bytes(t):
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def _stored(x, scale, cache):
    """32-bit rows as the cache holds them."""
    if cache.dtype == torch.float8_e4m3fn:
        return (x / scale[:, None]).clamp(-448.0, 448.0).to(cache.dtype)
    return x.to(cache.dtype)


def _plain_rope(s):
    s["q_out"].copy_(_norm_rope(s["q"], s["q_gamma"], s["eps"], s["pos"], s))
    s["k_out"].copy_(_norm_rope(s["k"], s["k_gamma"], s["eps"], s["pos"], s))
    return {"q": s["q_out"], "k": s["k_out"]}


def _plain_append(s):
    off = s["row_off"].long()
    count = off[1:] - off[:-1]
    seq = torch.repeat_interleave(torch.arange(count.numel(), device=off.device), count, output_size=s["n"])
    pos = s["kv_len"].long()[seq] - count[seq] + torch.arange(s["n"], device=off.device) - off[seq]
    page, at = s["table"][seq, pos // s["case"]["page"]].long(), pos % s["case"]["page"]
    s["q_out"].copy_(_norm_rope(s["q"], s["q_gamma"], s["eps"], pos, s))
    k = _norm_rope(s["k"], s["k_gamma"], s["eps"], pos, s)
    _bytes(s["k_cache"])[page, :, at] = _bytes(_stored(k, s["k_scale"], s["k_cache"]))
    _bytes(s["v_cache"])[page, :, at] = _bytes(_stored(s["v"].float(), s["v_scale"], s["v_cache"]))
    return {"q": s["q_out"], "k": s["k_cache"], "v": s["v_cache"]}


def _gathered(s, cache, scale):
    """[seqs, n_kv, length, dim] in 32 bits: every sequence's pages, one after another."""
    x = _bytes(cache)[s["table"].long()]
    x = (x.view(cache.dtype) if cache.dtype == torch.float8_e4m3fn else x).float()
    x = x.permute(0, 2, 1, 3, 4).flatten(2, 3)
    return x if scale is None else x * scale[:, None, None]


def _plain_attention(s):
    c, dev = s["case"], s["q"].device
    n_q, n_kv, group = c["n_q"], c["n_kv"], c["n_q"] // c["n_kv"]
    off, most = s["row_off"].long(), s["most_rows"]
    count = off[1:] - off[:-1]
    t = torch.arange(most, device=dev)
    held = t[None] < count[:, None]                                   # [seqs, most]
    at = (off[:-1, None] + t[None]).clamp(max=s["n"] - 1)
    q = s["q"][at].float().view(-1, most, n_kv, group, c["dim"]).permute(0, 2, 3, 1, 4).flatten(2, 3)
    k, v = _gathered(s, s["k_cache"], s["k_scale"]), _gathered(s, s["v_cache"], s["v_scale"])
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"])
    x = x.view(-1, n_kv, group, most, k.shape[2])
    j = torch.arange(k.shape[2], device=dev)
    i = s["kv_len"].long()[:, None] - count[:, None] + t[None]        # [seqs, most]
    seen = (j <= i[..., None]) & (j < s["kv_len"].long()[:, None, None])
    if c["window"]:
        seen &= (i[..., None] - j < c["window"]) | (j < c["sinks"])
    x = x.masked_fill_(~seen[:, None, None], float("-inf"))
    x = x.sub_(x.amax(-1, keepdim=True)).exp_()
    total = x.sum(-1, keepdim=True)
    y = torch.matmul(x.flatten(2, 3), v).view(-1, n_kv, group, most, c["dim"]) / total
    y = y.permute(0, 3, 1, 2, 4).reshape(-1, most, n_q, c["dim"])
    s["out"].copy_(y[held])
    return {"out": s["out"]}


# ------------------------------------------------------------ the library's
def _library(s):
    """The context of this geometry and the binding, as a serving program holds them."""
    c = s["case"]
    key = (c["n_q"], c["n_kv"], c["dim"], c["page"], c["cache"])
    if key not in _ctx:
        from sparse_moe_expert_gemv_b200 import binding as B
        ctx = B.moe_create(2048, 768, 512, 10, B.MOE_Q4_SYM_G32_F16)
        B.moe_attn_configure(ctx, c["n_q"], c["n_kv"], c["dim"], c["page"],
                             B.MOE_KV_E4M3 if c["cache"] == "e4m3" else B.MOE_KV_BF16)
        _ctx[key] = (B, ctx)
    return _ctx[key]


def _batch(B, s):
    return B.KvBatch(s["k_cache"], s["v_cache"], s["table"], s["row_off"], s["kv_len"], s["n"],
                     k_scale=s["k_scale"], v_scale=s["v_scale"])


def _handles(s):
    """The binding, the context, the layer's norms and rotation and the batch's view of the cache."""
    if "handles" not in s:
        B, ctx = _library(s)
        norm = rope = batch = None
        if s["case"]["op"] in ("rope", "append"):
            if s["q_gamma"] is not None:
                norm = B.QkNorm(s["q_gamma"], s["k_gamma"], s["eps"])
            rope = B.Rope(s["inv_freq_dev"], s["case"]["rot"], s["case"]["interleaved"])
        if s["case"]["op"] != "rope":
            batch = _batch(B, s)
        s["handles"] = (B, ctx, norm, rope, batch)
    return s["handles"]


def _own_rope(s):
    B, ctx, norm, rope, _ = _handles(s)
    B.moe_qk_norm_rope(ctx, s["n"], s["q"], s["k"], s["pos"], norm, rope, s["q_out"], s["k_out"])
    return {"q": s["q_out"], "k": s["k_out"]}


def _own_append(s):
    B, ctx, norm, rope, batch = _handles(s)
    B.moe_kv_append(ctx, batch, s["q"], s["k"], s["v"], norm, rope, s["q_out"])
    return {"q": s["q_out"], "k": s["k_cache"], "v": s["v_cache"]}


def _own_attention(s):
    B, ctx, _, _, batch = _handles(s)
    c = s["case"]
    if c["op"] == "forward":
        B.moe_attn_forward(ctx, batch, s["q"], s["most_rows"], s["scale"], c["window"], c["sinks"], s["out"])
    else:
        B.moe_attn_prefill(ctx, batch, s["q"], s["most_rows"], s["scale"], c["window"], c["sinks"], s["out"])
    return {"out": s["out"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return _own_rope(state) if op == "rope" else _own_append(state) if op == "append" else _own_attention(state)
    return _plain_rope(state) if op == "rope" else _plain_append(state) if op == "append" else _plain_attention(state)


# -------------------------------------------------------------------- work
def _seen(i, kv, window, sinks):
    """Keys that the row at position i of a sequence of kv cached tokens sees."""
    n = min(i + 1, kv)
    if not window or n <= window:
        return max(n, 0)
    low = i + 1 - window  # the first key inside the window
    return max(0, n - low) + min(sinks, low)


def work(case):
    c = case
    rows, kv = _plan(c)
    n, n_q, n_kv, dim = sum(rows), c["n_q"], c["n_kv"], c["dim"]
    if c["op"] == "rope":
        return {"bytes": 2 * n * (n_q + n_kv) * dim * 2 + 4 * n, "flops": 10 * n * (n_q + n_kv) * dim}
    held = 1 if c["cache"] == "e4m3" else 2
    if c["op"] == "append":
        return {"bytes": n * dim * (2 * n_q * 2 + 2 * n_kv * (2 + held)) + 4 * n,
                "flops": 10 * n * (n_q + n_kv) * dim}
    pairs = sum(_seen(b - a + t, b, c["window"], c["sinks"]) for a, b in zip(rows, kv) for t in range(a))
    touched = [0 if not a else b if not c["window"] else
               min(b, c["window"] + a - 1) + min(c["sinks"], max(0, b - c["window"] - a + 1))
               for a, b in zip(rows, kv)]
    return {"bytes": 2 * sum(touched) * n_kv * dim * held + 2 * n * n_q * dim * 2, "flops": 4 * pairs * n_q * dim}


# ----------------------------------------------------- values in 64 bits
def _rotated64(x, gamma, eps, pos, c):
    """One head row at a time seen as D numbers: norm, then each pair turned by its angle."""
    x = x.double()
    if gamma is not None:
        x = x / (x.square().sum(-1, keepdim=True) / x.shape[-1] + eps).sqrt() * gamma.double()
    half = c["rot"] // 2
    p = torch.arange(half, device=x.device)
    first, second = (2 * p, 2 * p + 1) if c["interleaved"] else (p, p + half)
    turn = torch.exp(-p.double() * 2 / c["rot"] * math.log(10000.0)) * pos.double().view(-1, 1, 1)
    z = torch.complex(x[..., first], x[..., second]) * torch.polar(torch.ones_like(turn), turn)
    x[..., first], x[..., second] = z.real, z.imag
    return x


def exact(case, seed):
    c, s = case, prepare(case, seed)
    rows, kv = _plan(c)
    if c["op"] == "rope":
        return {"q": _rotated64(s["q"], s["q_gamma"], s["eps"], s["pos"], c),
                "k": _rotated64(s["k"], s["k_gamma"], s["eps"], s["pos"], c)}
    if c["op"] == "append":
        pos = torch.tensor([b - a + t for a, b in zip(rows, kv) for t in range(a)], device="cuda")
        seq = torch.tensor([i for i, a in enumerate(rows) for _ in range(a)], device="cuda")
        k = _rotated64(s["k"], s["k_gamma"], s["eps"], pos, c)
        v = s["v"].double()
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        if s["k_scale"] is not None:
            k, v = k / s["k_scale"].double()[:, None], v / s["v_scale"].double()[:, None]
        where = s["table"].long()[seq, pos // c["page"]] * c["page"] + pos % c["page"]
        for cache, new in ((kc, k), (vc, v)):
            flat = cache.transpose(1, 2).reshape(-1, c["n_kv"], c["dim"])
            flat[where] = new.clamp(-448, 448) if c["cache"] == "e4m3" else new
            cache.copy_(flat.view(-1, c["page"], c["n_kv"], c["dim"]).transpose(1, 2))
        return {"q": _rotated64(s["q"], s["q_gamma"], s["eps"], pos, c), "k": kc, "v": vc}
    if 4 * sum(rows) * max(kv) * c["n_q"] * c["dim"] > 3e12:
        return None
    out = torch.zeros(s["n"], c["n_q"], c["dim"], dtype=torch.float64, device="cuda")
    group, begin = c["n_q"] // c["n_kv"], 0
    for b, (a, length) in enumerate(zip(rows, kv)):
        if a:
            pages = s["table"][b, :-(-length // c["page"])].long()
            j = torch.arange(length, device="cuda")
            i = torch.arange(length - a, length, device="cuda")[:, None]
            hidden = j > i
            if c["window"]:
                hidden = hidden | ((i - j >= c["window"]) & (j >= c["sinks"]))
            for h in range(c["n_kv"]):
                k = s["k_cache"][:, h][pages] if c["cache"] == "bf16" else \
                    s["k_cache"].view(torch.uint8)[:, h][pages].view(torch.float8_e4m3fn)
                v = s["v_cache"][:, h][pages] if c["cache"] == "bf16" else \
                    s["v_cache"].view(torch.uint8)[:, h][pages].view(torch.float8_e4m3fn)
                k, v = k.double().reshape(-1, c["dim"])[:length], v.double().reshape(-1, c["dim"])[:length]
                if s["k_scale"] is not None:
                    k, v = k * s["k_scale"][h].double(), v * s["v_scale"][h].double()
                for m in range(h * group, h * group + group):
                    w = (s["q"][begin:begin + a, m].double() @ k.T) * s["scale"]
                    w = torch.softmax(w.masked_fill(hidden, float("-inf")), -1)
                    out[begin:begin + a, m] = w @ v
        begin += a
    return {"out": out}
