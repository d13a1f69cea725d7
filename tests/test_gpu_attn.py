"""Attention calls on the GPU against 64-bit references: norms with rotary
positions, the append to the paged cache, window and chunk attention, and a
run of them together."""
import math

import pytest
import torch

from tests import _attn as A

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from sparse_moe_expert_gemv_b200 import binding
    return binding


@pytest.fixture(scope="module")
def make_ctx(B):
    made = {}

    def get(n_q, n_kv, dim, page, e4m3):
        key = (n_q, n_kv, dim, page, e4m3)
        if key not in made:
            ctx = B.moe_create(256, 128, 16, 2, B.MOE_Q4_SYM_G32_F16)
            B.moe_attn_configure(ctx, n_q, n_kv, dim, page, B.MOE_KV_E4M3 if e4m3 else B.MOE_KV_BF16)
            made[key] = ctx
        return made[key]

    yield get
    for ctx in made.values():
        B.moe_destroy(ctx)


def rnd(shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def close(got, want, tol):
    got, bad = got.double(), None
    assert torch.isfinite(got).all()
    over = (got - want).abs() - tol
    if (over > 0).any():
        bad = int((over > 0).sum()), float(over.max()), float((got - want).abs().max())
    assert bad is None, bad


# ------------------------------------------------------- norms and rotation
@pytest.mark.parametrize("n,n_q,n_kv,dim,rot,inter,norm,rope,far", [
    (1, 16, 2, 128, 128, False, True, True, 0),
    (4, 16, 4, 128, 128, True, True, True, 7),
    (5, 3, 3, 64, 32, False, True, True, 1000000),
    (37, 10, 2, 64, 64, True, False, True, 2000000000),
    (129, 8, 1, 128, 64, False, "one", True, 31000),
    (3, 1, 1, 64, 8, False, True, True, 12345),
    (1500, 12, 4, 128, 128, False, True, True, 100),
    (7, 16, 2, 128, 128, False, True, False, 0),
    (7, 16, 2, 128, 128, False, False, False, 0),
])
def test_qk_norm_rope(B, make_ctx, n, n_q, n_kv, dim, rot, inter, norm, rope, far):
    ctx = make_ctx(n_q, n_kv, dim, 64, False)
    qkv = rnd((n, n_q + 2 * n_kv, dim), 1)
    q, k = qkv[:, :n_q], qkv[:, n_q:n_q + n_kv]
    gq = 1 + 0.1 * rnd((dim,), 2).float() if norm is True else None
    gk = 1 + 0.1 * rnd((dim,), 3).float() if norm is True else None
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    pos = (far + torch.arange(n, device="cuda").flip(0)).to(torch.int32)
    N = B.QkNorm(gq, gk, 1e-6) if norm else None
    R = B.Rope(inv, rot, inter) if rope else None
    # outputs strided too; what lies between their rows stays
    qo, ko = torch.full((n + 1, n_q + 1, dim), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full(
        (n + 1, n_kv, dim), 7.0, dtype=torch.bfloat16, device="cuda")
    B.moe_qk_norm_rope(ctx, n, q, k, pos if rope else None, N, R, qo[:, :n_q], ko)
    for got, x, gm in ((qo[:n, :n_q], q, gq), (ko[:n], k, gk)):
        want, err = A.norm_rope64(x, gm, 1e-6 if norm else None, pos, inv if rope else None, rot, inter)
        close(got, want, err + (want.abs() + err) * 2.0 ** -8)
    assert (qo[:, n_q] == 7).all() and (qo[n] == 7).all() and (ko[n] == 7).all()
    # in place, on the fused projection's rows
    B.moe_qk_norm_rope(ctx, n, q, k, pos if rope else None, N, R, q, k)
    assert torch.equal(q, qo[:n, :n_q]) and torch.equal(k, ko[:n])
    B.moe_sync(ctx, 60000)


def test_qk_norm_rope_zero_rows_and_zero_heads(B, make_ctx):
    ctx = make_ctx(16, 2, 128, 64, False)
    z = torch.zeros((3, 16, 128), dtype=torch.bfloat16, device="cuda")
    zk = torch.zeros((3, 2, 128), dtype=torch.bfloat16, device="cuda")
    out, outk = torch.full_like(z, 5), torch.full_like(zk, 5)
    B.moe_qk_norm_rope(ctx, 0, z, zk, None, B.QkNorm(), None, out, outk)
    assert (out == 5).all() and (outk == 5).all()
    B.moe_qk_norm_rope(ctx, 3, z, zk, None, B.QkNorm(eps=1e-6), None, out, outk)
    assert (out == 0).all() and (outk == 0).all()


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("rows,kv,page,n_q,n_kv,dim", [
    ([1], [1], 16, 16, 2, 128),
    ([4, 0, 5, 1], [4, 9, 130, 64], 64, 16, 4, 128),
    ([33, 70], [40, 70], 16, 10, 2, 64),
    ([0, 3, 0, 0, 2, 0], [0, 3, 5, 0, 257, 1], 256, 8, 8, 64),
    ([1500], [1999], 32, 12, 4, 128),
    ([1] * 300, [1 + i % 40 for i in range(300)], 16, 4, 1, 64),
])
def test_append(B, make_ctx, e4m3, rows, kv, page, n_q, n_kv, dim):
    ctx = make_ctx(n_q, n_kv, dim, page, e4m3)
    cache = A.Cache(kv, n_kv, dim, page, e4m3, seed=5)
    n, extra = sum(rows), 3
    qkv = rnd((n + extra, n_q + 2 * n_kv, dim), 6)
    q, k, v = qkv[:, :n_q], qkv[:, n_q:n_q + n_kv], qkv[:, n_q + n_kv:]
    gq, gk = 1 + 0.1 * rnd((dim,), 2).float(), 1 + 0.1 * rnd((dim,), 3).float()
    inv = 10000.0 ** (-torch.arange(0, dim, 2, dtype=torch.float64, device="cuda") / dim)
    before = [A.as_bytes(cache.k).clone(), A.as_bytes(cache.v).clone()]
    batch = cache.batch(B, rows, extra)
    q_out = torch.full((n + extra, n_q, dim), 9.0, dtype=torch.bfloat16, device="cuda")
    B.moe_kv_append(ctx, batch, q, k, v, B.QkNorm(gq, gk, 1e-6), B.Rope(inv, dim), q_out)
    B.moe_sync(ctx, 60000)
    assert (q_out[n:] == 9).all()
    pos = torch.tensor([b - a + t for a, b in zip(rows, kv) for t in range(a)], device="cuda")
    seq = [b for b, a in enumerate(rows) for _ in range(a)]
    want, err = A.norm_rope64(q[:n], gq, 1e-6, pos, inv, dim, False)
    close(q_out[:n], want, err + (want.abs() + err) * 2.0 ** -8)
    wk, ek = A.norm_rope64(k[:n], gk, 1e-6, pos, inv, dim, False)
    wv, ev = v[:n].double(), torch.zeros_like(v[:n].double())
    touched = torch.zeros(before[0].shape[0], page, dtype=torch.bool, device="cuda")
    page_of = torch.tensor([cache.pages[b][p // page] for b, p in zip(seq, pos.tolist())], device="cuda")
    touched[page_of, pos % page] = True
    for got, w, e, sc, old in ((cache.k, wk, ek, cache.k_scale, before[0]), (cache.v, wv, ev, cache.v_scale, before[1])):
        stored = A.as_bytes(got)[page_of, :, pos % page]
        stored = (stored.view(A.E4M3) if e4m3 else stored).double()
        if e4m3:
            # one rounding of x / scale (itself rounded once): half a step, 2^-4
            # of a normal value, 2^-10 of a subnormal one
            w, e = w / sc.double()[:, None], e / sc.double()[:, None]
            w = w.clamp(-448, 448)
            close(stored, w, e + (w.abs() + e) * (2.0 ** -4 + 2.0 ** -23) + 2.0 ** -10)
        else:
            close(stored, w, e + (w.abs() + e) * 2.0 ** -8)
        same = A.as_bytes(got).permute(0, 2, 1, 3)[~touched]
        old = old.permute(0, 2, 1, 3)[~touched]
        assert torch.equal(same.contiguous().view(torch.uint8), old.contiguous().view(torch.uint8))


def test_append_saturates_and_keeps_nan(B, make_ctx):
    """e4m3: finite values past 448 and infinities are stored as +-448, NaN as NaN."""
    ctx = make_ctx(4, 1, 64, 16, True)
    cache = A.Cache([2], 1, 64, 16, True, seed=1)
    cache.k_scale.fill_(0.5)
    cache.v_scale.fill_(2.0)
    k = rnd((2, 1, 64), 1)
    v = rnd((2, 1, 64), 2)
    k[0, 0, :4] = torch.tensor([1e4, -1e4, float("inf"), float("nan")])
    v[1, 0, :3] = torch.tensor([896.0, -897.0, float("-inf")])
    B.moe_kv_append(ctx, cache.batch(B, [2]), None, k, v, None, None, None)
    B.moe_sync(ctx, 60000)
    p = cache.pages[0][0]
    assert cache.k[p, 0, 0, :3].float().tolist() == [448, -448, 448] and cache.k[p, 0, 0, 3].float().isnan()
    assert cache.v[p, 0, 1, :3].float().tolist() == [448, -448, -448]


# --------------------------------------------------------------- attention
SHAPES = [
    # rows, kv, page, n_q, n_kv, dim, window, sinks
    ([1], [1], 16, 16, 2, 128, 0, 0),
    ([1], [63], 64, 16, 4, 128, 0, 0),
    ([4], [64], 64, 16, 4, 128, 0, 0),
    ([5], [65], 16, 10, 2, 64, 0, 0),
    ([1, 3, 0, 5], [200, 3, 77, 129], 32, 24, 4, 128, 0, 0),
    ([0, 2, 0, 0, 32, 0], [0, 2, 5, 0, 900, 0], 256, 8, 8, 64, 0, 0),
    ([8], [5000], 128, 16, 2, 128, 0, 0),           # 64 rows: four row tiles, many parts
    ([3], [9001], 16, 4, 1, 64, 0, 0),              # one head over the whole GPU
    ([4, 4], [3000, 40], 64, 16, 4, 128, 256, 4),
    ([2, 5], [1000, 700], 16, 32, 4, 64, 1, 0),     # each row sees itself alone
    ([2, 5], [1000, 700], 32, 6, 2, 64, 1, 1),
    ([1, 4, 7], [4097, 500, 7], 64, 20, 4, 128, 100, 70),
    ([6], [2500], 64, 8, 1, 128, 2400, 63),
    ([7], [300], 64, 12, 12, 64, 100000, 5),        # a window past the start
    ([12, 9], [333, 1025], 64, 28, 4, 128, 0, 0),   # more than 64 rows per head: several blocks
    ([1] * 150, [1 + (i * 37) % 400 for i in range(150)], 16, 8, 2, 64, 0, 0),
]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("rows,kv,page,n_q,n_kv,dim,window,sinks", SHAPES)
def test_forward(B, make_ctx, e4m3, rows, kv, page, n_q, n_kv, dim, window, sinks):
    run_attention(B, make_ctx, B.moe_attn_forward, e4m3, rows, kv, page, n_q, n_kv, dim, window, sinks)


def run_attention(B, make_ctx, fn, e4m3, rows, kv, page, n_q, n_kv, dim, window, sinks, scale=None):
    ctx = make_ctx(n_q, n_kv, dim, page, e4m3)
    cache = A.Cache(kv, n_kv, dim, page, e4m3, seed=11)
    n, extra = sum(rows), 2
    if window:  # keys before every row's window hold anything
        for b, (r, length) in enumerate(zip(rows, kv)):
            for j in range(sinks, max(sinks, length - r - window + 1)):
                for t, x in ((cache.k, float("inf")), (cache.v, float("nan"))):
                    A.as_bytes(t)[cache.pages[b][j // page], :, j % page] = A.as_bytes(
                        torch.tensor(x, device="cuda").to(t.dtype))
        # and pages that hold no visible key are given back
        for b, (r, length) in enumerate(zip(rows, kv)):
            for i in range(len(cache.pages[b])):
                if r and i * page >= sinks and (i + 1) * page <= length - r - window + 1:
                    cache.table[b, i] = -1 - i
    wide = rnd((n + extra, n_q + 3, dim), 12, scale=2.0)
    q = wide[:, 1:n_q + 1]
    scale = scale or 1 / math.sqrt(dim)
    out = torch.full((n + extra, n_q, dim), 3.0, dtype=torch.bfloat16, device="cuda")
    batch = cache.batch(B, rows, extra)
    fn(ctx, batch, q, max(rows), scale, window, sinks, out)
    B.moe_sync(ctx, 60000)
    want, tol = A.attention64(q[:n], cache, rows, scale, window, sinks, chunk=max(rows) * (n_q // n_kv) > 64)
    close(out[:n], want, tol)
    assert (out[n:] == 3).all()
    # the same call again gives the same bits, and so does out = q
    again = torch.full_like(out, 3.0)
    fn(ctx, batch, q, max(rows), scale, window, sinks, again)
    assert torch.equal(again, out)
    fn(ctx, batch, q, max(rows), scale, window, sinks, q)
    B.moe_sync(ctx, 60000)
    assert torch.equal(q[:n], out[:n])


def test_forward_peaked_and_flat_scores(B, make_ctx):
    """Scores of hundreds (one key takes all) and of zero (the mean)."""
    ctx = make_ctx(8, 2, 128, 64, False)
    cache = A.Cache([777], 2, 128, 64, False, seed=3)
    batch = cache.batch(B, [2])
    for s in (0.0, 40.0):
        q = rnd((2, 8, 128), 4, scale=s)
        out = torch.empty_like(q)
        B.moe_attn_forward(ctx, batch, q, 2, 1 / math.sqrt(128), 0, 0, out)
        want, tol = A.attention64(q, cache, [2], 1 / math.sqrt(128), 0, 0)
        close(out, want, tol)


@pytest.mark.parametrize("e4m3", [False, True])
def test_more_rows_than_announced(B, make_ctx, e4m3):
    """max_T below a sequence's rows: the same results, in more row blocks."""
    ctx = make_ctx(16, 2, 128, 64, e4m3)
    rows = [20, 1, 41]
    cache = A.Cache([500, 90, 41], 2, 128, 64, e4m3, seed=3)
    q = rnd((sum(rows), 16, 128), 4, scale=2.0)
    out = torch.empty_like(q)
    for fn in (B.moe_attn_forward, B.moe_attn_prefill):
        out.fill_(float("nan"))
        fn(ctx, cache.batch(B, rows), q, 1, 0.09, 100, 3, out)
        want, tol = A.attention64(q, cache, rows, 0.09, 100, 3)
        close(out, want, tol)


def test_forward_nan_reaches_only_its_sequence(B, make_ctx):
    """A NaN that a row sees gives NaN there, and touches no other sequence."""
    ctx = make_ctx(8, 2, 64, 16, False)
    cache = A.Cache([100, 90], 2, 64, 16, False, seed=3)
    cache.v[cache.pages[0][2], 1, 3] = float("nan")
    q = rnd((2, 8, 64), 4)
    out = torch.empty_like(q)
    B.moe_attn_forward(ctx, cache.batch(B, [1, 1]), q, 1, 0.125, 0, 0, out)
    assert out[0, 4:].isnan().all() and out[0, :4].isfinite().all() and out[1].isfinite().all()


def test_tables_updated_in_place_under_a_graph(B, make_ctx):
    """A captured append and attention replay with the tables' new contents."""
    ctx = make_ctx(16, 4, 128, 64, False)
    full = A.Cache([700, 260], 4, 128, 64, False, seed=21)
    rows = [2, 1]
    n = 3
    batch = full.batch(B, rows)
    kv_len = batch.tensors[4]
    q, k, v = rnd((n, 16, 128), 1), rnd((n, 4, 128), 2), rnd((n, 4, 128), 3)
    q_out, out = torch.empty_like(q), torch.empty_like(q)
    inv = 10000.0 ** (-torch.arange(0, 128, 2, dtype=torch.float64, device="cuda") / 128)
    norm, rope = B.QkNorm(eps=1e-6), B.Rope(inv, 128)

    def step():
        B.moe_kv_append(ctx, batch, q, k, v, norm, rope, q_out)
        B.moe_attn_forward(ctx, batch, q_out, 2, 0.1, 0, 0, out)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for lens in ([700, 260], [64, 1], [129, 65]):
        kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        q.copy_(rnd(q.shape, sum(lens)))
        k.copy_(rnd(k.shape, sum(lens) + 1))
        if lens == [64, 1]:
            assert rows == [2, 1]
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        full.kv = lens
        # the cache now holds the appended rows: attention over it in 64 bits
        want, tol = A.attention64(q_out, full, rows, 0.1, 0, 0)
        close(got, want, tol)
        pos = torch.tensor([lens[0] - 2, lens[0] - 1, lens[1] - 1], device="cuda")
        wq, eq = A.norm_rope64(q, None, 1e-6, pos, inv, 128, False)
        close(q_out, wq, eq + (wq.abs() + eq) * 2.0 ** -8)
    B.moe_sync(ctx, 60000)


def test_bad_tables_are_reported_and_index_nothing(B, make_ctx):
    """Page ids, offsets and lengths the device finds wrong: the call's other
    sequences are right, the bad ones' rows are left, moe_sync says DEVICE."""
    ctx = make_ctx(8, 2, 64, 16, False)
    for what in ("page", "len", "off", "short"):
        cache = A.Cache([50, 60, 70], 2, 64, 16, False, seed=9)
        batch = cache.batch(B, [1, 2, 1])
        _, _, table, off, kv_len = batch.tensors[:5]
        if what == "page":
            table[1, 3] = 10 ** 6
        elif what == "len":
            kv_len[1] = 10 ** 6
        elif what == "off":
            off[2] = -5
        else:
            kv_len[1] = 1  # fewer tokens than rows
        k0, v0 = cache.k.clone(), cache.v.clone()
        q, k, v = rnd((4, 8, 64), 1), rnd((4, 2, 64), 2), rnd((4, 2, 64), 3)
        q_out = torch.full_like(q, 5.0)
        B.moe_kv_append(ctx, batch, q, k, v, None, None, q_out)
        with pytest.raises(B.MoeError) as ei:
            B.moe_sync(ctx, 60000)
        assert ei.value.status == B.MOE_ERR_DEVICE
        B.moe_sync(ctx, 60000)  # reported once
        cache.k.copy_(k0)
        cache.v.copy_(v0)
        out = torch.full_like(q, 5.0)
        B.moe_attn_forward(ctx, batch, q, 2, 0.1, 0, 0, out)
        with pytest.raises(B.MoeError) as ei:
            B.moe_sync(ctx, 60000)
        assert ei.value.status == B.MOE_ERR_DEVICE
        good = [0] if what == "off" else [0, 3]
        cache.table[cache.table > 1000] = 0
        want, tol = A.attention64(q, cache, [1, 2, 1], 0.1, 0, 0)
        for r in good:
            close(out[r], want[r], tol[r])
        if what != "page":
            assert (out[1:3] == 5).all() and (q_out[1:3] == 5).all()


def test_descending_offsets_leave_no_parts_counted(B, make_ctx):
    """Offsets that descend make more row blocks than the call has rows for:
    reported, and later calls whose keys are split over the SMs are right."""
    ctx = make_ctx(16, 4, 128, 64, False)
    bad = A.Cache([4608, 64, 4608], 4, 128, 64, False, seed=21)
    batch = bad.batch(B, [2560, 0, 2560], extra_rows=-2560)
    batch.tensors[3].copy_(torch.tensor([0, 2560, 0, 2560], dtype=torch.int32))
    q = rnd((2560, 16, 128), 1)
    B.moe_attn_prefill(ctx, batch, q, 2560, 0.1, 0, 0, torch.empty_like(q))
    with pytest.raises(B.MoeError) as ei:
        B.moe_sync(ctx, 60000)
    assert ei.value.status == B.MOE_ERR_DEVICE
    cache = A.Cache([4000], 4, 128, 64, False, seed=22)
    q = rnd((50, 16, 128), 2)
    out = torch.empty_like(q)
    B.moe_attn_prefill(ctx, cache.batch(B, [50]), q, 50, 0.1, 0, 0, out)
    B.moe_sync(ctx, 60000)
    close(out, *A.attention64(q, cache, [50], 0.1, 0, 0, chunk=True))


def test_refusals(B, make_ctx):
    ctx = make_ctx(8, 2, 64, 16, False)
    cache = A.Cache([50], 2, 64, 16, False, seed=9)
    batch = cache.batch(B, [2])
    q, k, v = rnd((2, 8, 64), 1), rnd((2, 2, 64), 2), rnd((2, 2, 64), 3)
    out = torch.empty_like(q)

    def refused(fn, *args, status=1):
        with pytest.raises(B.MoeError) as ei:
            fn(*args)
        assert ei.value.status == status

    refused(B.moe_attn_configure, ctx, 8, 2, 64, 16, 1, status=4)
    for bad in ((0, 0.1, 0, 0), (33, 0.1, 0, 0), (2, 0.0, 0, 0), (2, float("nan"), 0, 0), (2, float("inf"), 0, 0),
                (2, 0.1, -1, 0), (2, 0.1, 0, -1)):
        refused(B.moe_attn_forward, ctx, batch, q, *bad, out)
    refused(B.moe_attn_prefill, ctx, batch, q, 0, 0.1, 0, 0, out)
    odd = torch.empty(2 * 8 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(2, 8, 64)
    refused(B.moe_attn_forward, ctx, batch, odd, 2, 0.1, 0, 0, out)
    refused(B.moe_kv_append, ctx, batch, odd, k, v, None, None, out)
    refused(B.moe_kv_append, ctx, batch, None, k, v, None, None, out)
    refused(B.moe_qk_norm_rope, ctx, 2, q, k, None, None, B.Rope(torch.ones(4, dtype=torch.float64, device="cuda"), 8),
            out, k)
    refused(B.moe_qk_norm_rope, ctx, 2, q, k, None, B.QkNorm(eps=-1.0), None, out, k)
    refused(B.moe_qk_norm_rope, ctx, -1, q, k, None, None, None, out, k)
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    for rot in (4, 12, 72):
        refused(B.moe_qk_norm_rope, ctx, 2, q, k, pos, None,
                B.Rope(torch.ones(rot // 2, dtype=torch.float64, device="cuda"), rot), out, k)
    new = B.moe_create(256, 128, 16, 2, B.MOE_Q4_SYM_G32_F16)
    try:
        refused(B.moe_attn_forward, new, batch, q, 2, 0.1, 0, 0, out, status=4)
        refused(B.moe_attn_configure, new, 8, 3, 64, 16, 1)
        refused(B.moe_attn_configure, new, 8, 2, 64, 24, 1)
        refused(B.moe_attn_configure, new, 8, 2, 64, 512, 1)
        refused(B.moe_attn_configure, new, 8, 2, 64, 16, 3)
        refused(B.moe_attn_configure, new, 8, 2, 96, 16, 1, status=8)
    finally:
        B.moe_destroy(new)
    for bad in (q.cpu(), q.float(), q[:1], q.transpose(0, 1), q[..., :32]):
        with pytest.raises(ValueError):
            B.moe_attn_forward(ctx, batch, bad, 2, 0.1, 0, 0, out)
    other = A.Cache([50], 1, 64, 16, False, seed=9).batch(B, [2])
    with pytest.raises(ValueError):
        B.moe_attn_forward(ctx, other, q, 2, 0.1, 0, 0, out)
    B.moe_sync(ctx, 60000)


# ------------------------------------------------------------------ chunks
CHUNKS = [
    # rows, kv, page, n_q, n_kv, dim, window, sinks
    ([128], [128], 64, 16, 2, 128, 0, 0),
    ([65], [65], 16, 4, 4, 128, 0, 0),              # one head per tile
    ([33, 0, 100, 1], [33, 9, 357, 40], 32, 16, 4, 128, 0, 0),
    ([257, 300], [257, 1111], 128, 12, 4, 64, 0, 0),  # three heads a group
    ([1000], [3000], 256, 24, 4, 128, 0, 0),
    ([777, 5], [777, 130], 16, 10, 2, 64, 0, 0),
    ([300], [2000], 64, 28, 4, 128, 200, 4),
    ([513, 90], [1500, 90], 16, 8, 1, 64, 64, 0),
    ([200], [900], 32, 32, 2, 128, 1, 1),
    ([150], [150], 64, 8, 8, 64, 100000, 3),
    ([400, 400], [5000, 640], 64, 20, 4, 128, 130, 200),
    ([40], [10], 16, 16, 16, 64, 0, 0),             # replaced below by kv = rows
    ([2100], [2100], 64, 16, 4, 128, 1024, 70),
    ([70] * 20, [70 + 31 * i for i in range(20)], 32, 8, 2, 128, 0, 0),
    ([300], [900], 16, 16, 16, 128, 0, 0),          # one head per tile
    ([2000], [2500], 128, 3, 1, 64, 90, 5),
    ([520, 0, 1], [520, 0, 700], 16, 8, 2, 64, 0, 0),
    ([50], [9000], 64, 8, 2, 128, 0, 0),            # few blocks: their keys split over the SMs
    ([65, 33], [5000, 3333], 32, 12, 2, 64, 3000, 100),
    ([90], [20000], 128, 4, 1, 128, 0, 0),
    ([40] * 50, [40 + i for i in range(50)], 16, 16, 2, 64, 30, 1),  # more than 32 sequences
]
CHUNKS = [(r, [max(a, b) for a, b in zip(r, k)], *rest) for r, k, *rest in CHUNKS]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("rows,kv,page,n_q,n_kv,dim,window,sinks", CHUNKS)
def test_prefill(B, make_ctx, e4m3, rows, kv, page, n_q, n_kv, dim, window, sinks):
    run_attention(B, make_ctx, B.moe_attn_prefill, e4m3, rows, kv, page, n_q, n_kv, dim, window, sinks)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("rows", [2, 300])
def test_scores_that_keep_growing(B, make_ctx, e4m3, rows):
    """Later keys score higher and higher, so the running maximum moves in
    every tile; and the reverse, where the first keys hold everything."""
    ctx = make_ctx(8, 2, 128, 64, e4m3)
    for sign in (1.0, -1.0):
        cache = A.Cache([1500], 2, 128, 64, e4m3, seed=3)
        for i, p in enumerate(cache.pages[0]):
            ramp = (torch.arange(64, device="cuda") + 64 * i).float()[:, None] * (0.02 if not e4m3 else 0.2) * sign
            cache.k[p] = (cache.k[p].float() * 0.25 + ramp).to(cache.k.dtype)
        q = rnd((rows, 8, 128), 4).abs()
        out = torch.empty_like(q)
        fn = B.moe_attn_forward if rows <= 32 else B.moe_attn_prefill
        fn(ctx, cache.batch(B, [rows]), q, rows, 1 / math.sqrt(128), 0, 0, out)
        cache.kv = [1500]
        want, tol = A.attention64(q, cache, [rows], 1 / math.sqrt(128), 0, 0, chunk=rows > 32)
        close(out, want, tol)
    B.moe_sync(ctx, 60000)


@pytest.mark.parametrize("rows,window", [(1, 0), (3, 40), (70, 0)])
def test_hundreds_of_sequences(B, make_ctx, rows, window):
    """More sequences than a block has threads: every thread holds several."""
    n = 700 if rows < 10 else 400
    counts = [(i * 7) % (rows + 1) for i in range(n)]
    kv = [max(c, 1 + (i * 37) % 90) for i, c in enumerate(counts)]
    run_attention(B, make_ctx, B.moe_attn_prefill if rows > 32 else B.moe_attn_forward, False, counts, kv, 16, 8, 2,
                  64, window, 2 if window else 0)


def test_e4m3_without_scales(B, make_ctx):
    for rows in (2, 90):
        ctx = make_ctx(8, 2, 64, 16, True)
        cache = A.Cache([200], 2, 64, 16, True, seed=3)
        cache.k_scale = cache.v_scale = None
        q = rnd((rows, 8, 64), 4)
        out = torch.empty_like(q)
        # values of the type's own range: a scale of 1/64 in the softmax's
        B.moe_attn_prefill(ctx, cache.batch(B, [rows]), q, rows, 0.125 / 64, 0, 0, out)
        want, tol = A.attention64(q, cache, [rows], 0.125 / 64, 0, 0, chunk=rows * 4 > 64)
        close(out, want, tol)


@pytest.mark.parametrize("rows", [2, 100])
@pytest.mark.parametrize("e4m3", [False, True])
def test_rows_off_their_lines(B, make_ctx, e4m3, rows):
    """Rows that begin 16 bytes into a line and end anywhere."""
    ctx = make_ctx(6, 2, 64, 32, e4m3)
    cache = A.Cache([rows + 70], 2, 64, 32, e4m3, seed=8)
    wide = rnd((rows, 6 * 64 + 24), 4, scale=2.0)
    q = wide[:, 8:8 + 6 * 64]
    out = torch.full((rows, 6 * 64 + 8), 2.0, dtype=torch.bfloat16, device="cuda")
    B.moe_attn_prefill(ctx, cache.batch(B, [rows]), q, rows, 0.125, 0, 0, out[:, 8:])
    want, tol = A.attention64(q.reshape(rows, 6, 64), cache, [rows], 0.125, 0, 0, chunk=rows * 3 > 64)
    close(out[:, 8:].reshape(rows, 6, 64), want, tol)
    assert (out[:, :8] == 2).all()


def test_split_chunk_replays(B, make_ctx):
    """A captured chunk whose keys are split over the SMs, replayed with other
    lengths (other splits), on a stream of its own."""
    ctx = make_ctx(8, 2, 128, 64, False)
    cache = A.Cache([6000], 2, 128, 64, False, seed=8)
    batch = cache.batch(B, [100])
    q = rnd((100, 8, 128), 4, scale=2.0)
    out = torch.empty_like(q)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        B.moe_attn_prefill(ctx, batch, q, 100, 0.09, 0, 0, out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.moe_attn_prefill(ctx, batch, q, 100, 0.09, 0, 0, out)
    for length in (6000, 100, 3001, 6000):
        batch.tensors[4].fill_(length)
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        cache.kv = [length]
        want, tol = A.attention64(q, cache, [100], 0.09, 0, 0)
        close(out, want, tol)
    B.moe_sync(ctx, 60000)


def test_two_contexts_on_two_streams(B, make_ctx):
    """Calls of two contexts may overlap: each has its own scratch."""
    work = []
    for i, (n_kv, kv) in enumerate(((2, 5000), (4, 4000))):
        ctx = make_ctx(8, n_kv, 128, 64, False)
        cache = A.Cache([kv], n_kv, 128, 64, False, seed=i)
        for rows in (2, 60):
            q = rnd((rows, 8, 128), i + rows, scale=2.0)
            work.append((ctx, cache, rows, q, torch.empty_like(q), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for j in (0, 2, 1, 3):
            ctx, cache, rows, q, out, _ = work[j]
            s = work[j // 2 * 2][5]  # a stream per context
            with torch.cuda.stream(s):
                B.moe_attn_prefill(ctx, cache.batch(B, [rows]), q, rows, 0.09, 0, 0, out)
    torch.cuda.synchronize()
    for ctx, cache, rows, q, out, _ in work:
        want, tol = A.attention64(q, cache, [rows], 0.09, 0, 0)
        close(out, want, tol)


def test_empty_calls(B, make_ctx):
    ctx = make_ctx(8, 2, 64, 16, False)
    cache = A.Cache([50, 0], 2, 64, 16, False, seed=9)
    q, k = rnd((3, 8, 64), 1), rnd((3, 2, 64), 2)
    out = torch.full_like(q, 5.0)
    before = cache.k.clone().view(torch.int16)
    for batch in (cache.batch(B, [0, 0]), cache.batch(B, [0, 0], 3)):
        B.moe_kv_append(ctx, batch, q, k, k, None, None, out)
        B.moe_attn_forward(ctx, batch, q, 1, 0.1, 0, 0, out)
        B.moe_attn_prefill(ctx, batch, q, 100, 0.1, 5, 1, out)
    B.moe_sync(ctx, 60000)
    assert (out == 5).all() and torch.equal(cache.k.view(torch.int16), before)
