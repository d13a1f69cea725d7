"""Attention at the far ends: long flat tails, positions and cache offsets past
32 bits, scores without a finite value."""
import math

import pytest
import torch

from tests import _attn as A

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from sparse_moe_expert_gemv_b200 import binding
    return binding


@pytest.fixture
def make_ctx(B):
    made = []

    def get(n_q, n_kv, dim, page, e4m3):
        made.append(B.moe_create(256, 128, 16, 2, B.MOE_Q4_SYM_G32_F16))
        B.moe_attn_configure(made[-1], n_q, n_kv, dim, page, B.MOE_KV_E4M3 if e4m3 else B.MOE_KV_BF16)
        return made[-1]

    yield get
    for ctx in made:
        B.moe_destroy(ctx)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("e4m3", [False, True])
def test_a_long_flat_tail_behind_one_large_score(B, make_ctx, e4m3):
    """2^20 - 1 keys 25.2 octaves below the first one hold 2.6 % of the softmax
    together, each too small for fp16 beside a first term of 1.  Many
    sequences, so that a block walks a whole one; all of them share two pages."""
    page, n_seqs, kv, dim, group = 256, 300, 1 << 20, 64, 64
    below = 25.2
    ctx = make_ctx(group, 1, dim, page, e4m3)
    kind = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    k, v = (torch.zeros((2, 1, page, dim), device="cuda") for _ in range(2))
    k[0, 0, 0, 0] = 1.0
    v[..., :32] = 1.0           # what the tail holds
    v[0, 0, 0] = 0.0
    v[0, 0, 0, 32:] = 1.0       # what the first key holds
    table = torch.ones((n_seqs, kv // page), dtype=torch.int32, device="cuda")
    table[:, 0] = 0
    batch = B.KvBatch(k.to(kind), v.to(kind), table, ints(list(range(n_seqs + 1))), ints([kv] * n_seqs), n_seqs)
    q = torch.zeros((n_seqs, group, dim), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    out = torch.full_like(q, float("nan"))
    B.moe_attn_forward(ctx, batch, q, 1, below * math.log(2), 0, 0, out)
    B.moe_sync(ctx, 60000)
    tail = (kv - 1) * 2.0 ** -below
    for got, want in ((out[..., :32], tail / (1 + tail)), (out[..., 32:], 1 / (1 + tail))):
        # A term is rounded to 16 bits: bf16 by up to 2^-8 of it; fp16 by half
        # a step of its subnormals, 2^-25, where the largest term is 2^7.
        # The sums are fp32: o grows in 2^16 steps of 16 keys, each rounded or
        # cut by up to 2^-23 of the sum, 2^-7 in all; a tile's terms of a lane
        # (16 of them, 2^-21.2) are rounded by up to 2^-24 as they join a sum
        # of 1, in one lane of four: 4 % of the tail, 2^-9 of the whole.  One
        # rounding to bf16.
        terms = (kv - 1) * 2.0 ** -32 if e4m3 else tail * 2.0 ** -8
        tol = terms + want * (2.0 ** -7 + 2.0 ** -9 + 2.0 ** -8)
        assert (got.double() - want).abs().max() <= tol, (
            float(got.double().min()), float(got.double().max()), want, tol)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("rows", [3, 70])
def test_the_last_positions_below_2_31(B, make_ctx, e4m3, rows):
    """A sequence of almost 2^31 tokens with a sliding window and sinks: only
    its first and last pages are there, and what lies behind its end is NaN."""
    n_q, n_kv, dim, page, window, sinks, near = 4, 2, 128, 64, 100, 5, 6
    kv, most = 2 ** 31 - 100, 2 ** 25 - 1
    ctx = make_ctx(n_q, n_kv, dim, page, e4m3)
    # the same rows see the same keys in a short sequence without the pages between
    n_pages = -(-kv // page)
    short = A.Cache([kv - (n_pages - near - 1) * page], n_kv, dim, page, e4m3, seed=4)
    table = torch.full((1, most), -1, dtype=torch.int32, device="cuda")
    table[0, 0] = short.pages[0][0]
    table[0, n_pages - near:n_pages] = ints(short.pages[0][1:])
    batch = B.KvBatch(short.k, short.v, table, ints([0, rows]), ints([kv]), rows, k_scale=short.k_scale,
                      v_scale=short.v_scale)
    qkv = torch.randn((rows, n_q + 2 * n_kv, dim), device="cuda",
                      generator=torch.Generator(device="cuda").manual_seed(5)).bfloat16()
    q, k, v = qkv[:, :n_q], qkv[:, n_q:n_q + n_kv], qkv[:, n_q + n_kv:]
    out = torch.full((rows, n_q, dim), float("nan"), dtype=torch.bfloat16, device="cuda")
    B.moe_kv_append(ctx, batch, None, k, v, None, None, None)
    B.moe_attn_prefill(ctx, batch, q, rows, 0.09, window, sinks, out)
    B.moe_sync(ctx, 60000)
    for which, x, scale in (("k", k, short.k_scale), ("v", v, short.v_scale)):
        stored = short.rows64(0, which)[-rows:]
        if e4m3:  # one rounding, and one of x / scale before it
            tol = x.double().abs() * 2.0 ** -4 * (1 + 2.0 ** -19) + 2.0 ** -10 * scale.double()[:, None]
            assert ((stored - x.double()).abs() <= tol).all()
        else:
            assert torch.equal(stored, x.double())
    want, tol = A.attention64(q.contiguous(), short, [rows], 0.09, window, sinks,
                              chunk=rows * (n_q // n_kv) > 64)
    assert ((out.double() - want).abs() <= tol).all(), float((out.double() - want).abs().max())


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("rows,kv", [(1, 40), (1, 9000), (40, 40), (40, 9000)])
def test_scores_without_a_finite_value(B, make_ctx, e4m3, rows, kv):
    """A row whose visible scores are all -inf has no softmax: NaN, as the
    formula gives, not zeros; other rows are what they were."""
    n_q, n_kv, dim = 8, 2, 64
    ctx = make_ctx(n_q, n_kv, dim, 16, e4m3)
    cache = A.Cache([kv, 90], n_kv, dim, 16, e4m3, seed=6)
    A.as_bytes(cache.k)[cache.pages[0], ..., 0] = A.as_bytes(torch.tensor(-1.0, device="cuda").to(cache.k.dtype))
    q = torch.randn((rows + 1, n_q, dim), device="cuda",
                    generator=torch.Generator(device="cuda").manual_seed(5)).bfloat16()
    poisoned = q.clone()
    poisoned[rows - 1, 3, 0] = math.inf
    out = torch.zeros_like(q)
    B.moe_attn_prefill(ctx, cache.batch(B, [rows, 1]), poisoned, rows, 0.1, 0, 0, out)
    B.moe_sync(ctx, 60000)
    assert out[rows - 1, 3].isnan().all()
    want, tol = A.attention64(q, cache, [rows, 1], 0.1, 0, 0, chunk=rows * (n_q // n_kv) > 64)
    rest = torch.ones((rows + 1, n_q), dtype=torch.bool, device="cuda")
    rest[rows - 1, 3] = False
    assert ((out.double() - want).abs() <= tol)[rest].all()


@pytest.mark.parametrize("e4m3", [False, True])
def test_a_cache_past_2_31_elements(B, make_ctx, e4m3):
    """Pages whose elements lie past 2^31 (bf16) and 2^32 bytes into the cache:
    append, window and chunk attention."""
    n_q, n_kv, dim, page = 4, 2, 128, 64
    n_pages = (2 ** 32 if e4m3 else 2 ** 31) // (n_kv * page * dim) + 4000
    ctx = make_ctx(n_q, n_kv, dim, page, e4m3)
    rows = [3, 0, 70]
    small = A.Cache([200, 30, 333], n_kv, dim, page, e4m3, seed=8)
    k, v = (torch.empty((n_pages, *t.shape[1:]), dtype=t.dtype, device="cuda") for t in (small.k, small.v))
    at = n_pages - 1 - 100 * torch.arange(small.k.shape[0], device="cuda")  # where the small cache's pages lie
    assert int(at.min()) * n_kv * page * dim * k.element_size() > 2 ** 32
    A.as_bytes(k)[at], A.as_bytes(v)[at] = A.as_bytes(small.k), A.as_bytes(small.v)
    table = torch.where(small.table >= 0, at[small.table.clamp(min=0).long()].int(), -1)
    n = sum(rows)
    batch = B.KvBatch(k, v, table, ints([0, 3, 3, n]), ints(small.kv), n, k_scale=small.k_scale,
                      v_scale=small.v_scale)
    qkv = torch.randn((n, n_q + 2 * n_kv, dim), device="cuda",
                      generator=torch.Generator(device="cuda").manual_seed(5)).bfloat16()
    q, new_k, new_v = qkv[:, :n_q], qkv[:, n_q:n_q + n_kv], qkv[:, n_q + n_kv:]
    B.moe_kv_append(ctx, batch, None, new_k, new_v, None, None, None)
    same = small.batch(B, rows)  # the same append among few pages
    B.moe_kv_append(ctx, same, None, new_k, new_v, None, None, None)
    B.moe_sync(ctx, 60000)
    for big, few in ((k, small.k), (v, small.v)):
        assert torch.equal(A.as_bytes(big)[at].view(torch.uint8), A.as_bytes(few).view(torch.uint8))
    for max_T in (3, 70):  # the window and the chunk kernel
        out = torch.full((n, n_q, dim), float("nan"), dtype=torch.bfloat16, device="cuda")
        B.moe_attn_prefill(ctx, batch, q, max_T, 0.09, 0, 0, out)
        B.moe_sync(ctx, 60000)
        want, tol = A.attention64(q.contiguous(), small, rows, 0.09, 0, 0, chunk=max_T * (n_q // n_kv) > 64)
        assert ((out.double() - want).abs() <= tol).all(), float((out.double() - want).abs().max())


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("rows", [[2, 0, 3], [0, 40, 2]])
def test_rows_before_the_first_sequence(B, make_ctx, e4m3, rows):
    """Two batches may share one buffer of rows: offsets need not begin at 0.
    Rows of no sequence, in front and behind, are left and are no error."""
    n_q, n_kv, dim, page = 8, 2, 64, 16
    ctx = make_ctx(n_q, n_kv, dim, page, e4m3)
    cache = A.Cache([30, 7, 50] if rows[1] == 0 else [30, 70, 50], n_kv, dim, page, e4m3, seed=8)
    front, behind, n = 5, 2, sum(rows)
    batch = cache.batch(B, rows, front + behind)
    batch.tensors[3].add_(front)
    qkv = torch.randn((front + n + behind, n_q + 2 * n_kv, dim), device="cuda",
                      generator=torch.Generator(device="cuda").manual_seed(5)).bfloat16()
    q, k, v = qkv[:, :n_q], qkv[:, n_q:n_q + n_kv], qkv[:, n_q + n_kv:]
    q_out, out = (torch.full((front + n + behind, n_q, dim), 7.0, dtype=torch.bfloat16, device="cuda")
                  for _ in range(2))
    B.moe_kv_append(ctx, batch, q, k, v, None, None, q_out)
    B.moe_attn_prefill(ctx, batch, q_out, max(rows), 0.1, 0, 0, out)
    B.moe_sync(ctx, 60000)
    assert torch.equal(q_out[front:front + n], q[front:front + n])
    for t in (q_out, out):
        assert (t[:front] == 7).all() and (t[front + n:] == 7).all()
    want, tol = A.attention64(q[front:front + n].contiguous(), cache, rows, 0.1, 0, 0,
                              chunk=max(rows) * (n_q // n_kv) > 64)
    assert ((out[front:front + n].double() - want).abs() <= tol).all()
    at = front
    for b, r in enumerate(rows):  # the appended keys are where the sequence has them
        stored = cache.rows64(b, "k")[len(cache.rows64(b, "k")) - r:]
        x = k[at:at + r].double()
        if e4m3:
            s = cache.k_scale.double()[:, None]
            assert ((stored - x).abs() <= x.abs() * 2.0 ** -4 * (1 + 2.0 ** -19) + 2.0 ** -10 * s).all()
        else:
            assert torch.equal(stored, x)
        at += r
