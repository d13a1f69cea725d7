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
