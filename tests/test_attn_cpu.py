"""Attention calls without a GPU: the kernels' index arithmetic, compiled for
the host, and the refusals that need no device."""
import os
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def B():
    from sparse_moe_expert_gemv_b200 import build
    build.build()
    from sparse_moe_expert_gemv_b200 import binding
    return binding


def test_index_arithmetic_on_the_host(tmp_path):
    from sparse_moe_expert_gemv_b200 import build
    exe = str(tmp_path / "attn_host")
    subprocess.check_call([build.NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-std=c++17", "-O1",
                           "--expt-relaxed-constexpr", "-I", build.CSRC, "-o", exe,
                           os.path.join(ROOT, "tests", "attn_host.cu")])
    out = subprocess.run([exe], capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.stdout


def test_calls_without_a_context_are_refused(B):
    L = B.lib()
    assert L.moe_attn_configure(None, 8, 2, 64, 16, 1) == B.MOE_ERR_INVALID_ARG
    assert L.moe_qk_norm_rope(None, 1, None, 0, None, 0, None, None, None, None, 0, None, 0, None) == 1
    assert L.moe_kv_append(None, None, None, 0, None, 0, None, 0, None, None, None, 0, None) == 1
    assert L.moe_attn_forward(None, None, None, 0, 1, 1.0, 0, 0, None, 0, None) == 1
    assert L.moe_attn_prefill(None, None, None, 0, 1, 1.0, 0, 0, None, 0, None) == 1


def test_binding_refuses_what_the_library_cannot_see(B):
    """Host tensors, other types, shapes and strides never become addresses."""
    bf = torch.bfloat16
    cache = torch.zeros((4, 2, 16, 64), dtype=bf)
    table, off, kv = (torch.zeros(s, dtype=torch.int32) for s in ((1, 4), (2,), (1,)))
    for args in ((cache, cache, table, off, kv), (cache[0], cache[0], table, off, kv),
                 (cache, cache, table[0], off, kv)):
        with pytest.raises(ValueError):
            B.KvBatch(*args, 1)
    with pytest.raises(ValueError):
        B.Rope(torch.ones(32, dtype=torch.float64), 64)
    with pytest.raises(ValueError):
        B.QkNorm(torch.ones(64))
    m, batch = B._marshal(), 64  # no call gets as far as its batch
    good = torch.zeros((2, 8, 64), dtype=bf)  # but for where it lives
    for bad in (good, torch.zeros((2, 8, 64)), torch.zeros((2, 7, 64), dtype=bf), good.flatten(), 7, None,
                torch.zeros((2, 8, 128), dtype=bf)[..., ::2]):
        with pytest.raises(ValueError):
            m.attend(0, 8, 64, 0, 0, 2, batch, bad, 2, 0.1, 0, 0, good, 0)
        with pytest.raises(ValueError):
            m.kv_append(8, 8, 64, 0, 0, 2, batch, None, bad, good, None, None, None, 0)
        with pytest.raises(ValueError):
            m.qk_norm_rope(8, 8, 64, 0, 0, 2, bad, good, None, None, None, good, good, 0)
    with pytest.raises(OverflowError):
        m.attend(0, 8, 64, 0, 0, 2, batch, good, 2, 0.1, 1 << 31, 0, good, 0)
    with pytest.raises(TypeError):
        m.attend(0, 8, 64)
    with pytest.raises(B.MoeError) as ei:
        B.moe_qk_norm_rope(12345, 1, None, None, None, None, None, None, None)
    assert ei.value.status == B.MOE_ERR_STATE
