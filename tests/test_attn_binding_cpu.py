"""The attention calls' tensor checks without a GPU: tensors that say they are
on cuda:0 but hold no memory.  What the checks let through reaches the library
with a null context, which it refuses (INVALID_ARG)."""
import os
import subprocess
import sys

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
N, N_Q, N_KV, DIM = 2, 8, 4, 64
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def m():
    from sparse_moe_expert_gemv_b200 import build
    build.build()
    from sparse_moe_expert_gemv_b200 import binding
    return binding._marshal()


def fake(shape, dtype=BF16, device="cuda:0"):
    with FakeTensorMode():
        return torch.empty(shape, dtype=dtype, device=device)


def view_of(shape, take):
    with FakeTensorMode():
        return take(torch.empty(shape, dtype=BF16, device="cuda:0"))


# every call with its row arguments by name: (heads, call)
def attend(chunk):
    return {"q": N_Q, "out": N_Q}, lambda m, t: m.attend(chunk, N_Q, DIM, 0, 0, N, 64, t["q"], N, 0.1, 0, 0,
                                                         t["out"], 0)


CALLS = {
    "forward": attend(0),
    "prefill": attend(1),
    "append": ({"q": N_Q, "k": N_KV, "v": N_KV, "q_out": N_Q},
               lambda m, t: m.kv_append(N_Q, N_KV, DIM, 0, 0, N, 64, t["q"], t["k"], t["v"], None, None, t["q_out"],
                                        0)),
    "norm_rope": ({"q": N_Q, "k": N_KV, "q_out": N_Q, "k_out": N_KV},
                  lambda m, t: m.qk_norm_rope(N_Q, N_KV, DIM, 0, 0, N, t["q"], t["k"], None, None, None, t["q_out"],
                                              t["k_out"], 0)),
}


def bad_rows(heads):
    yield "float16", fake((N, heads, DIM), torch.float16)
    yield "int16", fake((N, heads, DIM), torch.int16)
    yield "uint16", fake((N, heads, DIM), torch.uint16)
    yield "float32", fake((N, heads, DIM), torch.float32)
    yield "e4m3", fake((N, heads, DIM), torch.float8_e4m3fn)
    yield "another device", fake((N, heads, DIM), device="cuda:1")
    yield "heads", fake((N, heads + 1, DIM))
    yield "width", fake((N, heads * DIM - 1))
    yield "head size", fake((N, heads, 2 * DIM))
    yield "1-D", fake((N * heads * DIM,))
    yield "4-D", fake((1, N, heads, DIM))
    yield "too few rows", fake((N - 1, heads, DIM))
    yield "strided within a head", view_of((N, heads, 2 * DIM), lambda t: t[..., ::2])
    yield "heads apart", view_of((N, 2 * heads, DIM), lambda t: t[:, ::2])
    yield "heads first", view_of((heads, N, DIM), lambda t: t.transpose(0, 1))


@pytest.mark.parametrize("call", CALLS)
def test_rows_are_checked_argument_by_argument(m, call):
    heads, run = CALLS[call]
    good = {name: fake((N, h, DIM)) for name, h in heads.items()}
    assert run(m, good) == 1  # the library's own refusal: no context
    assert run(m, {name: fake((N, h * DIM)) for name, h in heads.items()}) == 1
    assert run(m, {name: view_of((N, h + 3, DIM), lambda t: t[:, 1:-2]) for name, h in heads.items()}) == 1
    for name, h in heads.items():
        for what, bad in bad_rows(h):
            try:
                rc = run(m, {**good, name: bad})
            except ValueError as e:
                assert str(e).startswith(name + ":"), (what, e)
            else:
                raise AssertionError(f"{call}: {name} ({what}) was accepted: {rc}")


UNKNOWN_SIZE = """
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
from torch.fx.experimental.symbolic_shapes import ShapeEnv
from tests.test_attn_binding_cpu import CALLS, fake, N, DIM
from sparse_moe_expert_gemv_b200 import binding
m = binding._marshal()
mode = FakeTensorMode(shape_env=ShapeEnv())
for heads, run in CALLS.values():
    good = {name: fake((N, h, DIM)) for name, h in heads.items()}
    for name, h in heads.items():
        with mode:
            bad = torch.empty((mode.shape_env.create_unbacked_symint(), h, DIM), dtype=torch.bfloat16,
                              device="cuda:0")
        try:
            run(m, {**good, name: bad})
        except ValueError as e:
            assert "plain CUDA tensor" in str(e), e
        else:
            raise AssertionError(name)
print("refused")
"""


def test_a_tensor_that_throws_is_a_python_error(m):
    """Sizes that are no numbers: in a process of its own, which an exception
    through the interpreter's C frames would end."""
    r = subprocess.run([sys.executable, "-c", UNKNOWN_SIZE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("refused"), (r.returncode, r.stderr[-2000:])
