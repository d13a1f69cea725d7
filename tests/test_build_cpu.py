"""What build() makes where parts of its toolchain are missing, and when it
makes the marshalling again."""
import os

import pytest

from sparse_moe_expert_gemv_b200 import build


@pytest.fixture
def made(monkeypatch, tmp_path):
    """build()'s compilations, recorded instead of run, in a folder of their own."""
    made = []

    def compile(cmd):
        made.append(os.path.basename(cmd[0]))
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(build, "SO", str(tmp_path / "libmoe.so"))
    monkeypatch.setattr(build, "MARSHAL_SO", str(tmp_path / "_marshal.so"))
    monkeypatch.setattr(build.subprocess, "check_call", compile)
    return made


def test_both_once(made):
    assert build.build() == build.SO
    assert made == [os.path.basename(build.NVCC), "g++"]
    build.build()
    assert len(made) == 2


@pytest.mark.parametrize("missing", ["torch", "headers", "g++"])
def test_the_library_needs_nvcc_alone(made, monkeypatch, capfd, missing):
    if missing == "torch":
        monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: None)
    elif missing == "headers":
        monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": "/nowhere"})
    else:
        monkeypatch.setattr(build.shutil, "which", lambda name: None)
    assert build.build() == build.SO
    assert made == [os.path.basename(build.NVCC)]
    assert "_marshal.so is not built" in capfd.readouterr().err


def test_another_torch_makes_the_marshalling_again(made, monkeypatch):
    build.build()
    monkeypatch.setattr(build.importlib.metadata, "version", lambda name: "1.0")
    build.build()
    assert made[2:] == ["g++"]
    build.build()
    assert len(made) == 3
