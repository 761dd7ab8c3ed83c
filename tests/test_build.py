"""CPU tests of the build's order and paths, with the compiler calls replaced."""
import os

import pytest

from dispatch_expert_gemm_amd import build as b


@pytest.fixture
def calls(monkeypatch, tmp_path):
    """Commands that "build" into an empty folder; those that `fails` holds for fail."""
    ran = []

    def run(cmd):
        ran.append(cmd)
        if run.fails(cmd):
            return 1, "no"
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")
        return 0, ""

    run.fails = lambda cmd: False
    monkeypatch.setattr(b, "_run", run)
    monkeypatch.setattr(b, "LIBDIR", str(tmp_path))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libmoe.so"))
    monkeypatch.setattr(b, "TORCH_NODES", str(tmp_path / "moe_torch.so"))
    run.ran = ran
    return run


def test_both_libraries_are_built(calls, tmp_path):
    assert b.build() == str(tmp_path / "libmoe.so")
    assert os.path.exists(tmp_path / "libmoe.so") and os.path.exists(tmp_path / "moe_torch.so")
    assert len(calls.ran) == len(b.sources()) + 3


@pytest.mark.parametrize("how", ["compiler fails", "no compiler", "no headers", "link fails"])
def test_the_kernels_library_is_linked_where_the_nodes_cannot_be_built(calls, tmp_path, monkeypatch, how):
    if how == "compiler fails":
        calls.fails = lambda cmd: any(a.endswith("torch_nodes.cpp") for a in cmd)
    elif how == "link fails":
        calls.fails = lambda cmd: "-ltorch" in cmd
    else:
        def missing(*a):
            raise FileNotFoundError("g++") if how == "no compiler" else ImportError("torch")
        monkeypatch.setattr(b, "nodes_command", missing)
    (tmp_path / "moe_torch.so").write_text("an older one")
    with pytest.raises((RuntimeError, OSError, ImportError)):
        b.build()
    assert os.path.exists(tmp_path / "libmoe.so") and not os.path.exists(tmp_path / "moe_torch.so")


def test_a_kernel_that_does_not_compile_stops_the_build(calls, tmp_path):
    calls.fails = lambda cmd: any(a.endswith("gemm.hip") for a in cmd)
    with pytest.raises(RuntimeError, match="gemm.hip"):
        b.build()
    assert not os.path.exists(tmp_path / "libmoe.so") and not os.path.exists(tmp_path / "moe_torch.so")


def test_the_nodes_take_the_headers_of_the_chosen_hipcc(monkeypatch, tmp_path):
    (tmp_path / "bin").mkdir()
    (tmp_path / "include" / "hip").mkdir(parents=True)
    (tmp_path / "include" / "hip" / "hip_runtime.h").write_text("")
    (tmp_path / "bin" / "hipcc").write_text("")
    monkeypatch.setenv("HIPCC", str(tmp_path / "bin" / "hipcc"))
    assert str(tmp_path / "include") in b.nodes_command() and "/opt/rocm/include" not in b.nodes_command()
    monkeypatch.delenv("HIPCC")
    assert str(tmp_path / "include") not in b.nodes_command()
