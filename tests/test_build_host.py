"""When the binding module on torch's tensors is compiled again (no compiler is run)."""

import os

import pytest

from mixture_experts_ffn_14_b200 import build as B


@pytest.fixture
def compiled(tmp_path, monkeypatch):
    """Commands that the build runs; each leaves the module it names."""
    monkeypatch.setattr(B, "TORCH_CALLS", str(tmp_path / "_torch_calls.so"))
    monkeypatch.setattr(B, "TORCH_CALLS_TAG", str(tmp_path / "build" / "torch_calls.tag"))
    commands = []

    def run(cmd, check):
        assert check
        commands.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(B.subprocess, "run", run)
    return commands


def test_the_module_is_compiled_once_for_a_torch_and_a_python(compiled, monkeypatch):
    for _ in range(3):
        assert B.build_torch_calls() == B.TORCH_CALLS
    assert len(compiled) == 1
    monkeypatch.setattr(B.importlib.metadata, "version", lambda name: {"torch": "99.1+cu1"}[name])
    for _ in range(3):
        B.build_torch_calls()
    assert len(compiled) == 2
    monkeypatch.setattr(B.sysconfig, "get_config_var", lambda name: {"SOABI": "cpython-399-x86_64-linux-gnu"}[name])
    for _ in range(3):
        B.build_torch_calls()
    assert len(compiled) == 3


def test_the_module_is_compiled_again_without_its_record_or_after_its_sources(compiled):
    B.build_torch_calls()
    os.remove(B.TORCH_CALLS_TAG)                     # a module of unknown origin
    B.build_torch_calls()
    assert len(compiled) == 2
    os.utime(B.TORCH_CALLS, (0, 0))                  # older than its sources
    B.build_torch_calls()
    assert len(compiled) == 3
    B.build_torch_calls(force=True)
    assert len(compiled) == 4
    os.remove(B.TORCH_CALLS)
    B.build_torch_calls()
    assert len(compiled) == 5


def test_a_failed_compilation_leaves_no_record(compiled, monkeypatch):
    def fail(cmd, check):
        raise B.subprocess.CalledProcessError(1, cmd)

    monkeypatch.setattr(B.subprocess, "run", fail)
    with pytest.raises(B.subprocess.CalledProcessError):
        B.build_torch_calls()
    assert not os.path.exists(B.TORCH_CALLS_TAG)
