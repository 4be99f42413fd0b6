"""The build's parts, with a stand-in for the compilers: the library needs neither torch nor Python's headers."""
import importlib.machinery
import os
import subprocess
import sys

import pytest

from speculative_decoding_draft_lm_gb300 import build


@pytest.fixture
def commands(monkeypatch, tmp_path):
    """Runs of compilers, which write what -o names and fail where the test says so."""
    ran, fail = [], set()

    def run(cmd, **kw):
        ran.append(cmd)
        bad = any(f in " ".join(cmd) for f in fail)
        if not bad:
            open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, int(bad), "", "no" if bad else "")

    monkeypatch.setattr(subprocess, "run", run)
    monkeypatch.setattr(build, "PKG", str(tmp_path))
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "objects"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / os.path.basename(build.LIB)))
    monkeypatch.setattr(build, "ARGS", str(tmp_path / os.path.basename(build.ARGS)))
    return ran, fail


def test_library_and_module(commands):
    pytest.importorskip("torch")
    ran, _ = commands
    assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and os.path.exists(build.ARGS)
    assert len(ran) == len(build.sources()) + 2


def test_the_library_is_built_without_torch(commands, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)
    assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and not os.path.exists(build.ARGS)
    assert "torch" in capsys.readouterr().out


def test_the_library_is_built_where_the_module_is_not(commands):
    pytest.importorskip("torch")
    commands[1].add("optim_args.cpp")
    with pytest.raises(RuntimeError, match="optim_args.cpp"):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.ARGS)


def test_a_library_that_is_not_built_is_an_error(commands):
    commands[1].add("optim_api.cu")
    with pytest.raises(RuntimeError, match="optim_api.cu"):
        build.build()
    assert not os.path.exists(build.LIB)


def test_the_module_is_this_pythons_and_this_torchs(monkeypatch):
    torch = pytest.importorskip("torch")
    from speculative_decoding_draft_lm_gb300 import optim
    if not os.path.exists(build.ARGS):
        build.build()
    assert os.path.basename(build.ARGS) == "_optim_args" + importlib.machinery.EXTENSION_SUFFIXES[0]
    args = optim._load_args()
    assert os.path.realpath(args.__file__) == os.path.realpath(build.ARGS) and args.torch_version == torch.__version__
    monkeypatch.setattr(args, "torch_version", "0.0")
    with pytest.raises(ImportError, match="0.0"):
        optim._load_args()
    monkeypatch.setitem(sys.modules, "speculative_decoding_draft_lm_gb300._optim_args", None)
    monkeypatch.delattr("speculative_decoding_draft_lm_gb300._optim_args")
    with pytest.raises(ImportError, match="speculative_decoding_draft_lm_gb300.build"):
        optim._load_args()
