"""What is built, when it is built again, and what is loaded: no compiler runs here."""
import os
import subprocess
import sys

import pytest

mla = pytest.importorskip("mla_latent_kv_gb300")
from mla_latent_kv_gb300 import build  # noqa: E402


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """A build folder of its own with a library and a binding that are newer than every source."""
    for name, attr in (("libmla_latent_kv.so", "LIB"), ("_mla_torch.so", "BINDING")):
        (tmp_path / name).write_bytes(b"built")
        monkeypatch.setattr(build, attr, str(tmp_path / name))
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(mla, "BINDING_PATH", str(tmp_path / "_mla_torch.so"))
    monkeypatch.setattr(mla, "_torch_binding", None)
    return tmp_path


@pytest.mark.parametrize("stamp", [None, "", "torch 1.13.0, cpython-310-x86_64-linux-gnu"])
def test_a_binding_of_another_torch_is_built_again_and_not_loaded(elsewhere, stamp):
    """The binding reads torch's objects by the layouts of the headers it was compiled with."""
    pytest.importorskip("torch")
    mark = elsewhere / "_mla_torch.so.built_for"
    if stamp is not None:
        mark.write_text(stamp)
    assert not build.up_to_date()
    with pytest.raises(RuntimeError, match="built for"):
        mla._native()
    mark.write_text(build.built_for())
    assert build.up_to_date()
    os.utime(elsewhere / "_mla_torch.so", (0, 0))  # older than its source
    assert not build.up_to_date()


@pytest.fixture
def compilers(elsewhere, monkeypatch):
    """The commands that a build would run, which make empty files instead; those of the binding fail on demand."""
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        binding = any("binding.cpp" in x for x in cmd)
        if not (binding and run.broken):
            open(cmd[cmd.index("-o") + 1], "wb").close()
        return subprocess.CompletedProcess(cmd, int(binding and run.broken), "", "no headers" if binding else "")
    run.broken, run.ran = False, ran
    monkeypatch.setattr(build.subprocess, "run", run)
    for f in elsewhere.iterdir():
        f.unlink()
    return run


def test_the_library_is_built_without_torch(elsewhere, compilers, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)  # importing it raises
    assert not build.up_to_date()
    assert build.build() == str(elsewhere / "libmla_latent_kv.so")
    assert (elsewhere / "libmla_latent_kv.so").exists() and not (elsewhere / "_mla_torch.so").exists()
    assert len(compilers.ran) == len(build.sources()) + 1 and not any("binding" in " ".join(c) for c in compilers.ran)
    assert build.up_to_date()
    build.build()
    assert len(compilers.ran) == len(build.sources()) + 1  # nothing to do


def test_a_binding_that_does_not_compile_leaves_the_library(elsewhere, compilers):
    pytest.importorskip("torch")
    compilers.broken = True
    with pytest.raises(RuntimeError, match="compiler failed"):
        build.build()
    assert (elsewhere / "libmla_latent_kv.so").exists() and not (elsewhere / "_mla_torch.so").exists()
    assert not build.up_to_date()
    compilers.broken = False
    build.build()
    assert (elsewhere / "_mla_torch.so").exists() and build.up_to_date()
    assert build.binding_built_for() == build.built_for()
