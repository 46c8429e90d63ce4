"""What is built, when it is built again, and what is loaded: no compiler runs here."""
import os

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
