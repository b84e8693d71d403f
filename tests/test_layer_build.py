"""When the torch binding of the operators around the attention is built again, and when it is left out."""
import os

import pytest

from chunkwise_causal_linear_gb300 import build as la_build


@pytest.fixture(scope="module", autouse=True)
def _built():
    pytest.importorskip("torch")
    la_build.build()


def fake_torch(path, version="9.9.9", cuda=True):
    os.makedirs(path / "lib")
    (path / "version.py").write_text(f"__version__ = '{version}'\n")
    if cuda:
        (path / "lib" / "libc10_cuda.so").write_text("")
    return str(path)


def test_another_torch_makes_the_binding_stale(tmp_path, monkeypatch):
    assert la_build.up_to_date()
    monkeypatch.setattr(la_build, "TORCH", fake_torch(tmp_path / "torch"))
    assert not la_build.up_to_date()


def test_the_stamp_tells_versions_and_pythons_apart(tmp_path, monkeypatch):
    monkeypatch.setattr(la_build, "TORCH", fake_torch(tmp_path / "torch"))
    first = la_build.binding_stamp()
    (tmp_path / "torch" / "version.py").write_text("__version__ = '9.9.10'\n")
    second = la_build.binding_stamp()
    assert first != second
    monkeypatch.setattr(la_build.sysconfig, "get_config_var", lambda name: "cpython-399-somewhere")
    assert la_build.binding_stamp() not in (first, second)


def test_a_torch_without_cuda_is_no_reason_to_fail(tmp_path, monkeypatch):
    """The C library is built and up to date without a binding, which then says that it is missing."""
    assert la_build.cuda_torch(fake_torch(tmp_path / "cpu", cuda=False)) is None
    path = fake_torch(tmp_path / "cuda")
    assert la_build.cuda_torch(path) == path
    assert la_build.cuda_torch(None) is None
    monkeypatch.setattr(la_build, "TORCH", None)
    assert la_build.up_to_date()
