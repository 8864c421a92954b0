"""When the build is up to date: not with sources newer than what was built,
nor with a binding built against another PyTorch or Python. CPU only."""
import os
import sysconfig

import pytest

from row_wise_softmax_ce_gb300 import build as cuda_build


@pytest.fixture
def built(tmp_path, monkeypatch):
    """A finished build elsewhere, against a PyTorch of version 1."""
    torch = tmp_path / "torch"
    torch.mkdir()
    (torch / "version.py").write_text("__version__ = '1'\n")
    monkeypatch.setattr(cuda_build, "_torch_dir", lambda: str(torch))
    for name in ("LIB", "BINDING", "BINDING_FOR"):
        path = tmp_path / name
        path.write_text("")
        monkeypatch.setattr(cuda_build, name, str(path))
    (tmp_path / "BINDING_FOR").write_text(cuda_build._binding_for())
    assert cuda_build.up_to_date()
    return tmp_path


def test_another_pytorch_version(built):
    (built / "torch" / "version.py").write_text("__version__ = '2'\n")
    assert not cuda_build.up_to_date()


def test_pytorch_elsewhere(built, monkeypatch):
    other = built / "site" / "torch"
    other.mkdir(parents=True)
    (other / "version.py").write_text("__version__ = '1'\n")
    monkeypatch.setattr(cuda_build, "_torch_dir", lambda: str(other))
    assert not cuda_build.up_to_date()


def test_another_python(built, monkeypatch):
    real = sysconfig.get_config_var
    monkeypatch.setattr(sysconfig, "get_config_var", lambda name: "cpython-399" if name == "SOABI" else real(name))
    assert not cuda_build.up_to_date()


def test_no_record(built):
    os.remove(built / "BINDING_FOR")
    assert not cuda_build.up_to_date()


def test_a_newer_source(built):
    os.utime(built / "LIB", (1, 1))
    assert not cuda_build.up_to_date()


def test_the_real_build_is_recorded():
    cuda_build.build()
    assert cuda_build.up_to_date()
    with open(cuda_build.BINDING_FOR) as f:
        assert f.read() == cuda_build._binding_for()
    assert cuda_build._torch_dir() in cuda_build._binding_for()
