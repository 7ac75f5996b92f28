"""The build without a GPU: the Python extension's versions are in its name, and a machine that
cannot build it still gets the library."""
import os
import subprocess
import sysconfig

import pytest
import torch

from test_linear_forms import sv  # noqa: F401
from speculative_decoding_verification_31_gb300 import build


def test_the_name_holds_both_versions(monkeypatch):
    path = build.binding_path()
    assert path.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    monkeypatch.setattr(torch, "__version__", "99.1.2+cu999")
    other = build.binding_path()
    assert other != path and "99_1_2_cu999" in other
    assert not build.up_to_date(other, build.BINDING_DEPS)  # one built for this PyTorch does not count


@pytest.mark.parametrize("command", [["false"], ["/nonexistent/c++"]], ids=["fails", "no compiler"])
def test_the_library_is_built_without_the_extension(sv, monkeypatch, tmp_path, capfd, command):  # noqa: F811
    path = tmp_path / "_binding.so"
    path.write_bytes(b"an old one")
    os.utime(path, (0, 0))
    monkeypatch.setattr(build, "binding_path", lambda: str(path))
    monkeypatch.setattr(build, "binding_command", lambda: command)
    assert build.build() == build.LIB and not path.exists()
    assert "extension was not built" in capfd.readouterr().err


def test_a_failed_library_raises(monkeypatch, tmp_path):
    monkeypatch.setattr(build, "nvcc_command", lambda **_: ["false"])
    monkeypatch.setattr(build, "LIB", str(tmp_path / "lib.so"))
    with pytest.raises(subprocess.CalledProcessError):
        build.build()


def test_a_missing_extension_is_named_at_the_call(sv, monkeypatch, tmp_path):  # noqa: F811
    """The calls through ctypes do not need it; the others say what is missing."""
    monkeypatch.setattr(build, "binding_path", lambda: str(tmp_path / "_binding.so"))
    monkeypatch.setattr(sv.specverify, "_ops", None)
    with pytest.raises(RuntimeError, match="not built"):
        sv.spec_rms_norm(torch.zeros(2, 8), torch.zeros(8))
    assert sv.spec_verify_strerror(sv.SPEC_EBADLEN)
