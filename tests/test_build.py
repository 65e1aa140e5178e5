"""When the built files count as up to date, and what is built again."""
import os

import pytest

from gemm_conv_chains_gb300 import build


@pytest.fixture
def built(tmp_path, monkeypatch):
    """A tree of one source whose built files are newer, and what build() would run."""
    src = tmp_path / "a.cu"
    src.write_text("")
    os.utime(src, (1000, 1000))
    made = []

    def binding(obj):
        made.append("binding")
        (tmp_path / "_binding.so").write_text("")
        (tmp_path / "binding.for").write_text(build._binding_target())

    for name, value in (("BUILD_DIR", str(tmp_path)), ("LIB_PATH", str(tmp_path / "libb2b.so")),
                        ("BINDING_PATH", str(tmp_path / "_binding.so")),
                        ("BINDING_FOR", str(tmp_path / "binding.for")), ("_deps", lambda: [str(src)]),
                        ("_compile_binding", lambda: "binding.o"), ("_link_binding", binding)):
        monkeypatch.setattr(build, name, value)
    (tmp_path / "libb2b.so").write_text("")
    binding(None)
    made.clear()
    return tmp_path, made


def test_built_files_newer_than_the_sources_stay(built):
    assert build.up_to_date()
    assert build.build() == build.LIB_PATH and built[1] == []


@pytest.mark.parametrize("change", ["torch", "python", "unknown"])
def test_another_torch_or_python_has_the_binding_built_anew(built, monkeypatch, change):
    import sysconfig

    import torch
    if change == "torch":
        monkeypatch.setattr(torch, "__version__", "0.0.1")
    elif change == "python":
        real = sysconfig.get_config_var
        monkeypatch.setattr(sysconfig, "get_config_var", lambda n: "cp" if n == "SOABI" else real(n))
    else:
        os.remove(build.BINDING_FOR)
    assert not build.up_to_date()
    assert build.build() == build.LIB_PATH
    assert built[1] == ["binding"] and build.up_to_date()


@pytest.mark.parametrize("missing", ["libb2b.so", "_binding.so"])
def test_a_missing_or_older_file_is_not_up_to_date(built, missing):
    path = built[0] / missing
    os.utime(path, (500, 500))
    assert not build.up_to_date()
    os.remove(path)
    assert not build.up_to_date()
