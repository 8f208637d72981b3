"""The build of the C library without torch, and of the binding's native module beside it (CPU only; a small source of
its own, in a folder of its own)."""
import os

import pytest

from mamba_ssd_prefill_amd import build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    if not os.path.exists(build.HIPCC):
        pytest.skip("hipcc not available")
    (tmp_path / "include").mkdir()
    (tmp_path / "include" / "mamba_ssd.h").write_text("\n")
    (tmp_path / "one.cpp").write_text('extern "C" __attribute__((visibility("default"))) int one() { return 1; }\n')
    (tmp_path / "ssd_meta.cpp").write_text("int meta() { return 2; }\n")
    for name, value in (("SOURCES", ["one.cpp"]), ("CSRC", str(tmp_path)), ("ROOT", str(tmp_path)),
                        ("BUILD_DIR", str(tmp_path / "_build")), ("LIB", str(tmp_path / "libone.so")),
                        ("META", str(tmp_path / "_meta.so"))):
        monkeypatch.setattr(build, name, value)
    return tmp_path


def small_command(flag="-O0"):
    return lambda out: ["g++", flag, "-fPIC", "-shared", os.path.join(build.CSRC, "ssd_meta.cpp"), "-o", out]


def test_the_library_builds_without_torch(tree, monkeypatch, capsys):
    def no_torch(out):
        raise ImportError("No module named 'torch'")
    monkeypatch.setattr(build, "_meta_command", no_torch)
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert not os.path.exists(build.META) and "_meta" in capsys.readouterr().err
    assert sorted(f.name for f in tree.iterdir() if ".so" in f.name) == ["libone.so"]


def test_a_module_that_does_not_compile_leaves_the_library(tree, monkeypatch):
    (tree / "ssd_meta.cpp").write_text("no c++\n")
    monkeypatch.setattr(build, "_meta_command", small_command())
    with pytest.raises(RuntimeError, match="ssd_meta.cpp"):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.META)


def test_the_module_is_built_again_when_its_command_changes(tree, monkeypatch):
    """Another torch or Python gives another command (paths, versions, ABI): an incremental build notices."""
    monkeypatch.setattr(build, "_meta_command", small_command())
    build.build()
    first = os.stat(build.META).st_mtime_ns
    build.build(force=False)
    assert os.stat(build.META).st_mtime_ns == first
    monkeypatch.setattr(build, "_meta_command", small_command("-O1"))
    build.build(force=False)
    second = os.stat(build.META).st_mtime_ns
    assert second > first
    build.build(force=False)
    assert os.stat(build.META).st_mtime_ns == second
    build.build()
    assert os.stat(build.META).st_mtime_ns > second


def test_the_module_is_built_for_a_torch_and_a_python(monkeypatch):
    import torch
    made = build._meta_made_from(["g++"])
    monkeypatch.setattr(torch, "__version__", "0.0")
    assert made != build._meta_made_from(["g++"])
    assert "0.0" in build._meta_made_from(["g++"]) and "python" in made
