"""What building takes: libsmp.so needs nvcc alone; the extension module of the
cached step also PyTorch, headers and g++, and its absence is said when it is
asked for."""

import os
import sys

import pytest

from spec_verify_gb300 import binding, build


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """Builds of one source file into a folder of their own."""
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libsmp.so"))
    monkeypatch.setattr(build, "STEP_LIB", str(tmp_path / "smp_step_binding.so"))
    monkeypatch.setattr(build, "SOURCES", ["api.cu"])
    return tmp_path


def without(what, monkeypatch):
    if what == "PyTorch":
        for name in [n for n in sys.modules if n == "torch" or n.startswith("torch.")]:
            monkeypatch.delitem(sys.modules, name)
        monkeypatch.setitem(sys.modules, "torch", None)          # importing it fails
    elif what == "Python's headers":
        paths = dict(build.sysconfig.get_paths(), include="/nowhere")
        monkeypatch.setattr(build.sysconfig, "get_paths", lambda: paths)
    else:
        which = build.shutil.which
        monkeypatch.setattr(build.shutil, "which", lambda name: None if name == "g++" else which(name))


@pytest.mark.parametrize("what", ["PyTorch", "Python's headers", "g++"])
def test_libsmp_builds_without_what_the_extension_takes(what, elsewhere, monkeypatch, capsys):
    without(what, monkeypatch)
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert not os.path.exists(build.STEP_LIB)
    assert f"lacks {what}" in capsys.readouterr().err
    before = os.path.getmtime(build.LIB)
    assert build.up_to_date() and build.build() == build.LIB and os.path.getmtime(build.LIB) == before
    monkeypatch.setattr(binding, "_step", None)
    monkeypatch.setattr(binding, "_torch", lambda: None)
    monkeypatch.setattr(binding, "load", lambda: None)
    with pytest.raises(binding.SmpError, match=what):
        binding.step_module()


def test_an_extension_that_does_not_compile_leaves_libsmp_built(elsewhere, monkeypatch):
    pytest.importorskip("torch")
    source = elsewhere / "step_binding.cpp"
    source.write_text("#error not this one\n")
    monkeypatch.setattr(build, "STEP_SOURCE", str(source))
    with pytest.raises(RuntimeError, match="not this one"):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.STEP_LIB)


def test_an_extension_of_another_pytorch_is_not_loaded_but_built_again(elsewhere, monkeypatch):
    torch = pytest.importorskip("torch")
    for name in ("libsmp.so", "smp_step_binding.so"):
        (elsewhere / name).write_text("")
    stamp = elsewhere / "smp_step_binding.so.torch"
    stamp.write_text(str(torch.__version__))
    assert build.up_to_date()
    stamp.write_text("1.0.0")
    assert not build.up_to_date()
    monkeypatch.setattr(binding, "_step", None)
    monkeypatch.setattr(binding, "load", lambda: None)
    with pytest.raises(binding.SmpError, match="built against PyTorch 1.0.0"):
        binding.step_module()
    stamp.unlink()
    assert not build.up_to_date()
