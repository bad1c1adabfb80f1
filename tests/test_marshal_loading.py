"""Which file binding.load() takes as the compiled marshalling, on the CPU: one built
from these sources, and none that does not load."""
import os
import shutil
import subprocess
import sys
import sysconfig

import pytest

import __graft_entry__
from diffusion_transformer_joint_gb300 import binding, build


def test_a_module_of_other_sources_has_another_name(tmp_path, monkeypatch):
    """With a changed prototype, or changed marshalling, the module built before is
    not the one that load() looks for: it would call by the old prototypes."""
    before = build.marshal_path()
    include, pkg = tmp_path / "include", tmp_path / "pkg"
    shutil.copytree(build.INCLUDE, include)
    pkg.mkdir()
    shutil.copy(os.path.join(build.PKG, "marshal.cpp"), pkg)
    monkeypatch.setattr(build, "INCLUDE", str(include))
    monkeypatch.setattr(build, "PKG", str(pkg))
    assert build.marshal_path() == before  # (the same sources elsewhere)
    for changed in (include / "flux_attn.h", pkg / "marshal.cpp"):
        text = changed.read_text()
        changed.write_text(text.replace("mask_bs", "mask_stride"))
        assert build.marshal_path() != before
        assert os.path.dirname(build.marshal_path()) == os.path.dirname(before)
        changed.write_text(text)


def test_a_module_of_another_interpreter_has_another_name(monkeypatch):
    """Two interpreters with the same torch in one tree: extension modules are not
    theirs to share, and the name's ending says whose one is."""
    before = build.marshal_path()
    assert before.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    get = sysconfig.get_config_var
    monkeypatch.setattr(sysconfig, "get_config_var",
                        lambda n: ".cpython-399.so" if n == "EXT_SUFFIX" else get(n))
    assert build.marshal_path() != before and build.marshal_path().endswith(".cpython-399.so")

_LOAD = """
import sys, warnings
warnings.simplefilter("ignore")
from diffusion_transformer_joint_gb300 import binding, build
{}
lib = binding.load()
assert binding._compiled is None and binding._compiled_lib is None
assert lib.flux_status_string(0)
print("loaded")
"""


@pytest.mark.parametrize("spoil", [
    "open(sys.argv[1], 'w').write('no module'); build.marshal_path = lambda: sys.argv[1]",
    "open(sys.argv[1], 'w').close(); build.marshal_path = lambda: sys.argv[1]",
    "build.marshal_path = lambda: build.LIB_PATH",   # a library, but no module
    "sys.modules['torch'] = None",                   # no torch: the C functions alone
    "build.INCLUDE = sys.argv[1]",                   # no header beside the package
], ids=["text", "empty", "no-module", "no-torch", "no-header"])
def test_without_a_module_that_loads_the_library_is_there(spoil, tmp_path):
    """In a process of its own: load() returns the library, whose calls are marshalled
    in Python."""
    build.build()
    r = subprocess.run([sys.executable, "-c", _LOAD.format(spoil), str(tmp_path / "_marshal.so")],
                       capture_output=True, text=True, cwd=build.ROOT)
    assert r.stdout == "loaded\n", r.stderr


def test_a_module_that_does_not_load_is_said(tmp_path, monkeypatch):
    bad = tmp_path / "_marshal.so"
    bad.write_text("no module")
    monkeypatch.setattr(build, "marshal_path", lambda: str(bad))
    monkeypatch.setattr(binding, "_compiled", None)
    monkeypatch.setattr(binding, "_compiled_lib", None)
    with pytest.warns(RuntimeWarning, match="marshalled in Python"):
        binding._load_compiled(object())
    assert binding._compiled is None


@pytest.mark.parametrize("fault", [FileNotFoundError("g++"), RuntimeError("g++ failed"),
                                   ModuleNotFoundError("torch")], ids=lambda e: type(e).__name__)
def test_the_build_goes_on_without_the_marshalling(fault, monkeypatch, capsys):
    """Without g++ or torch's headers the library and the oracle are built all the
    same, and the message says what is missing."""
    def fail(force=False):
        raise fault

    monkeypatch.setattr(build, "build_marshal", fail)
    __graft_entry__.build()
    assert str(fault) in capsys.readouterr().err
    monkeypatch.setattr(sys, "argv", ["build.py"])
    assert build.main() == 0
    said = capsys.readouterr()
    assert said.out.strip() == build.LIB_PATH and str(fault) in said.err
