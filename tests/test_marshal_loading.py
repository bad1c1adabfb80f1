"""Which file binding.load() takes as the compiled marshalling, on the CPU: one built
from these sources."""
import os
import shutil
import sysconfig

from diffusion_transformer_joint_gb300 import build


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
