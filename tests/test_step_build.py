"""Building the libraries: the collectives' does not depend on the step operators' Python module."""
import importlib.util
import os
import subprocess
import sysconfig
from types import SimpleNamespace

import pytest

from all_gather_placement_amd import build


@pytest.fixture
def linked(monkeypatch):
    """The libraries that a build links, in order; nothing is compiled.  Sources in `broken` do not compile."""
    made, broken = [], set()

    class Compile:
        def __init__(self, args):
            self.args = args

        def wait(self):
            self.returncode = int(any(a.endswith(b) for a in self.args for b in broken))
            return self.returncode

    monkeypatch.setattr(build.subprocess, "Popen", Compile)
    monkeypatch.setattr(build.subprocess, "run", lambda *a, **k: None)
    monkeypatch.setattr(build.os, "replace", lambda tmp, out: made.append(out))
    return made, broken


def test_every_library_is_built(linked):
    made, _ = linked
    assert build.build() == build.LIB
    assert made[0] == build.LIB and set(made) == {build.LIB, build.PROBE_LIB, build.STEP_LIB, build.STEP_BINDING}
    assert made.index(build.STEP_LIB) < made.index(build.STEP_BINDING)  # which links it


def test_the_collectives_are_built_without_torch(linked, monkeypatch):
    made, _ = linked
    found = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else found(name, *a))
    assert build.build() == build.LIB
    assert made == [build.LIB, build.PROBE_LIB, build.STEP_LIB]
    # what cannot be built is not asked for
    asked = []
    monkeypatch.setattr(build, "is_current", lambda lib: asked.append(lib) or True)
    build.ensure_built()
    assert asked == [build.LIB, build.PROBE_LIB, build.STEP_LIB]


def test_the_collectives_are_built_where_the_module_is_not(linked):
    """Torch without its headers: the error is raised, the libraries are there."""
    made, broken = linked
    broken.add("step_binding.cpp")
    with pytest.raises(subprocess.CalledProcessError):
        build.build()
    assert made == [build.LIB, build.PROBE_LIB, build.STEP_LIB]


def test_the_modules_build_id_covers_torch_and_the_interpreter(monkeypatch, tmp_path):
    """Its compiled code fits one torch and one interpreter; the libraries' code depends on neither."""
    libs = (build.LIB, build.PROBE_LIB, build.STEP_LIB)
    ids, module = [build.source_hash(lib) for lib in libs], build.source_hash(build.STEP_BINDING)
    assert build.built_id(build.STEP_BINDING) == module
    torch = importlib.util.find_spec("torch").submodule_search_locations[0]
    (tmp_path / "version.py").write_bytes(open(os.path.join(torch, "version.py"), "rb").read())
    found = importlib.util.find_spec
    there = SimpleNamespace(submodule_search_locations=[str(tmp_path)])
    seen = {module}

    def changed():
        assert [build.source_hash(lib) for lib in libs] == ids
        now = build.source_hash(build.STEP_BINDING)
        new = now not in seen
        seen.add(now)
        return new

    with monkeypatch.context() as m:
        m.setattr(importlib.util, "find_spec", lambda name, *a: there if name == "torch" else found(name, *a))
        assert not changed()  # the same torch elsewhere
        (tmp_path / "version.py").write_text("__version__ = '99.0'\n")
        assert changed()
        assert not build.is_current(build.STEP_BINDING)
    config = sysconfig.get_config_var
    with monkeypatch.context() as m:
        m.setattr(sysconfig, "get_config_var", lambda name: "cpython-999" if name == "SOABI" else config(name))
        assert changed()
    with monkeypatch.context() as m:
        m.setattr(build, "MODULE_FLAGS", ["-O1"])
        assert changed()
