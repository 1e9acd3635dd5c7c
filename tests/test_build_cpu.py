"""The build on machines of other kinds: what is compiled and linked when, with the compilers
replaced by a function that writes the file they are asked for."""
import itertools
import os
import subprocess

import pytest

from int4_weight_only_matmulnbits_gb300 import _build


class Compilers:
    def __init__(self, where, monkeypatch):
        self.made, self.fail = [], None
        for name in ("OBJ_DIR", "LIB_PATH", "PY_PATH"):
            if hasattr(_build, name):
                path = str(where / os.path.basename(getattr(_build, name)))
                monkeypatch.setattr(_build, name, path)
        monkeypatch.setattr(_build, "_nvcc", lambda: "nvcc")
        monkeypatch.setattr(_build.subprocess, "run", self.run)
        self.clock = itertools.count(int(os.path.getmtime(_build.PY_SRC)) + 10 ** 6)

    def run(self, cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        name = os.path.basename(out).split(".tmp")[0]
        failed = self.fail is not None and self.fail in cmd[0] + " " + name
        if not failed:
            self.made.append(name)
            with open(out, "w") as f:
                f.write(" ".join(cmd))
            now = next(self.clock)  # every file is newer than the one before it
            os.utime(out, (now, now))
        return subprocess.CompletedProcess(cmd, int(failed), "", "no such compiler")

    def build(self):
        """What a build makes, in order; it may raise."""
        self.made.clear()
        _build.build_library()
        return list(self.made)


@pytest.fixture
def compilers(tmp_path, monkeypatch):
    return Compilers(tmp_path, monkeypatch)


def test_the_library_is_built_without_torch(compilers, monkeypatch):
    """A caller of the C ABI needs nvcc alone."""
    find = _build.importlib.util.find_spec
    monkeypatch.setattr(_build.importlib.util, "find_spec",
                        lambda name, *a: None if name == "torch" else find(name, *a))
    made = compilers.build()
    assert made[-1] == "libmnb.so" and not any("py" in n for n in made)
    assert os.path.exists(_build.LIB_PATH)
    assert compilers.build() == []


def test_the_library_is_linked_whatever_becomes_of_the_binding(compilers):
    """Without g++ or torch's headers the binding's native part fails, and says so; libmnb.so is
    there by then."""
    compilers.fail = "g++"
    with pytest.raises(RuntimeError, match="py_attn"):
        compilers.build()
    assert os.path.exists(_build.LIB_PATH)
    compilers.fail = None
    made = compilers.build()
    assert len(made) == 2 and made[0].startswith("py_attn.") and made[1].startswith("_mnb_py")
    assert compilers.build() == []


def test_each_torch_has_a_module_of_its_own(compilers, monkeypatch, tmp_path):
    """Built for one torch, then another, then the first again: what the binding would load is made
    for the torch of the process each time, and newer than its object."""
    for turn, version in enumerate(("1", "2", "1", "2")):
        torch_dir = tmp_path / f"torch{version}"
        torch_dir.mkdir(exist_ok=True)
        (torch_dir / "version.py").write_text(f"version = {version!r}\n")
        monkeypatch.setattr(_build, "_torch_dir", lambda: str(torch_dir))
        made = compilers.build()
        with open(_build.py_path()) as f:
            command = f.read()
        obj = [w for w in command.split() if "py_attn." in w][0]
        with open(obj) as f:
            assert str(torch_dir) in command and str(torch_dir) in f.read()
        assert os.path.getmtime(_build.py_path()) > os.path.getmtime(obj)
        assert [n for n in made if "py" in n] == (
            [os.path.basename(obj), os.path.basename(_build.py_path())] if turn < 2 else [])
