"""The build script: the library without torch, and one binding module a torch version."""
import os
import subprocess
import sys

import pytest

from normalisation_row_bf16_b200 import build as nbuild
from normalisation_row_bf16_b200 import ops

SCRIPT = """
import sys
sys.modules["torch"] = None                  # import torch raises ImportError
sys.path.insert(0, {root!r})
from normalisation_row_bf16_b200 import build as b
b.PKG, b.CSRC, b.LIB = {tmp!r}, {tmp!r}, {tmp!r} + "/libtiny.so"
print(b.build(verbose=True))
"""


def test_library_builds_without_torch(tmp_path):
    (tmp_path / "tiny.cu").write_text('extern "C" int tiny() { return 7; }\n')
    r = subprocess.run([sys.executable, "-c", SCRIPT.format(root=nbuild.ROOT, tmp=str(tmp_path))], capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert os.path.exists(tmp_path / "libtiny.so")
    assert not list(tmp_path.glob("_binding*"))


@pytest.mark.parametrize("broken", ["raises", "fails"])
def test_library_is_built_where_the_binding_is_not(broken, monkeypatch):
    built = []
    monkeypatch.setattr(nbuild, "_build_library", lambda force, verbose: built.append(1) or "lib")
    monkeypatch.setattr(nbuild, "binding_is_stale", lambda: True)

    def start(verbose):
        if broken == "raises":
            raise FileNotFoundError("no C++ compiler")
        return subprocess.Popen([sys.executable, "-c", "raise SystemExit(1)"]), "unused"
    monkeypatch.setattr(nbuild, "_start_binding", start)
    with pytest.raises(RuntimeError, match="binding"):
        nbuild.build()
    assert built


def test_binding_of_another_torch_is_not_taken(monkeypatch):
    import torch
    mine = nbuild.binding_path()
    assert torch.__version__ in mine
    monkeypatch.setattr(torch, "__version__", "1.0.0")
    assert nbuild.binding_path() != mine and nbuild.binding_is_stale()
    monkeypatch.setattr(ops, "_binding_module", None)
    with pytest.raises(RuntimeError, match="is missing"):
        ops._binding()


def test_a_changed_header_makes_the_library_stale(tmp_path, monkeypatch):
    for d, n in (("CSRC", "a.cu"), ("CSRC", "b.cuh"), ("CSRC", "c.h"), ("INCLUDE", "d.h")):
        at = tmp_path / d
        at.mkdir(exist_ok=True)
        (at / n).write_text("")
        os.utime(at / n, (1000, 1000))
        monkeypatch.setattr(nbuild, d, str(at))
    lib = tmp_path / "lib.so"
    lib.write_text("")
    os.utime(lib, (2000, 2000))
    monkeypatch.setattr(nbuild, "LIB", str(lib))
    assert not nbuild.is_stale()
    for p in ("CSRC/a.cu", "CSRC/b.cuh", "CSRC/c.h", "INCLUDE/d.h"):
        os.utime(tmp_path / p, (3000, 3000))
        assert nbuild.is_stale(), p
        os.utime(tmp_path / p, (1000, 1000))
