"""The C library is built by nvcc alone: neither torch nor the extension module
has a part in it."""
import os
import subprocess
import sys

import pytest

import paged_kv_cache_72_gb300.build as b

BLOCK = """
import sys, importlib.util
class NoTorch:
    def find_spec(self, name, path=None, target=None):
        if name.split('.')[0] == 'torch':
            raise ModuleNotFoundError('No module named torch')
sys.meta_path.insert(0, NoTorch())
spec = importlib.util.spec_from_file_location('build_alone', sys.argv[1])
m = importlib.util.module_from_spec(spec)
spec.loader.exec_module(m)
print(m.build_library())
"""


def test_library_builds_without_torch():
    b.build()
    r = subprocess.run([sys.executable, "-c", BLOCK, b.__file__], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert r.stdout.split()[-1] == b.LIB
    # nothing of torch in what it links
    names = subprocess.run(["readelf", "-d", b.LIB], capture_output=True, text=True).stdout
    assert "NEEDED" in names and "torch" not in names and "c10" not in names


def test_library_is_in_place_when_the_extension_module_fails(monkeypatch, tmp_path):
    # a stand-in library, an nvcc that writes its output file, and an extension module
    # whose source does not compile
    for name in ("csrc", "include", "build"):
        (tmp_path / name).mkdir()
    (tmp_path / "include" / "pa.h").write_text("")
    (tmp_path / "csrc" / "one.cu").write_text("")
    (tmp_path / "csrc" / b.CALL_SOURCE).write_text("this is not C++")
    nvcc = tmp_path / "bin" / "nvcc"
    nvcc.parent.mkdir()
    nvcc.write_text('#!/bin/sh\nwhile [ "$1" != "-o" ]; do shift; done\necho made > "$2"\n')
    nvcc.chmod(0o755)
    for name, value in (("CSRC", tmp_path / "csrc"), ("INCLUDE", tmp_path / "include"),
                        ("BUILD", tmp_path / "build"), ("PKG", tmp_path),
                        ("LIB", tmp_path / "libpa.so"), ("CALL", tmp_path / "_pa_call.so")):
        monkeypatch.setattr(b, name, str(value))
    monkeypatch.setattr(b, "SOURCES", ["one.cu"])
    monkeypatch.setattr(b, "_nvcc", lambda: str(nvcc))
    with pytest.raises(RuntimeError, match=b.CALL_SOURCE):
        b.build()
    assert (tmp_path / "libpa.so").read_text() == "made\n"
    assert not os.path.exists(b.CALL)
    # and the module's source is no reason to make the library again
    (tmp_path / "libpa.so").write_text("kept\n")
    (tmp_path / "csrc" / b.CALL_SOURCE).write_text("neither is this")
    with pytest.raises(RuntimeError, match=b.CALL_SOURCE):
        b.build()
    assert (tmp_path / "libpa.so").read_text() == "kept\n"
