"""Host: what is built and loaded when a part is missing (no compiler run but a C stub's, no GPU)."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_library_is_built_without_the_binding(tmp_path, monkeypatch):
    """No g++, no torch or Python headers: the C library is made all the same, and the failure is said."""
    from gated_deltanet_state_gdn_amd import build as b
    made = []
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libgdn.so"))
    monkeypatch.setattr(b, "BUILD", str(tmp_path))
    monkeypatch.setattr(b, "hipcc", lambda: "hipcc")
    monkeypatch.setattr(b, "_compile", lambda src: src + ".o")

    def link(cmd, *a, **kw):
        made.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(b.subprocess, "check_call", link)

    def no_headers():
        raise OSError("no g++ here")

    monkeypatch.setattr(b, "build_binding", no_headers)
    with pytest.raises(RuntimeError, match="no g\\+\\+ here"):
        b.build(verbose=False)
    assert os.path.exists(b.LIB) and len(made) == 1 and made[0][0] == "hipcc"
    os.remove(b.LIB)
    assert b.build_library(verbose=False) == b.LIB and os.path.exists(b.LIB)


def _load(tmp_path, source):
    if shutil.which("gcc") is None:
        pytest.skip("gcc not available")
    src, lib = tmp_path / "old.c", str(tmp_path / "libgdn.so")
    src.write_text(source)
    subprocess.check_call(["gcc", "-shared", "-fPIC", str(src), "-o", lib])
    code = ("import gated_deltanet_state_gdn_amd as gdn\n"
            "try:\n    gdn.load()\n"
            "except ImportError as e:\n    print('raised:', e)\n")
    p = subprocess.run([sys.executable, "-c", code], cwd=ROOT, env=dict(os.environ, GDN_LIB_PATH=lib), capture_output=True,
                       text=True, timeout=120)
    assert p.returncode == 0, p.stderr
    return p.stdout


def test_a_library_of_older_sources_is_refused(tmp_path):
    from gated_deltanet_state_gdn_amd import _lib
    old = [n for n in _lib.EXPORTS if not any(w in n for w in ("conv", "ssm", "step", "rope", "paged"))]
    said = _load(tmp_path, "int gdn_abi_version(void) { return %d; }\n" % _lib.ABI_VERSION +
                 "".join("void %s(void) {}\n" % n for n in old if n != "gdn_abi_version"))
    assert "raised:" in said and "gdn_conv" in said and "build" in said


def test_a_library_of_another_version_is_refused(tmp_path):
    said = _load(tmp_path, "int gdn_abi_version(void) { return 1; }\n")
    assert "raised:" in said and "version" in said
