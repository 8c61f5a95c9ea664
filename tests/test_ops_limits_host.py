"""Host-side limits of the suffix and decode operators: sizes whose products leave 64 bits, grids that
one launch does not hold.  No call here reaches a kernel.  Run once more against the library whose
argument validation is built with ASan and UBSan."""
import ctypes
import os
import subprocess
import sys

import pytest

from test_ops_host import N, SHAPE, _call, _paged, gdn  # noqa: F401 (gdn: the fixture)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("change", [dict(total_tokens=1 << 60, h_q=16), dict(total_tokens=1 << 62), dict(total_tokens=1 << 31),
                                    dict(total_tokens=(1 << 63) - 1), dict(total_tokens=0, n_seqs=0x7fffffff, h_q=1 << 30, h_kv=1 << 30)])
def test_paged_sizes_beyond_32_bits(gdn, change):  # noqa: F811
    d = _paged(gdn, **change)
    assert gdn.gdn_paged_workspace_bytes(d) == 0
    for name in ("gdn_paged_attn", "gdn_qk_norm_rope"):
        assert _call(gdn, name, d, N[name]) == SHAPE


def test_under_sanitizers():
    try:
        from gated_deltanet_state_gdn_amd import build as gbuild
        gbuild.hipcc()
        rt = gbuild.clang_asan_runtime()
    except Exception as e:   # no ROCm toolchain on this host
        pytest.skip(str(e))
    lib = gbuild.build_host_sanitized()
    env = dict(os.environ, LD_PRELOAD=rt, GDN_LIB_PATH=lib, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0:halt_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    p = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", "-k", "not sanitizers and not index",
                        "tests/test_ops_limits_host.py", "tests/test_ops_host.py"], cwd=ROOT, env=env, capture_output=True,
                       text=True, timeout=600)
    assert p.returncode == 0, p.stdout[-3000:] + p.stderr[-3000:]
    assert "passed" in p.stdout and "skipped" not in p.stdout
